"""Results of kvc_rotate that share memory with its operand: refused but in place.  The
test of layouts (csrc/kvc_overlap.h) against sets of bytes."""
import ctypes
import os
import random
import shutil
import subprocess
import time

import pytest

import kv_cache_compression_c128_gb300 as kvc

SHIM = """
#include "kvc_overlap.h"
extern "C" int meet(int64_t x, int64_t xt, int64_t xh, int64_t out, int64_t ot, int64_t oh, int64_t tokens, int64_t heads, int64_t size) {
  return kvc::rows_meet(reinterpret_cast<const void*>(x), {xt, xh}, reinterpret_cast<const void*>(out), {ot, oh}, tokens, heads, size, 1);
}
"""


@pytest.fixture(scope="module")
def meet(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("overlap")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", f"-I{kvc._CSRC}", str(d / "shim.cpp"), "-o", str(d / "shim.so")], check=True)
    f = ctypes.CDLL(str(d / "shim.so")).meet
    f.argtypes = [ctypes.c_int64] * 9
    return f


def _bytes(at, by_token, by_head, tokens, heads, size):
    return {at + t * by_token + h * by_head + i for t in range(tokens) for h in range(heads) for i in range(size)}


def test_layouts_against_sets_of_bytes(meet):
    rng = random.Random(1)
    seen = [0, 0]
    for _ in range(20000):
        tokens, heads, size = rng.randint(1, 5), rng.randint(1, 5), rng.randint(1, 4)
        stride = lambda: rng.choice((0, size, rng.randint(0, 40), rng.randint(0, 12) * size))
        x, out = [1000 + rng.randint(0, 60), stride(), stride()], [1000 + rng.randint(0, 60), stride(), stride()]
        if rng.random() < 0.3:
            out[1] = x[1]
        if rng.random() < 0.3:
            out[2] = x[2]
        want = not _bytes(*x, tokens, heads, size).isdisjoint(_bytes(*out, tokens, heads, size))
        assert bool(meet(*x, *out, tokens, heads, size)) == want, (x, out, tokens, heads, size)
        seen[want] += 1
    assert min(seen) > 3000


def test_large_layouts_are_told_apart_quickly(meet):
    T, H, W = 1 << 20, 64, 128 * (512 + 64)  # queries [T, H, 512] and turned dims [T, H, 64] in the rows of one tensor
    began = time.perf_counter()
    base = 1 << 40
    assert not meet(base + 896, W, 1024, base + H * 1024, W, 128, T, H, 128)
    assert meet(base + 896, W, 1024, base + H * 1024 - 16, W, 128, T, H, 128)
    assert not meet(base + 896, W, 1024, base, W, 1024, T, H, 128)            # other dims of the same rows
    assert meet(base + 896, W, 1024, base + 880, W, 1024, T, H, 128)
    assert meet(base + 896, W, 1024, base + 896 + W, W, 1024, T, H, 128)      # a token on
    assert meet(base, W, 0, base + 5 * W, W, 128, T, H, 128)                  # one row for all heads
    assert meet(base + 896, W, 1024, base, H * 128, 128, T, H, 128)           # closed up in place
    assert not meet(base, W, 1024, base + T * W, H * 128, 128, T, H, 128)
    assert not meet(base + 896, W, 1024, base + 128 * T, 1024, 1 << 36, T, H, 128)  # between the rows for a long way
    assert meet(base + 896, W, 1024, base + 128 * T - 16, 1024, 1 << 36, T, H, 128)
    assert not meet(base, 1 << 62, 1 << 62, base + 128, 128, 1 << 32, T, H, 128)  # (beyond any memory, but not a number too large)
    assert meet(base, 1 << 62, 1 << 62, base - 64, 128, 1 << 32, T, H, 128)
    assert time.perf_counter() - began < 2


_X = 0x10000000
_ROTATE = dict(x=_X, dtype=1, x_token_stride=8 * 512, x_head_stride=512, num_tokens=10, num_heads=8, positions=0x40000,
               positions_token_stride=1, positions_axis_stride=0, num_axes=1, pair_axes=None, cos_sin_cache=0x50000,
               num_positions=100, inverse=0, stream=0)


@pytest.mark.parametrize("out,by_token,by_head", [
    (_X + 16, 8 * 512, 512), (_X - 16, 8 * 512, 512), (_X + 1024, 8 * 512, 512), (_X + 8 * 1024, 8 * 512, 512), (_X, 8 * 64, 64),
    (_X, 8 * 512, 64), (_X, 512, 10 * 512), (_X + 7 * 1024 + 112, 8 * 512, 64), (_X + 9 * 8 * 1024 + 7 * 1024, 8 * 64, 64),
    (_X - 128 * 79 + 16, 8 * 64, 64)])
def test_results_over_other_rows_are_refused(out, by_token, by_head):
    kvc.build()
    assert kvc.kvc_rotate(**_ROTATE, out=out, out_token_stride=by_token, out_head_stride=by_head) == kvc.KVC_ERR_INVALID_ARG
