"""kvc.join against a 64-bit form."""
import numpy as np
import pytest
import torch

import slots_testlib as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_compression_c128_gb300 as kvc

    kvc.build()
    return kvc


def _parts(seed, parts, shape, dtype, empty=0.2):
    rng = np.random.default_rng(seed)
    outs = [torch.from_numpy(rng.standard_normal(shape + (512,)).astype(np.float32)).to(dtype) for _ in range(parts)]
    lses = [torch.from_numpy((4 * rng.standard_normal(shape)).astype(np.float32)) for _ in range(parts)]
    for x in lses:
        x[torch.from_numpy(rng.random(shape) < empty)] = -np.inf
    return outs, lses


def _check(out, lse, outs, lses, dtype):
    want, want_lse, away = plain.join([o.double().numpy() for o in outs], [x.numpy() for x in lses])
    n = len(outs)
    # weights: a difference of two fp32 numbers (a half step of the larger), exp and the sum;
    # then a step per part in each sum and one rounding to the type
    big = np.max(np.stack([np.where(np.isinf(x.numpy()), 0, np.abs(x.numpy())) for x in lses]), 0)
    rel = (2 * (big + 4) + 2 * n + 8) * plain.STEP_F32
    half = plain.HALF_BF16 if dtype == torch.bfloat16 else plain.STEP_F32 / 2
    tol = away * rel[..., None] + half * np.abs(want) * 1.01 + 1e-37
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all()
    g = lse.double().cpu().numpy()
    same = g == want_lse
    assert (same | (np.abs(np.where(same, 0, g - np.where(same, 0, want_lse))) <= rel + 4 * plain.STEP_F32 * (big + 4))).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("parts,shape", [(1, (3, 5)), (2, (8, 64)), (3, (1,)), (5, (129, 3)), (8, (7, 2, 3)), (2, (1031,)),
                                         (4, (611, 17))])
def test_join(kvc, parts, shape, dtype):
    outs, lses = _parts(parts + len(shape), parts, shape, dtype)
    out, lse = kvc.join([o.cuda() for o in outs], [x.cuda() for x in lses])
    _check(out, lse, outs, lses, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_that_no_part_holds(kvc, dtype):
    outs, lses = _parts(1, 3, (10,), dtype, empty=0.0)
    for x in lses:
        x[4] = -np.inf
    lses[1][6] = -np.inf
    outs[1][6] = float("nan")                # not read into the sum
    out, lse = kvc.join([o.cuda() for o in outs], [x.cuda() for x in lses])
    assert (out[4] == 0).all() and lse[4] == -np.inf
    outs[1][6] = 0
    _check(out, lse, outs, lses, dtype)


def test_far_apart_and_large(kvc):
    outs, lses = _parts(2, 2, (6,), torch.float32, empty=0.0)
    lses[0][:3], lses[1][:3] = 1e30, -1e30
    lses[0][3:], lses[1][3:] = -3e38, -3e38
    out, lse = kvc.join([o.cuda() for o in outs], [x.cuda() for x in lses])
    assert torch.equal(out[:3].cpu(), outs[0][:3])
    assert torch.equal(out[3:].cpu(), (outs[0][3:] + outs[1][3:]) * 0.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_and_zero_rows(kvc, dtype):
    outs, lses = _parts(3, 4, (333,), dtype)
    o, x = [t.cuda() for t in outs], [t.cuda() for t in lses]
    want = kvc.join(o, x)
    got = kvc.join(o, x, out=o[2], lse=x[1])
    assert got[0] is o[2] and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    empty = kvc.join([t[:0] for t in o], [t[:0] for t in x])
    assert empty[0].shape == (0, 512) and empty[1].shape == (0,)


def test_stream_and_graph(kvc):
    outs, lses = _parts(4, 2, (50,), torch.bfloat16)
    o, x = [t.cuda() for t in outs], [t.cuda() for t in lses]
    want = kvc.join(o, x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = kvc.join(o, x, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = kvc.join(o, x)
    g.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
