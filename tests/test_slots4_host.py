"""4-bit slots, vectors into slots and rotary positions without a device: refusals of
the C entry points and the wrappers, and what their plain forms promise."""
import os
import shutil

import numpy as np
import pytest
import torch

import slots4_testlib as four

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")


@pytest.fixture(scope="module")
def kvc():
    import kv_cache_compression_c128_gb300 as kvc

    kvc.build()
    return kvc


AXES = bytes([0] * 16 + [1] * 16)
_STORE = dict(x=0x10000, x_dtype=1, x_row_stride=512, num_rows=10, kv_cache=0x20000, kv_format=1, num_kv_pages=4,
              slots=0x30000, positions=0x40000, positions_row_stride=2, positions_axis_stride=1, num_axes=2,
              pair_axes=AXES, cos_sin_cache=0x50000, num_positions=100, stream=0)


@pytest.mark.parametrize("change", [
    dict(x=0), dict(x=0x10008), dict(x_dtype=2), dict(x_dtype=-1), dict(x_row_stride=-512), dict(x_row_stride=516),
    dict(x_dtype=0, x_row_stride=514), dict(num_rows=-1), dict(num_rows=1 << 33), dict(kv_cache=0), dict(kv_cache=0x20004),
    dict(kv_format=2), dict(kv_format=-1), dict(num_kv_pages=0), dict(num_kv_pages=-3), dict(slots=0), dict(slots=0x30004),
    dict(positions=0), dict(positions=0x40004), dict(positions_row_stride=-1), dict(positions_axis_stride=-1),
    dict(num_axes=5), dict(num_axes=-1), dict(num_axes=1), dict(pair_axes=None), dict(pair_axes=bytes([2] * 32)),
    dict(cos_sin_cache=0), dict(cos_sin_cache=0x50004), dict(num_positions=0), dict(num_axes=0),
    dict(num_axes=0, positions=0), dict(num_axes=0, pair_axes=None)])
def test_store_refuses(kvc, change):
    assert kvc.kvc_store(**dict(_STORE, **change)) == kvc.KVC_ERR_INVALID_ARG


def test_store_of_no_row_is_a_no_op(kvc):
    assert kvc.kvc_store(**dict(_STORE, num_rows=0)) == kvc.KVC_OK
    assert kvc.kvc_store(**dict(_STORE, num_rows=0, x=0, slots=0, positions=0)) == kvc.KVC_OK


_ROTATE = dict(x=0x10000, dtype=1, x_token_stride=8 * 512, x_head_stride=512, num_tokens=10, num_heads=8, positions=0x40000,
               positions_token_stride=2, positions_axis_stride=1, num_axes=2, pair_axes=AXES, cos_sin_cache=0x50000,
               num_positions=100, inverse=0, out=0x60000, out_token_stride=8 * 64, out_head_stride=64, stream=0)


@pytest.mark.parametrize("change", [
    dict(x=0), dict(x=0x10002), dict(dtype=2), dict(x_token_stride=-8), dict(x_token_stride=4), dict(x_head_stride=4),
    dict(dtype=0, x_head_stride=66), dict(num_tokens=-1), dict(num_heads=-1), dict(num_tokens=1 << 33), dict(num_heads=65536),
    dict(positions=0), dict(positions=0x40002), dict(positions_token_stride=-2), dict(positions_axis_stride=-2),
    dict(num_axes=0), dict(num_axes=5), dict(num_axes=1), dict(pair_axes=None), dict(cos_sin_cache=0),
    dict(cos_sin_cache=0x50008), dict(num_positions=-1), dict(inverse=2), dict(out=0), dict(out=0x60008),
    dict(out_token_stride=8 * 64 - 8), dict(out_head_stride=56), dict(out_head_stride=0), dict(out_token_stride=0),
    dict(out_token_stride=32), dict(out_token_stride=64, out_head_stride=64 * 10 - 8), dict(out_head_stride=-64)])
def test_rotate_refuses(kvc, change):
    assert kvc.kvc_rotate(**dict(_ROTATE, **change)) == kvc.KVC_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(num_tokens=0), dict(num_heads=0), dict(num_tokens=0, x=0, out=0, positions=0)])
def test_rotate_of_nothing_is_a_no_op(kvc, change):
    assert kvc.kvc_rotate(**dict(_ROTATE, **change)) == kvc.KVC_OK


@pytest.mark.parametrize("change", [
    dict(kv_format=2), dict(kv_cache=0), dict(kv_cache=0x10004), dict(num_kv_pages=0), dict(slots=0), dict(slots=0x20004),
    dict(num_slots=-1), dict(num_slots=1 << 33), dict(out=0), dict(out=0x30008), dict(out_dtype=7)])
def test_dequantize_refuses(kvc, change):
    args = dict(kv_cache=0x10000, kv_format=1, num_kv_pages=3, slots=0x20000, num_slots=5, out=0x30000, out_dtype=1, stream=0)
    assert kvc.kvc_dequantize_format(**dict(args, **change)) == kvc.KVC_ERR_INVALID_ARG
    assert kvc.kvc_dequantize_format(**dict(args, num_slots=0)) == kvc.KVC_OK


def test_attend_and_evict_refuse_other_forms(kvc):
    from test_slots_host import _ATTEND, _EVICT

    for form in (-1, 2):
        assert kvc.kvc_attend_format(**_ATTEND, kv_format=form) == kvc.KVC_ERR_INVALID_ARG
        assert kvc.kvc_evict_format(**_EVICT, kv_format=form) == kvc.KVC_ERR_INVALID_ARG
    for form in (0, 1):
        assert kvc.kvc_attend_format(**dict(_ATTEND, num_reqs=0), kv_format=form) == kvc.KVC_OK
        assert kvc.kvc_attend_format(**dict(_ATTEND, q=0), kv_format=form) == kvc.KVC_ERR_INVALID_ARG
        assert kvc.kvc_evict_format(**dict(_EVICT, num_reqs=0), kv_format=form) == kvc.KVC_OK
        assert kvc.kvc_evict_format(**dict(_EVICT, keep=-1), kv_format=form) == kvc.KVC_ERR_INVALID_ARG


def test_wrappers_refuse_cpu_tensors(kvc):
    assert kvc.KV4_PAGE_BYTES == four.PAGE4_BYTES
    kv = torch.zeros((2, kvc.KV4_PAGE_BYTES), dtype=torch.uint8)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="no CPU path"):
        kvc.store(torch.zeros((3, 512)), kv, slots)
    with pytest.raises(ValueError, match="no CPU path"):
        kvc.dequantize(kv, slots)
    with pytest.raises(ValueError, match="no CPU path"):
        kvc.rotate(torch.zeros((3, 2, 64)), slots, torch.zeros((5, 64)))
    with pytest.raises(ValueError, match="no CPU path"):
        kvc.attend(torch.zeros((1, 8, 512), dtype=torch.bfloat16), kv, torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32))


def test_axes_are_32_numbers_whatever_holds_them(kvc):
    names = [0, 2, 1, 1] * 8
    want = (3, bytes(names))
    for held in (names, tuple(names), bytes(names), bytearray(names), iter(names), torch.tensor(names)):
        assert kvc._axes(held) == want
    for dtype in (np.uint8, np.int32, np.int64, ">i2"):
        assert kvc._axes(np.array(names, dtype)) == want
    # neither a number of axes nor 32 bytes of fewer numbers
    for bad in (32, None, [0.0] * 32, "0" * 32):
        with pytest.raises(TypeError):
            kvc._axes(bad)
    for bad in (np.zeros(4, np.int64), np.zeros(32 * 8, np.uint8), names[:31], [-1] * 32, [256] * 32):
        with pytest.raises(ValueError):
            kvc._axes(bad)


def test_a_code_is_within_half_a_scale_and_uses_all_seven():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((300, 512)) * 10.0 ** rng.uniform(-3, 4, (300, 1))).astype(np.float32)
    payload, scales = four.slot_bytes(x, 4)
    off = np.abs(four.decode4(payload, scales) - x)[:, :448].reshape(-1, 14, 32)
    s = four.SCALE_OF_BYTE[scales[:, :14]][..., None]
    a = np.abs(four.bf16(x[:, :448])).reshape(-1, 14, 32).max(-1)
    assert (off <= s / 2 + 2.0 ** -8 * a[..., None]).all()   # and the rounding of x to bf16
    assert (7 * s[..., 0] >= a).all() and (7 * s[..., 0] < a * 1.125 + 7 * 2.0 ** -16).all()
    codes, _ = four.codes4(x)
    assert codes.max() == 7 and codes.min() == -7


def test_halves_are_rounded_away_from_zero():
    x = np.zeros((1, 512), np.float32)
    x[0, :9] = [7, 0.5, -0.5, 1.5, -1.5, 2.5, -6.5, 6.4375, -0.498046875]
    codes, byte = four.codes4(x)
    assert four.SCALE_OF_BYTE[byte[0, 0]] == 1 and codes[0, :9].tolist() == [7, 1, -1, 2, -2, 3, -7, 6, 0]


def test_the_order_of_codes_in_a_word():
    x = np.zeros((1, 512), np.float32)
    x[0, :8] = [-7, -6, -5, -4, -3, -2, -1, 7]
    payload, scales = four.slot_bytes(x, 4)
    # even dims 0, 2, 4, 6 in the low half from the lowest bits on, odd ones in the high half
    assert payload[0, :4].tolist() == [0x31, 0x75, 0x42, 0xF6] and scales[0, 0] == 16 * 8 and (scales[0, 14:] == 0).all()


def test_turning_back_gives_the_rows_again():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 3, 64)).astype(np.float32)
    p, table, axes = rng.integers(0, 90, (5, 3)), four.table_of(90), rng.integers(0, 3, 32)
    there, _ = four.turn(x, p, table, axes)
    back, _ = four.turn(there, p, table, axes, inverse=True)
    assert np.abs(back - x).max() < 1e-6                     # (the table's cos^2 + sin^2 is 1 in fp32 only)
    # the inverse is the transpose: <turn x, g> = <x, inverse g>
    g = rng.standard_normal(x.shape)
    assert abs((there * g).sum() - (x * four.turn(g, p, table, axes, inverse=True)[0]).sum()) < 1e-9
