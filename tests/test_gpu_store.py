"""kvc.store and kvc.dequantize: vectors into 8-bit and 4-bit slots, byte by byte against
64-bit forms, and 4-bit slots read back."""
import numpy as np
import pytest
import torch

import slots4_testlib as four
from kvc_testlib import PAGE_BYTES, SCALE_BASE, SCALE_DIM, TOKEN_STRIDE, bf16_bits_to_f32

pytestmark = pytest.mark.gpu
FORMS = {8: (PAGE_BYTES, TOKEN_STRIDE, SCALE_BASE, SCALE_DIM, 448),
         4: (four.PAGE4_BYTES, four.STRIDE4, four.SCALE_BASE4, four.SCALES4, 224)}


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_compression_c128_gb300 as kvc

    kvc.build()
    return kvc


def _error(kvc):
    return kvc.kvc_get_device_error(torch.cuda.current_stream().cuda_stream)


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _vectors(rng, n, spread=True):
    x = rng.standard_normal((n, 512)).astype(np.float32)
    return x * (10.0 ** rng.uniform(-6, 5, (n, 1))).astype(np.float32) if spread else x


def _put(kv, slots, payload, scales, bits):
    """The bytes of `slots` (numpy, in place)."""
    _, stride, base, width, _ = FORMS[bits]
    for i, s in enumerate(slots):
        if s < 0 or s // 64 >= len(kv):
            continue
        p, o = divmod(int(s), 64)
        kv[p, o * stride:(o + 1) * stride] = payload[i]
        kv[p, base + o * width:base + (o + 1) * width] = scales[i]


def _rope(kv, slots, bits):
    _, stride, _, _, codes = FORMS[bits]
    rows = kv[:, :64 * stride].reshape(len(kv), 64, stride)[slots // 64, slots % 64, codes:]
    return bf16_bits_to_f32(np.ascontiguousarray(rows).view("<u2")).astype(np.float64)


def _as(x, dtype):
    t = torch.from_numpy(x).to(dtype)
    return t, t.float().numpy()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [0, 1, 2, 7, 8, 9, 64, 65, 1000, 5003])
def test_the_bytes_of_every_slot(kvc, bits, dtype, n):
    rng = np.random.default_rng(n + bits)
    pages = n // 64 + 3
    x, seen = _as(_vectors(rng, n), dtype)
    slots = rng.permutation(64 * pages)[:n].astype(np.int64)
    kv = rng.integers(0, 256, (pages, FORMS[bits][0]), dtype=np.uint8)
    got = cuda(kv)
    assert kvc.store(x.cuda(), got, cuda(slots)) is got
    assert _error(kvc) == 0
    _put(kv, slots, *four.slot_bytes(seen, bits), bits)
    assert np.array_equal(got.cpu().numpy(), kv)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("axes", [1, 2, 3, 4, "mixed", "unused"])
def test_rows_turned_to_their_positions(kvc, bits, dtype, axes):
    rng = np.random.default_rng(bits)
    n, table = 333, four.table_of(700)
    count = axes if isinstance(axes, int) else 4
    names = (rng.integers(0, 4, 32) if axes == "mixed" else np.repeat([1, 3], 16) if axes == "unused" else np.arange(32) * count // 32)
    p = rng.integers(0, 700, (n, count))
    if axes == "unused":
        p[:, 0] = -5                                    # of an axis that no pair has
    x, seen = _as(_vectors(rng, n), dtype)
    slots = rng.permutation(64 * 7)[:n].astype(np.int64)
    kv = rng.integers(0, 256, (7, FORMS[bits][0]), dtype=np.uint8)
    got = cuda(kv)
    kvc.store(x.cuda(), got, cuda(slots), positions=cuda(p if count > 1 else p[:, 0]), cos_sin_cache=cuda(table),
              axes=None if count == 1 else names.tolist())
    assert _error(kvc) == 0
    payload, scales = four.slot_bytes(seen, bits)
    _put(kv, slots, payload, scales, bits)
    got = got.cpu().numpy()
    want, tol = four.turn(seen[:, 448:], p, table, names)
    off = np.abs(_rope(got, slots, bits) - want)
    assert (off <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()
    # everything but the turned words is as without positions
    _, stride, _, _, codes = FORMS[bits]
    for a in (got, kv):
        a[:, :64 * stride].reshape(len(a), 64, stride)[slots // 64, slots % 64, codes:] = 0
    assert np.array_equal(got, kv)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_values_at_the_borders(kvc, bits, dtype):
    rng = np.random.default_rng(3)
    x = np.zeros((200, 512), np.float32)
    # whole and half multiples of scales, of all sizes: codes at and next to the border
    s = four.SCALE_OF_BYTE[rng.integers(0, 256, (100, 512))].astype(np.float32)
    x[:100] = rng.integers(-14, 15, (100, 512)) / 2 * s
    x[100:140] = rng.integers(-14, 15, (40, 512)) / 2 * s[:40, :1]
    x[140, :448] = 1e-45
    x[141, ::3] = 2.0 ** -16 * 7
    x[142, ::3] = np.float32(61440) * 7                 # what the largest scale holds
    x[143, ::3] = 3e38
    x[144, ::5] = np.inf
    x[144, 1::5] = -np.inf
    x[145, ::5] = np.nan
    x[145, 1::5] = 1.5
    x[146, :448] = np.nan
    x[147, :448:7], x[147, 1:448:7] = np.nan, -np.inf
    x[148] = -0.0
    x[149, :448] = 127 * 2.0 ** -9
    x[150, :448] = np.float32(127.5 * 2.0 ** -9)
    x[151, :448] = 1e-4
    x[152, 10], x[152, 11] = 100, -1e-3
    x[153:] = rng.standard_normal((47, 512)) * 10.0 ** rng.uniform(-40, 38, (47, 512))
    x[:, 448:][np.isnan(x[:, 448:])] = 0                # (a NaN's bits are the conversion's own)
    t, seen = _as(x, dtype)
    kv = np.full((4, FORMS[bits][0]), 0xAB, np.uint8)
    got, slots = cuda(kv), rng.permutation(256)[:200].astype(np.int64)
    kvc.store(t.cuda(), got, cuda(slots))
    assert _error(kvc) == 0
    with np.errstate(invalid="ignore", over="ignore"):
        _put(kv, slots, *four.slot_bytes(seen, bits), bits)
    got = got.cpu().numpy()
    assert np.array_equal(got, kv), np.argwhere(got != kv)[:5]


def test_the_compressor_stores_the_same_for_its_vectors(kvc):
    # a window's normalised vector, written by store, gives the bytes that the
    # compressor has written: codes, scales, and words turned to the window's position
    from kv_cache_compression_c128_gb300 import inputs
    from kvc_testlib import slots_of_case

    case = inputs.make_case(2, 2048, 16, seed=inputs.BASE_SEED + 5)
    dev = torch.device("cuda")
    t = lambda a: torch.from_numpy(a).to(dev)
    state = torch.from_numpy(case.state_bits.view(np.int16)).view(torch.bfloat16).to(dev)
    kv, y = t(case.kv_cache.copy()), torch.empty((case.num_outputs, 512), device=dev)
    kvc.c128_256_512_compress(state, t(case.token_to_req), t(case.positions), t(case.boundary_token_indices),
                              t(case.block_table), t(case.rms_norm_weight), t(case.cos_sin_cache), t(case.kv_slot_mapping),
                              kv, 8, 16, case.rms_norm_eps, y_out=y)
    slots = np.array(slots_of_case(case), np.int64)
    written = slots >= 0
    at = case.positions[case.boundary_token_indices] // 16 * 16
    again = t(case.kv_cache.copy())
    kvc.store(y[t(written)], again, t(slots[written]), positions=t(at[written]), cos_sin_cache=t(case.cos_sin_cache))
    assert _error(kvc) == 0 and torch.equal(again, kv)


@pytest.mark.parametrize("bits", [8, 4])
def test_strides_and_skipped_rows(kvc, bits):
    rng = np.random.default_rng(4)
    wide = torch.from_numpy(rng.standard_normal((90, 3, 520)).astype(np.float32)).to(torch.bfloat16)
    x = wide.cuda()[::2, 1, 8:]
    seen = wide[::2, 1, 8:].float().numpy()
    slots = rng.permutation(128)[:45].astype(np.int64)
    slots[[0, 7, 44]] = [-1, -(1 << 62), -3]
    p = torch.from_numpy(rng.integers(0, 50, (2, 90)))
    kv = rng.integers(0, 256, (2, FORMS[bits][0]), dtype=np.uint8)
    got, table = cuda(kv), four.table_of(50)
    kvc.store(x, got, cuda(slots), positions=p.cuda()[:, ::2].T, cos_sin_cache=cuda(table), axes=[0] * 8 + [1] * 24)
    assert _error(kvc) == 0
    want, tol = four.turn(seen[:, 448:], p.numpy()[:, ::2].T, table, [0] * 8 + [1] * 24)
    _put(kv, slots, *four.slot_bytes(seen, bits), bits)
    got, there = got.cpu().numpy(), slots[slots >= 0]
    assert (np.abs(_rope(got, there, bits) - want[slots >= 0]) <= (tol + 2.0 ** -8 * (np.abs(want) + tol))[slots >= 0]).all()
    # one row for all slots
    one = cuda(kv)
    kvc.store(x[3:4].expand(45, 512), one, cuda(slots))
    _put(kv, slots, *four.slot_bytes(np.repeat(seen[3:4], 45, 0), bits), bits)
    assert np.array_equal(one.cpu().numpy(), kv)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("where", ["slot", "far slot", "position", "negative position"])
def test_bad_indices_leave_their_slot_alone(kvc, bits, where):
    rng = np.random.default_rng(5)
    x, seen = _as(_vectors(rng, 70), torch.float32)
    slots = rng.permutation(128)[:70].astype(np.int64)
    p = rng.integers(0, 30, (70, 2))
    kept = slots.copy()
    kept[11] = -1
    if where == "slot":
        slots[11] = 128
    elif where == "far slot":
        slots[11] = (1 << 63) - 1
    else:
        p[11, 1] = 30 if where == "position" else -1
    kv = rng.integers(0, 256, (2, FORMS[bits][0]), dtype=np.uint8)
    got, same = cuda(kv), cuda(kv)
    args = dict(cos_sin_cache=cuda(four.table_of(30)), axes=bytes([0] * 31 + [1]))
    kvc.store(x.cuda(), got, cuda(slots), positions=cuda(p), **args)
    assert _error(kvc) == kvc.KVC_ERR_BAD_INDEX
    kvc.store(x.cuda(), same, cuda(kept), positions=cuda(p.clip(0, 29)), **args)
    assert _error(kvc) == 0 and torch.equal(got, same)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [0, 1, 5, 64, 1000, 20011])
def test_reading_4_bit_slots_back(kvc, dtype, n):
    rng = np.random.default_rng(n)
    kv = four.random_cache(rng, 40, 0, 255)
    slots = rng.integers(0, 64 * 40, n).astype(np.int64)    # the same slot more than once, too
    slots[::13] = -1
    out = torch.full((n, 512), 7.0, dtype=dtype, device="cuda")
    assert kvc.dequantize(cuda(kv), cuda(slots), dtype, out=out) is out
    assert _error(kvc) == 0
    rows = kv[:, :four.SCALE_BASE4].reshape(-1, four.STRIDE4)[slots]
    want = four.decode4(rows, kv[:, four.SCALE_BASE4:].reshape(-1, four.SCALES4)[slots])
    want[slots < 0] = 0
    assert np.array_equal(out.double().cpu().numpy(), want)


def test_reading_beyond_the_cache(kvc):
    kv = cuda(four.random_cache(np.random.default_rng(6), 2))
    slots = torch.tensor([3, 128, 1 << 62, 127], device="cuda")
    out = kvc.dequantize(kv, slots)
    assert _error(kvc) == kvc.KVC_ERR_BAD_INDEX
    assert (out[1:3] == 0).all() and torch.equal(out[[0, 3]], kvc.dequantize(kv, slots[[0, 3]]))


@pytest.mark.parametrize("bits", [8, 4])
def test_slots_and_rows_beyond_four_gigabytes(kvc, bits):
    rng = np.random.default_rng(7)
    width = FORMS[bits][0]
    pages = (1 << 32) // width + 40
    pool = torch.empty((pages, width), dtype=torch.uint8, device="cuda")
    pool[-2:] = 0xAB
    n = (1 << 31) // 512 + 9                              # more than 2^31 elements
    x = torch.empty((n, 512), dtype=torch.bfloat16, device="cuda")
    t, seen = _as(_vectors(rng, 5), torch.bfloat16)
    x[-5:] = t.cuda()
    slots = torch.full((n,), -1, device="cuda")
    last = 64 * pages - np.array([1, 100, 64, 65, 7], np.int64)
    slots[-5:] = cuda(last)
    kvc.store(x, pool, slots)
    assert _error(kvc) == 0
    kv = np.full((2, width), 0xAB, np.uint8)
    _put(kv, last - 64 * (pages - 2), *four.slot_bytes(seen, bits), bits)
    assert np.array_equal(pool[-2:].cpu().numpy(), kv)
    got = kvc.dequantize(pool, slots, torch.bfloat16)     # 4 GB of them
    assert _error(kvc) == 0
    assert torch.equal(got[-5:], kvc.dequantize(pool[-2:].contiguous(), cuda(last - 64 * (pages - 2)), torch.bfloat16))
    assert (got[-5:] != 0).any(1).all() and (got[:9] == 0).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_streams_and_graphs(kvc, bits):
    rng = np.random.default_rng(8)
    x, _ = _as(_vectors(rng, 300), torch.bfloat16)
    slots = cuda(rng.permutation(320)[:300].astype(np.int64))
    x = x.cuda()
    kv = torch.zeros((5, FORMS[bits][0]), dtype=torch.uint8, device="cuda")
    want = kvc.store(x, kv.clone(), slots)
    read = kvc.dequantize(want, slots)
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), kv.clone()
    torch.cuda.synchronize()
    kvc.store(x, got, slots, stream=side)
    back = kvc.dequantize(got, slots, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(back, read)
    graph, got, y = torch.cuda.CUDAGraph(), kv.clone(), torch.zeros_like(x)
    with torch.cuda.graph(graph):
        kvc.store(y, got, slots)
        back = kvc.dequantize(got, slots)
    y.copy_(x)
    for _ in range(3):
        got.zero_()
        graph.replay()
        assert torch.equal(got, want) and torch.equal(back, read)
    # rows written one call after the other, each read at once
    got.zero_()
    for i in range(0, 300, 20):
        kvc.store(x[i:i + 20], got, slots[i:i + 20])
        back[i:i + 20] = kvc.dequantize(got, slots[i:i + 20])
    assert torch.equal(got, want) and torch.equal(back, read) and _error(kvc) == 0


def test_refusals_of_the_wrappers(kvc):
    kv = torch.zeros((4, kvc.KV4_PAGE_BYTES), dtype=torch.uint8, device="cuda")
    x, slots = torch.zeros((3, 512), device="cuda"), torch.arange(3, device="cuda")
    p, table = torch.zeros((3, 2), dtype=torch.int64, device="cuda"), torch.zeros((9, 64), device="cuda")
    axes = bytes(32)
    store = lambda **more: kvc.store(**dict(dict(x=x, kv_cache=kv, slots=slots), **more))
    for error, more in [
            (TypeError, dict(x=x.half())), (TypeError, dict(x=[0])), (ValueError, dict(x=x.cpu())), (ValueError, dict(x=x[:, :448])),
            (ValueError, dict(x=x.T.contiguous().T)), (ValueError, dict(x=x[0])), (ValueError, dict(kv_cache=kv[:, :23551])),
            (TypeError, dict(kv_cache=kv.to(torch.int8))), (ValueError, dict(slots=slots[:2])), (TypeError, dict(slots=slots.int())),
            (ValueError, dict(positions=p, cos_sin_cache=table)), (ValueError, dict(positions=p[:2], cos_sin_cache=table, axes=axes)),
            (TypeError, dict(positions=p.int(), cos_sin_cache=table, axes=axes)), (ValueError, dict(axes=axes)),
            (ValueError, dict(positions=p, cos_sin_cache=table, axes=axes[:31])),
            (ValueError, dict(positions=p, cos_sin_cache=table, axes=[2] * 32)),
            (TypeError, dict(positions=p, axes=axes)), (ValueError, dict(cos_sin_cache=table)),
            (ValueError, dict(positions=p, cos_sin_cache=table[:, :32], axes=axes)),
            (TypeError, dict(positions=p, cos_sin_cache=table.double(), axes=axes)),
            (kvc.KvcError, dict(positions=p, cos_sin_cache=table[:0], axes=axes)),
            (kvc.KvcError, dict(x=torch.zeros(3 * 513 + 1, device="cuda")[:1539].view(3, 513)[:, :512])),
            (kvc.KvcError, dict(x=torch.zeros(3 * 512 + 1, device="cuda")[1:].view(3, 512)))]:
        with pytest.raises(error):
            store(**more)
    with pytest.raises(ValueError):
        kvc.dequantize(kv, slots, out=torch.zeros((2, 512), device="cuda"))
    assert store() is kv and _error(kvc) == 0
