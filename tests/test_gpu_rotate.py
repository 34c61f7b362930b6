"""kvc.rotate against complex products in 64 bits."""
import numpy as np
import pytest
import torch

import slots4_testlib as four

pytestmark = pytest.mark.gpu


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


def _x(rng, shape, dtype):
    t = torch.from_numpy((3 * rng.standard_normal(shape)).astype(np.float32)).to(dtype)
    return t, t.double().numpy()


def _check(got, seen, p, table, axes, inverse=False):
    want, tol = four.turn(seen, p, table, axes, inverse)
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    off = np.abs(got.double().cpu().numpy() - want)
    assert (off <= tol).all(), off.max()


DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])


@DTYPES
@pytest.mark.parametrize("T,H", [(1, 1), (1, 128), (3, 5), (7, 64), (129, 4), (1000, 17), (2049, 1), (0, 4), (5, 0), (2, 1000)])
@pytest.mark.parametrize("inverse", [False, True])
def test_sizes(kvc, dtype, T, H, inverse):
    rng = np.random.default_rng(T + H)
    table = four.table_of(3000)
    x, seen = _x(rng, (T, H, 64), dtype)
    p = rng.integers(0, 3000, T)
    got = kvc.rotate(x.cuda(), cuda(p), cuda(table), inverse=inverse)
    assert _error(kvc) == 0 and got.shape == x.shape
    _check(got, seen, p, table, np.zeros(32, int), inverse)


@DTYPES
@pytest.mark.parametrize("axes", ["runs 2", "runs 3", "runs 4", "turns 3", "mixed 4", "unused"])
def test_axes(kvc, dtype, axes):
    rng = np.random.default_rng(1)
    T, H, table = 57, 11, four.table_of(500)
    count = 4 if axes == "unused" else int(axes[-1])
    names = {"runs": np.arange(32) * count // 32, "turn": np.arange(32) % count, "mixe": rng.integers(0, 4, 32), "unus": np.full(32, 2)}[axes[:4]]
    p = rng.integers(0, 500, (T, count))
    if axes == "unused":
        p[:, [0, 1, 3]] = 1 << 40
    x, seen = _x(rng, (T, H, 64), dtype)
    got = kvc.rotate(x.cuda(), cuda(p), cuda(table), axes=names.tolist())
    assert _error(kvc) == 0
    _check(got, seen, p, table, names)
    assert torch.equal(got, kvc.rotate(x.cuda(), cuda(p), cuda(table), axes=bytes(names.tolist())))


@DTYPES
def test_strides_and_in_place(kvc, dtype):
    # the last dims of whole queries, every second head, positions down the columns
    rng = np.random.default_rng(2)
    table = four.table_of(900)
    whole, _ = _x(rng, (23, 12, 512), dtype)
    p = torch.from_numpy(rng.integers(0, 900, (3, 46)))
    at, names = p.cuda()[:, ::2].T, [0] * 11 + [1] * 11 + [2] * 10
    q = whole.cuda()
    before = q.clone()
    view = q[:, 1::2, 448:]
    out = torch.full((12, 23, 72), 7.0, dtype=dtype, device="cuda")
    kvc.rotate(view, at, cuda(table), axes=names, out=out.transpose(0, 1)[:, ::2, 8:])
    seen = whole[:, 1::2, 448:].double().numpy()
    _check(out.transpose(0, 1)[:, ::2, 8:], seen, at.cpu().numpy(), table, names)
    assert (out[1::2] == 7).all() and (out[:, :, :8] == 7).all()
    assert kvc.rotate(view, at, cuda(table), axes=names, out=view) is view
    assert torch.equal(view, out.transpose(0, 1)[:, ::2, 8:])
    assert torch.equal(q[:, ::2], before[:, ::2]) and torch.equal(q[..., :448], before[..., :448])
    # rows without heads, and one row for every token and head
    two = kvc.rotate(view[:, 0], at, cuda(table), axes=names)
    assert torch.equal(two, kvc.rotate(view[:, :1], at, cuda(table), axes=names)[:, 0])
    one = kvc.rotate(view[:1, :1].expand(23, 6, 64), at, cuda(table), axes=names)
    assert torch.equal(one, kvc.rotate(view[:1, :1].expand(23, 6, 64).contiguous(), at, cuda(table), axes=names))
    assert _error(kvc) == 0


@DTYPES
def test_the_inverse_is_the_gradient(kvc, dtype):
    rng = np.random.default_rng(3)
    table, names = four.table_of(64), np.arange(32) % 3
    p = rng.integers(0, 64, (9, 3))
    x, seen = _x(rng, (9, 4, 64), dtype)
    g, grad = _x(rng, (9, 4, 64), dtype)
    got = kvc.rotate(g.cuda(), cuda(p), cuda(table), axes=names.tolist(), inverse=True)
    _check(got, grad, p, table, names, inverse=True)
    # against differences of <g, rotate(x)> in 64 bits: the map is linear, so that a
    # step of 1 in one dim gives its derivative up to the two sums' rounding
    for _ in range(20):
        t, h, d = rng.integers(9), rng.integers(4), rng.integers(64)
        step = np.zeros_like(seen)
        step[t, h, d] = 1
        more = (grad * (four.turn(seen + step, p, table, names)[0] - four.turn(seen, p, table, names)[0])).sum()
        tol = four.turn(grad, p, table, names, inverse=True)[1][t, h, d] + 1e-9
        tol += (2.0 ** -8 * (abs(more) + tol) if dtype == torch.bfloat16 else 0)
        assert abs(float(got[t, h, d]) - more) <= tol


@DTYPES
@pytest.mark.parametrize("bad", [500, -1, 1 << 62, -(1 << 62)])
@pytest.mark.parametrize("several", [False, True])
def test_bad_positions_leave_their_token_alone(kvc, dtype, bad, several):
    rng = np.random.default_rng(4)
    table, names = four.table_of(500), (np.arange(32) == 31).astype(int)
    p = rng.integers(0, 500, (20, 2))
    x, seen = _x(rng, (20, 70, 64), dtype)
    p[7, 1 if several else 0] = bad
    out = torch.full((20, 70, 64), 3.0, dtype=dtype, device="cuda")
    kvc.rotate(x.cuda(), cuda(p), cuda(table), axes=names.tolist(), out=out)
    assert _error(kvc) == kvc.KVC_ERR_BAD_INDEX
    assert (out[7] == 3).all()
    rest = np.arange(20) != 7
    _check(out[cuda(rest)], seen[rest], p[rest], table, names)


def test_infinities_and_nan_stay_in_their_pair(kvc):
    rng = np.random.default_rng(5)
    table = four.table_of(100)
    x, _ = _x(rng, (3, 2, 64), torch.float32)
    x[1, 1, 6], x[2, 0, 33] = float("nan"), float("inf")
    got = kvc.rotate(x.cuda(), cuda(np.array([5, 6, 7])), cuda(table)).cpu()
    broken = ~torch.isfinite(got)
    assert broken[1, 1, 6:8].all() and broken[2, 0, 32:34].all() and broken.sum() == 4


def test_rows_beyond_four_gigabytes(kvc):
    table = four.table_of(50)
    T, H = 70000, 64                                     # 8.6 GB at 512 dims a head
    q = torch.empty((T, H, 512), dtype=torch.float32, device="cuda")
    x, seen = _x(np.random.default_rng(6), (3, H, 64), torch.float32)
    q[-3:, :, 448:] = x.cuda()
    p = torch.arange(T, device="cuda") % 50
    kvc.rotate(q[..., 448:], p, cuda(table), out=q[..., 448:])
    assert _error(kvc) == 0
    _check(q[-3:, :, 448:], seen, p[-3:].cpu().numpy(), table, np.zeros(32, int))


def test_streams_and_graphs(kvc):
    rng = np.random.default_rng(7)
    table = cuda(four.table_of(100))
    x, _ = _x(rng, (33, 16, 64), torch.bfloat16)
    x, p = x.cuda(), cuda(rng.integers(0, 100, 33))
    want = kvc.rotate(x, p, table)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = kvc.rotate(x, p, table, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph, y, at = torch.cuda.CUDAGraph(), torch.zeros_like(x), torch.zeros_like(p)
    with torch.cuda.graph(graph):
        kvc.rotate(y, at, table, out=y)
        got = kvc.rotate(y, at, table, inverse=True)
    for _ in range(3):
        y.copy_(x)
        at.copy_(p)
        graph.replay()
        assert torch.equal(y, want) and torch.equal(got, kvc.rotate(want, p, table, inverse=True))


def test_refusals_of_the_wrapper(kvc):
    x, p, table = torch.zeros((4, 2, 64), device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros((9, 64), device="cuda")
    rotate = lambda **more: kvc.rotate(**dict(dict(x=x, positions=p, cos_sin_cache=table), **more))
    for error, more in [
            (TypeError, dict(x=x.half())), (ValueError, dict(x=x.cpu())), (ValueError, dict(x=x[..., :32])),
            (ValueError, dict(x=x.transpose(1, 2).contiguous().transpose(1, 2))), (ValueError, dict(x=x[0, 0])),
            (ValueError, dict(positions=p[:3])), (TypeError, dict(positions=p.int())), (ValueError, dict(positions=p.cpu())),
            (ValueError, dict(positions=p[:, None, None])), (ValueError, dict(positions=p[:, None].expand(4, 5))),
            (ValueError, dict(positions=p[:, None].expand(4, 2))), (ValueError, dict(positions=p[:, None][:, :0])),
            (ValueError, dict(axes=[0] * 33)), (ValueError, dict(axes=[1] * 32)), (ValueError, dict(axes=[300] * 32)),
            (TypeError, dict(cos_sin_cache=table.double())), (ValueError, dict(cos_sin_cache=table[:, :32])),
            (ValueError, dict(out=x[:3])), (TypeError, dict(out=x.bfloat16())), (ValueError, dict(out=x.cpu())),
            (kvc.KvcError, dict(out=torch.zeros((4, 1, 64), device="cuda").expand(4, 2, 64))),
            (kvc.KvcError, dict(x=torch.zeros((4, 2, 65), device="cuda")[..., :64])),
            (kvc.KvcError, dict(x=torch.zeros((4, 2, 68), device="cuda")[..., 1:65]))]:
        with pytest.raises(error):
            rotate(**more)
    assert torch.equal(rotate(), torch.zeros_like(x)) and _error(kvc) == 0
