"""kvc.evict against sorting on the CPU: the bytes of the whole cache, and every array, exactly."""
import numpy as np
import pytest
import torch

import slots_testlib as plain
from kvc_testlib import PAGE_BYTES

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


def _case(seed, lengths, kind="spread", extra_pages=2):
    rng = np.random.default_rng(seed)
    table, pool = plain.page_tables(rng, lengths, extra_pages)
    kv = rng.integers(0, 256, (pool, PAGE_BYTES), dtype=np.uint8)
    S = max(1, max(lengths))
    if kind == "spread":
        w = np.exp(2 * rng.standard_normal((len(lengths), S))).astype(np.float32)
    elif kind == "ties":
        w = rng.integers(0, 4, (len(lengths), S)).astype(np.float32)
    elif kind == "equal":
        w = np.full((len(lengths), S), 0.25, np.float32)
    elif kind == "signs":
        w = rng.choice(np.array([0.0, -0.0, 1e-45, -1e-45, -1, 1, 2.5, np.inf, -np.inf], np.float32), (len(lengths), S))
    else:
        w = rng.standard_normal((len(lengths), S)).astype(np.float32)
        w[rng.random(w.shape) < 0.3] = np.nan
        w[rng.random(w.shape) < 0.1] = -np.inf
    births = np.stack([rng.permutation(S) for _ in lengths]).astype(np.int32)
    return kv, table, np.array(lengths, np.int32), w, births


def _compare(kvc, kv, table, lengths, w, births, keep, recent):
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    want_kv, want_len, want_kept = plain.evict(kv, table, lengths, w, keep, recent, births)
    d_kv, d_w, d_b = cuda(kv), cuda(w), None if births is None else cuda(births)
    w_out = torch.full((len(lengths), max(1, keep) + 3), 7.0, device="cuda")
    b_out = torch.full((len(lengths), max(1, keep) + 3), 7, dtype=torch.int32, device="cuda")
    new, kept = kvc.evict(d_kv, cuda(table), cuda(lengths), d_w, keep, recent=recent, births=d_b, slot_weights_out=w_out,
                          births_out=None if births is None else b_out)
    assert _error(kvc) == 0
    assert np.array_equal(new.cpu().numpy(), want_len)
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(d_kv.cpu().numpy(), want_kv)
    for r, n in enumerate(want_len):
        assert np.array_equal(w_out[r, :n].cpu().numpy(), w[r, want_kept[r, :n]], equal_nan=True)
        assert (w_out[r, n:] == 7).all()
        if births is not None:
            assert np.array_equal(b_out[r, :n].cpu().numpy(), births[r, want_kept[r, :n]])
            assert (b_out[r, n:] == 7).all()


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "signs", "nan"])
@pytest.mark.parametrize("keep,recent", [(100, 0), (100, 7), (100, 100), (1, 1), (0, 0), (257, 32)])
def test_kinds_of_weights(kvc, kind, keep, recent):
    kv, table, lengths, w, births = _case(keep + recent, [257, 0, 1, 64, 101, 256], kind)
    _compare(kvc, kv, table, lengths, w, births, keep, recent)


@pytest.mark.parametrize("n", [1, 31, 32, 63, 64, 65, 1023, 1024, 1025, 2047, 4099, 8192])
def test_lengths(kvc, n):
    kv, table, lengths, w, births = _case(n, [n, max(0, n - 1), n // 2])
    for keep in sorted({max(0, n - 1), n // 2, n // 3 + 1, n, n + 5}):
        _compare(kvc, kv, table, lengths, w, births, keep, min(5, keep))


@pytest.mark.parametrize("keep", [11, 20000, 44000])
def test_longer_than_the_keys_that_stay_on_chip(kvc, keep):
    kv, table, lengths, w, births = _case(keep, [50001, 40961], "ties")
    _compare(kvc, kv, table, lengths, w, births, keep, min(keep, 1000))


def test_without_births(kvc):
    kv, table, lengths, w, _ = _case(3, [500, 100])
    _compare(kvc, kv, table, lengths, w, None, 99, 0)


def test_births_of_any_sign_and_repeated(kvc):
    kv, table, lengths, w, births = _case(4, [300, 200])
    births = (births // 3 - 1000).astype(np.int32)
    births[0, 5], births[0, 9] = np.iinfo(np.int32).max, np.iinfo(np.int32).min
    births[1, 7] = np.iinfo(np.int32).min
    for recent in (1, 40, 150):
        _compare(kvc, kv, table, lengths, w, births, 150, recent)


def test_in_place_arrays_and_repeats(kvc):
    kv, table, lengths, w, births = _case(5, [700, 650, 3])
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    want_kv, want_len, want_kept = plain.evict(kv, table, lengths, w, 400, 10, births)
    d_kv, d_t, d_l, d_w, d_b = (cuda(a) for a in (kv, table, lengths, w, births))
    # again from the same lengths and weights: the same bytes
    for _ in range(3):
        _, kept = kvc.evict(d_kv, d_t, d_l, d_w, 400, recent=10, births=d_b)
    assert np.array_equal(d_kv.cpu().numpy(), want_kv)
    new, kept = kvc.evict(d_kv, d_t, d_l, d_w, 400, recent=10, births=d_b, lengths_out=d_l, slot_weights_out=d_w, births_out=d_b)
    assert new is d_l and np.array_equal(d_l.cpu().numpy(), want_len)
    assert np.array_equal(d_kv.cpu().numpy(), want_kv)
    for r, n in enumerate(want_len):
        assert np.array_equal(d_w[r, :n].cpu().numpy(), w[r, want_kept[r, :n]])
        assert np.array_equal(d_w[r, n:].cpu().numpy(), w[r, n:])
        assert np.array_equal(d_b[r, :n].cpu().numpy(), births[r, want_kept[r, :n]])
    # and on from there
    w2, b2, len2 = d_w.cpu().numpy(), d_b.cpu().numpy(), d_l.cpu().numpy()
    want_kv2, want_len2, want_kept2 = plain.evict(want_kv, table, len2, w2, 123, 10, b2)
    new, kept = kvc.evict(d_kv, d_t, d_l, d_w, 123, recent=10, births=d_b)
    assert np.array_equal(kept.cpu().numpy(), want_kept2) and np.array_equal(d_kv.cpu().numpy(), want_kv2)


def test_strides(kvc):
    kv, table, lengths, w, births = _case(6, [200, 150])
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    wide = lambda a, fill: torch.cat([torch.full_like(cuda(a), fill), cuda(a), torch.full_like(cuda(a), fill)], 1)[:, a.shape[1]:2 * a.shape[1]]
    want_kv, want_len, want_kept = plain.evict(kv, table, lengths, w, 90, 8, births)
    d_kv = cuda(kv)
    new, kept = kvc.evict(d_kv, wide(table, -1), cuda(lengths), wide(w, 1e9), 90, recent=8, births=wide(births, 10 ** 6))
    assert np.array_equal(kept.cpu().numpy(), want_kept) and np.array_equal(d_kv.cpu().numpy(), want_kv)


@pytest.mark.parametrize("where", ["length", "negative", "page", "weights"])
def test_bad_indices_leave_their_request_alone(kvc, where):
    kv, table, lengths, w, births = _case(7, [200, 250, 130])
    want_kv, want_len, want_kept = plain.evict(kv, table, lengths, w, 60, 4, births)
    own = table[1].copy()
    w = np.ascontiguousarray(np.pad(w, ((0, 0), (0, 6))))
    births = np.ascontiguousarray(np.pad(births, ((0, 0), (0, 6))))
    if where == "length":
        lengths[1] = 64 * table.shape[1] + 1
    elif where == "negative":
        lengths[1] = -3
    elif where == "page":
        table[1, 3] = len(kv)
    else:
        w, births = np.ascontiguousarray(w[:, :249]), np.ascontiguousarray(births[:, :249])
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    d_kv = cuda(kv)
    new = torch.full((3,), 77, dtype=torch.int32, device="cuda")
    kept = torch.full((3, 60), 77, dtype=torch.int32, device="cuda")
    kvc.evict(d_kv, cuda(table), cuda(lengths), cuda(w), 60, recent=4, births=cuda(births), lengths_out=new, kept=kept)
    assert _error(kvc) == kvc.KVC_ERR_BAD_INDEX
    assert new[1] == 77 and (kept[1] == 77).all()
    got = d_kv.cpu().numpy()
    assert np.array_equal(got[own], kv[own])
    others = np.setdiff1d(np.arange(len(kv)), own)
    assert np.array_equal(got[others], want_kv[others])
    for r in (0, 2):
        assert new[r] == want_len[r] and np.array_equal(kept[r].cpu().numpy(), want_kept[r])


def test_many_requests(kvc):
    rng = np.random.default_rng(8)
    kv, table, lengths, w, births = _case(8, [int(x) for x in rng.integers(0, 150, 400)])
    _compare(kvc, kv, table, lengths, w, births, 40, 5)


def test_pages_beyond_four_gigabytes(kvc):
    pages = (1 << 32) // PAGE_BYTES + 40
    kv, table, lengths, w, births = _case(9, [200], extra_pages=0)
    want_kv, want_len, want_kept = plain.evict(kv, table, lengths, w, 90, 8, births)
    pool = torch.zeros((pages, PAGE_BYTES), dtype=torch.uint8, device="cuda")
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    pool[-len(kv):] = cuda(kv)
    new, kept = kvc.evict(pool, cuda(table + pages - len(kv)).int(), cuda(lengths), cuda(w), 90, recent=8, births=cuda(births))
    assert _error(kvc) == 0
    assert np.array_equal(pool[-len(kv):].cpu().numpy(), want_kv) and not pool[:-len(kv)].any()


def test_stream_and_graph(kvc):
    kv, table, lengths, w, births = _case(10, [300, 200])
    want_kv, want_len, want_kept = plain.evict(kv, table, lengths, w, 90, 0)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    a, b, t, n, ww = cuda(kv), cuda(kv), cuda(table), cuda(lengths), cuda(w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    new, kept = kvc.evict(a, t, n, ww, 90, stream=s)
    s.synchronize()
    assert np.array_equal(a.cpu().numpy(), want_kv) and np.array_equal(kept.cpu().numpy(), want_kept)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        new, kept = kvc.evict(b, t, n, ww, 90)
    g.replay()
    g.replay()
    assert np.array_equal(b.cpu().numpy(), want_kv) and np.array_equal(kept.cpu().numpy(), want_kept)


def test_refusals_of_the_wrapper(kvc):
    kv = torch.zeros((4, PAGE_BYTES), dtype=torch.uint8, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    n, w = torch.ones(2, dtype=torch.int32, device="cuda"), torch.ones((2, 128), device="cuda")
    births = torch.zeros((2, 128), dtype=torch.int32, device="cuda")
    evict = lambda **more: kvc.evict(**dict(dict(kv_cache=kv, page_table=table, lengths=n, slot_weights=w, keep=4), **more))
    for error, more in [
            (ValueError, dict(keep=-1)), (ValueError, dict(recent=5, births=births)), (ValueError, dict(recent=1)),
            (ValueError, dict(births_out=births)), (TypeError, dict(slot_weights=w.double())), (ValueError, dict(slot_weights=w[:1])),
            (ValueError, dict(slot_weights=w.t().contiguous().t())), (ValueError, dict(births=births[:, :64])),
            (ValueError, dict(slot_weights_out=w[:, :3])), (kvc.KvcError, dict(slot_weights_out=w[0].expand(2, 128))),
            (ValueError, dict(kept=torch.zeros((2, 3), dtype=torch.int32, device="cuda"))), (TypeError, dict(workspace=3)),
            (ValueError, dict(page_table=table[:, :0])), (TypeError, dict(lengths=n.float()))]:
        with pytest.raises(error):
            evict(**more)
    new, kept = evict()
    assert new.tolist() == [1, 1] and kept.tolist() == [[0, -1, -1, -1]] * 2
