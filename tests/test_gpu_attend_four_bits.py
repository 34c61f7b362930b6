"""kvc.attend and kvc.evict over 4-bit slots against 64-bit forms."""
import numpy as np
import pytest
import torch

import slots4_testlib as four
import slots_testlib as plain

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


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
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _q(rng, R, H, spread=2.0):
    return torch.from_numpy((spread * rng.standard_normal((R, H, 512))).astype(np.float32)).to(torch.bfloat16)


def _case(seed, lengths, H, sinks=False, extra_pages=3):
    rng = np.random.default_rng(seed)
    table, pool = plain.page_tables(rng, lengths, extra_pages)
    s = rng.standard_normal(H).astype(np.float32) * 3 if sinks else None
    return rng, four.random_cache(rng, pool), table, np.array(lengths, np.int32), _q(rng, len(lengths), H), s


def _check(got, want, tol, what):
    got = got.double().cpu().numpy()
    off = np.abs(got - want)
    off[(got == want)] = 0      # infinities that agree
    assert np.isfinite(off).all(), what
    assert (off <= tol).all(), f"{what}: {off.max()} at {np.unravel_index((off - tol).argmax(), off.shape)}"


def _compare(kvc, kv, table, lengths, q, sinks=None, weights=False, scale=SCALE, **more):
    want = four.attend(q.double().numpy(), kv, table, lengths, scale, None if sinks is None else sinks.astype(np.float64))
    w = torch.full((len(lengths), int(max(lengths)) + 5), 7.0, device="cuda") if weights else None
    out, lse = kvc.attend(q.cuda(), cuda(kv), cuda(table), cuda(lengths), scale, sinks=cuda(sinks), slot_weights=w, **more)
    assert _error(kvc) == 0
    _check(out, want[0], want[3], "out")
    _check(lse, want[1], want[4], "lse")
    if weights:
        S = want[2].shape[1]
        there = np.arange(S + 5) < lengths[:, None]
        g = w.cpu().numpy()
        assert (g[~there] == 7.0).all(), "entries behind the length were written"
        _check(torch.from_numpy(np.where(there[:, :S], g[:, :S], 0)), want[2], want[5], "slot_weights")
    return out, lse, w


@pytest.mark.parametrize("H", [1, 3, 8, 16, 17, 32, 33, 48, 64, 65, 100, 128])
def test_heads(kvc, H):
    _, kv, table, lengths, q, sinks = _case(H, [130, 64, 0, 1, 77], H, sinks=H % 2 == 1)
    _compare(kvc, kv, table, lengths, q, sinks, weights=True)


@pytest.mark.parametrize("lengths", [[0], [1], [63], [64], [65], [127, 128, 129], [1000], [2049, 0, 0, 511],
                                     [0, 0, 0], [1] * 70, [300, 1, 64, 4097, 0, 128, 640]])
@pytest.mark.parametrize("H", [8, 24, 64])
def test_lengths(kvc, lengths, H):
    _, kv, table, lengths, q, sinks = _case(sum(lengths) + H, lengths, H, sinks=True)
    _compare(kvc, kv, table, lengths, q, sinks, weights=True)
    _compare(kvc, kv, table, lengths, q)


def test_every_byte_decodes_exactly(kvc):
    # one slot alone has weight 1: out is the slot itself, for every scale byte and code
    rng = np.random.default_rng(8)
    for b in range(0, 256, 3):
        kv = four.random_cache(rng, 1, b, b)
        kv[0, :224] = (np.arange(224) * 37 + b).astype(np.uint8)
        q = torch.zeros((1, 3, 512), dtype=torch.bfloat16, device="cuda")
        out, lse = kvc.attend(q, cuda(kv), torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                              torch.ones(1, dtype=torch.int32, device="cuda"))
        want = four.slot_vectors(kv, np.zeros(1, np.int64), 1)
        assert np.array_equal(out.double().cpu().numpy(), np.broadcast_to(want, (1, 3, 512))), b
        assert (lse == 0).all()


def test_what_lies_behind_a_length_does_not_count(kvc):
    rng, kv, table, lengths, q, _ = _case(9, [70, 1, 0, 129], 20, extra_pages=9)
    ref = _compare(kvc, kv, table, lengths, q, weights=True)
    dirty = np.full_like(kv, 0xFF)                      # NaN words, the largest scale, code 7
    rows, scales = dirty[:, :four.SCALE_BASE4].reshape(-1, four.STRIDE4), dirty[:, four.SCALE_BASE4:].reshape(-1, 16)
    for r, n in enumerate(lengths):
        at = table[r, np.arange(n) // 64].astype(np.int64) * 64 + np.arange(n) % 64
        rows2, scales2 = kv[:, :four.SCALE_BASE4].reshape(-1, four.STRIDE4), kv[:, four.SCALE_BASE4:].reshape(-1, 16)
        rows[at], scales[at] = rows2[at], scales2[at]
    dirty = np.concatenate([rows.reshape(len(kv), -1), scales.reshape(len(kv), -1)], 1)
    got = _compare(kvc, dirty, table, lengths, q, weights=True)
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


def test_words_of_large_values(kvc):
    # RoPE words on both sides of 2^65, where the reference begins to follow the maximum
    rng, kv, table, lengths, q, _ = _case(10, [300, 200], 40)
    words = kv[:, :four.SCALE_BASE4].reshape(-1, 64, four.STRIDE4)[..., 224:]
    big = (rng.standard_normal(words.shape[:-1] + (64,)) * 2.0 ** rng.integers(60, 70, words.shape[:-1] + (1,))).astype(np.float32)
    kv[:, :four.SCALE_BASE4].reshape(-1, 64, four.STRIDE4)[..., 224:] = (big.view(np.uint32) >> 16).astype("<u2").view(np.uint8)
    q[..., 448:] = 0                                    # scores of ordinary size
    _compare(kvc, kv, table, lengths, q, weights=True)


def test_scores_that_grow_along_the_slots(kvc):
    rng, kv, table, lengths, q, _ = _case(7, [640, 640], 24)
    for i in range(10):
        for r, p in ((0, table[0][i]), (1, table[1][9 - i])):
            kv[p, four.SCALE_BASE4:].reshape(64, 16)[:, :14] = 90 + 8 * i
    _compare(kvc, kv, table, lengths, q, weights=True)


def test_strides_and_shared_pages(kvc):
    rng, kv, table, lengths, q, _ = _case(10, [200, 200, 90], 12)
    table[1] = table[0]
    R, H = q.shape[:2]
    wide = torch.zeros((R, 2 * H + 1, 520), dtype=torch.bfloat16)
    wide[:, 1:2 * H + 1:2, :512] = q
    big = np.full((R, table.shape[1] + 3), 99999, np.int32)
    big[:, :table.shape[1]] = table
    want = four.attend(q.double().numpy(), kv, table, lengths, SCALE)
    w = torch.full((R, 300), 7.0, device="cuda")
    out, lse = kvc.attend(wide.cuda()[:, 1:2 * H + 1:2, :512], cuda(kv), cuda(big)[:, :table.shape[1]], cuda(lengths),
                          slot_weights=w[:, 20:220])
    assert _error(kvc) == 0
    _check(out, want[0], want[3], "out")
    _check(w[:, 20:220], np.where(np.arange(200) < lengths[:, None], want[2], 7.0), want[5], "weights")
    assert (w[:, :20] == 7).all() and (w[:, 220:] == 7).all()


def test_sinks_alone_above_and_below(kvc):
    _, kv, table, lengths, q, _ = _case(14, [100, 0], 6)
    sinks = np.array([-np.inf, -1e30, 0, 80, 1e4, -80], np.float32)
    _compare(kvc, kv, table, lengths, q, sinks=sinks, weights=True)


@pytest.mark.parametrize("where", ["length", "page", "page -1", "weights"])
def test_bad_indices_leave_their_request_alone(kvc, where):
    rng, kv, table, lengths, q, _ = _case(16, [300, 400, 120], 70)
    want = four.attend(q.double().numpy(), kv, table, lengths, SCALE)
    table, lengths, cols = table.copy(), lengths.copy(), 448
    if where == "length":
        lengths[1] = 64 * table.shape[1] + 1
    elif where == "page":
        table[1, 5] = len(kv)
    elif where == "page -1":
        table[1, 2] = -1
    else:
        cols = 399
    out = torch.full((3, 70, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, 70), 3.0, device="cuda")
    w = torch.full((3, cols), 7.0, device="cuda")
    kvc.attend(q.cuda(), cuda(kv), cuda(table), cuda(lengths), out=out, lse=lse, slot_weights=w)
    assert _error(kvc) == kvc.KVC_ERR_BAD_INDEX
    assert (out[1] == 3).all() and (lse[1] == 3).all() and (w[1] == 7).all()
    for r in (0, 2):
        _check(out[r], want[0][r], want[3][r], "out")
        n = int(lengths[r])
        _check(w[r, :n], want[2][r, :n], want[5][r, :n], "weights")


@pytest.mark.parametrize("ctas", [1, 2, 7, 40])
@pytest.mark.parametrize("H", [5, 32, 64, 128])
def test_any_number_of_shares(kvc, ctas, H):
    _, kv, table, lengths, q, sinks = _case(21 + ctas, [700, 64, 0, 1, 130, 65, 333, 1291], H, sinks=True)
    _compare(kvc, kv, table, lengths, q, sinks, weights=True, flags=ctas)


@pytest.mark.parametrize("H", [8, 24, 64])
@pytest.mark.parametrize("R,top,flags", [(5, 3000, 9), (20, 1500, 0), (40, 900, 61), (161, 300, 0)])
def test_ragged_batches(kvc, R, top, flags, H):
    rng = np.random.default_rng(R + top)
    lengths = rng.integers(0, top + 1, R).tolist()
    lengths[R // 2], lengths[-1] = 0, top
    _, kv, table, n, q, s = _case(31, lengths, H, sinks=True)
    _compare(kvc, kv, table, n, q, s, weights=True, flags=flags)


def test_pages_beyond_four_gigabytes(kvc):
    pages = (1 << 32) // four.PAGE4_BYTES + 40
    rng = np.random.default_rng(18)
    kv = four.random_cache(rng, 4)
    pool = torch.empty((pages, four.PAGE4_BYTES), dtype=torch.uint8, device="cuda")
    pool[-4:] = cuda(kv)
    table, lengths, q = np.array([[3, 0, 2]], np.int32), np.array([150], np.int32), _q(rng, 1, 16)
    want = four.attend(q.double().numpy(), kv, table, lengths, SCALE)
    out, lse = kvc.attend(q.cuda(), pool, cuda(table + pages - 4).int(), cuda(lengths))
    assert _error(kvc) == 0
    _check(out, want[0], want[3], "out")


@pytest.mark.parametrize("limit", [1, 3000])
@pytest.mark.parametrize("H", [16, 32, 64])
def test_waits_that_run_out(kvc, limit, H):
    _, kv, table, lengths, q, sinks = _case(25, [1000, 90, 700], H, sinks=True)
    try:
        assert kvc.kvc_selftest_set_wait_limit(limit) == 0
        w = torch.zeros((3, 1000), device="cuda")
        kvc.attend(q.cuda(), cuda(kv), cuda(table), cuda(lengths), sinks=cuda(sinks), slot_weights=w)
        assert _error(kvc) == kvc.KVC_ERR_TIMEOUT
    finally:
        kvc.kvc_selftest_set_wait_limit(0)
    _compare(kvc, kv, table, lengths, q, sinks, weights=True)


@pytest.mark.parametrize("lengths,H", [([64 * 152 * 4], 64), ([410, 2199, 1464, 1083, 965, 724, 826, 1673], 88), ([8192], 128),
                                       ([2000] * 20, 32), ([900] * 40, 16)])
def test_many_calls_give_the_same_bits(kvc, lengths, H):
    # every place of the rings is used again; one given back too early shows as rare differences
    _, kv, table, lengths, q, _ = _case(60 + H, lengths, H)
    args = (q.cuda(), cuda(kv), cuda(table), cuda(lengths))
    ws = torch.empty(kvc.kvc_attend_workspace_bytes(len(lengths), H, table.shape[1], True), dtype=torch.uint8, device="cuda")
    w = torch.zeros((len(lengths), int(max(lengths))), device="cuda")
    first = kvc.attend(*args, slot_weights=w, workspace=ws) + (w.clone(),)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        out, lse = kvc.attend(*args, slot_weights=w, workspace=ws)
        differ += (out != first[0]).any() | (lse != first[1]).any() | (w != first[2]).any()
    assert int(differ) == 0
    want = four.attend(q.double().numpy(), kv, table, lengths, SCALE)
    _check(out, want[0], want[3], "out")
    _check(w, np.where(np.arange(w.shape[1]) < lengths[:, None], want[2], 0), want[5], "weights")


def test_streams_and_graphs_at_once(kvc):
    cases = [_case(5, [1500, 3, 0, 900, 2000], 64, sinks=True), _case(6, list(range(0, 700, 9)), 8), _case(7, [8000], 128)]
    given = [(q.cuda(), cuda(kv), cuda(table), cuda(n), cuda(s)) for _, kv, table, n, q, s in cases]
    alone = [kvc.attend(q, kv, table, n, sinks=s) for q, kv, table, n, s in given]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in given]
    graphs, kept = [], []
    for q, kv, table, n, s in given:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kept.append(kvc.attend(q, kv, table, n, sinks=s))
        graphs.append(g)
    got = []
    for _ in range(20):
        for (q, kv, table, n, s), stream, g in zip(given, streams, graphs):
            got.append(kvc.attend(q, kv, table, n, sinks=s, stream=stream))
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    assert _error(kvc) == 0
    for i, (out, lse) in enumerate(got + kept):
        want, want_lse = alone[i % 3]
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, want_lse)


def _evict_case(seed, lengths):
    rng = np.random.default_rng(seed)
    table, pool = plain.page_tables(rng, lengths, 2)
    kv = rng.integers(0, 256, (pool, four.PAGE4_BYTES), dtype=np.uint8)
    S = max(1, max(lengths))
    return (kv, table, np.array(lengths, np.int32), rng.integers(0, 50, (len(lengths), S)).astype(np.float32),
            np.stack([rng.permutation(S) for _ in lengths]).astype(np.int32))


@pytest.mark.parametrize("lengths,keep,recent", [([257, 0, 1, 64, 101, 256], 100, 7), ([257, 0, 1, 64, 101, 256], 0, 0), ([65], 64, 64),
                                                 ([1025] * 9, 1024, 30), ([4099, 1, 3000, 4000], 1000, 64), ([8192, 8000], 4096, 0),
                                                 ([9000, 20, 8193], 5000, 10), ([130, 70], 200, 3), ([3] * 400, 2, 1)])
def test_evict(kvc, lengths, keep, recent):
    kv, table, n, w, births = _evict_case(keep + len(lengths), lengths)
    want_kv, want_len, want_kept = four.evict(kv, table, n, w, keep, recent, births)
    d_kv = cuda(kv)
    new, kept = kvc.evict(d_kv, cuda(table), cuda(n), cuda(w), keep, recent=recent, births=cuda(births))
    assert _error(kvc) == 0
    assert np.array_equal(new.cpu().numpy(), want_len) and np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(d_kv.cpu().numpy(), want_kv)


def test_evict_leaves_a_request_with_a_bad_page_alone(kvc):
    kv, table, n, w, births = _evict_case(3, [300, 200, 100])
    table[1, 2] = len(kv)
    d_kv = cuda(kv)
    new = torch.full((3,), 7, dtype=torch.int32, device="cuda")
    kvc.evict(d_kv, cuda(table), cuda(n), cuda(w), 50, lengths_out=new)
    assert _error(kvc) == kvc.KVC_ERR_BAD_INDEX and new.tolist() == [50, 7, 50]
    rest = [0, 2]
    want_kv, _, _ = four.evict(kv, table[rest], n[rest], w[rest], 50)
    assert np.array_equal(d_kv.cpu().numpy(), want_kv)


def test_evict_beyond_four_gigabytes(kvc):
    kv, table, n, w, _ = _evict_case(4, [700])
    pages = (1 << 32) // four.PAGE4_BYTES + 20
    pool = torch.empty((pages, four.PAGE4_BYTES), dtype=torch.uint8, device="cuda")
    pool[-len(kv):] = cuda(kv)
    kvc.evict(pool, cuda(table + pages - len(kv)).int(), cuda(n), cuda(w), 300)
    want_kv, _, _ = four.evict(kv, table, n, w, 300)
    assert _error(kvc) == 0 and np.array_equal(pool[-len(kv):].cpu().numpy(), want_kv)
