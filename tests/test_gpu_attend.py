"""kvc.attend against a 64-bit form: one new token per request over packed slots."""
import numpy as np
import pytest
import torch

import slots_testlib as plain
from kvc_testlib import PAGE_BYTES, SCALE_BASE, SCALE_DIM, TOKEN_STRIDE

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


def _q(rng, R, H, spread=2.0):
    return torch.from_numpy((spread * rng.standard_normal((R, H, 512))).astype(np.float32)).to(torch.bfloat16)


def _case(seed, lengths, H, sinks=False, extra_pages=3, width=None):
    rng = np.random.default_rng(seed)
    table, pool = plain.page_tables(rng, lengths, extra_pages, width)
    kv = plain.random_cache(rng, pool)
    q = _q(rng, len(lengths), H)
    s = rng.standard_normal(H).astype(np.float32) * 3 if sinks else None
    return rng, kv, table, np.array(lengths, np.int32), q, s


def _check(got, want, tol, what):
    got = got.double().cpu().numpy()
    off = np.abs(got - want)
    off[(got == want)] = 0      # infinities that agree
    assert np.isfinite(off).all(), what
    assert (off <= tol).all(), f"{what}: {off.max()} at {np.unravel_index((off - tol).argmax(), off.shape)}"


def _compare(kvc, kv, table, lengths, q, sinks=None, weights=False, scale=SCALE, **more):
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    want = plain.attend(q.double().numpy(), kv, table, lengths, scale, None if sinks is None else sinks.astype(np.float64))
    w = torch.full((len(lengths), int(max(lengths)) + 5), 7.0, device="cuda") if weights else None
    out, lse = kvc.attend(q.cuda(), cuda(kv), cuda(table), cuda(lengths), scale,
                          sinks=None if sinks is None else cuda(sinks), slot_weights=w, **more)
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
@pytest.mark.parametrize("H", [8, 64])
def test_lengths(kvc, lengths, H):
    _, kv, table, lengths, q, sinks = _case(sum(lengths) + H, lengths, H, sinks=True)
    _compare(kvc, kv, table, lengths, q, sinks, weights=True)
    _compare(kvc, kv, table, lengths, q)


@pytest.mark.parametrize("H", [16, 128])
def test_more_requests_than_sms(kvc, H):
    rng = np.random.default_rng(5)
    lengths = [int(x) for x in rng.integers(0, 200, 333)]
    _, kv, table, lengths, q, _ = _case(6, lengths, H)
    _compare(kvc, kv, table, lengths, q, weights=True)


def test_scores_that_grow_along_the_slots(kvc):
    # the running maximum rises by far more than a factor of 2^64 from page to page
    rng, kv, table, lengths, q, _ = _case(7, [640, 640], 24)
    page_of = table[0]
    for i in range(10):
        scales = kv[page_of[i], SCALE_BASE:].reshape(64, SCALE_DIM)
        scales[:, :7] = 120 + i
        scales = kv[table[1][9 - i], SCALE_BASE:].reshape(64, SCALE_DIM)
        scales[:, :7] = 120 + i
    _compare(kvc, kv, table, lengths, q, weights=True)


def test_every_scale_byte_decodes_exactly(kvc):
    # one slot alone has weight 1: out is the slot itself
    rng = np.random.default_rng(8)
    kv = plain.random_cache(rng, 4)
    scales = kv[:, SCALE_BASE:].reshape(256, SCALE_DIM)
    scales[:, :7] = np.arange(256, dtype=np.uint8)[:, None]
    rows = kv[:, :SCALE_BASE].reshape(256, TOKEN_STRIDE)
    rows[249:, :448] = rng.integers(0, 2, (7, 448))    # 2^122 and above: codes that stay finite
    rows[255, :448] = 0
    # a table of one page per request, and the slot moved to place 0
    for b in range(0, 256, 5):
        one = kv[:1].copy()
        one[0, :TOKEN_STRIDE] = rows[b]
        one[0, SCALE_BASE:SCALE_BASE + SCALE_DIM] = scales[b]
        q = torch.zeros((1, 3, 512), dtype=torch.bfloat16, device="cuda")
        out, lse = kvc.attend(q, torch.from_numpy(one).cuda(), torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                              torch.ones(1, dtype=torch.int32, device="cuda"))
        want = plain.slot_vectors(one, np.zeros(1, np.int64), 1)
        assert np.array_equal(out.double().cpu().numpy(), np.broadcast_to(want, (1, 3, 512))), b
        assert (lse == 0).all()


def test_what_lies_behind_a_length_does_not_count(kvc):
    rng, kv, table, lengths, q, _ = _case(9, [70, 1, 0, 129], 20, extra_pages=9)
    ref = _compare(kvc, kv, table, lengths, q, weights=True)
    bad = np.full((1, PAGE_BYTES), 0xFF, np.uint8)     # NaN words, scale byte 255
    dirty = np.repeat(bad, len(kv), 0)
    for r, n in enumerate(lengths):
        for i in range(int(n)):
            p, o = table[r, i // 64], i % 64
            dirty[p, o * TOKEN_STRIDE:(o + 1) * TOKEN_STRIDE] = kv[p, o * TOKEN_STRIDE:(o + 1) * TOKEN_STRIDE]
            dirty[p, SCALE_BASE + o * 8:SCALE_BASE + o * 8 + 8] = kv[p, SCALE_BASE + o * 8:SCALE_BASE + o * 8 + 8]
    got = _compare(kvc, dirty, table, lengths, q, weights=True)
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


def test_strides_and_shared_pages(kvc):
    rng, kv, table, lengths, q, _ = _case(10, [200, 200, 90], 12)
    table[1] = table[0]                                # two requests read the same pages
    R, H = q.shape[:2]
    wide = torch.zeros((R, 2 * H + 1, 520), dtype=torch.bfloat16)
    wide[:, 1:2 * H + 1:2, :512] = q
    big = np.full((R, table.shape[1] + 3), 99999, np.int32)
    big[:, :table.shape[1]] = table
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    want = plain.attend(q.double().numpy(), kv, table, lengths, SCALE)
    w = torch.full((R, 300), 7.0, device="cuda")
    out, lse = kvc.attend(wide.cuda()[:, 1:2 * H + 1:2, :512], cuda(kv), cuda(big)[:, :table.shape[1]], cuda(lengths),
                          slot_weights=w[:, 20:220])
    assert _error(kvc) == 0
    _check(out, want[0], want[3], "out")
    _check(lse, want[1], want[4], "lse")
    _check(w[:, 20:220], np.where(np.arange(200) < lengths[:, None], want[2], 7.0), want[5], "weights")
    assert (w[:, :20] == 7).all() and (w[:, 220:] == 7).all()


def test_queries_shared_by_heads_and_requests(kvc):
    rng, kv, table, lengths, q, _ = _case(11, [150, 40], 1)
    q = q[:1].expand(2, 9, 512)                        # strides of zero
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    want = plain.attend(q.double().numpy(), kv, table, lengths, SCALE)
    one = q[:1, :1].contiguous().cuda()
    out, lse = kvc.attend(one.expand(2, 9, 512), cuda(kv), cuda(table), cuda(lengths))
    _check(out, want[0], want[3], "out")
    _check(lse, want[1], want[4], "lse")


def test_weights_accumulate_in_place(kvc):
    rng, kv, table, lengths, q, sinks = _case(12, [150, 0, 64], 16, sinks=True)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    args = (q.cuda(), cuda(kv), cuda(table), cuda(lengths))
    w = torch.rand((3, 150), device="cuda")
    before = w.clone()
    kvc.attend(*args, sinks=cuda(sinks), slot_weights=w, slot_weights_in=w)
    alone = torch.zeros((3, 150), device="cuda")
    kvc.attend(*args, sinks=cuda(sinks), slot_weights=alone)
    there = torch.arange(150, device="cuda") < args[3][:, None]
    assert torch.equal(w, torch.where(there, before + alone, before))


@pytest.mark.parametrize("scale", [0.0, -SCALE, 1.0, 1e-30])
def test_scales(kvc, scale):
    _, kv, table, lengths, q, _ = _case(13, [100, 257], 10)
    _compare(kvc, kv, table, lengths, q, scale=scale, weights=True)


def test_sinks_alone_above_and_below(kvc):
    _, kv, table, lengths, q, _ = _case(14, [100, 0], 6)
    sinks = np.array([-np.inf, -1e30, 0, 80, 1e4, -80], np.float32)
    _compare(kvc, kv, table, lengths, q, sinks=sinks, weights=True)


def test_scores_that_overflow_to_minus_infinity(kvc):
    # q . k below the fp32 range on every slot: a row without a key
    kv = np.zeros((1, PAGE_BYTES), np.uint8)
    kv[0, :SCALE_BASE].reshape(64, TOKEN_STRIDE)[:, :448] = 100
    kv[0, SCALE_BASE:].reshape(64, 8)[:, :7] = 127
    q = torch.full((1, 2, 512), -3e38, device="cuda").to(torch.bfloat16)
    q[0, 1] = 1e-3
    w = torch.full((1, 64), 7.0, device="cuda")
    out, lse = kvc.attend(q, torch.from_numpy(kv).cuda(), torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                          torch.tensor([40], dtype=torch.int32, device="cuda"), 1.0, slot_weights=w)
    assert (out[0, 0] == 0).all() and lse[0, 0] == -np.inf
    # the other head spreads its weight 1 evenly over 40 slots
    assert torch.allclose(w[0, :40], torch.full((40,), 1 / 40, device="cuda"), rtol=64 * 2.0 ** -23, atol=0)
    assert (out[0, 1, :448] == 100).all() and (out[0, 1, 448:] == 0).all()


def test_nan_stays_with_its_row(kvc):
    rng, kv, table, lengths, q, _ = _case(15, [70, 70], 8)
    q[0, 3, 5] = float("nan")
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    out, lse = kvc.attend(q.cuda(), cuda(kv), cuda(table), cuda(lengths))
    nan = torch.isnan(out).all(-1)
    assert nan[0, 3] and nan.sum() == 1 and torch.isnan(lse).sum() == 1


@pytest.mark.parametrize("where", ["length", "negative", "page", "page -1", "weights"])
def test_bad_indices_leave_their_request_alone(kvc, where):
    rng, kv, table, lengths, q, _ = _case(16, [300, 400, 120], 70)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    want = plain.attend(q.double().numpy(), kv, table, lengths, SCALE)
    table, lengths = table.copy(), lengths.copy()
    cols = 448
    if where == "length":
        lengths[1] = 64 * table.shape[1] + 1
    elif where == "negative":
        lengths[1] = -1
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
        _check(lse[r], want[1][r], want[4][r], "lse")
        n = int(lengths[r])
        _check(w[r, :n], want[2][r, :n], want[5][r, :n], "weights")


def test_same_bits_on_every_call(kvc):
    _, kv, table, lengths, q, sinks = _case(17, [3000, 10, 700], 64, sinks=True)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    args = (q.cuda(), cuda(kv), cuda(table), cuda(lengths))
    got = []
    for _ in range(20):
        w = torch.zeros((3, 3000), device="cuda")
        got.append(kvc.attend(*args, sinks=cuda(sinks), slot_weights=w) + (w,))
    for g in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(g, got[0]))


def test_pages_beyond_four_gigabytes(kvc):
    pages = (1 << 32) // PAGE_BYTES + 40
    rng = np.random.default_rng(18)
    kv = plain.random_cache(rng, 4)
    pool = torch.empty((pages, PAGE_BYTES), dtype=torch.uint8, device="cuda")
    pool[-4:] = torch.from_numpy(kv).cuda()
    table = np.array([[3, 0, 2]], np.int32)
    lengths = np.array([150], np.int32)
    q = _q(rng, 1, 16)
    want = plain.attend(q.double().numpy(), kv, table, lengths, SCALE)
    out, lse = kvc.attend(q.cuda(), pool, torch.from_numpy(table + pages - 4).int().cuda(), torch.from_numpy(lengths).cuda())
    assert _error(kvc) == 0
    _check(out, want[0], want[3], "out")


def test_streams_and_graphs(kvc):
    _, kv, table, lengths, q, _ = _case(19, [500, 90], 40)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    args = [q.cuda(), cuda(kv), cuda(table), cuda(lengths)]
    other = [-args[0]] + args[1:]
    want, want2 = kvc.attend(*args), kvc.attend(*other)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = kvc.attend(*args, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # two graphs without a workspace of their own given, replayed at once
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for a in (args, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(kvc.attend(*a))
        graphs.append(g)
    for _ in range(30):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, (want, want2)):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_lengths_change_between_replays(kvc):
    _, kv, table, lengths, q, _ = _case(20, [640, 640, 640], 32)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    args = (q.cuda(), cuda(kv), cuda(table), cuda(lengths))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = kvc.attend(*args)
    for now in ([640, 640, 640], [1, 0, 640], [0, 0, 0], [65, 300, 2]):
        args[3].copy_(torch.tensor(now, dtype=torch.int32))
        g.replay()
        want = plain.attend(q.double().numpy(), kv, table, np.array(now), SCALE)
        _check(out, want[0], want[3], "out")
        _check(lse, want[1], want[4], "lse")


@pytest.mark.parametrize("ctas", [1, 2, 7, 40])
@pytest.mark.parametrize("H", [5, 32, 64, 128])
def test_any_number_of_shares(kvc, ctas, H):
    # few CTAs: many segments each; 40: units cut in places of all kinds
    _, kv, table, lengths, q, sinks = _case(21 + ctas, [700, 64, 0, 1, 130, 65, 333, 1291], H, sinks=True)
    _compare(kvc, kv, table, lengths, q, sinks, weights=True, flags=ctas)


@pytest.mark.parametrize("R,H", [(33, 64), (1500, 8)])
def test_requests_beyond_a_warp_and_a_block(kvc, R, H):
    rng = np.random.default_rng(22)
    lengths = [int(x) for x in rng.integers(0, 3, R)]
    lengths[R // 2] = 200
    _, kv, table, lengths, q, _ = _case(23, lengths, H)
    _compare(kvc, kv, table, lengths, q, weights=True)


def test_bad_pages_in_a_divided_request(kvc):
    # a bad page in the middle of a request that many CTAs share
    rng, kv, table, lengths, q, _ = _case(24, [64 * 90, 64 * 70, 100], 64)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    want = plain.attend(q.double().numpy(), kv, table, lengths, SCALE)
    table = table.copy()
    table[0, 41] = 1 << 30
    out = torch.full((3, 64, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, 64), 3.0, device="cuda")
    w = torch.full((3, 64 * 90), 7.0, device="cuda")
    kvc.attend(q.cuda(), cuda(kv), cuda(table), cuda(lengths), out=out, lse=lse, slot_weights=w)
    assert _error(kvc) == kvc.KVC_ERR_BAD_INDEX
    assert (out[0] == 3).all() and (lse[0] == 3).all() and (w[0] == 7).all()
    for r in (1, 2):
        n = int(lengths[r])
        _check(out[r], want[0][r], want[3][r], "out")
        _check(w[r, :n], want[2][r, :n], want[5][r, :n], "weights")


@pytest.mark.parametrize("limit", [1, 3000])
def test_waits_that_run_out(kvc, limit):
    # shortened pipeline waits make the call give up: the error is reported, the
    # context stays usable and the next call is right
    _, kv, table, lengths, q, sinks = _case(25, [1000, 90, 700], 64, sinks=True)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    try:
        assert kvc.kvc_selftest_set_wait_limit(limit) == 0
        w = torch.zeros((3, 1000), device="cuda")
        kvc.attend(q.cuda(), cuda(kv), cuda(table), cuda(lengths), sinks=cuda(sinks), slot_weights=w)
        assert _error(kvc) == kvc.KVC_ERR_TIMEOUT
    finally:
        kvc.kvc_selftest_set_wait_limit(0)
    _compare(kvc, kv, table, lengths, q, sinks, weights=True)


def test_calls_in_a_row_share_a_workspace(kvc):
    # 40 calls of different shapes on one workspace, nothing waited for between
    cases, got = [], []
    ws = torch.empty(kvc.kvc_attend_workspace_bytes(8, 128, 40, True), dtype=torch.uint8, device="cuda")
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    for i in range(8):
        rng = np.random.default_rng(26 + i)
        lengths = [int(x) for x in rng.integers(0, 64 * 40, rng.integers(1, 9))]
        _, kv, table, lengths, q, _ = _case(40 + i, lengths, int(rng.integers(1, 129)))
        cases.append((q, kv, table, lengths, [q.cuda(), cuda(kv), cuda(table), cuda(lengths)]))
    torch.cuda.synchronize()
    for _ in range(5):
        for c in cases:
            w = torch.zeros((len(c[3]), 64 * 40), device="cuda")
            got.append(kvc.attend(*c[4], slot_weights=w, workspace=ws) + (w,))
    assert _error(kvc) == 0
    for i, (q, kv, table, lengths, _) in enumerate(cases):
        want = plain.attend(q.double().numpy(), kv, table, lengths, SCALE)
        _check(got[i][0], want[0], want[3], "out")
        _check(got[i][1], want[1], want[4], "lse")
        for again in got[i::8]:
            assert all(torch.equal(a, b) for a, b in zip(again, got[i]))


def test_keys_of_large_values(kvc):
    # The sum of a row is formed in fp32 before it is divided, so 64 slots of
    # 128 * 2^(b - 127) have to stay below 2^128: b up to 241 (7 + 114 + 6 = 127).
    rng = np.random.default_rng(27)
    kv = plain.random_cache(rng, 1)
    rows = kv[0, :SCALE_BASE].reshape(64, TOKEN_STRIDE)
    rows[:, :448] = 0
    rows[:, :64] = rng.integers(0, 256, (64, 64), dtype=np.uint8)
    kv[0, SCALE_BASE:].reshape(64, SCALE_DIM)[:, :7] = rng.integers(231, 242, (64, 7), dtype=np.uint8)
    lengths = np.array([64], np.int32)
    q = torch.zeros((1, 4, 512), dtype=torch.bfloat16)
    q[:, :, 448:] = torch.from_numpy(rng.standard_normal((1, 4, 64)).astype(np.float32)).to(torch.bfloat16)
    _compare(kvc, kv, np.zeros((1, 1), np.int32), lengths, q)


@pytest.mark.parametrize("lengths,H", [([64 * 152 * 4], 64), ([410, 2199, 1464, 1083, 965, 724, 826, 1673], 88), ([8192], 128),
                                       ([2000] * 20, 32), ([900] * 40, 16)])
def test_many_calls_give_the_same_bits(kvc, lengths, H):
    # several pages a CTA, so that every place of the rings is used again; a place
    # given back too early shows as rare differences between calls
    _, kv, table, lengths, q, _ = _case(60 + H, lengths, H)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    args = (q.cuda(), cuda(kv), cuda(table), cuda(lengths))
    ws = torch.empty(kvc.kvc_attend_workspace_bytes(len(lengths), H, table.shape[1], True), dtype=torch.uint8, device="cuda")
    w = torch.zeros((len(lengths), int(max(lengths))), device="cuda")
    first = kvc.attend(*args, slot_weights=w, workspace=ws) + (w.clone(),)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        out, lse = kvc.attend(*args, slot_weights=w, workspace=ws)
        differ += (out != first[0]).any() | (lse != first[1]).any() | (w != first[2]).any()
    assert int(differ) == 0
    want = plain.attend(q.double().numpy(), kv, table, lengths, SCALE)
    _check(out, want[0], want[3], "out")
    _check(w, np.where(np.arange(w.shape[1]) < lengths[:, None], want[2], 0), want[5], "weights")


def test_refusals_of_the_wrapper(kvc):
    kv = torch.zeros((4, PAGE_BYTES), dtype=torch.uint8, device="cuda")
    table, n = torch.zeros((2, 2), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    q = torch.zeros((2, 8, 512), dtype=torch.bfloat16, device="cuda")
    attend = lambda **more: kvc.attend(**dict(dict(q=q, kv_cache=kv, page_table=table, lengths=n), **more))
    for error, more in [
            (TypeError, dict(q=q.float())), (ValueError, dict(q=q[:, :, :256])), (ValueError, dict(q=q[:1])),
            (ValueError, dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))), (ValueError, dict(kv_cache=kv[:, :64])),
            (TypeError, dict(page_table=table.long())), (ValueError, dict(page_table=table[:, :0])),
            (TypeError, dict(lengths=n.long())), (ValueError, dict(lengths=n[:1])), (TypeError, dict(lengths=[1, 1])),
            (ValueError, dict(sinks=torch.zeros(7, device="cuda"))), (ValueError, dict(lse=torch.zeros(2, 8))),
            (ValueError, dict(slot_weights=torch.zeros((2, 0), device="cuda"))),
            (ValueError, dict(slot_weights=torch.zeros((3, 128), device="cuda"))),
            (kvc.KvcError, dict(slot_weights=torch.zeros(128, device="cuda").expand(2, 128))),
            (ValueError, dict(slot_weights_in=torch.zeros((2, 128), device="cuda"))),
            (TypeError, dict(workspace=[0])), (kvc.KvcError, dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))),
            (kvc.KvcError, dict(scale=3e38)), (kvc.KvcError, dict(flags=1 << 16))]:
        with pytest.raises(error):
            attend(**more)
    out, lse = attend()
    assert _error(kvc) == 0 and torch.equal(out, torch.zeros_like(out)) and torch.equal(lse, torch.zeros_like(lse))


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("lengths,H", [([0, 100, 0, 192], 64), ([0] * 9 + [1] + [0] * 200, 8), ([64, 0, 33], 100), ([0, 0], 128)])
def test_short_requests_beside_empty_ones(kvc, lengths, H, sinks):
    _, kv, table, n, q, s = _case(77, lengths, H, sinks=sinks)
    _compare(kvc, kv, table, n, q, s)
    _compare(kvc, kv, table, n, q, s, flags=1)


@pytest.mark.parametrize("H", [8, 24, 64])
@pytest.mark.parametrize("R,top,flags", [(5, 3000, 0), (5, 3000, 9), (20, 1500, 0), (20, 1500, 33), (40, 900, 0), (40, 900, 61),
                                         (100, 700, 0), (160, 300, 0), (161, 300, 0)])
def test_ragged_batches(kvc, R, top, flags, H):
    rng = np.random.default_rng(R + top)
    lengths = rng.integers(0, top + 1, R).tolist()
    lengths[R // 2], lengths[-1] = 0, top
    _, kv, table, n, q, s = _case(31, lengths, H, sinks=True)
    _compare(kvc, kv, table, n, q, s, weights=True, flags=flags)


def test_calls_on_several_streams_at_once(kvc):
    cases = [_case(5, [1500, 3, 0, 900, 2000], 64, sinks=True), _case(6, list(range(0, 700, 9)), 8), _case(7, [8000], 128)]
    cuda = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
    given = [(q.cuda(), cuda(kv), cuda(table), cuda(n), cuda(s)) for _, kv, table, n, q, s in cases]
    alone = [kvc.attend(q, kv, table, n, sinks=s) for q, kv, table, n, s in given]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in given]
    got = []
    for _ in range(30):
        got.append([kvc.attend(q, kv, table, n, sinks=s, stream=stream) for (q, kv, table, n, s), stream in zip(given, streams)])
    torch.cuda.synchronize()
    assert _error(kvc) == 0
    for turn in got:
        for (out, lse), (want, want_lse) in zip(turn, alone):
            assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, want_lse)
