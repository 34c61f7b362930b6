"""kvc.attend at the ends of the fp32 range: scores far beyond what a difference resolves."""
import numpy as np
import pytest
import torch

import slots_testlib as plain
from kvc_testlib import PAGE_BYTES, SCALE_BASE, SCALE_DIM, TOKEN_STRIDE

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


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _equal_slots(rng, first):
    """A page of 64 equal slots whose dim 0 is `first` (scale byte 127: 2^0)."""
    kv = plain.random_cache(rng, 1)
    rows, scales = kv[0, :SCALE_BASE].reshape(64, TOKEN_STRIDE), kv[0, SCALE_BASE:].reshape(64, SCALE_DIM)
    rows[:], scales[:] = rows[0], scales[0]
    rows[:, 0], scales[:, 0] = np.int8(first).view(np.uint8), 127
    return kv


def _one_score(rng, H, size):
    """Queries that are zero but for dim 0: `size` to twice that in bf16, each head its own."""
    q = torch.zeros((1, H, 512))
    q[0, :, 0] = torch.from_numpy((size * (1 + rng.random(H))).astype(np.float32))
    return q.to(torch.bfloat16)


@pytest.mark.parametrize("size", [1e5, 2.0 ** 31, 3e9, 1e10, 1e20, 1e30, 1e37, -1e5, -(2.0 ** 31), -3e9, -1e10, -1e20, -1e37])
@pytest.mark.parametrize("n,flags", [(1, 0), (2, 0), (64, 0), (200, 1), (3000, 0), (3000, 7)])
def test_equal_slots_of_large_scores(kvc, n, flags, size):
    # Every weight is 2^0 before the division, the sums n and n k_d are whole
    # numbers of units that fp32 holds (8 bits of k_d, 12 of n), and the
    # quotient is k_d again once rounded to bf16.
    rng = np.random.default_rng(n)
    kv = _equal_slots(rng, 1)
    q = _one_score(rng, 40, size)
    table = torch.zeros((1, -(-n // 64)), dtype=torch.int32, device="cuda")
    scale = float(np.float32(0.7))
    out, lse = kvc.attend(q.cuda(), _cuda(kv), table, torch.tensor([n], dtype=torch.int32, device="cuda"), scale, flags=flags)
    assert _error(kvc) == 0
    slot = plain.slot_vectors(kv, np.zeros(1, np.int64), 1)[0]
    assert np.array_equal(out.double().cpu().numpy(), np.broadcast_to(slot, (1, 40, 512)))
    # scale log2(e), its product with the dot product, + log2(n), / log2(e): half a step each
    # (log2(e) itself is the same fp32 number both times), and the steps of log2(n)
    want = scale * q[0, :, 0].double().numpy() + np.log(n)
    off = np.abs(lse[0].double().cpu().numpy() - want)
    assert (off <= 2.5 * plain.STEP_F32 * np.abs(want) + 2.0 ** -19).all(), off


@pytest.mark.parametrize("size", [1e10, -1e10, 1e20, -1e20, 1e35])
@pytest.mark.parametrize("n", [2, 130, 900])
def test_the_largest_of_large_scores_takes_all(kvc, n, size):
    rng = np.random.default_rng(n)
    best = n - 1 if size > 0 else 0
    kv = np.concatenate([_equal_slots(rng, 3)] * -(-n // 64))
    one = plain.random_cache(rng, 1)[0]
    page, at = divmod(best, 64)
    kv[page, at * TOKEN_STRIDE:(at + 1) * TOKEN_STRIDE] = one[:TOKEN_STRIDE]
    kv[page, at * TOKEN_STRIDE] = 4 if size > 0 else 2
    table = np.arange(len(kv), dtype=np.int32)[None]
    q = _one_score(rng, 64, size)
    out, lse = kvc.attend(q.cuda(), _cuda(kv), _cuda(table), torch.tensor([n], dtype=torch.int32, device="cuda"), 1.0)
    assert _error(kvc) == 0
    slot = plain.slot_vectors(kv, table[0], n)[best]
    assert np.array_equal(out.double().cpu().numpy(), np.broadcast_to(slot, (1, 64, 512)))
    want = slot[0] * q[0, :, 0].double().numpy()
    assert (np.abs(lse[0].double().cpu().numpy() - want) <= 2.5 * plain.STEP_F32 * np.abs(want)).all()


def _rising(rng, pages, rise, where, large):
    """Pages of slots that a query of 1 in dim 448 scores 0, rise, 2 rise, ...
    (in nats, before the slots' own spread of 1), whose values in the pages
    `large` reach 2^112: as codes (where "codes") or as RoPE words ("rope")."""
    kv = plain.random_cache(rng, pages)
    rows = kv[:, :SCALE_BASE].reshape(pages, 64, TOKEN_STRIDE)
    scales = kv[:, SCALE_BASE:].reshape(pages, 64, SCALE_DIM)
    words = np.ascontiguousarray(rows[..., 448:]).view("<u2").reshape(pages, 64, 64).copy()
    bits = lambda x: (np.asarray(x, np.float32).view(np.uint32) >> 16).astype("<u2")
    if where == "codes":
        scales[large, :, :7] = rng.integers(222, 233, scales[large, :, :7].shape, dtype=np.uint8)  # 2^95 .. 2^105
    else:
        words[large, :, 1:] = bits(rng.standard_normal((len(large), 64, 63)) * 2.0 ** rng.integers(95, 110, (len(large), 64, 63)))
    words[..., 0] = bits(rise * np.arange(pages)[:, None] + rng.random((pages, 64)))
    rows[..., 448:] = words.view(np.uint8).reshape(pages, 64, 128)
    return kv


@pytest.mark.parametrize("where", ["codes", "rope"])
@pytest.mark.parametrize("H,n,rise,large,flags", [
    (8, 128, 20.0, [0, 1], 1), (64, 128, 20.0, [1], 1), (24, 200, 9.0, [0, 3], 0), (64, 64 * 12 - 5, 7.0, list(range(12)), 1),
    (16, 64 * 12 - 5, 20.0, [4, 5, 11], 2), (100, 64 * 12 - 5, -20.0, list(range(12)), 5), (64, 2500, 3.0, [10, 20, 39], 3),
    (32, 2500, 0.0, list(range(40)), 0)])
def test_values_near_the_end_of_the_range(kvc, where, H, n, rise, large, flags):
    # Scores that rise by less than 2^32 (in weight) from page to page, under
    # values whose sum stays in range: 40 pages of 64 values below 2^115 are
    # below 2^127, and so is every sum of them times weights of at most 1.
    rng = np.random.default_rng(H + n)
    kv = _rising(rng, -(-n // 64), rise, where, large)
    table = rng.permutation(len(kv)).astype(np.int32)[None]
    kv[table[0]] = kv.copy()
    q = torch.zeros((1, H, 512))
    q[0, :, 448] = torch.from_numpy(rng.choice([-1.0, 0.5, 1.0, 1.0, 1.0625], H).astype(np.float32))
    q = q.to(torch.bfloat16)
    lengths = np.array([n], np.int32)
    want = plain.attend(q.double().numpy(), kv, table, lengths, 1.0)
    out, lse = kvc.attend(q.cuda(), _cuda(kv), _cuda(table), _cuda(lengths), 1.0, flags=flags)
    assert _error(kvc) == 0
    off = np.abs(out.double().cpu().numpy() - want[0])
    assert np.isfinite(off).all()
    assert (off <= want[3]).all()
    assert (np.abs(lse.double().cpu().numpy() - want[1]) <= want[4]).all()


@pytest.mark.parametrize("size", [30.0, 1e5, 1e6, 1e10, 1e37, -1e5, -1e6, -1e10, -1e37])
@pytest.mark.parametrize("H", [1, 8, 40, 100])
@pytest.mark.parametrize("n,flags", [(1, 0), (2, 0), (64, 0), (200, 1), (3000, 0), (3000, 7)])
def test_weights_of_equal_slots(kvc, n, flags, H, size):
    # each of n equal slots gets 1 / n of every head, in undivided requests and in
    # divided ones: half a step for the quotient and one for each head added
    rng = np.random.default_rng(n)
    kv = _equal_slots(rng, 1)
    q = _one_score(rng, H, size)
    table = torch.zeros((1, -(-n // 64)), dtype=torch.int32, device="cuda")
    w = torch.full((1, n + 3), 7.0, device="cuda")
    kvc.attend(q.cuda(), _cuda(kv), table, torch.tensor([n], dtype=torch.int32, device="cuda"), 0.7, slot_weights=w, flags=flags)
    assert _error(kvc) == 0 and (w[0, n:] == 7).all()
    off = np.abs(w[0, :n].double().cpu().numpy() - H / n)
    assert (off <= (H + 1) / 2 * plain.STEP_F32 * H / n).all(), off.max() * n / H


@pytest.mark.parametrize("lengths,flags", [([1, 64, 150], 0), ([3000], 0), ([700, 30], 3)])
@pytest.mark.parametrize("spread", [1.0, 1e3, 1e6])
def test_weights_of_a_request_sum_up_to_its_heads(kvc, lengths, flags, spread):
    # Whatever rounding did to the scores, the weights and the sum that divides
    # them are formed from the same ones: off by the steps of the exponentials
    # (2 each), of the sums (one a slot, and one a head) and of the quotient.
    rng = np.random.default_rng(len(lengths))
    table, pool = plain.page_tables(rng, lengths)
    H = 24
    q = torch.from_numpy((spread * rng.standard_normal((len(lengths), H, 512))).astype(np.float32)).to(torch.bfloat16)
    sinks = np.full(H, -np.inf, np.float32)
    w = torch.zeros((len(lengths), max(lengths)), device="cuda")
    kvc.attend(q.cuda(), _cuda(plain.random_cache(rng, pool)), _cuda(table), _cuda(np.array(lengths, np.int32)), sinks=_cuda(sinks),
               slot_weights=w, flags=flags)
    assert _error(kvc) == 0
    got = w.double().sum(1).cpu().numpy()
    assert (np.abs(got - H) <= H * (np.array(lengths) + H + 8) * plain.STEP_F32).all(), got
