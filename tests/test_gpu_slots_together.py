"""The operators on packed slots together, as a decoding program uses them:
compress windows into slots, attend over them while their weights add up,
join with the part that is not packed, evict, and attend again."""
import numpy as np
import pytest
import torch

import slots_testlib as plain
from kv_cache_compression_c128_gb300 import inputs
from kvc_testlib import run_gpu, slots_of_case

pytestmark = pytest.mark.gpu


def test_compress_attend_join_evict(oracle_mod):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_compression_c128_gb300 as kvc

    kvc.build()
    R, H, scale = 2, 24, 512 ** -0.5
    # every slot of one page pair per request: 2 x 128 windows of 16 tokens
    case = inputs.make_case(R, 2 * 2048, 16, seed=inputs.BASE_SEED + 77)
    kv, _, err = run_gpu(case)
    assert err == 0
    # the mapping of outputs to slots is a permutation of the pool: request r takes pages 2r, 2r + 1
    table = np.array([[0, 1], [2, 3]], np.int32)
    lengths = np.array([128, 117], np.int32)
    assert sorted(slots_of_case(case)) == list(range(256))
    rng = np.random.default_rng(3)
    q = [torch.from_numpy((2 * rng.standard_normal((R, H, 512))).astype(np.float32)).to(torch.bfloat16) for _ in range(4)]
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    d_kv, d_t, d_l = cuda(kv), cuda(table), cuda(lengths)
    weights = torch.zeros((R, 128), device="cuda")
    births = torch.arange(128, dtype=torch.int32, device="cuda").repeat(R, 1)
    total, tol = np.zeros((R, 128)), np.zeros((R, 128))
    for step in range(3):
        out, lse = kvc.attend(q[step].cuda(), d_kv, d_t, d_l, scale, slot_weights=weights, slot_weights_in=weights)
        want = plain.attend(q[step].double().numpy(), kv, table, lengths, scale)
        assert (np.abs(out.double().cpu().numpy() - want[0]) <= want[3]).all()
        total += want[2]
        tol += want[5] + plain.STEP_F32 * total
    assert (np.abs(weights.double().cpu().numpy() - total) <= tol).all()
    # the same attention as two halves of the slots, joined
    half = torch.full_like(d_l, 64)
    a = kvc.attend(q[0].cuda(), d_kv, d_t, half, scale)
    b = kvc.attend(q[0].cuda(), d_kv, d_t[:, 1:], d_l - 64, scale)
    out, lse = kvc.join([a[0], b[0]], [a[1], b[1]])
    want = plain.attend(q[0].double().numpy(), kv, table, lengths, scale)
    pa = plain.attend(q[0].double().numpy(), kv, table, half.cpu().numpy(), scale)
    pb = plain.attend(q[0].double().numpy(), kv, table[:, 1:], lengths - 64, scale)
    assert (np.abs(lse.double().cpu().numpy() - want[1]) <= pa[4] + pb[4] + 16 * plain.STEP_F32 * (1 + np.abs(want[1]))).all()
    wa, wb = (np.exp(p[1] - want[1])[..., None] for p in (pa, pb))
    off = wa * pa[3] + wb * pb[3] + (pa[4] + pb[4] + 2 ** -18)[..., None] * (wa * np.abs(pa[0]) + wb * np.abs(pb[0]))
    assert (np.abs(out.double().cpu().numpy() - want[0]) <= off + plain.HALF_BF16 * (np.abs(want[0]) + off)).all()
    # evict by the weights that the GPU summed, then attend over what stays
    w_host = weights.cpu().numpy()
    want_kv, want_len, want_kept = plain.evict(kv, table, lengths, w_host, 80, 16, births.cpu().numpy())
    kvc.evict(d_kv, d_t, d_l, weights, 80, recent=16, births=births, lengths_out=d_l, slot_weights_out=weights, births_out=births)
    assert np.array_equal(d_kv.cpu().numpy(), want_kv) and np.array_equal(d_l.cpu().numpy(), want_len)
    for r in range(R):
        assert np.array_equal(weights[r, :80].cpu().numpy(), w_host[r, want_kept[r]])
    out, lse = kvc.attend(q[3].cuda(), d_kv, d_t, d_l, scale, slot_weights=weights, slot_weights_in=weights)
    want = plain.attend(q[3].double().numpy(), want_kv, table, want_len, scale)
    assert (np.abs(out.double().cpu().numpy() - want[0]) <= want[3]).all()
    assert (np.abs(lse.double().cpu().numpy() - want[1]) <= want[4]).all()
    assert kvc.kvc_get_device_error(torch.cuda.current_stream().cuda_stream) == 0
