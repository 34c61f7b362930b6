"""kvc.attend where the reference of the softmax moves, with tolerances that a
row of zeros, or one that a move left as it was, does not meet
(test_slots_rescale_host.py shows that on the CPU)."""
import numpy as np
import pytest
import torch

import slots_rescale_testlib as cases

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_compression_c128_gb300 as kvc

    kvc.build()
    return kvc


@pytest.mark.parametrize("name", cases.HEIGHTS)
@pytest.mark.parametrize("H", [9, 24, 64, 100])
@pytest.mark.parametrize("repeat,flags", [(1, 1), (1, 0), (3, 1), (3, 2), (9, 4)])
def test_the_reference_moves(kvc, name, H, repeat, flags):
    q, kv = cases.case(H + repeat, cases.HEIGHTS[name], H, repeat)
    n = 64 * len(kv) - 9
    table = np.random.default_rng(H).permutation(len(kv)).astype(np.int32)
    kv[table] = kv.copy()
    out, lse, weights, tol_out, tol_lse, tol_w = cases.expected(q, kv, table, n, len(kv))
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    w = torch.zeros((1, n), device="cuda")
    got, got_lse = kvc.attend(cuda(q).to(torch.bfloat16), cuda(kv), cuda(table[None]), cuda(np.array([n], np.int32)), 1.0,
                              slot_weights=w, flags=flags)
    assert kvc.kvc_get_device_error(torch.cuda.current_stream().cuda_stream) == 0
    off = np.abs(got[0].double().cpu().numpy() - out)
    assert (off <= tol_out).all(), (off / tol_out).max()
    off = np.abs(got_lse[0].double().cpu().numpy() - lse)
    assert (off <= tol_lse).all(), (off / tol_lse).max()
    off = np.abs(w[0].double().cpu().numpy() - weights)
    assert (off <= tol_w).all(), (off / tol_w).max()
