"""kvc.attend of several tokens of one request: a row for each, over one page table."""
import numpy as np
import pytest
import torch

import slots_testlib as plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,tokens,H", [(70, 4, 16), (1000, 7, 64), (300, 33, 100)])
def test_tokens_of_one_request_share_its_pages(n, tokens, H):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_compression_c128_gb300 as kvc

    kvc.build()
    rng = np.random.default_rng(n)
    table, pool = plain.page_tables(rng, [n], extra_pages=2)
    kv = plain.random_cache(rng, pool)
    q = torch.from_numpy((2 * rng.standard_normal((tokens, H, 512))).astype(np.float32)).to(torch.bfloat16)
    lengths = np.maximum(0, n - rng.integers(0, 70, tokens)).astype(np.int32)  # what each token may see
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    w = torch.zeros((tokens, n), device="cuda")
    out, lse = kvc.attend(q.cuda(), cuda(kv), cuda(table).expand(tokens, -1), cuda(lengths), slot_weights=w)
    assert kvc.kvc_get_device_error(torch.cuda.current_stream().cuda_stream) == 0
    want = plain.attend(q.double().numpy(), kv, np.repeat(table, tokens, 0), lengths, 512 ** -0.5)
    assert (np.abs(out.double().cpu().numpy() - want[0]) <= want[3]).all()
    assert (np.abs(lse.double().cpu().numpy() - want[1]) <= want[4]).all()
    S = want[2].shape[1]
    assert (np.abs(w[:, :S].double().cpu().numpy() - want[2]) <= want[5]).all() and (w[:, S:] == 0).all()
