"""kvc.attend calls that give up in the middle of long shares.

Shares of many pages take every place of the rings again and again.  Whichever wait runs
out, the call ends with its error and no copy of its own on the way, and the next call
is right; a limit that was long enough gives the usual bits."""
import numpy as np
import pytest
import torch

import slots4_testlib as four
import slots_testlib as plain

pytestmark = pytest.mark.gpu
LIMITS = [1, 150, 400, 700, 1000, 1300, 1600, 2000, 2500, 3000, 4000, 6000, 10000, 30000]


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_compression_c128_gb300 as kvc

    kvc.build()
    return kvc


@pytest.mark.parametrize("form", [plain, four], ids=["8bit", "4bit"])
@pytest.mark.parametrize("H", [16, 32, 64, 100])
@pytest.mark.parametrize("lengths,ctas,weights", [([64 * 41 - 3], 1, False), ([1700, 64 * 3, 900, 333], 2, True), ([2200] * 3, 3, False)])
def test_long_shares_that_give_up(kvc, form, H, lengths, ctas, weights):
    rng = np.random.default_rng(len(lengths) + H)
    table, pool = plain.page_tables(rng, lengths)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    R = len(lengths)
    q = torch.from_numpy((2 * rng.standard_normal((R, H, 512))).astype(np.float32)).to(torch.bfloat16).cuda()
    args = (q, cuda(form.random_cache(rng, pool)), cuda(table), cuda(np.array(lengths, np.int32)))
    space = torch.empty(kvc.kvc_attend_workspace_bytes(R, H, table.shape[1], weights), dtype=torch.uint8, device="cuda")

    def call():
        w = torch.zeros((R, max(lengths)), device="cuda") if weights else None
        got = kvc.attend(*args, slot_weights=w, flags=ctas, workspace=space) + ((w,) if weights else ())
        return got, kvc.kvc_get_device_error(torch.cuda.current_stream().cuda_stream)

    want, error = call()
    assert error == 0 and torch.isfinite(want[1]).all()
    gave_up = 0
    try:
        for limit in LIMITS:
            assert kvc.kvc_selftest_set_wait_limit(limit) == 0
            for _ in range(3):
                got, error = call()
                assert error in (0, kvc.KVC_ERR_TIMEOUT) and (limit > 1 or error), limit
                gave_up += error != 0
                assert error or all(torch.equal(g, w) for g, w in zip(got, want)), limit
            assert kvc.kvc_selftest_set_wait_limit(0) == 0
            got, error = call()
            assert error == 0 and all(torch.equal(g, w) for g, w in zip(got, want)), limit
    finally:
        kvc.kvc_selftest_set_wait_limit(0)
    assert gave_up >= 3
