"""Evictions and attention one behind the other on a stream, nothing waited for
between: each call reads what the one before it has just written in place."""
import numpy as np
import pytest
import torch

import slots_testlib as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_compression_c128_gb300 as kvc

    kvc.build()
    return kvc


@pytest.mark.parametrize("lengths,H,step", [([1025, 640, 64, 900], 64, 1), ([2000, 1300], 64, 150), ([500] * 30, 16, 40),
                                            ([9000, 200], 100, 900)])
def test_evictions_and_attention_in_a_row(kvc, lengths, H, step):
    rng = np.random.default_rng(len(lengths) + H)
    table, pool = plain.page_tables(rng, lengths)
    kv = torch.from_numpy(plain.random_cache(rng, pool)).cuda()
    q = torch.from_numpy((2 * rng.standard_normal((8, len(lengths), H, 512))).astype(np.float32)).to(torch.bfloat16).cuda()
    table = torch.from_numpy(table).cuda()
    start = torch.from_numpy(np.exp(rng.standard_normal((len(lengths), max(lengths)))).astype(np.float32)).cuda()

    def run(wait):
        cache, n, w = kv.clone(), torch.tensor(lengths, dtype=torch.int32, device="cuda"), start.clone()
        births = torch.arange(w.shape[1], dtype=torch.int32, device="cuda").repeat(len(lengths), 1)
        got, keep = [], max(lengths)
        for i in range(8):
            keep -= step
            got.append(kvc.attend(q[i], cache, table, n, slot_weights=w, slot_weights_in=w))
            wait()
            kvc.evict(cache, table, n, w, keep, recent=10, births=births, lengths_out=n, slot_weights_out=w, births_out=births)
            wait()
            got.append(kvc.attend(q[i], cache, table, n))
            wait()
        torch.cuda.synchronize()
        return [t for pair in got for t in pair] + [cache, n, w, births]

    want = run(torch.cuda.synchronize)
    for _ in range(10):
        for a, b in zip(run(lambda: None), want):
            assert torch.equal(a, b)
    assert kvc.kvc_get_device_error(torch.cuda.current_stream().cuda_stream) == 0
