"""Stores and reads of the same slots one behind the other on a stream, nothing waited
for between: each read returns what the store before it has just written."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_compression_c128_gb300 as kvc

    kvc.build()
    return kvc


@pytest.mark.parametrize("four", [False, True], ids=["8bit", "4bit"])
@pytest.mark.parametrize("M", [7, 1000, 20011])
@pytest.mark.parametrize("into", ["fp32", "bf16", "bf16 at 8 bytes"])
def test_reads_see_the_store_before_them(kvc, M, into, four):
    if four and into == "bf16 at 8 bytes":
        pytest.skip("4-bit slots are read into 16-byte aligned rows")
    gen = torch.Generator("cuda").manual_seed(M)
    pages, rounds = (M + 63) // 64 + 2, 6
    x = torch.randn((rounds, M, 512), device="cuda", generator=gen)
    slots = torch.stack([torch.randperm(64 * pages, device="cuda", generator=gen)[:M] for _ in range(rounds)])
    dtype = torch.float32 if into == "fp32" else torch.bfloat16

    def run(wait):
        kv = torch.zeros((pages, kvc.KV4_PAGE_BYTES if four else kvc.KV_PAGE_BYTES), dtype=torch.uint8, device="cuda")
        got = torch.zeros(2 * rounds * (M * 512 + 8), dtype=dtype, device="cuda").view(2 * rounds, -1)
        out = got[:, 4:4 + M * 512] if into.endswith("8 bytes") else got[:, :M * 512]
        for i in range(rounds):
            kvc.store(x[i], kv, slots[i])
            wait()
            kvc.dequantize(kv, slots[i], dtype, out=out[2 * i].view(M, 512))
            wait()
            kvc.dequantize(kv, slots[i - 1], dtype, out=out[2 * i + 1].view(M, 512))
            wait()
        torch.cuda.synchronize()
        return kv, got

    want = run(torch.cuda.synchronize)
    read = want[1][0, :M * 512] if not into.endswith("8 bytes") else want[1][0, 4:4 + M * 512]
    assert (read.view(M, 512).float() - x[0]).abs().max() < (0.5 if four else 0.1)  # what was stored, not zeros
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))
    assert kvc.kvc_get_device_error(torch.cuda.current_stream().cuda_stream) == 0
