"""What kvc.dequantize refuses before it makes a call: caches whose pages are of neither
form (their slots would be looked for at other places, and beyond the cache) and results
that are too small.  Tensors without memory stand for the device's."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import kv_cache_compression_c128_gb300 as kvc

PAGES, M = 3, 5
WIDTHS = [kvc.KV_PAGE_BYTES, kvc.KV4_PAGE_BYTES]


@pytest.fixture(autouse=True)
def no_call(monkeypatch):
    called = []
    kvc._load_torch()
    monkeypatch.setattr(kvc, "_quick", None)
    monkeypatch.setattr(kvc, "_run", lambda call, device, stream: called.append(device) or kvc.KVC_OK)
    return called


def _tensor(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("shape", [
    (PAGES, 64, 368), (PAGES, 64, 352), (PAGES, kvc.KV4_PAGE_BYTES - 16), (PAGES, kvc.KV_PAGE_BYTES + 8), (PAGES, kvc.KV_PAGE_BYTES, 2),
    (PAGES * kvc.KV_PAGE_BYTES,), (PAGES * kvc.KV4_PAGE_BYTES,), (PAGES, 512), ()])
def test_pages_of_neither_form_are_refused(no_call, shape):
    with FakeTensorMode():
        kv, slots = _tensor(shape, torch.uint8), _tensor((M,), torch.int64)
        for out in (None, _tensor((M, 512), torch.float32)):
            with pytest.raises(ValueError, match="kv_cache must be"):
                kvc.dequantize(kv, slots, out=out)
    assert not no_call


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("shape", [(M - 1, 512), (M, 511), (M * 512 - 1,), (0,)])
def test_short_results_are_refused(no_call, width, shape, dtype):
    with FakeTensorMode():
        with pytest.raises(ValueError, match="out must hold"):
            kvc.dequantize(_tensor((PAGES, width), torch.uint8), _tensor((M,), torch.int64), dtype, out=_tensor(shape, dtype))
    assert not no_call


@pytest.mark.parametrize("shape", [(PAGES, w) for w in WIDTHS] + [(PAGES, 64, 584), (PAGES, 8, 4672)])
@pytest.mark.parametrize("out", [None, (M, 512), (M * 512,), (M + 2, 512), (2, M, 512)])
def test_what_has_room_is_taken(no_call, shape, out):
    # an 8-bit page may be split into several dimensions, results be larger or of other dimensions
    with FakeTensorMode():
        kvc.dequantize(_tensor(shape, torch.uint8), _tensor((M,), torch.int64), out=None if out is None else _tensor(out, torch.float32))
        kvc.dequantize(_tensor(shape, torch.uint8), _tensor((0,), torch.int64), out=_tensor((0, 512), torch.float32))
    assert no_call == [0, 0]
