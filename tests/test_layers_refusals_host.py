"""What kvc.compress_layers refuses before it makes a call: tensors that the kernel would
read or write beyond, caches of 4-bit slots among them (their pages are shorter than the
ones it fills).  Tensors without memory stand for the device's."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import kv_cache_compression_c128_gb300 as kvc

L, BLOCKS, T, N, PAGES, P = 2, 64, 256, 2, 3, 300


def _arguments(**shapes):
    t = lambda name, shape, dtype: torch.empty(shapes.get(name, shape), dtype=dtype, device="cuda")
    return dict(state_caches=[t("state_caches", (BLOCKS, 8, 1024), torch.bfloat16) for _ in range(L)],
                token_to_req=t("token_to_req", (T,), torch.int32), positions=t("positions", (T,), torch.int64),
                boundary_token_indices=t("boundary_token_indices", (N,), torch.int64),
                block_table=t("block_table", (1, 32), torch.int32),
                rms_norm_weights=[t("rms_norm_weights", (512,), torch.float32) for _ in range(L)],
                cos_sin_cache=t("cos_sin_cache", (P, 64), torch.float32), kv_slot_mapping=t("kv_slot_mapping", (T,), torch.int64),
                kv_caches=[t("kv_caches", (PAGES, kvc.KV_PAGE_BYTES), torch.uint8) for _ in range(L)],
                block_size=8, compress_ratio=128)


@pytest.mark.parametrize("name,shape", [
    ("kv_caches", (PAGES, kvc.KV4_PAGE_BYTES)), ("kv_caches", (PAGES, 64, 368)), ("kv_caches", (PAGES * kvc.KV_PAGE_BYTES,)),
    ("kv_caches", ()), ("rms_norm_weights", (511,)), ("cos_sin_cache", (P, 32)), ("cos_sin_cache", (P * 64,)), ("cos_sin_cache", ()),
    ("token_to_req", (T - 1,)), ("state_caches", (BLOCKS, 7, 1024)), ("block_table", (32,))])
def test_tensors_too_small_are_refused(name, shape):
    with FakeTensorMode():
        with pytest.raises(ValueError):
            kvc.compress_layers(**_arguments(**{name: shape}))


def test_what_has_room_comes_to_the_call(monkeypatch):
    # (an older form: pages in several dimensions, weights of more than 512 entries)
    class Called(Exception):
        pass

    def call(*_):
        raise Called

    monkeypatch.setattr(torch.cuda, "device", call)
    for shapes in ({}, dict(kv_caches=(PAGES, 64, 584)), dict(rms_norm_weights=(600,)), dict(token_to_req=(T + 1,)),
                   dict(state_caches=(BLOCKS, 16, 1024))):
        with FakeTensorMode(), pytest.raises(Called):
            kvc.compress_layers(**_arguments(**shapes))
