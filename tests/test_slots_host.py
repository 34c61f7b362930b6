"""Refusals of the operators on packed slots, on the host before any CUDA call."""
import os
import shutil

import pytest
import torch

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")


@pytest.fixture(scope="module")
def kvc():
    import kv_cache_compression_c128_gb300 as kvc

    kvc.build()
    return kvc


_ATTEND = dict(q=0x10000, q_req_stride=64 * 512, q_head_stride=512, num_reqs=4, num_heads=64, kv_cache=0x20000,
               num_kv_pages=100, page_table=0x30000, max_pages_per_req=8, page_table_row_stride=8, lengths=0x40000,
               scale=0.04, sinks=None, out=0x50000, lse=0x60000, slot_weights_in=None, slot_weights_in_row_stride=0,
               slot_weights=None, slot_weights_row_stride=0, max_slots=0, workspace=0x70000, workspace_bytes=1 << 40,
               flags=0, stream=0)


@pytest.mark.parametrize("change", [
    dict(q=0), dict(q=0x10008), dict(q_req_stride=4), dict(q_head_stride=513), dict(q_head_stride=-512), dict(q_head_stride=0), dict(num_reqs=-1),
    dict(num_reqs=65536), dict(num_heads=0), dict(num_heads=129), dict(kv_cache=0), dict(kv_cache=0x20004),
    dict(num_kv_pages=0), dict(num_kv_pages=1 << 31), dict(page_table=0), dict(page_table=0x30002),
    dict(max_pages_per_req=0), dict(max_pages_per_req=1 << 40), dict(page_table_row_stride=-1), dict(lengths=0),
    dict(lengths=0x40001), dict(scale=float("nan")), dict(scale=float("inf")), dict(sinks=0x90002), dict(out=0),
    dict(out=0x50008), dict(lse=0x60002), dict(slot_weights_in=0xA0000), dict(slot_weights=0xA0002, max_slots=512),
    dict(slot_weights=0xA0000, max_slots=-1), dict(slot_weights=0xA0000, slot_weights_row_stride=-1),
    dict(workspace=0), dict(workspace=0x70004), dict(workspace_bytes=8), dict(flags=1 << 16)])
def test_attend_refuses(kvc, change):
    assert kvc.kvc_attend(**dict(_ATTEND, **change)) == kvc.KVC_ERR_INVALID_ARG


def test_attend_of_no_request_is_a_no_op(kvc):
    assert kvc.kvc_attend(**dict(_ATTEND, num_reqs=0)) == kvc.KVC_OK


_JOIN = dict(outs=[0x10000, 0x20000], lses=[0x30000, 0x40000], num_rows=10, dtype=1, out=0x50000, lse=0x60000, stream=0)


@pytest.mark.parametrize("change", [
    dict(outs=[], lses=[]), dict(outs=[0x10000] * 9, lses=[0x30000] * 9), dict(outs=[0x10000, 0]),
    dict(outs=[0x10008, 0x20000]), dict(lses=[0, 0x40000]), dict(lses=[0x30002, 0x40000]), dict(num_rows=-1),
    dict(num_rows=1 << 40), dict(dtype=2), dict(out=0), dict(out=0x50004), dict(lse=0x60002)])
def test_join_refuses(kvc, change):
    assert kvc.kvc_join(**dict(_JOIN, **change)) == kvc.KVC_ERR_INVALID_ARG


def test_join_of_no_row_is_a_no_op(kvc):
    assert kvc.kvc_join(**dict(_JOIN, num_rows=0)) == kvc.KVC_OK


_EVICT = dict(kv_cache=0x10000, num_kv_pages=100, page_table=0x20000, num_reqs=4, max_pages_per_req=8,
              page_table_row_stride=8, lengths=0x30000, slot_weights=0x40000, slot_weights_row_stride=512, max_slots=512,
              births=0x50000, births_row_stride=512, keep=100, recent=8, lengths_out=0x60000, kept=0x70000,
              slot_weights_out=None, slot_weights_out_row_stride=0, births_out=None, births_out_row_stride=0,
              workspace=0x80000, workspace_bytes=1 << 40, stream=0)


@pytest.mark.parametrize("change", [
    dict(kv_cache=0), dict(kv_cache=0x10008), dict(num_kv_pages=0), dict(page_table=0), dict(num_reqs=-1),
    dict(num_reqs=65536), dict(max_pages_per_req=0), dict(page_table_row_stride=-8), dict(lengths=0),
    dict(slot_weights=0), dict(slot_weights=0x40002), dict(slot_weights_row_stride=-1), dict(max_slots=-1),
    dict(births=None), dict(births=0x50001), dict(births_row_stride=-1), dict(keep=-1), dict(keep=1 << 31),
    dict(recent=-1), dict(recent=101), dict(lengths_out=0), dict(lengths_out=0x60002), dict(kept=0x70002),
    dict(slot_weights_out=0x90002), dict(births_out=0x90001), dict(births=None, recent=0, births_out=0x90000),
    dict(workspace=0), dict(workspace=0x80008), dict(workspace_bytes=16)])
def test_evict_refuses(kvc, change):
    assert kvc.kvc_evict(**dict(_EVICT, **change)) == kvc.KVC_ERR_INVALID_ARG


def test_evict_of_no_request_is_a_no_op(kvc):
    assert kvc.kvc_evict(**dict(_EVICT, num_reqs=0)) == kvc.KVC_OK


def test_workspace_sizes(kvc):
    assert kvc.kvc_attend_workspace_bytes(0, 0, 0) == 0 and kvc.kvc_attend_workspace_bytes(1, 129, 1) == 0
    assert kvc.kvc_attend_workspace_bytes(8, 64, 2) > 0
    assert kvc.kvc_evict_workspace_bytes(-1, 1, 1) == 0
    assert kvc.kvc_evict_workspace_bytes(8, 4, 100) >= 8 * 4 + 8 * 2 * 4 * 100


def test_wrappers_refuse_cpu_tensors_and_wrong_types(kvc):
    kv = torch.zeros((2, kvc.KV_PAGE_BYTES), dtype=torch.uint8)
    t, n = torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="no CPU path"):
        kvc.attend(torch.zeros((1, 8, 512), dtype=torch.bfloat16), kv, t, n)
    with pytest.raises(ValueError, match="no CPU path"):
        kvc.evict(kv, t, n, torch.zeros((1, 64)), 3)
    with pytest.raises(ValueError, match="no CPU path"):
        kvc.join([torch.zeros(1, 512)], [torch.zeros(1)])
    with pytest.raises(ValueError, match="one entry per part"):
        kvc.join([torch.zeros(1, 512)], [])


@pytest.mark.parametrize("change", [dict(scale=3e38), dict(slot_weights=0xA0000, slot_weights_row_stride=0, max_slots=512),
                                    dict(slot_weights=0xA0000, slot_weights_row_stride=511, max_slots=512)])
def test_attend_refuses_scales_near_the_end_and_rows_that_overlap(kvc, change):
    assert kvc.kvc_attend(**dict(_ATTEND, **change)) == kvc.KVC_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(slot_weights_out=0x90000, slot_weights_out_row_stride=99), dict(births_out=0x90000, births_out_row_stride=0),
    dict(births_out=0x90000, births_out_row_stride=49, max_slots=50, keep=64)])
def test_evict_refuses_rows_that_overlap(kvc, change):
    assert kvc.kvc_evict(**dict(_EVICT, **change)) == kvc.KVC_ERR_INVALID_ARG


def test_workspace_sizes_beyond_the_limits_are_zero(kvc):
    for args in [(65536, 8, 8), (8, 1 << 58, 8), (8, 8, 1 << 62)]:
        assert kvc.kvc_evict_workspace_bytes(*args) == 0
    assert kvc.kvc_evict_workspace_bytes(65535, (1 << 30) // 64, 1 << 29) >= 65535 * (16 << 29)
