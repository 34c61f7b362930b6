"""kvc.rotate into memory that its operand lies in too: in place and between its rows as
into memory of its own, over other rows refused."""
import numpy as np
import pytest
import torch

import slots4_testlib as four

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", params=["quick", "python"])
def kvc(request):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_compression_c128_gb300 as kvc

    kvc.build()
    kvc._load_torch()
    quick = kvc._quick
    if request.param == "python":
        kvc._quick = None
    yield kvc
    kvc._quick = quick


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 6), (37, 1), (37, 6)])
def test_shared_memory(kvc, T, H, dtype):
    rng = np.random.default_rng(T + H)
    table = torch.from_numpy(four.table_of(90)).cuda()
    positions = torch.from_numpy(rng.integers(0, 90, T)).cuda()
    # the rows of one tensor: queries of 512 dims a head, then 64 turned ones a head
    whole = torch.from_numpy(rng.standard_normal((T, H * 576)).astype(np.float32)).to(dtype).cuda()

    def views():
        w = whole.clone()
        q, packed = w[:, :H * 512].view(T, H, 512), w[:, H * 512:].view(T, H, 64)
        return w, q, packed

    w, q, packed = views()
    want = kvc.rotate(q[..., 448:].clone(), positions, table)
    for to in (lambda q, packed: packed, lambda q, packed: q[..., 64:128], lambda q, packed: q[..., 448:]):
        w, q, packed = views()
        out = to(q, packed)
        assert kvc.rotate(q[..., 448:], positions, table, out=out) is out
        assert torch.equal(out, want)
        out.copy_(to(*views()[1:]))
        assert torch.equal(w, whole)                          # and nothing else was written
    w, q, packed = views()
    step = 16 // w.element_size()
    refused = [q[..., 448 - step:512 - step]]                  # 16 bytes before
    if T > 1:
        flat = torch.as_strided(w, (T - 1, H, 64), (H * 576, 512, 1), 448)
        on = torch.as_strided(w, (T - 1, H, 64), (H * 576, 512, 1), 448 + H * 576)
        with pytest.raises(kvc.KvcError):                      # the next token's rows
            kvc.rotate(flat, positions[1:], table, out=on)
    if H > 1:
        refused.append(torch.as_strided(w, (T, H, 64), (H * 576, 64, 1), 448))
    if T > 1 and H > 1:
        refused.append(torch.as_strided(w, (T, H, 64), (H * 64, 64, 1), 448))
    for out in refused:
        with pytest.raises(kvc.KvcError, match="invalid argument"):
            kvc.rotate(q[..., 448:], positions, table, out=out)
    if H > 1:                                                  # one row for all heads, turned into another tensor's or over itself
        one = q[:, :1, 448:].expand(T, H, 64)
        assert torch.equal(kvc.rotate(one, positions, table, out=packed), want[:, :1].expand(T, H, 64))
        with pytest.raises(kvc.KvcError):
            kvc.rotate(one, positions, table, out=q[..., 448:])
    w, q, packed = views()
    assert kvc.kvc_get_device_error(torch.cuda.current_stream().cuda_stream) == 0
