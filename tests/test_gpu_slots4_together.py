"""The operators around a 4-bit cache together, as a decoding program uses them, one
behind the other on a stream: vectors are written to their positions as they come,
queries are turned, attend over the slots, their rows are turned back, and slots are
evicted; every call reads what the one before it has written."""
import numpy as np
import pytest
import torch

import slots4_testlib as four
import slots_testlib as plain
from kvc_testlib import bf16_bits_to_f32, torch_bf16_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,attend,width", [(4, four.attend, four.PAGE4_BYTES), (8, plain.attend, 37376)])
@pytest.mark.parametrize("captured", [False, True])
def test_decode_steps(bits, attend, width, captured):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_compression_c128_gb300 as kvc

    kvc.build()
    rng = np.random.default_rng(bits)
    R, H, steps, start = 3, 20, 6, 90
    table = np.array([[4, 1], [0, 5], [2, 3]], np.int32)
    turns, names = four.table_of(4000), (np.arange(32) * 3 // 32).tolist()
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    d_turns, d_table = cuda(turns), cuda(table)
    kv = torch.zeros((6, width), dtype=torch.uint8, device="cuda")
    # a prompt of `start` rows each
    slot = lambda n: (table[:, n // 64].astype(np.int64) * 64 + n % 64)
    x0 = rng.standard_normal((R, start, 512)).astype(np.float32)
    p0 = rng.integers(0, 4000, (R, start, 3))
    slots0 = np.stack([slot(n) for n in range(start)], 1)
    kvc.store(cuda(x0.reshape(-1, 512)), kv, cuda(slots0.reshape(-1)), positions=cuda(p0.reshape(-1, 3)), cos_sin_cache=d_turns, axes=names)
    x = rng.standard_normal((steps, R, 512)).astype(np.float32)
    p = rng.integers(0, 4000, (steps, R, 3))
    q = torch.from_numpy(rng.standard_normal((steps, R, H, 512)).astype(np.float32)).to(torch.bfloat16)
    d_x, d_p, d_q = cuda(x).to(torch.bfloat16), cuda(p), q.cuda()
    now_x, now_p, now_q = torch.empty_like(d_x[0]), torch.empty_like(d_p[0]), torch.empty_like(d_q[0])
    now_slots, lengths = torch.empty(R, dtype=torch.int64, device="cuda"), torch.full((R,), start, dtype=torch.int32, device="cuda")
    weights = torch.zeros((R, 128), device="cuda")
    rows, lse = torch.empty((R, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((R, H), device="cuda")

    def step():
        kvc.store(now_x, kv, now_slots, positions=now_p, cos_sin_cache=d_turns, axes=names)
        kvc.rotate(now_q[..., 448:], now_p, d_turns, axes=names, out=now_q[..., 448:])
        kvc.attend(now_q, kv, d_table, lengths, out=rows, lse=lse, slot_weights=weights, slot_weights_in=weights)
        kvc.rotate(rows[..., 448:], now_p, d_turns, axes=names, inverse=True, out=rows[..., 448:])

    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph):
            step()
    got, seen = [], []
    for i in range(steps):
        now_x.copy_(d_x[i]), now_p.copy_(d_p[i]), now_q.copy_(d_q[i])
        now_slots.copy_(cuda(slot(start + i)))
        lengths += 1
        graph.replay() if captured else step()
        got.append((rows.clone(), lse.clone()))
        seen.append((now_q.clone(), kv.clone()))
    assert kvc.kvc_get_device_error(torch.cuda.current_stream().cuda_stream) == 0
    total, tol = np.zeros((R, 128)), np.zeros((R, 128))
    for i, ((out, l), (turned, cache)) in enumerate(zip(got, seen)):
        n = np.full(R, start + 1 + i, np.int32)
        turned, cache = turned.double().cpu().numpy(), cache.cpu().numpy()
        # the queries as they were turned, the cache as it was written
        want_q, off = four.turn(q[i, ..., 448:].double().numpy(), p[i], turns, names)
        assert (np.abs(turned[..., 448:] - want_q) <= off + 2.0 ** -8 * (np.abs(want_q) + off)).all()
        want = attend(turned, cache, table, n, 512 ** -0.5)
        assert (np.abs(l.double().cpu().numpy() - want[1]) <= want[4]).all()
        out = out.double().cpu().numpy()
        assert (np.abs(out - want[0]) <= want[3])[..., :448].all()
        # rows turned back: both dims of a pair carry their tolerance over, and are rounded again
        back, off = four.turn(want[0][..., 448:], p[i], turns, names, inverse=True)
        pair = want[3][..., 448:].reshape(R, H, 32, 2).sum(-1, keepdims=True).repeat(2, -1).reshape(R, H, 64)
        off = off * 2 + pair
        assert (np.abs(out[..., 448:] - back) <= off + 2.0 ** -8 * (np.abs(back) + off)).all()
        total[:, :start + 1 + i] += want[2]
        tol[:, :start + 1 + i] += want[5] + plain.STEP_F32 * total[:, :start + 1 + i]
    assert (np.abs(weights.double().cpu().numpy() - total) <= tol).all()
    # what was written is what the vectors quantise to: the last step's rows, read back
    last = kvc.dequantize(kv, cuda(slot(start + steps - 1))).double().cpu().numpy()
    payload, scales = four.slot_bytes(bf16_bits_to_f32(torch_bf16_bits(x[-1])).reshape(x[-1].shape), bits)
    nope = four.decode4(payload, scales) if bits == 4 else np.ascontiguousarray(payload[:, :448]).view(np.int8) * np.repeat(
        np.ldexp(1.0, scales[:, :7].astype(int) - 127), 64, 1)
    assert np.array_equal(last[:, :448], nope[:, :448])
    # the slots that few looked at go, and attention over the others is as in 64 bits
    before, w_host = kv.cpu().numpy(), weights.cpu().numpy()
    want_kv, want_len, _ = (four.evict if bits == 4 else plain.evict)(before, table, np.full(R, start + steps), w_host, 50)
    kvc.evict(kv, d_table, lengths, weights, 50, lengths_out=lengths, slot_weights_out=weights)
    out, l = kvc.attend(now_q, kv, d_table, lengths)
    assert np.array_equal(kv.cpu().numpy(), want_kv) and np.array_equal(lengths.cpu().numpy(), want_len)
    want = attend(now_q.double().cpu().numpy(), want_kv, table, want_len, 512 ** -0.5)
    assert (np.abs(out.double().cpu().numpy() - want[0]) <= want[3]).all()
