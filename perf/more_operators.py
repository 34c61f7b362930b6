"""The cases on which the operators around a cache held in 4 bits are measured.

A slot can be held in 8 bits a value (448 int8 codes, 64 bf16 words, 8 scale bytes: 584 bytes) or
in 4 (448 codes of 4 bits, 64 bf16 words, 16 scale bytes: 368 bytes). What a program does beside
compressing windows: it writes vectors into slots as they come, rotated to their positions and
quantised (store), reads slots back (dequantize), lets each request's new token attend over its
slots (attend), and turns queries to their positions and attention's rows back (rotate); positions
have one axis (text) or several (time, height and width of images and video).

`run` computes them in elementary torch operations, or, where `own` is true, through the package.

The 4-bit slot: dims 0 .. 447 in groups of 32. With z = bf16(x) and a = max |z| of a group, its
scale s is the smallest of (1 + m / 8) 2^(e - 16), e < 32, m < 8, that 7 s >= a holds for (the
largest if none does), the byte 8 e + m, and a code is z / s rounded to the nearest whole number, halves
away from zero, at most 7 in size. A 32-bit word holds 8 codes plus 8 each: those of even dims in
its low half, of odd ones in its high half. Dims 448 .. 511 are 32 pairs, rotated and kept in bf16.
"""
import math
import random

import torch

own = False

HEAD_DIM, NOPE, ROPE, PAIRS = 512, 448, 64, 32
PAGE = 64
GROUP4, PAYLOAD4, SCALES4 = 32, 352, 16
GROUP8, PAYLOAD8, SCALES8 = 64, 576, 8
POSITIONS = 32768
LARGEST_SLOTS, LARGEST_HEADS = 64 * 8192, 64
LARGEST_ROWS, LARGEST_READ, LARGEST_TURNED = 65537, 262144, 16384 * 64


def listed():
    return [
        # The new tokens of a decode batch, one row each, at scattered places.
        dict(name="write 8 bf16 4-bit", op="write", rows=8, bits=4, dtype="bf16", axes=1, scattered=True),
        # A prompt with images: rows in the order of their pages, three axes of positions.
        dict(name="write 16384 bf16 4-bit 3 axes", op="write", rows=16384, bits=4, dtype="bf16", axes=3, scattered=False),
        # The compressor's normalised vectors of many prompts (32 bits, already rotated elsewhere), in 8 bits.
        dict(name="write 65537 fp32 8-bit", op="write", rows=65537, bits=8, dtype="fp32", axes=0, scattered=False),
        # A few hundred selected slots of one request.
        dict(name="read 509 4-bit fp32", op="read", rows=509, dtype="fp32", scattered=True),
        # The selected slots of a whole batch.
        dict(name="read 262144 4-bit bf16", op="read", rows=262144, dtype="bf16", scattered=True),
        # One conversation of 8192 tokens at 128 tokens a slot: nothing but latency.
        dict(name="attend 1x64 h64", op="attend", reqs=1, slots=64, ragged=False, heads=64, sinks=False, weights=False),
        # A serving batch of mixed lengths, heads spread over four cards.
        dict(name="attend 32x<=4099 h16", op="attend", reqs=32, slots=4099, ragged=True, heads=16, sinks=True, weights=False),
        # Eviction to come: the weight that each slot got is summed up as well.
        dict(name="attend 24x<=2050 h32 weights", op="attend", reqs=24, slots=2050, ragged=True, heads=32, sinks=True, weights=True),
        # 64 contexts of a million tokens: the whole cache is read.
        dict(name="attend 64x8192 h64", op="attend", reqs=64, slots=8192, ragged=False, heads=64, sinks=True, weights=False),
        # A decode batch's queries.
        dict(name="rotate 8x64 bf16", op="rotate", tokens=8, heads=64, dtype="bf16", axes=1, inverse=False),
        # The gradient of a prompt's queries in 32 bits, two axes.
        dict(name="rotate 4099x16 fp32 inverse", op="rotate", tokens=4099, heads=16, dtype="fp32", axes=2, inverse=True),
        # A prompt with video: three axes, all heads.
        dict(name="rotate 16384x64 bf16 3 axes", op="rotate", tokens=16384, heads=64, dtype="bf16", axes=3, inverse=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("write", "read", "attend", "attend", "rotate"))
    dtype = rng.choice(("bf16", "fp32"))
    if op == "write":
        rows = _log_int(rng, 1, LARGEST_ROWS)
        return dict(op=op, rows=rows, bits=rng.choice((4, 4, 8)), dtype=dtype, axes=rng.randint(0, 3), scattered=rng.random() < 0.5)
    if op == "read":
        return dict(op=op, rows=_log_int(rng, 1, LARGEST_READ), dtype=dtype, scattered=rng.random() < 0.5)
    if op == "rotate":
        heads = rng.choice((1, 8, 16, 64, 128, rng.randint(1, 128)))
        tokens = _log_int(rng, 1, min(16384, LARGEST_TURNED // heads // (2 if dtype == "fp32" else 1)))
        return dict(op=op, tokens=tokens, heads=heads, dtype=dtype, axes=rng.randint(1, 4), inverse=rng.random() < 0.5)
    reqs = _log_int(rng, 1, 128)
    slots = _log_int(rng, 40, min(8192, LARGEST_SLOTS // reqs))
    most = LARGEST_SLOTS * LARGEST_HEADS // (reqs * slots)
    heads = min(most, rng.choice((8, 16, 32, 64, 128, rng.randint(1, 128))))
    return dict(op=op, reqs=reqs, slots=slots, ragged=rng.random() < 0.6, heads=heads, sinks=rng.random() < 0.5, weights=rng.random() < 0.4)


def lengths_of(case):
    """Slots of each request: all of them, or spread from none to all."""
    reqs, slots = case["reqs"], case["slots"]
    if not case["ragged"]:
        return [slots] * reqs
    rng = random.Random(1000003 * reqs + slots)
    return [slots] + [rng.choice((0, 1, rng.randint(1, slots), rng.randint(1, slots), rng.randint(1, slots), _log_int(rng, 1, slots)))
                      for _ in range(reqs - 1)]


def axes_of(axes):
    """The axis of each of the 32 pairs: runs of nearly equal length, one for each axis."""
    return [i * axes // PAIRS for i in range(PAIRS)]


# ---- the inputs ------------------------------------------------------------------


def _vectors(count, gen):
    """Rows as the compressor leaves them: normalised, with weights near 1."""
    weight = 1 + 0.1 * torch.randn(HEAD_DIM, device="cuda", generator=gen)
    y = torch.randn((count, HEAD_DIM), device="cuda", generator=gen)
    return y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight


def _table():
    """cos and sin of every position and pair, formed in 64 bits."""
    angle = torch.arange(POSITIONS, device="cuda", dtype=torch.float64)[:, None]
    angle = angle * 10000.0 ** (-torch.arange(PAIRS, device="cuda", dtype=torch.float64) / PAIRS)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _positions(count, axes, gen):
    """Places in a sequence for one axis, or in a clip's frames, rows and columns."""
    first = torch.randint(0, POSITIONS // 2, (1,), device="cuda", generator=gen)
    p = first + torch.randint(0, POSITIONS // 2, (count, 1), device="cuda", generator=gen)
    if axes == 1:
        return p
    return torch.cat([p, torch.randint(0, 128, (count, axes - 1), device="cuda", generator=gen)], 1)


def _slots(count, scattered, gen):
    """(pages of the pool, slots): places anywhere, or one after the other in pages of any order."""
    pages = -(-count // PAGE) * (4 if scattered and count <= 4096 else 1) + 1
    if scattered:
        return pages, torch.randperm(pages * PAGE, device="cuda", generator=gen)[:count]
    order = torch.randperm(pages, device="cuda", generator=gen)
    n = torch.arange(count, device="cuda")
    return pages, order[n // PAGE] * PAGE + n % PAGE


def _fill(cache, gen):
    for at in range(0, len(cache), 2048):
        part = cache[at:at + 2048]
        payload, scales = _pack4(_vectors(len(part) * PAGE, gen))
        part[:, :PAGE * PAYLOAD4] = payload.view(len(part), -1)
        part[:, PAGE * PAYLOAD4:] = scales.view(len(part), -1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case=case)
    dtype = torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16
    if case["op"] in ("write", "rotate") and case["axes"]:
        s["axes"] = bytes(axes_of(case["axes"]))
        s["axis"] = torch.tensor(axes_of(case["axes"]), device="cuda")
        s["table"] = _table()
        s["positions"] = _positions(case.get("rows", case.get("tokens")), case["axes"], gen)
    if case["op"] == "write":
        pages, s["slots"] = _slots(case["rows"], case["scattered"], gen)
        s["cache"] = torch.zeros((pages, PAGE * (PAYLOAD4 + SCALES4 if case["bits"] == 4 else PAYLOAD8 + SCALES8)), dtype=torch.uint8, device="cuda")
        s["x"] = _vectors(case["rows"], gen).to(dtype)
        s["out"] = torch.empty((case["rows"], HEAD_DIM), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "read":
        pages, s["slots"] = _slots(case["rows"], case["scattered"], gen)
        s["cache"] = torch.empty((pages, PAGE * (PAYLOAD4 + SCALES4)), dtype=torch.uint8, device="cuda")
        _fill(s["cache"], gen)
        s["out"] = torch.empty((case["rows"], HEAD_DIM), dtype=dtype, device="cuda")
    elif case["op"] == "rotate":
        shape = (case["tokens"], case["heads"])
        # the rotated dims of whole queries, as a projection leaves them and attention takes them
        s["x"] = torch.empty(shape + (HEAD_DIM,), dtype=dtype, device="cuda")[..., NOPE:]
        s["x"].copy_(torch.randn(shape + (ROPE,), device="cuda", generator=gen))
        s["out"] = torch.empty(shape + (HEAD_DIM,), dtype=dtype, device="cuda")[..., NOPE:]
    else:
        reqs, slots, heads = case["reqs"], case["slots"], case["heads"]
        lengths = lengths_of(case)
        width = -(-slots // PAGE)
        pages = [-(-n // PAGE) for n in lengths]
        pool = max(1, sum(pages))
        s["cache"] = torch.empty((pool, PAGE * (PAYLOAD4 + SCALES4)), dtype=torch.uint8, device="cuda")
        _fill(s["cache"], gen)
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        pages = torch.tensor(pages, dtype=torch.int64, device="cuda")
        column = torch.arange(width, device="cuda")
        order = torch.randperm(pool, device="cuda", generator=gen)
        at = (pages.cumsum(0) - pages)[:, None] + column
        s["pages"] = torch.where(column < pages[:, None], order[at.clamp_max(pool - 1)], -1).to(torch.int32)
        s["q"] = (3 * torch.randn((reqs, heads, HEAD_DIM), device="cuda", generator=gen)).to(torch.bfloat16)
        s["sinks"] = torch.randn(heads, device="cuda", generator=gen) if case["sinks"] else None
        s["out"] = torch.empty((reqs, heads, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((reqs, heads), device="cuda")
        if case["weights"]:
            s["weights"] = torch.exp(2 * torch.randn((reqs, slots), device="cuda", generator=gen))
            s["sums"] = torch.zeros_like(s["weights"])
        if own:
            import kv_cache_compression_c128_gb300 as kvc

            need = kvc.kvc_attend_workspace_bytes(reqs, heads, width, case["weights"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# ---- the plain forms -------------------------------------------------------------


def _pack4(x):
    """[slots, 512] vectors, rotated, as payload and scale bytes of 4-bit slots."""
    z = x[:, :NOPE].to(torch.bfloat16).float().unflatten(1, (NOPE // GROUP4, GROUP4))
    # (a / 7 in 64 bits: where 7 s = a holds it is s in 32, elsewhere a step of a bf16 number or more away)
    bits = (z.abs().amax(-1).double() / 7).float().view(torch.int32)
    byte = (((bits + 0xFFFFF) >> 20) - (127 - 16) * 8).clamp_(0, 255)
    s = ((byte + (127 - 16) * 8) << 20).view(torch.float32)[..., None]
    u = (torch.floor(z.abs() / s + 0.5).clamp_max_(7) * z.sign()).to(torch.int64) + 8
    u = u.view(-1, NOPE // 8, 4, 2)
    shift = 4 * torch.arange(4, device=x.device)[:, None] + 16 * torch.arange(2, device=x.device)
    words = (u << shift).sum((2, 3))
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    payload = torch.cat([words.view(torch.uint8), x[:, NOPE:].to(torch.bfloat16).contiguous().view(torch.uint8)], 1)
    return payload, torch.cat([byte.to(torch.uint8), torch.zeros_like(payload[:, :2])], 1)


def _pack8(x):
    """The same of 8-bit slots, as the compressor stores them."""
    z = x[:, :NOPE].to(torch.bfloat16).float().unflatten(1, (NOPE // GROUP8, GROUP8))
    # (in 64 bits: next to a power of two the logarithm decides)
    e = torch.ceil(torch.log2(z.abs().amax(-1).clamp_min(1e-4).double() / 127)).float()
    codes = torch.trunc(z * torch.exp2(-e)[..., None]).clamp_(-127, 127).to(torch.int8).flatten(1)
    payload = torch.cat([codes.view(torch.uint8), x[:, NOPE:].to(torch.bfloat16).contiguous().view(torch.uint8)], 1)
    return payload, torch.cat([(e + 127).to(torch.uint8), torch.zeros_like(payload[:, :1])], 1)


def _unpack(payload, scales):
    """The vectors of packed slots, in 32 bits."""
    if payload.shape[-1] == PAYLOAD4:
        words = payload[..., :NOPE // 2].contiguous().view(torch.int32)[..., None, None]
        shift = 4 * torch.arange(4, device=words.device)[:, None] + 16 * torch.arange(2, device=words.device)
        codes = (((words >> shift) & 15) - 8).float().flatten(-3).unflatten(-1, (NOPE // GROUP4, GROUP4))
        s = ((scales[..., :NOPE // GROUP4].to(torch.int32) + (127 - 16) * 8) << 20).view(torch.float32)
    else:
        codes = payload[..., :NOPE].view(torch.int8).float().unflatten(-1, (NOPE // GROUP8, GROUP8))
        s = torch.exp2(scales[..., :NOPE // GROUP8].float() - 127)
    rope = payload[..., -2 * ROPE:].contiguous().view(torch.bfloat16).float()
    return torch.cat([(codes * s[..., None]).flatten(-2), rope], -1)


def _places(cache, slots):
    """What lies in a cache's slots: payload and scale bytes."""
    payload = PAYLOAD4 if cache.shape[1] == PAGE * (PAYLOAD4 + SCALES4) else PAYLOAD8
    rows = cache[:, :PAGE * payload].unflatten(1, (PAGE, payload))
    scales = cache[:, PAGE * payload:].unflatten(1, (PAGE, -1))
    return rows, scales, slots // PAGE, slots % PAGE


def _turn(x, s, inverse=False):
    """Pairs (2 i, 2 i + 1) of the last dims, in 32 bits, by the angles of their axes' positions."""
    at = s["positions"][:, s["axis"]]  # [tokens, 32]
    pair = torch.arange(PAIRS, device=x.device)
    cos, sin = s["table"][at, pair], s["table"][at, PAIRS + pair]
    sin = -sin if inverse else sin
    while cos.dim() < x.dim():
        cos, sin = cos[:, None], sin[:, None]
    a, b = x.float().unflatten(-1, (PAIRS, 2)).unbind(-1)
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _write(s):
    x = s["x"].float()
    if s["case"]["axes"]:
        x = torch.cat([x[:, :NOPE], _turn(x[:, NOPE:], s)], 1)
    rows, scales, page, place = _places(s["cache"], s["slots"])
    rows[page, place], scales[page, place] = _pack4(x) if s["case"]["bits"] == 4 else _pack8(x)
    return _read(s)


def _read(s):
    rows, scales, page, place = _places(s["cache"], s["slots"])
    return s["out"].copy_(_unpack(rows[page, place], scales[page, place]))


def _attend(s):
    case, slots = s["case"], s["case"]["slots"]
    n = torch.arange(slots, device="cuda")
    there = n < s["lengths"][:, None]
    rows, scales, page, place = _places(s["cache"], s["pages"].long().clamp_min(0)[:, n // PAGE] * PAGE + n % PAGE)
    kv = torch.where(there[..., None], _unpack(rows[page, place], scales[page, place]), 0)
    scores = s["q"].float() @ kv.transpose(1, 2) / math.sqrt(HEAD_DIM)
    scores = torch.where(there[:, None], scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        top = torch.maximum(top, s["sinks"][:, None])
    top = torch.where(top == -math.inf, 0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + torch.exp(s["sinks"][:, None] - top)
    p = p / torch.where(total == 0, 1, total)
    s["out"].copy_(p @ kv)
    s["lse"].copy_((top + torch.log(total))[..., 0])
    if not case["weights"]:
        return s["out"], s["lse"]
    s["sums"].copy_(torch.where(there, s["weights"] + p.sum(1), s["sums"]))
    return s["out"], s["lse"], s["sums"]


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "rotate":
            return s["out"].copy_(_turn(s["x"], s, case["inverse"]))
        return {"write": _write, "read": _read, "attend": _attend}[case["op"]](s)
    import kv_cache_compression_c128_gb300 as kvc

    if case["op"] == "write":
        kvc.store(s["x"], s["cache"], s["slots"], positions=s.get("positions"), cos_sin_cache=s.get("table"), axes=s.get("axes"))
        return kvc.dequantize(s["cache"], s["slots"], dtype=torch.bfloat16, out=s["out"])
    if case["op"] == "read":
        return kvc.dequantize(s["cache"], s["slots"], dtype=s["out"].dtype, out=s["out"])
    if case["op"] == "rotate":
        return kvc.rotate(s["x"], s["positions"], s["table"], axes=s["axes"], inverse=case["inverse"], out=s["out"])
    got = kvc.attend(s["q"], s["cache"], s["pages"], s["lengths"], sinks=s["sinks"], out=s["out"], lse=s["lse"],
                     slot_weights=s.get("sums"), slot_weights_in=s.get("weights"), workspace=s["workspace"])
    return got + (s["sums"],) if case["weights"] else got


# ---- what a pass cannot do without --------------------------------------------------


def work(case):
    size = 4 if case.get("dtype") == "fp32" else 2
    if case["op"] == "read":
        return dict(bytes=case["rows"] * (8 + PAYLOAD4 + SCALES4 + HEAD_DIM * size), flops=case["rows"] * NOPE)
    if case["op"] in ("write", "rotate"):
        count = case.get("rows", case.get("tokens"))
        angles = (8 * case["axes"] + 8 * PAIRS) * count if case["axes"] else 0
        if case["op"] == "rotate":
            return dict(bytes=angles + count * case["heads"] * 2 * ROPE * size, flops=6 * PAIRS * count * case["heads"])
        slot = PAYLOAD4 + SCALES4 if case["bits"] == 4 else PAYLOAD8 + SCALES8
        # the rows in, the slots out and back in, the values out
        return dict(bytes=angles + count * (8 + HEAD_DIM * size + 2 * slot + HEAD_DIM * 2), flops=count * (5 * NOPE + (6 * PAIRS if case["axes"] else 0)))
    lengths = lengths_of(case)
    total, rows = sum(lengths), case["reqs"] * case["heads"]
    there = total * (PAYLOAD4 + SCALES4) + 4 * sum(-(-n // PAGE) for n in lengths) + 4 * case["reqs"] + rows * (2 * 2 * HEAD_DIM + 4)
    there += 4 * case["heads"] if case["sinks"] else 0
    there += 8 * total if case["weights"] else 0
    return dict(bytes=there, flops=4 * HEAD_DIM * case["heads"] * total)


# ---- 64 bits -------------------------------------------------------------------------


def _exact_slots(cache, slots):
    """Slots of a 4-bit cache, decoded byte by byte."""
    flat = cache[slots // PAGE]
    place = (slots % PAGE)[:, None]
    out = torch.empty((len(slots), HEAD_DIM), dtype=torch.float64, device="cuda")
    dims = torch.arange(NOPE, device="cuda")
    # dim d: word d / 8, nibble (d % 8) / 2 of its half d % 2; a byte holds two nibbles
    nibble = dims % 8 // 2
    byte = flat.gather(1, place * PAYLOAD4 + dims // 8 * 4 + dims % 2 * 2 + nibble // 2).long()
    scale = flat.gather(1, PAGE * PAYLOAD4 + place * SCALES4 + dims // GROUP4).long()
    out[:, :NOPE] = (byte // 16 ** (nibble % 2) % 16 - 8).double() * (8 + scale % 8).double() * torch.pow(2.0, (scale // 8 - 19).double())
    words = flat.gather(1, place * PAYLOAD4 + NOPE // 2 + torch.arange(2 * ROPE, device="cuda"))
    out[:, NOPE:] = words.contiguous().view(torch.bfloat16).double()
    return out


def _exact_turn(x, s, sign):
    z = torch.view_as_complex(x.double().unflatten(-1, (PAIRS, 2)).contiguous())
    angles = torch.stack([torch.complex(s["table"][s["positions"][:, axis], i].double(), sign * s["table"][s["positions"][:, axis], PAIRS + i].double())
                          for i, axis in enumerate(axes_of(s["case"]["axes"]))], 1)
    if z.dim() == 3:
        angles = angles[:, None]
    return torch.view_as_real(z * angles).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "read":
        return _exact_slots(s["cache"], s["slots"])
    if case["op"] == "rotate":
        return _exact_turn(s["x"], s, -1 if case["inverse"] else 1)
    if case["op"] == "write":
        answer = s["x"].double()
        z = s["x"][:, :NOPE].to(torch.bfloat16).double()
        if case["bits"] == 4:
            scales = (1 + torch.arange(8, device="cuda", dtype=torch.float64) / 8) * torch.pow(2.0, torch.arange(-16, 16, device="cuda", dtype=torch.float64))[:, None]
            scales = scales.flatten()
            z = z.unflatten(1, (-1, GROUP4))
            most = z.abs().amax(-1)
            step = scales[torch.searchsorted(7 * scales, most.contiguous()).clamp_max(255)][..., None]
            down = (z / step).abs().floor()
            code = torch.where((z / step).abs() - down >= 0.5, down + 1, down).clamp(max=7)
        else:
            z = z.unflatten(1, (-1, GROUP8))
            most = z.abs().amax(-1, keepdim=True).clamp_min(1e-4)
            mantissa, power = torch.frexp(most)  # most = mantissa 2^power, 0.5 <= mantissa < 1
            step = torch.pow(2.0, power.double() - 7 + (mantissa > 127 / 128).double())
            code = (z / step).abs().floor().clamp(max=127)
        answer[:, :NOPE] = (torch.where(z < 0, -code, code) * step).flatten(1)
        if case["axes"]:
            answer[:, NOPE:] = _exact_turn(s["x"][:, NOPE:], s, 1)
        return answer
    heads, lengths = case["heads"], lengths_of(case)
    out = torch.zeros((case["reqs"], heads, HEAD_DIM), dtype=torch.float64, device="cuda")
    lse = torch.full((case["reqs"], heads), -math.inf, dtype=torch.float64, device="cuda")
    sums = torch.zeros((case["reqs"], case["slots"]), dtype=torch.float64, device="cuda")
    for r, n in enumerate(lengths):
        i = torch.arange(n, device="cuda")
        kv = _exact_slots(s["cache"], s["pages"][r, i // PAGE].long() * PAGE + i % PAGE)
        e = torch.exp(s["q"][r].double() @ kv.T / HEAD_DIM ** 0.5)  # far from the largest that 64 bits hold
        total = e.sum(1) + (torch.exp(s["sinks"].double()) if case["sinks"] else 0)
        if n:
            out[r] = e @ kv / total[:, None]
            sums[r, :n] = (e / total[:, None]).sum(0) + (s["weights"][r, :n].double() if case["weights"] else 0)
        lse[r] = torch.log(total)
    return (out, lse, sums) if case["weights"] else (out, lse)
