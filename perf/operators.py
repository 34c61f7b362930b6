"""The cases on which the operators that read and thin out a packed kv_cache are measured.

A program that decodes with a compressed cache does three things to it, step after step: the new
token of every request attends over the request's packed slots (attend), the result is joined with
the attention over the tokens that are not in the cache yet (join), and when a request outgrows its
share of the pool, the slots that gathered the least attention are thrown out (evict).

`run` computes them in elementary torch operations, or, where `own` is true, through the package.
A slot is 576 payload bytes (448 int8 codes, 64 bf16) and 8 scale bytes; 64 of them make a page.
A slot stands for 128 tokens or more, so 8192 slots are a context of a million tokens.
"""
import math
import random

import torch

own = False

HEAD_DIM, NOPE, GROUP = 512, 448, 64
PAGE, PAYLOAD, SCALES = 64, 576, 8
PAGE_BYTES = PAGE * (PAYLOAD + SCALES)
LARGEST_SLOTS, LARGEST_HEADS = 64 * 8192, 64


def listed():
    return [
        # One conversation of 8192 tokens at 128 tokens a slot: nothing but latency.
        dict(name="attend 1x64 h64", op="attend", reqs=1, slots=64, ragged=False, heads=64, sinks=False, weights=False),
        # The package's headline batch, 8 requests of 16384 tokens.
        dict(name="attend 8x128 h64", op="attend", reqs=8, slots=128, ragged=False, heads=64, sinks=False, weights=False),
        # One context of a million tokens and all heads on one card: few rows, a long axis.
        dict(name="attend 1x8192 h128", op="attend", reqs=1, slots=8192, ragged=False, heads=128, sinks=False, weights=False),
        # A serving batch of mixed lengths, heads spread over four cards.
        dict(name="attend 32x<=4099 h16", op="attend", reqs=32, slots=4099, ragged=True, heads=16, sinks=True, weights=False),
        # The same with eviction to come: the weight that each slot got is summed up as well.
        dict(name="attend 24x<=2050 h32 weights", op="attend", reqs=24, slots=2050, ragged=True, heads=32, sinks=True, weights=True),
        # Many short conversations, few heads a card.
        dict(name="attend 128x1000 h8 weights", op="attend", reqs=128, slots=1000, ragged=False, heads=8, sinks=False, weights=True),
        # 64 contexts of a million tokens: the whole cache is read.
        dict(name="attend 64x8192 h64", op="attend", reqs=64, slots=8192, ragged=False, heads=64, sinks=True, weights=False),
        # The cache's part and the recent tokens' part of a decode batch.
        dict(name="join 2 of 8 h64 bf16", op="join", parts=2, rows=8, heads=64, dtype="bf16"),
        # A cache spread over several owners, partial results in 32 bits.
        dict(name="join 5 of 509 h64 fp32", op="join", parts=5, rows=509, heads=64, dtype="fp32"),
        # The steady state: each request has outgrown its share by one slot.
        dict(name="evict 8x1025 to 1024", op="evict", reqs=8, slots=1025, ragged=False, keep=1024, recent=32, fresh=False),
        # A mixed batch is cut down for the first time.
        dict(name="evict 32x<=4099 to 1000", op="evict", reqs=32, slots=4099, ragged=True, keep=1000, recent=64, fresh=True),
        # Long contexts halved at once.
        dict(name="evict 64x8192 to 4096", op="evict", reqs=64, slots=8192, ragged=False, keep=4096, recent=64, fresh=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "join", "evict"))
    if op == "join":
        parts = rng.randint(2, 6)
        rows = _log_int(rng, 1, 500)
        return dict(op=op, parts=parts, rows=rows, heads=rng.randint(1, 64), dtype=rng.choice(("bf16", "fp32")))
    reqs = _log_int(rng, 1, 128)
    slots = _log_int(rng, 40, min(8192, LARGEST_SLOTS // reqs))
    case = dict(op=op, reqs=reqs, slots=slots, ragged=rng.random() < 0.6)
    if op == "evict":
        keep = rng.randint(1, slots)
        return dict(case, keep=keep, recent=rng.randint(0, min(keep, 128)), fresh=rng.random() < 0.5)
    most = LARGEST_SLOTS * LARGEST_HEADS // (reqs * slots)
    heads = min(most, rng.choice((8, 16, 32, 64, 128, rng.randint(1, 128))))
    return dict(case, heads=heads, sinks=rng.random() < 0.5, weights=rng.random() < 0.4)


def lengths_of(case):
    """Slots of each request: all of them, or spread from none to all."""
    reqs, slots = case["reqs"], case["slots"]
    if not case["ragged"]:
        return [slots] * reqs
    rng = random.Random(1000003 * reqs + slots)
    return [slots] + [rng.choice((0, 1, rng.randint(1, slots), rng.randint(1, slots), rng.randint(1, slots), _log_int(rng, 1, slots)))
                      for _ in range(reqs - 1)]


# ---- the inputs ------------------------------------------------------------------


def _pack(values):
    """[slots, 512] vectors as payload and scale bytes, the way the compressor stores them."""
    z = values[:, :NOPE].to(torch.bfloat16).float().view(-1, NOPE // GROUP, GROUP)
    e = torch.ceil(torch.log2(z.abs().amax(-1).clamp_min(1e-4) / 127))
    codes = torch.trunc(z * torch.exp2(-e)[..., None]).clamp_(-127, 127).to(torch.int8).view(-1, NOPE)
    rope = values[:, NOPE:].to(torch.bfloat16).contiguous()
    payload = torch.cat([codes.view(torch.uint8), rope.view(torch.uint8)], 1)
    scales = torch.cat([(e + 127).to(torch.uint8), torch.zeros_like(payload[:, :1])], 1)
    return payload, scales


def _cache(case, gen):
    """A pool of pages in random order, each request's pages in a table, and the lengths."""
    lengths = lengths_of(case)
    width = -(-case["slots"] // PAGE)
    pages = [-(-n // PAGE) for n in lengths]
    pool = max(1, sum(pages))
    cache = torch.empty((pool, PAGE_BYTES), dtype=torch.uint8, device="cuda")
    weight = 1 + 0.1 * torch.randn(HEAD_DIM, device="cuda", generator=gen)
    for at in range(0, pool, 2048):
        part = cache[at:at + 2048]
        y = torch.randn((len(part) * PAGE, HEAD_DIM), device="cuda", generator=gen)
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight
        payload, scales = _pack(y)
        part[:, :PAGE * PAYLOAD] = payload.view(len(part), -1)
        part[:, PAGE * PAYLOAD:] = scales.view(len(part), -1)
    lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    pages = torch.tensor(pages, dtype=torch.int64, device="cuda")
    column = torch.arange(width, device="cuda")
    order = torch.randperm(pool, device="cuda", generator=gen)
    at = (pages.cumsum(0) - pages)[:, None] + column
    table = torch.where(column < pages[:, None], order[at.clamp_max(pool - 1)], -1).to(torch.int32)
    return cache, table, lengths


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    state = dict(case=case)
    if case["op"] == "join":
        shape = (case["rows"], case["heads"])
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        state["outs"] = [torch.randn(shape + (HEAD_DIM,), device="cuda", generator=gen).to(dtype) for _ in range(case["parts"])]
        state["lses"] = [torch.randn(shape, device="cuda", generator=gen) * 2 + 5 for _ in range(case["parts"])]
        for i, lse in enumerate(state["lses"]):  # a part that held nothing for a row
            lse.masked_fill_(torch.rand(shape, device="cuda", generator=gen) < 0.05, -math.inf)
        state["out"] = torch.empty(shape + (HEAD_DIM,), dtype=dtype, device="cuda")
        state["lse"] = torch.empty(shape, device="cuda")
        return state
    reqs, slots = case["reqs"], case["slots"]
    cache, table, lengths = _cache(case, gen)
    state.update(cache=cache, table=table, lengths=lengths)
    weights = torch.exp(2 * torch.randn((reqs, slots), device="cuda", generator=gen))
    if case["op"] == "attend":
        heads = case["heads"]
        state["q"] = (3 * torch.randn((reqs, heads, HEAD_DIM), device="cuda", generator=gen)).to(torch.bfloat16)
        state["sinks"] = torch.randn(heads, device="cuda", generator=gen) if case["sinks"] else None
        state["out"] = torch.empty((reqs, heads, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
        state["lse"] = torch.empty((reqs, heads), device="cuda")
        if case["weights"]:
            state["weights"], state["sums"] = weights, torch.zeros_like(weights)
        if own:
            import kv_cache_compression_c128_gb300 as kvc

            need = kvc.kvc_attend_workspace_bytes(reqs, heads, table.shape[1], case["weights"])
            state["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        return state
    births = torch.arange(slots, device="cuda").expand(reqs, slots)
    if not case["fresh"]:  # earlier evictions left the slots in any order
        chance = torch.rand((reqs, slots), device="cuda", generator=gen)
        chance += 2 * (births >= lengths[:, None])
        births = chance.argsort(1).argsort(1)
    state["weights"], state["births"] = weights, births.to(torch.int32).contiguous()
    keep = case["keep"]
    state["lengths_out"] = torch.empty_like(lengths)
    state["kept"] = torch.empty((reqs, keep), dtype=torch.int32, device="cuda")
    state["weights_out"] = torch.zeros((reqs, keep), device="cuda")
    state["births_out"] = torch.zeros((reqs, keep), dtype=torch.int32, device="cuda")
    if own:
        import kv_cache_compression_c128_gb300 as kvc

        need = kvc.kvc_evict_workspace_bytes(reqs, table.shape[1], keep)
        state["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return state


# ---- the plain forms -------------------------------------------------------------


def _slot_ids(table, count):
    """The slot in the pool of each request's slots 0 .. count - 1; of page 0 where there is none."""
    n = torch.arange(count, device=table.device)
    return table.long().clamp_min(0)[:, n // PAGE] * PAGE + n % PAGE


def _read(cache, ids):
    """The vectors of packed slots, in 32 bits."""
    payload = cache[:, :PAGE * PAYLOAD].reshape(-1, PAYLOAD)[ids]
    scales = cache[:, PAGE * PAYLOAD:].reshape(-1, SCALES)[ids]
    codes = payload[..., :NOPE].view(torch.int8).float().unflatten(-1, (NOPE // GROUP, GROUP))
    nope = codes * torch.exp2(scales[..., :NOPE // GROUP].float() - 127)[..., None]
    rope = payload[..., NOPE:].contiguous().view(torch.bfloat16).float()
    return torch.cat([nope.flatten(-2), rope], -1)


def _attend(s):
    case, slots = s["case"], s["case"]["slots"]
    lengths = s["lengths"]
    there = torch.arange(slots, device="cuda") < lengths[:, None]
    kv = torch.where(there[..., None], _read(s["cache"], _slot_ids(s["table"], slots)), 0)
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


def _join(s):
    lses = torch.stack(s["lses"])
    top = lses.amax(0)
    top = torch.where(top == -math.inf, 0, top)
    p = torch.exp(lses - top)
    total = p.sum(0)
    p = p / torch.where(total == 0, 1, total)
    s["out"].copy_((p[..., None] * torch.stack(s["outs"]).float()).sum(0))
    s["lse"].copy_(top + torch.log(total))
    return s["out"], s["lse"]


def _evict(s):
    case, keep, slots = s["case"], s["case"]["keep"], s["case"]["slots"]
    cache, table, lengths = s["cache"], s["table"], s["lengths"].long()[:, None]
    n = torch.arange(slots, device="cuda")
    there = n < lengths
    births = s["births"].long()
    newest = torch.where(there, births, -1).amax(1, keepdim=True)
    bits = (s["weights"] + 0.0).view(torch.int32).long()  # order of the values as order of whole numbers
    rank = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    rank = torch.where(s["weights"].isnan(), -(1 << 33), rank)
    rank = torch.where(births > newest - case["recent"], 1 << 33, rank)
    rank = torch.where(there, rank, -(1 << 34))
    best = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :keep]
    new = lengths.clamp_max(keep)
    kept = torch.zeros_like(there).scatter_(1, best, n[:keep] < new)
    hole, mover = ~kept & (n < new), kept & (n >= new)
    # the i-th hole takes the i-th slot that is kept from behind the new length
    order = torch.where(mover, n, slots).sort(1).values
    moved = order.gather(1, (hole.cumsum(1) - 1).clamp_min(0))
    source = torch.where(n >= new, -1, torch.where(hole, moved, n))[:, :keep]
    s["lengths_out"].copy_(new[:, 0])
    s["kept"].copy_(source)
    at = source.clamp_min(0)
    s["weights_out"].copy_(torch.where(source >= 0, s["weights"].gather(1, at), s["weights_out"]))
    s["births_out"].copy_(torch.where(source >= 0, s["births"].gather(1, at), s["births_out"]))
    ids = _slot_ids(table, slots)
    to, of = ids[:, :keep][hole[:, :keep]], ids.gather(1, at)[hole[:, :keep]]
    for lo, size in ((0, PAYLOAD), (PAGE * PAYLOAD, SCALES)):
        rows = cache[:, lo:lo + PAGE * size].unflatten(1, (PAGE, size))
        rows[to // PAGE, to % PAGE] = rows[of // PAGE, of % PAGE]
    return cache, s["lengths_out"], s["kept"], s["weights_out"], s["births_out"]


def run(s):
    case = s["case"]
    if not own:
        return {"attend": _attend, "join": _join, "evict": _evict}[case["op"]](s)
    import kv_cache_compression_c128_gb300 as kvc

    if case["op"] == "join":
        return kvc.join(s["outs"], s["lses"], out=s["out"], lse=s["lse"])
    if case["op"] == "attend":
        got = kvc.attend(s["q"], s["cache"], s["table"], s["lengths"], sinks=s["sinks"], out=s["out"], lse=s["lse"],
                         slot_weights=s.get("sums"), slot_weights_in=s.get("weights"), workspace=s["workspace"])
        return got + (s["sums"],) if case["weights"] else got
    kvc.evict(s["cache"], s["table"], s["lengths"], s["weights"], case["keep"], recent=case["recent"], births=s["births"],
              lengths_out=s["lengths_out"], kept=s["kept"], slot_weights_out=s["weights_out"], births_out=s["births_out"],
              workspace=s["workspace"])
    return s["cache"], s["lengths_out"], s["kept"], s["weights_out"], s["births_out"]


# ---- what a pass cannot do without --------------------------------------------------


def work(case):
    if case["op"] == "join":
        rows = case["rows"] * case["heads"]
        size = 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=rows * (case["parts"] + 1) * (HEAD_DIM * size + 4), flops=2 * rows * case["parts"] * HEAD_DIM)
    lengths = lengths_of(case)
    total, reqs = sum(lengths), case["reqs"]
    pages = sum(-(-n // PAGE) for n in lengths)
    if case["op"] == "attend":
        rows = reqs * case["heads"]
        there = total * (PAYLOAD + SCALES) + 4 * pages + 4 * reqs + rows * (2 * 2 * HEAD_DIM + 4)
        there += 4 * case["heads"] if case["sinks"] else 0
        there += 8 * total if case["weights"] else 0
        return dict(bytes=there, flops=4 * HEAD_DIM * case["heads"] * total)
    keep, recent = case["keep"], case["recent"]
    moves = 0.0  # as many as chance leaves behind the new length
    for n in lengths:
        if n > keep:
            if case["fresh"]:  # the newest lie at the end
                tail = min(recent, n - keep)
                moves += tail + (keep - recent) * max(0, n - recent - keep) / max(1, n - recent)
            else:
                moves += keep * (n - keep) / n
    new = sum(min(n, keep) for n in lengths)
    return dict(bytes=int(8 * total + 4 * 2 * reqs + 4 * pages + new * 8 + 4 * reqs * keep + moves * 2 * (PAYLOAD + SCALES)), flops=total)


# ---- 64 bits -------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "join":
        weight = [torch.exp(x.double()) for x in s["lses"]]
        total = sum(weight)
        out = sum(w[..., None] * x.double() for w, x in zip(weight, s["outs"])) / total.clamp_min(1e-300)[..., None]
        return out, torch.log(total)
    if case["op"] == "evict":
        answer = s["weights_out"].double().cpu().numpy()
        weights, births = s["weights"].cpu().numpy(), s["births"].cpu().numpy()
        for r, n in enumerate(lengths_of(case)):
            new = min(n, case["keep"])
            newest = births[r, :n].max(initial=-1)
            ranked = sorted(range(n), key=lambda i: (not births[r, i] > newest - case["recent"], -weights[r, i], i)
                            if not births[r, i] > newest - case["recent"] else (False, 0.0, i))[:new]
            kept = set(ranked)
            behind = iter(sorted(i for i in kept if i >= new))
            for j in range(new):
                answer[r, j] = weights[r, j if j in kept else next(behind)]
        return None, None, None, answer, None
    heads, lengths = case["heads"], lengths_of(case)
    out = torch.zeros((case["reqs"], heads, HEAD_DIM), dtype=torch.float64, device="cuda")
    lse = torch.full((case["reqs"], heads), -math.inf, dtype=torch.float64, device="cuda")
    sums = torch.zeros((case["reqs"], case["slots"]), dtype=torch.float64, device="cuda")
    for r, n in enumerate(lengths):
        pages = s["cache"][s["table"][r, :-(-n // PAGE)].long()]
        payload = pages[:, :PAGE * PAYLOAD].reshape(-1, PAYLOAD)[:n]
        scales = pages[:, PAGE * PAYLOAD:].reshape(-1, SCALES)[:n, :NOPE // GROUP]
        codes = payload[:, :NOPE].to(torch.float64)
        codes = codes - 256 * (codes > 127)
        kv = torch.empty((n, HEAD_DIM), dtype=torch.float64, device="cuda")
        kv[:, :NOPE] = codes * torch.pow(2.0, scales.double() - 127).repeat_interleave(GROUP, 1)
        kv[:, NOPE:] = payload[:, NOPE:].contiguous().view(torch.bfloat16).double()
        e = torch.exp(s["q"][r].double() @ kv.T / HEAD_DIM ** 0.5)  # far from the largest that 64 bits hold
        total = e.sum(1) + (torch.exp(s["sinks"].double()) if case["sinks"] else 0)
        if n:
            out[r] = e @ kv / total[:, None]
            sums[r, :n] = (e / total[:, None]).sum(0) + (s["weights"][r, :n].double() if case["weights"] else 0)
        lse[r] = torch.log(total)
    return (out, lse, sums) if case["weights"] else (out, lse)
