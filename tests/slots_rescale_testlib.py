"""Cases for attention whose reference has to move: scores that rise from page
to page by some 2^33 and more in weight, under values that fall by as much, so
that every page counts in the result.  Scores come from one dim alone and are
exact, values of a dim have one sign: tolerances stay at the roundings of the
softmax weights and of the result, below 1 % of every value.  (127 * 2^106, the
largest value, times the 2304 slots of the longest case stays below 2^127.)
"""
from __future__ import annotations

import numpy as np

from kvc_testlib import SCALE_BASE, SCALE_DIM, TOKEN_STRIDE
from slots_testlib import HALF_BF16, STEP_F32, random_cache, slot_vectors

HEIGHTS = {
    "one step": [0, 34],
    "steps, some below 2^32": [0, 33, 36, 56],
    "steps to values beyond 2^64": [0, 33, 67, 70, 104],
    "up, down and up": [10, 0, 45, 3, 60],
    "a step a page": [0, 36, 72, 106],
}


def bf16(a):
    """float32 values rounded to bf16 (to nearest, ties to even)."""
    b = np.asarray(a, np.float32).view(np.uint32)
    return ((b + 0x7FFF + (b >> 16 & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def case(seed, heights, H, repeat=1):
    """(q float32 [1, H, 512], kv): a page for each height, `repeat` of them in a row."""
    rng = np.random.default_rng(seed)
    heights = np.repeat(heights, repeat)
    kv = random_cache(rng, len(heights))
    rows = kv[:, :SCALE_BASE].reshape(-1, 64, TOKEN_STRIDE)
    scales = kv[:, SCALE_BASE:].reshape(-1, 64, SCALE_DIM)
    sign = rng.choice([-1, 1], 512)
    rows[..., :448] = (sign[:448] * rng.integers(1, 128, (len(heights), 64, 448))).astype(np.int8).view(np.uint8)
    rows[..., 0] = heights[:, None]
    fall = int(max(heights)) - heights
    scales[..., 0] = 127
    scales[..., 1:7] = (127 + fall)[:, None, None]
    words = bf16(sign[448:] * (1 + rng.random((len(heights), 64, 64))) * 2.0 ** fall[:, None, None])
    rows[..., 448:] = np.ascontiguousarray(words.view(np.uint32) >> 16).astype("<u2").view(np.uint8).reshape(-1, 64, 128)
    q = np.zeros((1, H, 512), np.float32)
    # ln(2) and up to 5 % more or less, in steps of 1 %, so that neighbours' factors differ;
    # every seventh head falls where the others rise
    q[0, :, 0] = bf16(np.log(2) * (1 + 0.01 * (np.arange(H) * 5 % 11 - 5)) * np.where(np.arange(H) % 7 == 6, -0.5, 1))
    return q, kv


def expected(q, kv, table, n, pages):
    """(out, lse, weights, tolerances of the three) in float64 for one request, scale 1.

    In powers of two a score is off by two half steps (log2(e), the product), its
    distance from the reference by one more, the exponential by 2 steps; each move
    of the reference multiplies what is there by another such number.  The sums
    take a step for each slot.  The weight and the result are rounded to bf16.
    """
    k = slot_vectors(kv, table, n)
    s = q[0].astype(np.float64) @ k.T
    top = s.max(1, keepdims=True)
    e = np.exp(s - top)
    total = e.sum(1, keepdims=True)
    p, lse = e / total, (top + np.log(total))[:, 0]
    out, away = p @ k, p @ np.abs(k)
    x = np.abs(s).max(1) / np.log(2)
    rel = STEP_F32 * (np.log(2) * x + (pages + 1) * (2 + np.log(2) / 2 * x) + n + 16)
    first = away * (HALF_BF16 + rel[:, None]) * 1.01
    tol_out = first + HALF_BF16 * (np.abs(out) + first)
    tol_w = (p * 2 * rel[:, None]).sum(0) + len(p) * STEP_F32 * p.sum(0)
    return out, lse, p.sum(0), tol_out, rel + 3 * STEP_F32 * np.abs(lse), tol_w


def walk(q, kv, table, n, mistake=None):
    """(out, lse) page by page with a reference that moves where a score passes it
    by 2^32, as the operator forms them, in float64; `mistake` plants one."""
    k = slot_vectors(kv, table, n)
    s = q[0].astype(np.float64) @ k.T / np.log(2)
    H = len(s)
    ref, total, acc = np.full(H, -np.inf), np.zeros(H), np.zeros((H, 512))
    for at in range(0, n, 64):
        x, v = s[:, at:at + 64], k[at:at + 64]
        if (x.max(1) - ref > 32).any():
            new = np.maximum(ref, x.max(1))
            f = np.where(np.isinf(ref), 0.0, np.exp2(np.where(np.isinf(ref), 0, ref - new)))
            ref = new
            if mistake != "sum left":
                total = total * f
            if mistake == "rows left":
                pass
            elif mistake == "half the dims left":
                acc[:, :256] *= f[:, None]
            elif mistake == "the next head's factor":
                acc *= np.roll(f, 1)[:, None]
            elif mistake == "rows dropped":
                acc *= 0
            else:
                acc *= f[:, None]
        e = np.exp2(x - ref[:, None])
        total, acc = total + e.sum(1), acc + e @ v
    return acc / total[:, None], (ref + np.log2(total)) * np.log(2)
