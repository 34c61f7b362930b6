"""Plain 64-bit forms of the operators on packed slots, for their tests.

Everything here is numpy in float64, written from the definitions: the slot
layout of kvc_testlib, softmax over a request's slots, the join of parts by
their log-sum-exp, and eviction by sorting.
"""
from __future__ import annotations

import numpy as np

from kvc_testlib import PAGE_BYTES, PAGE_SLOTS, SCALE_BASE, SCALE_DIM, TOKEN_STRIDE, bf16_bits_to_f32

HALF_BF16 = 2.0 ** -8      # half a step of bf16, relative
STEP_F32 = 2.0 ** -23      # a step of fp32, relative


def random_cache(rng, pages, e_lo=-8, e_hi=-3):
    """Packed pages of random codes, scales 2^e_lo .. 2^e_hi and N(0, 1) bf16 words."""
    kv = np.zeros((pages, PAGE_BYTES), np.uint8)
    rows = kv[:, :SCALE_BASE].reshape(pages, PAGE_SLOTS, TOKEN_STRIDE)
    rows[..., :448] = rng.integers(0, 256, rows[..., :448].shape, dtype=np.uint8)
    rope = rng.standard_normal((pages, PAGE_SLOTS, 64)).astype(np.float32)
    bits = (rope.view(np.uint32) >> 16).astype("<u2")
    rows[..., 448:] = bits.view(np.uint8)
    scales = kv[:, SCALE_BASE:].reshape(pages, PAGE_SLOTS, SCALE_DIM)
    scales[..., :7] = rng.integers(127 + e_lo, 128 + e_hi, scales[..., :7].shape, dtype=np.uint8)
    return kv


def page_tables(rng, lengths, extra_pages=0, width=None):
    """(table int32 [R, width], pages in the pool): disjoint pages in random order, -1 behind."""
    counts = [-(-int(n) // PAGE_SLOTS) for n in lengths]
    width = max(1, max(counts)) if width is None else width
    pool = max(1, sum(counts) + extra_pages)
    order = rng.permutation(pool).astype(np.int32)
    table = np.full((len(lengths), width), -1, np.int32)
    at = 0
    for r, c in enumerate(counts):
        table[r, :c] = order[at:at + c]
        at += c
    return table, pool


def slot_vectors(kv, table_row, length):
    """The first `length` slots of a request as float64 [length, 512]."""
    pages = kv[table_row[:-(-length // PAGE_SLOTS)]]
    payload = pages[:, :SCALE_BASE].reshape(-1, TOKEN_STRIDE)[:length]
    scales = pages[:, SCALE_BASE:].reshape(-1, SCALE_DIM)[:length, :7].astype(np.int64) - 127
    codes = np.ascontiguousarray(payload[:, :448]).view(np.int8).astype(np.float64)
    out = np.empty((length, 512))
    out[:, :448] = codes * np.repeat(np.ldexp(1.0, scales), 64, axis=1)
    out[:, 448:] = bf16_bits_to_f32(np.ascontiguousarray(payload[:, 448:]).view("<u2"))
    return out


def attend(q, kv, table, lengths, scale, sinks=None):
    """(out, lse, weights, tolerances of the three) in float64.

    Tolerances count the roundings on the way.  A score is a sum of 512
    products in fp32, each addition off by at most a step of the running sum:
    off by d = 520 steps of scale * sum|q k| at most (8 more for the scaling
    and the subtraction of the maximum).  A softmax weight then is off by 2 d
    (its numerator and the sum) and a few steps for exp, and is rounded to
    bf16 once before the product; the product's sum adds a step per slot, and
    out is rounded to bf16 once.  A weight below 2^-126, the smallest normal
    fp32, may be flushed to zero: off by up to that much for each slot and
    head, and, where it is flushed before the division by a sum of at least 1,
    no more.
    """
    R, H, _ = q.shape
    S = int(max(lengths)) if len(lengths) else 0
    out, lse = np.zeros((R, H, 512)), np.full((R, H), -np.inf)
    weights = np.zeros((R, S))
    tol_out, tol_lse, tol_w = np.zeros((R, H, 512)), np.zeros((R, H)), np.zeros((R, S))
    for r in range(R):
        n = int(lengths[r])
        k = slot_vectors(kv, table[r], n)
        s = scale * (q[r] @ k.T)
        d = 520 * STEP_F32 * abs(scale) * (np.abs(q[r]) @ np.abs(k).T).max(1, initial=0.0)
        d = d + 4 * STEP_F32 * np.abs(s).max(1, initial=0.0)
        all_s = s if sinks is None else np.concatenate([s, sinks[:, None]], 1)
        if all_s.shape[1] == 0:
            continue
        top = all_s.max(1)
        top = np.where(np.isinf(top), 0, top)
        total = np.exp(all_s - top[:, None]).sum(1)
        with np.errstate(divide="ignore"):
            lse[r] = top + np.log(total)
        p = np.exp(s - top[:, None]) / np.where(total == 0, 1, total)[:, None]
        out[r] = p @ k
        away = p @ np.abs(k)
        tol_out[r] = away * (HALF_BF16 + 2 * d + (n + 16) * STEP_F32)[:, None] * 1.01
        tol_out[r] += n * 2.0 ** -126 * np.abs(k).max(initial=0.0)
        tol_out[r] += HALF_BF16 * (np.abs(out[r]) + tol_out[r]) + 2.0 ** -126
        tol_lse[r] = d + (8 + n) * STEP_F32 + 4 * STEP_F32 * np.abs(np.where(np.isinf(lse[r]), 0, lse[r]))
        weights[r, :n] = p.sum(0)
        tol_w[r, :n] = (p * (2 * d + (n + 16) * STEP_F32)[:, None]).sum(0) * 1.01 + H * STEP_F32 * p.sum(0) + H * 2.0 ** -126
    return out, lse, weights, tol_out, tol_lse, tol_w


def join(outs, lses):
    lses = np.stack([np.asarray(x, np.float64) for x in lses])
    top = lses.max(0)
    top = np.where(np.isinf(top), 0, top)
    w = np.exp(lses - top)
    total = w.sum(0)
    safe = np.where(total == 0, 1, total)
    out = sum(np.where((wi > 0)[..., None], np.asarray(o, np.float64), 0) * (wi / safe)[..., None]
              for wi, o in zip(w, outs))
    away = sum(np.where((wi > 0)[..., None], np.abs(np.asarray(o, np.float64)), 0) * (wi / safe)[..., None]
               for wi, o in zip(w, outs))
    with np.errstate(divide="ignore"):
        return out, top + np.log(total), away


def evict(kv, table, lengths, weights, keep, recent=0, births=None):
    """(kv, lengths, kept) after eviction, by sorting each request's slots."""
    kv = kv.copy()
    new_lengths, kept_out = [], np.full((len(lengths), keep), -1, np.int32)

    def rows(slot, r):
        page, off = int(table[r, slot // PAGE_SLOTS]), slot % PAGE_SLOTS
        return (page, slice(off * TOKEN_STRIDE, (off + 1) * TOKEN_STRIDE),
                slice(SCALE_BASE + off * SCALE_DIM, SCALE_BASE + (off + 1) * SCALE_DIM))

    for r, n in enumerate(int(x) for x in lengths):
        new = min(n, keep)
        w = weights[r, :n].astype(np.float64)
        protected = np.zeros(n, bool)
        if births is not None and recent > 0 and n:
            b = births[r, :n].astype(np.int64)
            protected = b > b.max() - recent
        order = sorted(range(n), key=lambda i: (not protected[i],
                                                0.0 if protected[i] else (1 if np.isnan(w[i]) else 0),
                                                0.0 if protected[i] or np.isnan(w[i]) else -w[i], i))
        stay = set(order[:new])
        holes = [i for i in range(new) if i not in stay]
        movers = sorted(i for i in stay if i >= new)
        kept_out[r, :new] = np.arange(new)
        for to, of in zip(holes, movers):
            kept_out[r, to] = of
            tp, ta, tb = rows(to, r)
            fp, fa, fb = rows(of, r)
            kv[tp, ta], kv[tp, tb] = kv[fp, fa], kv[fp, fb]
        new_lengths.append(new)
    return kv, np.array(new_lengths, np.int32), kept_out
