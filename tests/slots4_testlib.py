"""Plain 64-bit forms of 4-bit slots, of vectors written into slots and of rotary
positions, for their tests.

Everything here is numpy, written from the definitions: scales are looked up in
a list of all 256, codes are found among the halves, angles are complex numbers.
"""
from __future__ import annotations

from unittest import mock

import numpy as np

import slots_testlib as plain
from kvc_testlib import PAGE_SLOTS, bf16_bits_to_f32, torch_bf16_bits

STRIDE4, SCALES4, GROUP4 = 352, 16, 32
SCALE_BASE4 = PAGE_SLOTS * STRIDE4
PAGE4_BYTES = PAGE_SLOTS * (STRIDE4 + SCALES4)
SCALE_OF_BYTE = np.array([(1 + b % 8 / 8) * 2.0 ** (b // 8 - 16) for b in range(256)])
HALF_F32 = 2.0 ** -24


def bf16(x):
    """x (fp32) rounded to bf16, as float64."""
    return bf16_bits_to_f32(torch_bf16_bits(np.asarray(x, np.float32))).reshape(np.shape(x)).astype(np.float64)


def codes4(x):
    """(codes -7 .. 7, scale bytes) of the first 448 dims of fp32 vectors [n, 512]."""
    z = bf16(x[:, :448]).reshape(-1, 14, GROUP4)
    z = np.where(np.isnan(z), 0, z)
    byte = np.minimum(255, np.searchsorted(7 * SCALE_OF_BYTE, np.abs(z).max(-1)))
    size = np.abs(z) / SCALE_OF_BYTE[byte][..., None]
    whole = np.floor(np.minimum(size, 7))
    whole += (size - whole >= 0.5) & (whole < 7)
    return np.where(z < 0, -whole, whole).astype(np.int64).reshape(-1, 448), byte.astype(np.uint8)


def codes8(x):
    """(codes -127 .. 127, scale bytes) of 8-bit slots."""
    z = bf16(x[:, :448]).reshape(-1, 7, 64)
    z = np.where(np.isnan(z), 0, z)
    a = np.maximum(np.abs(z).max(-1), np.float64(np.float32(1e-4)))
    powers = 127 * 2.0 ** np.arange(-130, 123)          # the last: what holds infinities
    e = np.minimum(np.searchsorted(powers, a) - 130, 122)
    q = np.minimum(np.floor(np.abs(z) / 2.0 ** e[..., None]), 127)
    return np.where(z < 0, -q, q).astype(np.int64).reshape(-1, 448), (e + 127).astype(np.uint8)


def slot_bytes(x, bits):
    """(payload, scale record) of vectors that are not turned."""
    rope = np.ascontiguousarray(torch_bf16_bits(x[:, 448:]).reshape(-1, 64)).view(np.uint8)
    if bits == 8:
        q, s = codes8(x)
        return np.concatenate([q.astype(np.int8).view(np.uint8), rope], 1), np.concatenate([s, np.zeros((len(x), 1), np.uint8)], 1)
    q, s = codes4(x)
    u = (q + 8).reshape(-1, 56, 4, 2).astype(np.uint32)
    words = sum(u[:, :, i, p] << np.uint32(4 * i + 16 * p) for i in range(4) for p in range(2)).astype("<u4")
    return (np.concatenate([np.ascontiguousarray(words).view(np.uint8), rope], 1),
            np.concatenate([s, np.zeros((len(x), 2), np.uint8)], 1))


def random_cache(rng, pages, lo=90, hi=118):
    """Packed 4-bit pages of random codes, scale bytes lo .. hi and N(0, 1) bf16 words."""
    kv = np.zeros((pages, PAGE4_BYTES), np.uint8)
    rows = kv[:, :SCALE_BASE4].reshape(pages, PAGE_SLOTS, STRIDE4)
    rows[..., :224] = rng.integers(0, 256, rows[..., :224].shape, dtype=np.uint8)
    rope = rng.standard_normal((pages, PAGE_SLOTS, 64)).astype(np.float32)
    rows[..., 224:] = (rope.view(np.uint32) >> 16).astype("<u2").view(np.uint8)
    scales = kv[:, SCALE_BASE4:].reshape(pages, PAGE_SLOTS, SCALES4)
    scales[..., :14] = rng.integers(lo, hi + 1, scales[..., :14].shape, dtype=np.uint8)
    return kv


def decode4(payload, scales):
    """Vectors of 4-bit slots, float64 [n, 512], dim by dim."""
    out = np.empty((len(payload), 512))
    words = np.ascontiguousarray(payload[:, :224]).view("<u4")
    for d in range(448):
        u = words[:, d // 8] >> np.uint32(4 * (d % 8 // 2) + 16 * (d % 2)) & 15
        out[:, d] = (u.astype(np.float64) - 8) * SCALE_OF_BYTE[scales[:, d // GROUP4]]
    out[:, 448:] = bf16_bits_to_f32(np.ascontiguousarray(payload[:, 224:]).view("<u2"))
    return out


def slot_vectors(kv, table_row, length):
    pages = kv[table_row[:-(-length // PAGE_SLOTS)]]
    payload = pages[:, :SCALE_BASE4].reshape(-1, STRIDE4)[:length]
    return decode4(payload, pages[:, SCALE_BASE4:].reshape(-1, SCALES4)[:length])


def attend(*args, **more):
    """plain.attend over 4-bit slots."""
    with mock.patch.object(plain, "slot_vectors", slot_vectors):
        return plain.attend(*args, **more)


def evict(*args, **more):
    """plain.evict over 4-bit slots."""
    with mock.patch.multiple(plain, TOKEN_STRIDE=STRIDE4, SCALE_BASE=SCALE_BASE4, SCALE_DIM=SCALES4):
        return plain.evict(*args, **more)


def table_of(positions, theta=10000.0):
    """cos and sin of so many positions, fp32 [positions, 64]."""
    angle = np.arange(positions)[:, None] * theta ** (-np.arange(32) / 32)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def turn(x, positions, table, axes, inverse=False):
    """(values, tolerances before a last rounding) of rows [t, ..., 64] at positions
    [t, axes], in 64 bits.  Two products and their sum in fp32: half a step each of
    what they are."""
    positions = np.asarray(positions)
    at = (positions[:, None] if positions.ndim == 1 else positions)[:, np.asarray(axes)]
    c, s = table[at, np.arange(32)].astype(np.float64), table[at, 32 + np.arange(32)].astype(np.float64)
    z = x.astype(np.float64).reshape(*x.shape[:-1], 32, 2)
    w = (c + 1j * (-s if inverse else s)).reshape(len(x), *[1] * (x.ndim - 2), 32)
    got = (z[..., 0] + 1j * z[..., 1]) * w
    out = np.stack([got.real, got.imag], -1)
    size = np.stack([np.abs(z[..., 0] * w.real) + np.abs(z[..., 1] * w.imag),
                     np.abs(z[..., 1] * w.real) + np.abs(z[..., 0] * w.imag)], -1)
    tol = HALF_F32 * (size + np.abs(out)) * 1.0001 + 2.0 ** -148
    return out.reshape(x.shape), tol.reshape(x.shape)
