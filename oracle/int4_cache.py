"""The four-bit K/V cache and the pass before it, in float64 numpy.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Written from the
definitions: a row of D values x is held as whole numbers n in 0..15 with an
fp16 scale and zero point,

    zero = min x,  scale = fp16(fp32((max x - zero) / 15)),
    n = (x - zero) / scale to the nearest whole number, halves to even,

packed two to a byte (value 2j in the low half of byte j), and stands for
zero + scale * n.  A pool is uint8 [N, H, B * (D/2 + 4)]: the B rows of a
(block, head), then their B (scale, zero) pairs.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from . import attention


def quantise_rows(x: np.ndarray):
    """(n uint8 [..., D], scale fp16 [...], zero fp16 [...]) of finite fp16 rows x [..., D]."""
    x = np.asarray(x, dtype=np.float16)
    lo, hi = x.min(-1), x.max(-1)
    scale = ((hi.astype(np.float32) - lo.astype(np.float32)) / np.float32(15)).astype(np.float16)
    d = x.astype(np.float64) - lo.astype(np.float64)[..., None]        # exact: 40 bits at most
    s = scale.astype(np.float64)[..., None]
    n = np.floor(d / np.where(s == 0, 1, s))
    n = np.clip(n, 0, 15)
    # n and n + 1 by the exact remainder (n * s has 15 bits)
    r = 2 * (d - n * s)
    n = n + ((r > s) | ((r == s) & (n % 2 == 1)))
    n = np.where(s == 0, 0, np.clip(n, 0, 15))
    return n.astype(np.uint8), scale, lo


def empty_pool(num_blocks: int, num_heads: int, block_size: int, head_dim: int) -> np.ndarray:
    return np.zeros((num_blocks, num_heads, block_size * (head_dim // 2 + 4)), dtype=np.uint8)


def store(pool: np.ndarray, rows: np.ndarray, slots, block_size: int) -> None:
    """rows [T, H, D] to their slots (negative: none), one row at a time."""
    T, H, D = rows.shape
    n, scale, zero = quantise_rows(rows)
    for t in range(T):
        slot = int(slots[t])
        if slot < 0:
            continue
        blk, r = divmod(slot, block_size)
        for h in range(H):
            tile = pool[blk, h]
            tile[r * (D // 2):(r + 1) * (D // 2)] = n[t, h, 0::2] | (n[t, h, 1::2] << 4)
            at = block_size * (D // 2) + 4 * r
            tile[at:at + 4] = np.array([scale[t, h], zero[t, h]], dtype=np.float16).view(np.uint8)


def pool_values(pool: np.ndarray, block_size: int) -> np.ndarray:
    """What every row of a pool stands for: float64 [N, H, B, D]."""
    N, H, tile = pool.shape
    half = tile // block_size - 4
    data = pool[:, :, :block_size * half].reshape(N, H, block_size, half)
    meta = np.ascontiguousarray(pool[:, :, block_size * half:]).view(np.float16).reshape(N, H, block_size, 2)
    n = np.empty((N, H, block_size, 2 * half), dtype=np.float64)
    n[..., 0::2], n[..., 1::2] = data & 15, data >> 4
    meta = meta.astype(np.float64)
    with np.errstate(invalid="ignore"):
        return meta[..., 1:2] + meta[..., 0:1] * n


def paged_decode_attention(q, k_pool, v_pool, block_tables, context_lens, scale, block_size):
    """Decode attention with grouped heads over two four-bit pools: float64 [S, Hq, D]."""
    S, Hq, D = q.shape
    group = Hq // k_pool.shape[1]
    k = np.repeat(pool_values(k_pool, block_size), group, axis=1)
    v = np.repeat(pool_values(v_pool, block_size), group, axis=1)
    return attention.paged_decode_attention(np.asarray(q, np.float64), k, v, block_tables, context_lens, scale)


def prompt_attention(q, k, v, query_start, key_start, scale):
    """Causal attention of packed sequences with grouped heads, float64 [Tq, Hq, D] (rows in no
    sequence are zero)."""
    out = np.zeros(q.shape, dtype=np.float64)
    group = q.shape[1] // k.shape[1]
    for s in range(len(query_start) - 1):
        q0, q1, k0, k1 = (int(x) for x in (query_start[s], query_start[s + 1], key_start[s], key_start[s + 1]))
        ks = np.repeat(k[k0:k1].astype(np.float64), group, axis=1)
        vs = np.repeat(v[k0:k1].astype(np.float64), group, axis=1)
        for i in range(q1 - q0):
            p = (k1 - k0) - (q1 - q0) + i
            out[q0 + i] = attention.contiguous_attention(q[q0 + i], ks[:p + 1], vs[:p + 1], scale)
    return out


def turns_of(inv_freq: float) -> Fraction:
    """inv_freq / (2 pi) turns per position, with 2 pi to 60 digits."""
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021164194989")
    return Fraction(float(inv_freq)) / two_pi


def norm_rope(x, weight, eps, positions, inv_freq, pair_axis, interleaved):
    """x [T, H, D] normalised (where weight is given) and turned; positions [A, T].  The angle of
    position p is taken modulo one turn in exact arithmetic.  Returns (y, |a| + |b| per value)."""
    x = np.asarray(x, dtype=np.float64)
    T, H, D = x.shape
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    y, size = x.copy(), np.abs(x)
    R = 2 * len(inv_freq)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        turns = turns_of(f)
        for t in range(T):
            part = float((int(positions[pair_axis[i], t]) * turns) % 1)
            c, s = math.cos(2 * math.pi * part), math.sin(2 * math.pi * part)
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
        size[:, :, a] = size[:, :, b] = np.abs(x[:, :, a]) + np.abs(x[:, :, b])
    return y, size
