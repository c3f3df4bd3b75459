"""The operators around verification in 64 bits, from their definitions: the
gated delta rule over a sequence's tokens (TreeWY paper §1 Eq. (1)), the norm
and rotation of query and key heads, and moves between state slots.  Plain
numpy; shares nothing with the CUDA library.
"""
from __future__ import annotations

import numpy as np


def extend(S, q, k, v, alpha, beta):
    """One sequence: S [H][dv][dk], q, k [n][Hk][dk], v [n][H][dv], gates
    [n][H].  Returns (o [n][H][dv], the last state)."""
    S = np.array(S, dtype=np.float64)
    n, H, dv = v.shape
    rep = H // q.shape[1]
    o = np.zeros((n, H, dv))
    for t in range(n):
        for h in range(H):
            kt, qt = k[t, h // rep].astype(np.float64), q[t, h // rep].astype(np.float64)
            a, b = float(alpha[t, h]), float(beta[t, h])
            S[h] = a * (S[h] - b * np.outer(S[h] @ kt, kt)) + b * np.outer(v[t, h].astype(np.float64), kt)
            o[t, h] = S[h] @ qt
    return o, S


def norm_rotate(x, norm, eps, weight=None, scale=1.0, rope=None, position=None, interleaved=False, repeat=1):
    """Rows x [T][heads][d] normed, weighted, scaled, rotated and repeated."""
    x = np.asarray(x, dtype=np.float64)
    total = np.square(x).sum(axis=-1, keepdims=True)
    y = scale * x / np.sqrt((total if norm == "l2" else total / x.shape[2]) + eps)
    if weight is not None:
        y = y * np.asarray(weight, dtype=np.float64)
    if rope is not None:
        r = rope.shape[1]
        i = np.arange(r // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        table = np.asarray(rope, dtype=np.float64)[position][:, None]
        c, s = table[..., :r // 2], table[..., r // 2:]
        u, w = y[..., a], y[..., b]
        y[..., a], y[..., b] = u * c - w * s, w * c + u * s
    return np.repeat(y, repeat, axis=1)


def move_slots(pool, src, dst):
    """pool [layers][slots][...]: (the pool after the moves, status per move):
    bit 8 for an index outside the pool, bit 128 for moves that meet."""
    out = pool.copy()
    n, slots = len(src), pool.shape[1]
    status = np.zeros(n, dtype=np.int32)
    for i in range(n):
        if src[i] != dst[i]:
            for j in range(n):
                if j != i and src[j] != dst[j] and (dst[j] == dst[i] or (dst[j] == src[i] and src[i] >= 0)):
                    status[i] |= 128
        if not (-1 <= src[i] < slots and 0 <= dst[i] < slots):
            status[i] |= 8
        if status[i] == 0 and src[i] != dst[i]:
            out[:, dst[i]] = pool[:, src[i]] if src[i] >= 0 else 0
    return out, status
