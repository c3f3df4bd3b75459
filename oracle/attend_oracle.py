"""Attention over an 8-bit paged cache, the cache's append and the residual
norm, from their definitions in 64 bits (numpy, one request at a time).

``attend``: o_n = sum_j softmax_j(scale q_n . k_j) v_j over the context and the
nodes on n's path.  ``append``: rows into pages of e4m3 codes with a power of
two as the scale of each page and head.  ``add_norm``: z = x + residual,
y = w z / sqrt(mean z^2 + eps), and y in e4m3 with a scale per row or group.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
LEAST_EXPONENT = -40


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes: sign, four bits of exponent (bias 7), three of significand; 127 is NaN."""
    code = np.arange(256)
    exponent, part = (code >> 3) & 15, code & 7
    size = np.where(exponent == 0, part * 2.0 ** -9, (8 + part) * 2.0 ** (exponent - 10.0))
    size[(code & 127) == 127] = np.nan
    return np.where(code >= 128, -size, size)


_VALUES = e4m3_values()
_SORTED = np.arange(127)  # codes of the values 0 .. 448, ascending


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """Codes of x, rounded to nearest (ties to the even code), beyond 448 to 448; what is not finite becomes NaN."""
    x = np.asarray(x, np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    up = np.searchsorted(_VALUES[_SORTED], a).clip(0, 126)
    down = (up - 1).clip(0)
    lo, hi = a - _VALUES[down], _VALUES[up] - a
    take = (hi < lo) | ((hi == lo) & (up % 2 == 0)) | (up == 0)
    code = np.where(take, up, down)
    code = np.where(a >= E4M3_MAX, 126, code)
    code = np.where(np.isfinite(x), code, 127)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def from_e4m3(code: np.ndarray) -> np.ndarray:
    return _VALUES[code]


def page_scale(amax: float) -> float:
    """The least power of two, 2^-40 at least, with amax <= 448 times it."""
    e = LEAST_EXPONENT
    while amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def path(parent, node: int) -> list:
    """The nodes from the root to ``node``."""
    out = []
    while node >= 0:
        out.append(node)
        node = int(parent[node])
    return out[::-1]


def gather(codes, scale, pages, length: int) -> np.ndarray:
    """[heads][length][d] of a cache's codes [num_pages][heads][page_len][d] and scales [num_pages][heads]."""
    P = codes.shape[2]
    pages = np.asarray(pages[:-(-length // P)], np.int64)
    x = from_e4m3(codes[pages]) * np.asarray(scale, np.float64)[pages][..., None, None]
    return x.transpose(1, 0, 2, 3).reshape(codes.shape[1], -1, codes.shape[3])[:, :length]


def attend(q, k, v, parent, context_k, context_v, scale: float) -> np.ndarray:
    """q [N][Hq][d], k and v [N][Hkv][d] of one request's nodes, the context [Hkv][length][d]; o [N][Hq][d]."""
    N, Hq, d = q.shape
    G = Hq // k.shape[1]
    o = np.zeros((N, Hq, d))
    for n in range(N):
        on = path(parent, n)
        for h in range(Hq):
            keys = np.concatenate([context_k[h // G], k[on, h // G]])
            values = np.concatenate([context_v[h // G], v[on, h // G]])
            s = keys @ q[n, h] * scale
            w = np.exp(s - s.max())
            o[n, h] = w @ values / w.sum()
    return o


def append(codes, scale, pages, length: int, rows) -> None:
    """Rows [m][heads][d] behind a request's tokens, in place: codes uint8, scales float64."""
    P = codes.shape[2]
    m, at = rows.shape[0], 0
    while at < m:
        page, lo = int(pages[(length + at) // P]), (length + at) % P
        n = min(P - lo, m - at)
        for h in range(codes.shape[1]):
            new = rows[at:at + n, h]
            finite = np.abs(new[np.isfinite(new)])
            amax = float(finite.max()) if finite.size else 0.0
            was = float(scale[page, h])
            now = page_scale(amax) if lo == 0 else was if amax <= E4M3_MAX * was else max(was, page_scale(amax))
            if lo and now != was:
                codes[page, h, :lo] = to_e4m3(from_e4m3(codes[page, h, :lo]) * (was / now))
            codes[page, h, lo:lo + n] = to_e4m3(new / now)
            scale[page, h] = now
        at += n


def add_norm(x, residual, weight, eps: float):
    """z and y of the rows [T][n]."""
    z = x + residual if residual is not None else x
    y = z / np.sqrt((z * z).mean(axis=1, keepdims=True) + eps)
    return z, y * weight if weight is not None else y


def group_scales(y, group: int) -> np.ndarray:
    """Each row's scales: the largest |y| of every group of columns (0: the row) over 448, 2^-126 at least, 1 where that is 0."""
    n = y.shape[1]
    group = group or n
    top = np.stack([np.abs(y[:, i:i + group]).max(axis=1) for i in range(0, n, group)], axis=1)
    return np.where(top > 0, np.maximum(top / E4M3_MAX, 2.0 ** -126), 1.0)
