"""Paged 8-bit caches for the tests of the softmax layers' operators, made on the host, and comparisons with the
definitions in 64 bits."""
from __future__ import annotations

import numpy as np
import torch

from gdn_speculative_tree_gb300 import binding
from oracle import attend_oracle as orc

E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(x):
    return x.detach().cpu().to(torch.float64).numpy()


def rows(T, heads, d, dtype, pad, g, size=1.0, shift=0):
    """[T][heads][d] on the GPU; `pad` NaN elements between the token rows, the first `shift` elements in."""
    x = (torch.randn(T, heads, d, generator=g) * size).to(dtype)
    wide = torch.full((T * (heads * d + pad) + shift,), float("nan"), dtype=dtype)
    out = wide[shift:].view(T, heads * d + pad)[:, :heads * d].view(T, heads, d)
    out.copy_(x)
    dev = wide.cuda()
    return dev[shift:].view(T, heads * d + pad)[:, :heads * d].view(T, heads, d)


class Cache:
    """Pages of random tokens up to each length, their table in random order, anything behind the tokens."""

    def __init__(self, lengths, Hkv, d, page, room=0, seed=0, spread=0.0, pages=None, size=1.0, quick=False):
        r = np.random.RandomState(seed)
        self.lengths, self.P, self.Hkv, self.d = list(lengths), page, Hkv, d
        need = [-(-(n + room) // page) for n in lengths]
        num = pages or sum(need) + 3
        order = r.permutation(num)
        self.table_np = np.full((len(lengths), max([1] + need)), -1, np.int32)
        codes = r.randint(0, 256, (2, num, Hkv, page, d)).astype(np.uint8)  # NaN codes among them
        scale = (2.0 ** r.randint(-30, 30, (2, num, Hkv))).astype(np.float32)
        at = 0
        for i, n in enumerate(lengths):
            self.table_np[i, :need[i]] = order[at:at + need[i]]
            at += need[i]
            for p in range(0 if quick else -(-n // page)):
                m = min(page, n - p * page)
                x = r.randn(2, Hkv, m, d) * size * 2.0 ** (spread * r.randn(2, 1, 1, 1))
                for s in range(2):
                    for h in range(Hkv):
                        f = orc.page_scale(np.abs(x[s, h]).max())
                        scale[s, self.table_np[i, p], h] = f
                        codes[s, self.table_np[i, p], h, :m] = orc.to_e4m3(x[s, h] / f)
        if quick:  # codes of any size but NaN, one exponent's scales: many tokens in little time
            codes = np.where((codes & 127) == 127, 0x30, codes)
            scale = (2.0 ** r.randint(-8, -6, scale.shape)).astype(np.float32)
        self.k, self.v = (torch.from_numpy(c).cuda().view(E4M3) for c in codes)
        self.ks, self.vs = (torch.from_numpy(c).cuda() for c in scale)
        self.table = torch.from_numpy(self.table_np).cuda()
        self.length = torch.tensor(self.lengths, dtype=torch.int32, device="cuda")

    def made(self):
        return binding.make_cache(k=self.k, v=self.v, k_scale=self.ks, v_scale=self.vs, page_table=self.table,
                                  length=self.length)

    def context(self, r, length=None):
        """Keys and values of request r in 64 bits."""
        n = self.lengths[r] if length is None else length
        pages = self.table.cpu().numpy()[r]
        return tuple(orc.gather(c.cpu().view(torch.uint8).numpy(), f64(s), pages, n)
                     for c, s in ((self.k, self.ks), (self.v, self.vs)))


def trees(nodes, kind, seed=0):
    """Parents of each request's nodes."""
    r = np.random.RandomState(seed)
    out = []
    for n in nodes:
        if kind == "chain":
            out.append(np.arange(n) - 1)
        elif kind == "star":
            out.append(np.full(n, -1))
        else:
            out.append(np.array([r.randint(-1, i) if i else -1 for i in range(n)], np.int64))
    return out


class Attend:
    """One call of treewy_attend."""

    def __init__(self, lengths, nodes, *, Hq=4, Hkv=2, d=128, page=64, kind="tree", dtype="bf16", out="bf16", pad=0, shift=0,
                 scale=None, flags=0, max_context=None, max_nodes=None, seed=0, spread=0.0, size=1.0, null_parent=False,
                 quick=False):
        g = torch.Generator().manual_seed(seed)
        self.cache = Cache(lengths, Hkv, d, page, seed=seed, spread=spread, quick=quick)
        self.Hq, self.Hkv, self.d, self.nodes = Hq, Hkv, d, list(nodes)
        self.scale = d ** -0.5 if scale is None else scale
        self.off = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        T = int(self.off[-1])
        self.parents = trees(nodes, kind, seed)
        flat = np.concatenate([np.zeros(0)] + self.parents).astype(np.int32)
        self.parent = None if null_parent else torch.from_numpy(flat).cuda()
        self.node_offset = torch.from_numpy(self.off).cuda()
        t = TYPES[dtype]
        self.q = rows(T, Hq, d, t, pad, g, 1.5 * size, shift)
        self.k = rows(T, Hkv, d, t, pad, g, 1.0, shift)
        self.v = rows(T, Hkv, d, t, pad, g, 1.0, shift)
        self.o = torch.full((T, Hq, d), -7.0, dtype=TYPES[out], device="cuda")
        self.status = torch.zeros(len(nodes), dtype=torch.int32, device="cuda")
        self.more = dict(max_nodes=max_nodes or max([1] + self.nodes), flags=flags,
                         max_context=max([0] + list(lengths)) if max_context is None else max_context)
        self.tensor = dtype == "bf16" and out == "bf16" and d % 16 == 0 and not flags

    def make(self, **more):
        return binding.make_attn(cache=self.cache.made(), node_offset=self.node_offset, parent=self.parent, q=self.q, k=self.k,
                                 v=self.v, o=self.o, status=self.status, scale=self.scale, **{**self.more, **more})

    def run(self, stream=None):
        self.call = self.make()
        binding.treewy_attend(self.call, stream)
        torch.cuda.synchronize()
        return self

    def check(self, requests=None):
        """Each node against the definition.  Tolerances: a score's error is that of its products and of their sum; a
        weight's is that of its score, and on the tensor cores that of its two terms besides."""
        q, k, v, o = (f64(x) for x in (self.q, self.k, self.v, self.o))
        for r in range(len(self.nodes)) if requests is None else requests:
            at = slice(self.off[r], self.off[r + 1])
            if self.nodes[r] == 0:
                continue
            ck, cv = self.cache.context(r)
            want = orc.attend(q[at], k[at], v[at], self.parents[r], ck, cv, self.scale)
            keys, values = np.concatenate([ck, k[at].swapaxes(0, 1)], 1), np.concatenate([cv, v[at].swapaxes(0, 1)], 1)
            n, G = keys.shape[1], self.Hq // self.Hkv
            for h in range(self.Hq):
                size = np.abs(q[at][:, h]) @ np.abs(keys[h // G]).T * self.scale     # sum of |q k|, [N][n]
                score = self.d * 2.0 ** -24 * size.max()                              # f32 sums
                top = np.abs(values[h // G]).max()
                tol = 2 * score + n * 2.0 ** -24
                if self.tensor:
                    # queries, and the draft's keys, to 2^-17 of a row's largest; weights to 2^-8 of themselves or 2^-16
                    # of the largest of their row; the draft's values to 2^-17 of a row's largest
                    lengths = np.abs(keys[h // G]).sum(1).max() * np.abs(q[at][:, h]).max()
                    lengths += np.abs(q[at][:, h]).sum(1).max() * np.abs(keys[h // G]).max()
                    s = q[at][:, h] @ keys[h // G].T * self.scale
                    flat = np.minimum(1.0, n * 2.0 ** -16 / np.exp(s - s.max(1, keepdims=True)).sum(1).min())
                    tol += 2 * self.scale * 2.0 ** -17 * lengths + 2.0 ** -8 + flat + 2.0 ** -17
                err = np.abs(o[at][:, h] - want[:, h])
                half = 2.0 ** -8 if self.o.dtype == torch.bfloat16 else 2.0 ** -24
                assert (err <= tol * top + half * np.abs(want[:, h])).all(), (r, h, err.max(), tol * top)
        return self
