"""The operators around verification against their definitions in 64 bits.

Tolerances, from the number formats alone.  f32 results of ``treewy_extend``:
a product on the tensor cores takes f32 operands as two bf16 terms, 2^-17 of
an operand off at most, and a pseudo-value passes through at most four such
operands before the state or the output takes it in once more, so with a
factor of two for what a sequence adds up, 2 * 8 * 2^-17 / 2 = 2^-14 of the
largest value.  bf16 results add half a unit of their own last place, 2^-9
relative, doubled (2^-8) because a value beside a rounding boundary may go
the other way.  ``treewy_qk_norm``: 512 f32 roundings at most in a sum of 256
squares weigh half in the root, and a handful follow: 2^-24 * 64 of a row's
largest value covers the sum's error in the mean with room, and bf16 adds
2^-8.  Moves between slots are exact.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gdn_speculative_tree_gb300 import binding
from oracle import serving_oracle as orc

pytestmark = pytest.mark.gpu

F32_TOL = 2.0 ** -14
BF16_TOL = 2.0 ** -8
NORM_TOL = 2.0 ** -18
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(x):
    return x.detach().cpu().to(torch.float64).numpy()


def assert_near(got, ref, tol, rel=0.0, label=""):
    got, ref = f64(got), np.asarray(ref)
    bound = tol * max(float(np.abs(ref).max(initial=0)), 1e-30) + rel * np.abs(ref)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (label, int(bad.sum()), float(np.abs(got - ref).max()), float(np.abs(ref).max()))


# ------------------------------------------------------------------ extend

class Case:
    """Seeded inputs of one treewy_extend call on the GPU."""

    def __init__(self, lens, H=2, Hk=None, dk=128, dv=128, qkv="bf16", out="f32", pool="f32", alpha=(0.9, 0.999),
                 beta=None, fresh=(), pad=0, shift=0, seed=0, max_len=None, slots=None):
        Hk = Hk or H
        g = torch.Generator().manual_seed(seed)
        R, T = len(lens), int(sum(lens))
        self.lens, self.H, self.Hk, self.dk, self.dv = list(lens), H, Hk, dk, dv

        def rows(heads, d, unit):
            x = torch.randn(T, heads, d, generator=g)
            x = (x / x.norm(dim=-1, keepdim=True) if unit else x).to(DT[qkv])
            wide = torch.full((T * (heads * d + pad) + shift,), float("nan"), dtype=DT[qkv], device="cuda")
            view = wide[shift:].view(T, heads * d + pad)[:, :heads * d].view(T, heads, d)
            view.copy_(x)
            return view

        self.q, self.k, self.v = rows(Hk, dk, True), rows(Hk, dk, True), rows(H, dv, False)
        self.alpha = (alpha[0] + (alpha[1] - alpha[0]) * torch.rand(T, H, generator=g)).cuda()
        self.beta = (torch.sigmoid(torch.randn(T, H, generator=g)) if beta is None
                     else torch.full((T, H), float(beta))).cuda()
        num = R + 2
        self.slot = (torch.randperm(num, generator=g)[:R] if slots is None else torch.tensor(slots)).to(torch.int32).cuda()
        self.pool = (0.05 * torch.randn(num, H, dv, dk, generator=g)).to(DT[pool]).cuda()
        self.fresh = torch.zeros(R, dtype=torch.uint8)
        for r in fresh:
            self.fresh[r] = 1
        self.fresh = self.fresh.cuda()
        self.off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
        self.o = torch.full((T, H, dv), 7.0, device="cuda", dtype=DT[out])
        self.status = torch.zeros(R, dtype=torch.int32, device="cuda")
        self.max_len = max(lens, default=0) if max_len is None else max_len
        self.before = self.pool.clone()

    def seqs(self, flags=0):
        return binding.make_seqs(seq_offset=self.off, q=self.q, k=self.k, v=self.v, alpha=self.alpha, beta=self.beta,
                                 state=self.pool, state_slot=self.slot, fresh=self.fresh, o=self.o,
                                 status=self.status, max_len=self.max_len, flags=flags)

    def run(self, flags=0):
        binding.treewy_extend(self.seqs(flags))
        torch.cuda.synchronize()
        return self

    def check(self, skip=()):
        """Outputs and states against the definition; skipped sequences untouched."""
        ref_o = np.full(tuple(self.o.shape), 7.0)
        ref_s = f64(self.before)
        lo = 0
        for r, n in enumerate(self.lens):
            hi = lo + n
            if r not in skip:
                s = int(self.slot[r])
                S = np.zeros_like(ref_s[s]) if int(self.fresh[r]) else ref_s[s]
                ref_o[lo:hi], ref_s[s] = orc.extend(S, f64(self.q[lo:hi]), f64(self.k[lo:hi]), f64(self.v[lo:hi]),
                                                    f64(self.alpha[lo:hi]), f64(self.beta[lo:hi]))
            lo = hi
        assert_near(self.o, ref_o, F32_TOL, BF16_TOL if self.o.dtype == torch.bfloat16 else 0.0, "o")
        assert_near(self.pool, ref_s, F32_TOL, BF16_TOL if self.pool.dtype == torch.bfloat16 else 0.0, "state")
        used = {int(self.slot[r]) for r in range(len(self.lens)) if r not in skip
                and (self.lens[r] > 0 or int(self.fresh[r]))}
        for s in range(self.pool.shape[0]):
            if s not in used:
                assert torch.equal(self.pool[s], self.before[s]), f"slot {s} was written"
        return self


@pytest.mark.parametrize("pool", ["f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[1], [1, 1, 0, 1, 1], [2], [3, 17], [63], [64], [65], [128, 0, 1, 129, 66],
                                  [300, 191]])
def test_extend_lengths(cuda_lib, lens, out, pool):
    Case(lens, H=3, out=out, pool=pool, seed=len(lens) + sum(lens)).run().check()


@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 1), (6, 2), (4, 4)])
@pytest.mark.parametrize("n", [1, 150])
def test_extend_shared_key_heads(cuda_lib, H, Hk, n):
    Case([n, max(1, n // 3)], H=H, Hk=Hk, seed=H * 10 + Hk).run().check()


@pytest.mark.parametrize("dk,dv", [(1, 1), (16, 16), (64, 64), (48, 80), (80, 48), (7, 128), (128, 5), (100, 36)])
@pytest.mark.parametrize("qkv,pool", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
def test_extend_head_sizes(cuda_lib, dk, dv, qkv, pool):
    Case([1], dk=dk, dv=dv, qkv=qkv, pool=pool, seed=dk).run().check()
    Case([70, 1, 0, 33], dk=dk, dv=dv, qkv=qkv, pool=pool, seed=dv).run().check()


@pytest.mark.parametrize("n", [1, 90])
@pytest.mark.parametrize("pad,shift", [(8, 0), (64, 8), (3, 0), (0, 1), (5, 3)])
def test_extend_strides_and_alignment(cuda_lib, n, pad, shift):
    Case([n, n], H=2, Hk=1, pad=pad, shift=shift, seed=pad + shift).run().check()
    Case([n, n], H=2, Hk=1, pad=pad, shift=shift, seed=pad + shift, qkv="f32").run().check()


@pytest.mark.parametrize("n", [1, 100])
@pytest.mark.parametrize("alpha", [(0.0, 0.0), (1.0, 1.0), (1e-30, 1e-3), (0.0, 1.0), (1e-45, 1e-44)])
@pytest.mark.parametrize("beta", [0.0, 1.0, None])
def test_extend_extreme_gates(cuda_lib, n, alpha, beta):
    c = Case([n, n], alpha=alpha, beta=beta, seed=3)
    if alpha == (0.0, 1.0) and n > 1:  # resets inside a chunk
        c.alpha[::7] = 0.0
    c.run().check()


@pytest.mark.parametrize("n", [0, 1, 80])
def test_extend_fresh_state_is_not_read(cuda_lib, n):
    c = Case([n, n, n], fresh=(0, 2), seed=4)
    c.pool[c.slot[0].long()] = float("nan")
    c.pool[c.slot[2].long()] = float("inf")
    c.before = c.pool.clone()
    clean = c.before.clone()
    clean[c.slot[0].long()] = 0
    clean[c.slot[2].long()] = 0
    c.run()
    c.before = clean
    c.check()


@pytest.mark.parametrize("n", [1, 70])
def test_extend_nan_stays_in_its_sequence(cuda_lib, n):
    """NaN in one sequence's inputs reaches no other sequence or head."""
    c = Case([n, n, n], H=2, seed=5)
    c.v[n:2 * n, 1] = float("nan")
    c.run()
    ok = Case([n, n, n], H=2, seed=5).run()
    assert torch.equal(c.o[:n], ok.o[:n]) and torch.equal(c.o[2 * n:], ok.o[2 * n:])
    assert torch.equal(c.o[n:2 * n, 0], ok.o[n:2 * n, 0])
    assert torch.isnan(c.o[n:2 * n, 1]).any()
    assert torch.equal(c.pool[c.slot[1].long(), 0], ok.pool[c.slot[1].long(), 0])


@pytest.mark.parametrize("n", [1, 2, 70])
def test_extend_infinite_rows_past_a_sequence(cuda_lib, n):
    """A sequence's last chunk reaches over its neighbour's rows: nothing of them comes in."""
    c = Case([n, 3], H=1, seed=6)
    c.q[n:], c.k[n:], c.v[n:] = float("inf"), float("nan"), float("inf")
    c.alpha[n:], c.beta[n:] = float("nan"), float("nan")
    c.run()
    ok = Case([n, 3], H=1, seed=6).run()
    assert torch.equal(c.o[:n], ok.o[:n])
    assert torch.equal(c.pool[c.slot[0].long()], ok.pool[c.slot[0].long()])


@pytest.mark.parametrize("n", [1, 90])
def test_extend_bad_sequences_are_skipped(cuda_lib, n):
    c = Case([n, n, n, n], seed=7, max_len=n)
    c.slot[1] = 99
    c.run().check(skip=(1,))
    assert c.status.tolist() == [0, binding.STATUS_BAD_SLOT, 0, 0]
    c = Case([n, n + 1, n], seed=7, max_len=n).run().check(skip=(1,))
    assert c.status.tolist() == [0, binding.STATUS_TOO_MANY_NODES, 0]
    c = Case([n, n], seed=7, max_len=n)
    c.off[2] += 1
    c.max_len += 1
    c.run().check(skip=(1,))
    assert c.status.tolist() == [0, binding.STATUS_BAD_TREE]
    c = Case([n, n], seed=7, max_len=n)
    c.off[0] = -1
    c.max_len += 1
    c.run().check(skip=(0,))
    assert c.status.tolist() == [binding.STATUS_BAD_TREE, 0]
    c = Case([n, n, n], seed=7, max_len=2 * n)
    c.off[1] = 3 * n  # lengths 3n, -n, n
    c.run()
    assert c.status.tolist() == [binding.STATUS_TOO_MANY_NODES, binding.STATUS_TOO_MANY_NODES, 0]


def test_extend_bound_above_the_lengths(cuda_lib):
    Case([1, 1, 0], max_len=5000, seed=8).run().check()
    Case([0, 0], max_len=0, fresh=(1,), seed=8).run().check()


def test_extend_in_pieces_equals_whole(cuda_lib):
    """A prompt in two chunks and a decode step is the prompt in one go."""
    n = 200
    whole = Case([n], H=2, seed=9, fresh=(0,)).run()
    part = Case([n], H=2, seed=9, fresh=(0,))
    for lo, hi in ((0, 77), (77, 199), (199, 200)):
        off = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        binding.treewy_extend(binding.make_seqs(
            seq_offset=off, q=part.q[lo:hi], k=part.k[lo:hi], v=part.v[lo:hi], alpha=part.alpha[lo:hi],
            beta=part.beta[lo:hi], state=part.pool, state_slot=part.slot, fresh=part.fresh, o=part.o[lo:hi],
            status=part.status, max_len=hi - lo))
        part.fresh.zero_()
    torch.cuda.synchronize()
    assert_near(part.o, f64(whole.o), F32_TOL)
    assert_near(part.pool, f64(whole.pool), F32_TOL)


@pytest.mark.parametrize("n", [1, 140])
def test_extend_forced_generic_and_repeatable(cuda_lib, n):
    a = Case([n, 5], H=2, seed=10).run()
    b = Case([n, 5], H=2, seed=10).run()
    assert torch.equal(a.o, b.o) and torch.equal(a.pool, b.pool)
    Case([n, 5], H=2, seed=10).run(binding.FLAG_FORCE_GENERIC).check()


@pytest.mark.parametrize("n", [1, 140])
def test_extend_on_another_stream_and_in_a_graph(cuda_lib, n):
    ref = Case([n], seed=11).run()
    c = Case([n], seed=11)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    binding.treewy_extend(c.seqs(), side)
    side.synchronize()
    assert torch.equal(c.o, ref.o) and torch.equal(c.pool, ref.pool)
    c = Case([n], seed=11)
    s = c.seqs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.treewy_extend(s)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.o, ref.o) and torch.equal(c.pool, ref.pool)


def test_extend_many_sequences(cuda_lib):
    lens = [int(x) for x in np.random.RandomState(1).randint(0, 90, 120)]
    Case(lens, H=3, Hk=1, out="bf16", seed=12, fresh=range(0, 120, 3)).run().check()
    Case([1] * 200, H=3, Hk=1, out="bf16", seed=12).run().check()


def test_extend_long_sequence(cuda_lib):
    Case([3001], H=1, seed=13, alpha=(0.98, 0.9999)).run().check()


def test_extend_rows_past_32_bit_offsets(cuda_lib):
    """Token rows whose element offsets pass 2^31."""
    c = Case([1, 40], H=1, seed=14)
    wide = 70_000_000
    rows = []
    for x in (c.q, c.k, c.v):
        big = torch.empty(40 * wide + 128, dtype=torch.bfloat16, device="cuda")
        view = big.as_strided((41, 1, 128), (wide, 128, 1))
        view.copy_(x)
        rows.append(view)
    c.q, c.k, c.v = rows
    c.run().check()


def test_extend_feeds_verification(cuda_lib):
    """A chain of draft nodes verified from the state that extend left equals extending over them."""
    n, m = 100, 6
    c = Case([n], H=2, seed=15).run().check()
    d = Case([m], H=2, seed=16)
    d.pool[:] = c.pool
    slot = c.slot.clone()
    o, U = torch.empty_like(d.o), torch.empty_like(d.o)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    parent = torch.arange(-1, m - 1, dtype=torch.int32, device="cuda")
    b = binding.make_batch(node_offset=d.off, parent=parent, q=d.q.contiguous(), k=d.k.contiguous(),
                           v=d.v.contiguous(), alpha=d.alpha, beta=d.beta, state=c.pool, state_slot=slot, o=o, U=U,
                           status=status, max_nodes=m)
    binding.treewy_verify(b)
    binding.treewy_commit(b, torch.tensor([m - 1], dtype=torch.int32, device="cuda"))
    d.slot = slot
    d.run()
    # the verification's own bounds: 2e-3 of the outputs, 1e-3 of the state
    assert_near(o, f64(d.o), 2e-3)
    assert_near(c.pool, f64(d.pool), 1e-3)


@pytest.mark.parametrize("n", [1, 26, 70])
def test_extend_f32_outputs_over_a_rounded_state(cuda_lib, n):
    """A second call on the bf16 state that the first one rounded, its outputs in f32.

    An error e of the state lets a share e / 2^-8 of its values, doubled, round the other way, each 2^-8 off:
    eight f32 roundings, e = 2^-21 at most and 2^-22 in the mean, give sqrt(2^-13) 2^-8 of the state, and of the
    outputs read from it, in the norm: 2^-14.5, below 2^-14."""
    c = Case([n, n], H=8, alpha=(0.97, 0.999), out="f32", pool="bf16", seed=17)
    S = f64(c.pool)
    ref = np.zeros(tuple(c.o.shape))
    for _ in range(2):
        c.run()
        for r in range(2):
            s, rows = int(c.slot[r]), slice(r * n, (r + 1) * n)
            ref[rows], new = orc.extend(S[s], f64(c.q[rows]), f64(c.k[rows]), f64(c.v[rows]), f64(c.alpha[rows]),
                                        f64(c.beta[rows]))
            S[s] = f64(torch.from_numpy(new).to(torch.bfloat16))
    assert np.linalg.norm(f64(c.o) - ref) <= 2.0 ** -14 * np.linalg.norm(ref)


@pytest.mark.parametrize("R", [128, 129])
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
def test_extend_order_of_sequences(cuda_lib, R, qkv):
    """Equal, empty and refused lengths among as many sequences as are put in order, and one more."""
    lens = [int(x) for x in np.random.RandomState(2).choice([0, 1, 7, 40, 40, 66], R)]
    c = Case(lens, H=1, dk=32, dv=32, qkv=qkv, seed=21, max_len=60).run()
    bad = [r for r, n in enumerate(lens) if n > 60]
    c.check(skip=bad)
    assert c.status.tolist() == [binding.STATUS_TOO_MANY_NODES if r in bad else 0 for r in range(R)]


@pytest.mark.parametrize("lens", [[5, 0, 9, 16], [17, 3, 0, 38]])
@pytest.mark.parametrize("H", [1, 24])
@pytest.mark.parametrize("dk,dv", [(128, 128), (52, 71)])
@pytest.mark.parametrize("qkv,pool", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
def test_extend_token_by_token_splits(cuda_lib, lens, H, dk, dv, qkv, pool):
    """Few and many heads, below and above the lengths that are staged."""
    Case(lens, H=H, dk=dk, dv=dv, qkv=qkv, pool=pool, fresh=(2,), seed=18).run(binding.FLAG_FORCE_GENERIC).check()


@pytest.mark.parametrize("n", [9, 30])
@pytest.mark.parametrize("what", ["k", "v", "alpha"])
@pytest.mark.parametrize("at", [4, 6, 8])
def test_extend_token_by_token_nan_goes_forward_only(cuda_lib, n, what, at):
    ok = Case([n], H=2, seed=19).run(binding.FLAG_FORCE_GENERIC)
    c = Case([n], H=2, seed=19)
    getattr(c, what)[at] = float("nan")
    c.run(binding.FLAG_FORCE_GENERIC)
    assert torch.equal(c.o[:at], ok.o[:at]) and torch.isnan(c.o[at:]).all()


@pytest.mark.parametrize("n", [3, 18])
def test_extend_token_by_token_infinite_last_token(cuda_lib, n):
    """What fills a block of tokens up behind a sequence's end adds nothing, not even to an infinite state."""
    c = Case([n], H=1, seed=20)
    c.alpha[n - 1], c.beta[n - 1], c.v[n - 1] = 1.0, 1.0, float("inf")
    c.k[n - 1] = 0
    c.k[n - 1, :, 5] = 1.0
    before = Case([n - 1], H=1, seed=20)
    for x in ("q", "k", "v", "alpha", "beta"):
        getattr(before, x).copy_(getattr(c, x)[:n - 1])
    before.pool.copy_(c.before)
    before.slot = c.slot
    before.run(binding.FLAG_FORCE_GENERIC)
    c.run(binding.FLAG_FORCE_GENERIC)
    got, ref = c.pool[c.slot[0].long(), 0], before.pool[c.slot[0].long(), 0]
    assert torch.isinf(got[:, 5]).all() and torch.isnan(got[:, [4, 6]]).all()
    assert torch.isfinite(ref).all()


# ------------------------------------------------------------------ qk_norm

def qk_case(T, Hq, Hk, d, dtype="bf16", norm="l2", rope=0, interleaved=False, repeat=(1, 1), pad=0, shift=0,
            weight=False, eps=1e-6, scale=(1.0, 1.0), seed=0, inplace=False):
    g = torch.Generator().manual_seed(seed)

    def rows(heads):
        x = (3 * torch.randn(T, heads, d, generator=g)).to(DT[dtype])
        if T > 2:
            x[1] = 0  # rows of zeros
        wide = torch.full((T * (heads * d + pad) + shift,), float("nan"), dtype=DT[dtype], device="cuda")
        view = wide[shift:].view(T, heads * d + pad)[:, :heads * d].view(T, heads, d)
        view.copy_(x)
        return view

    q, k = rows(Hq), rows(Hk)
    w = [torch.randn(d, generator=g).cuda() if weight else None for _ in range(2)]
    tab = pos = None
    if rope:
        ang = torch.rand(50, rope // 2, generator=g, dtype=torch.float64) * 6
        tab = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
        pos = torch.randint(0, 50, (T,), generator=g, dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = [orc.norm_rotate(f64(x), norm, eps, None if y is None else f64(y), s, None if tab is None else f64(tab),
                           None if pos is None else pos.cpu().numpy(), interleaved, r)
           for x, y, s, r in zip((q, k), w, scale, repeat)]
    outs = [q, k] if inplace else [torch.full((T, h * r, d), 7.0, device="cuda", dtype=DT[dtype])
                                   for h, r in zip((Hq, Hk), repeat)]
    binding.treewy_qk_norm(binding.make_qk(
        q=q, k=k, q_out=outs[0], k_out=outs[1], norm=norm, eps=eps, q_weight=w[0], k_weight=w[1], q_scale=scale[0],
        k_scale=scale[1], rope=tab, position=pos, interleaved=interleaved, status=status))
    torch.cuda.synchronize()
    assert int(status) == 0
    for got, want, label in zip(outs, ref, "qk"):
        assert_near(got, want, NORM_TOL, BF16_TOL if dtype == "bf16" else 0.0, label)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [1, 8, 64, 72, 80, 100, 128, 200, 255, 256])
@pytest.mark.parametrize("norm", ["l2", "rms"])
def test_qk_norm_sizes(cuda_lib, dtype, d, norm):
    qk_case(5, 3, 2, d, dtype, norm, weight=norm == "rms", scale=(0.25, 1.0), seed=d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rope", [(64, 64), (64, 16), (128, 32), (128, 128), (256, 64), (256, 256), (80, 80),
                                    (80, 20), (128, 2), (128, 126), (66, 66), (256, 240)])
def test_qk_norm_rotation(cuda_lib, dtype, interleaved, d, rope):
    qk_case(7, 4, 1, d, dtype, "rms", rope=rope, interleaved=interleaved, weight=True, seed=rope)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (16, 8), (1, 0), (0, 1), (200, 0)])
def test_qk_norm_strides(cuda_lib, dtype, pad, shift):
    qk_case(9, 2, 3, 128, dtype, pad=pad, shift=shift, rope=64, seed=pad)


@pytest.mark.parametrize("T", [0, 1, 2, 63, 300])
@pytest.mark.parametrize("repeat", [(1, 1), (2, 2), (3, 1)])
def test_qk_norm_tokens_and_repeats(cuda_lib, T, repeat):
    qk_case(T, 4, 2, 128, repeat=repeat, seed=T)


@pytest.mark.parametrize("d,rope", [(128, 32), (100, 20)])
def test_qk_norm_in_place(cuda_lib, d, rope):
    qk_case(33, 4, 2, d, rope=rope, inplace=True, seed=1)


def test_qk_norm_one_side_only(cuda_lib):
    x = torch.randn(6, 2, 128, device="cuda")
    for side in ("q", "k"):
        out = torch.empty_like(x)
        binding.treewy_qk_norm(binding.make_qk(**{side: x, side + "_out": out}))
        torch.cuda.synchronize()
        assert_near(out, orc.norm_rotate(f64(x), "l2", 1e-6), NORM_TOL)


@pytest.mark.parametrize("d", [128, 100])
def test_qk_norm_bad_positions(cuda_lib, d):
    x = torch.randn(5, 2, d, device="cuda")
    tab = torch.cat([torch.ones(4, 16), torch.zeros(4, 16)], 1).cuda()
    pos = torch.tensor([0, 4, 1, -1, 3], dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.treewy_qk_norm(binding.make_qk(q=x, q_out=out, rope=tab, position=pos, status=status))
    torch.cuda.synchronize()
    assert int(status) == binding.STATUS_BAD_POSITION
    ref = orc.norm_rotate(f64(x), "l2", 1e-6)
    ref[[1, 3]] = 7.0
    assert_near(out, ref, NORM_TOL)


def test_qk_norm_extreme_rows(cuda_lib):
    """Rows whose squares leave f32 behave as the formula in f32 does; others are untouched by them."""
    x = torch.randn(4, 1, 128, device="cuda")
    x[1] = float("nan")
    x[2, 0, 5] = float("inf")
    out = torch.empty_like(x)
    binding.treewy_qk_norm(binding.make_qk(k=x, k_out=out))
    torch.cuda.synchronize()
    assert torch.isnan(out[1]).all() and torch.isnan(out[2, 0, 5])
    assert (out[2, 0, :5] == 0).all()
    assert_near(out[[0, 3]], orc.norm_rotate(f64(x[[0, 3]]), "l2", 1e-6), NORM_TOL)


# ------------------------------------------------------------------ copy_slots

def slots_case(src, dst, slots=9, layers=2, shape=(2, 8, 16), dtype=torch.float32, stride=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    pool = torch.randn(layers, slots + stride, *shape, generator=g).to(dtype).cuda()[:, :slots]
    before = pool.clone()
    status = torch.zeros(len(src), dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    binding.treewy_copy_slots(binding.make_slots(state=pool, src=torch.tensor(src, **i32),
                                                 dst=torch.tensor(dst, **i32), status=status, layers=layers))
    torch.cuda.synchronize()
    ref, bits = orc.move_slots(f64(before), src, dst)
    assert status.tolist() == bits.tolist()
    np.testing.assert_array_equal(f64(pool), ref)
    return bits


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(2, 8, 16), (1, 1), (3, 5), (7,), (1, 128, 128), (3, 128, 128)])
@pytest.mark.parametrize("src,dst", [([0], [1]), ([0, 0, 0], [1, 5, 8]), ([3, 7, -1, 2], [0, 1, 4, 6]), ([], []),
                                     ([-1], [8])])
def test_copy_slots(cuda_lib, dtype, shape, src, dst):
    bits = slots_case(src, dst, shape=shape, dtype=dtype)
    assert not bits.any()


@pytest.mark.parametrize("src,dst", [
    ([0, 1], [1, 2]),            # a source that is written
    ([0, 1], [1, 0]),            # a swap
    ([0, 3], [5, 5]),            # one destination twice
    ([0, -1], [5, 5]), ([0, -1], [5, 0]),
    ([9, 0], [1, 2]), ([0], [9]), ([-2], [1]), ([0], [-1]),
    ([4, 4], [4, 2]), ([4, 3], [4, 4]), ([9], [9]),   # moves onto themselves
    ([9, 1], [1, 3]),            # a move that is not made still counts
])
def test_copy_slots_refusals(cuda_lib, src, dst):
    slots_case(src, dst)


def test_copy_slots_many_and_strided(cuda_lib):
    rng = np.random.RandomState(0)
    at = rng.permutation(700)
    src, dst = [int(x) for x in at[:300]], [int(x) for x in at[300:600]]
    src[::11] = [-1] * len(src[::11])
    assert not slots_case(src, dst, slots=700, layers=3, shape=(1, 4, 4), stride=5).any()


def test_copy_slots_past_4_gb(cuda_lib):
    """Blocks whose byte offsets pass 2^32."""
    pool = torch.zeros(5, 1 << 28, device="cuda")
    pool[4, -7:] = 3.0
    pool[0, :5] = 2.0
    i32 = dict(dtype=torch.int32, device="cuda")
    status = torch.zeros(2, **i32)
    binding.treewy_copy_slots(binding.make_slots(state=pool, src=torch.tensor([4, 0], **i32),
                                                 dst=torch.tensor([1, 3], **i32), status=status))
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0]
    assert torch.equal(pool[1], pool[4]) and torch.equal(pool[3], pool[0]) and float(pool[2].abs().max()) == 0.0
