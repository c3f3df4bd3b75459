"""The operators around verification over more of their range: f32 rows over a bf16 pool, and more rows of
treewy_qk_norm than there are warps, so that a warp takes several parts of tokens in turn."""
from __future__ import annotations

import pytest
import torch

from gdn_speculative_tree_gb300 import binding
from oracle import serving_oracle as orc
from tests.test_gpu_serving import BF16_TOL, DT, NORM_TOL, Case, assert_near, f64

pytestmark = pytest.mark.gpu

# -------------------------------------------------- f32 q, k and v over a bf16 pool

@pytest.mark.parametrize("dk,dv", [(16, 16), (64, 64), (7, 128), (128, 5), (100, 36), (128, 128)])
def test_extend_f32_rows_over_a_bf16_pool(cuda_lib, dk, dv):
    Case([1, 1, 0], dk=dk, dv=dv, qkv="f32", pool="bf16", seed=dk).run().check()
    Case([70, 1, 0, 33], dk=dk, dv=dv, qkv="f32", pool="bf16", seed=dv).run().check()


@pytest.mark.parametrize("lens", [[5, 0, 9, 16], [17, 3, 0, 38]])
@pytest.mark.parametrize("H", [1, 24])
@pytest.mark.parametrize("dk,dv", [(128, 128), (52, 71)])
def test_extend_f32_rows_over_a_bf16_pool_splits(cuda_lib, lens, H, dk, dv):
    Case(lens, H=H, dk=dk, dv=dv, qkv="f32", pool="bf16", fresh=(2,), seed=34).run().check()


@pytest.mark.parametrize("n", [1, 6, 90])
@pytest.mark.parametrize("pad,shift", [(4, 0), (64, 4), (3, 0), (0, 1), (5, 3)])
def test_extend_f32_rows_over_a_bf16_pool_strides(cuda_lib, n, pad, shift):
    Case([n, n], H=2, Hk=1, qkv="f32", pool="bf16", pad=pad, shift=shift, seed=pad + shift).run().check()


# -------------------------------------------------- a step of prompts and single tokens as two calls

@pytest.mark.parametrize("pool", ["f32", "bf16"])
def test_extend_prompts_and_single_tokens_in_two_calls(cuda_lib, pool):
    c = Case([200, 90, 1, 1, 0, 1], H=4, Hk=2, out="bf16", pool=pool, fresh=(1, 3), seed=35)
    for lo, hi, most in ((0, 2, 200), (2, 6, 1)):
        binding.treewy_extend(binding.make_seqs(
            seq_offset=c.off[lo:hi + 1], q=c.q, k=c.k, v=c.v, alpha=c.alpha, beta=c.beta, state=c.pool,
            state_slot=c.slot[lo:hi], fresh=c.fresh[lo:hi], o=c.o, status=c.status[lo:hi], max_len=most))
    torch.cuda.synchronize()
    c.check()
    assert c.status.tolist() == [0] * 6


# -------------------------------------------------- qk_norm: several parts of tokens per warp

def norm_case(dtype, d, Hq, Hk, T, rope, interleaved, norm="rms", repeat=1, pad=0):
    g = torch.Generator().manual_seed(d + Hq)

    def rows(heads):
        wide = (3 * torch.randn(T, heads * d + pad, generator=g)).to(DT[dtype]).cuda()
        return wide[:, :heads * d].view(T, heads, d)

    q, k = rows(Hq), rows(Hk)
    w = [torch.randn(d, generator=g).cuda() for _ in range(2)]
    ang = 6 * torch.rand(50, rope // 2, generator=g, dtype=torch.float64)
    tab = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    pos = torch.randint(0, 50, (T,), generator=g, dtype=torch.int32)
    bad = torch.randperm(T, generator=g)[:T // 50]
    pos[bad] = torch.where(bad % 2 == 0, -1, 50).int()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.full((T, h * repeat, d), 7.0, device="cuda", dtype=DT[dtype]) for h in (Hq, Hk)]
    binding.treewy_qk_norm(binding.make_qk(q=q, k=k, q_out=outs[0], k_out=outs[1], norm=norm, q_weight=w[0],
                                           k_weight=w[1], q_scale=0.5, rope=tab, position=pos.cuda(),
                                           interleaved=interleaved, status=status))
    torch.cuda.synchronize()
    assert int(status) == binding.STATUS_BAD_POSITION
    safe = pos.clone()
    safe[bad] = 0
    for x, y, out, scale, label in ((q, w[0], outs[0], 0.5, "q"), (k, w[1], outs[1], 1.0, "k")):
        ref = orc.norm_rotate(f64(x), norm, 1e-6, f64(y), scale, f64(tab), safe.numpy(), interleaved, repeat)
        ref[bad.numpy()] = 7.0
        assert_near(out, ref, NORM_TOL, BF16_TOL if dtype == "bf16" else 0.0, label)


# heads per part: bf16 8, 16 and 32 of 256, 128 and 64 elements, f32 half of that; so two parts of q and one of k, the
# last ones not full, over about twice as many parts as there are warps (4,256: no multiple of 3)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,d,Hq,Hk", [("bf16", 256, 12, 5), ("bf16", 128, 20, 7), ("bf16", 64, 40, 9),
                                           ("f32", 256, 6, 3), ("f32", 128, 10, 3), ("f32", 64, 20, 5)])
def test_qk_norm_many_rows(cuda_lib, dtype, d, Hq, Hk, interleaved):
    norm_case(dtype, d, Hq, Hk, 3001, d // 4, interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hk,rope,interleaved", [(10, 3, 20, False), (34, 9, 20, True), (10, 3, 80, True)])
def test_qk_norm_many_rows_odd_pairs(cuda_lib, dtype, Hq, Hk, rope, interleaved):
    norm_case(dtype, 80, Hq, Hk, 3001, rope, interleaved, norm="l2")


def test_qk_norm_many_rows_repeated_and_strided(cuda_lib):
    norm_case("bf16", 128, 33, 2, 4001, 128, False, repeat=2, pad=72)
