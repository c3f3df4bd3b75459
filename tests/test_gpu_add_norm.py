"""treewy_add_norm against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from gdn_speculative_tree_gb300 import binding
from oracle import attend_oracle as orc
from tests.cache_helpers import E4M3, TYPES, f64

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def strided(T, n, dtype, pad, shift, g, size=1.0):
    wide = torch.full((T * (n + pad) + shift,), float("nan"), dtype=dtype)
    wide[shift:].view(T, n + pad)[:, :n] = (torch.randn(T, n, generator=g) * size).to(dtype)
    return wide.cuda()[shift:].view(T, n + pad)[:, :n]


def run(T, n, *, dtype="bf16", residual="bf16", group=128, both=True, eight=True, weight=True, pad=0, shift=0, eps=1e-6, seed=0,
        size=1.0):
    g = torch.Generator().manual_seed(seed)
    x = strided(T, n, TYPES[dtype], pad, shift, g, size)
    res = strided(T, n, TYPES[residual], pad, shift, g, 3 * size) if residual else None
    w = 1 + 0.3 * torch.randn(n, generator=g).cuda() if weight else None
    m = -(-n // group) if group else 1
    out = torch.full((T, n), -7.0, dtype=TYPES[residual], device="cuda") if residual else None
    y = torch.full((T, n), -7.0, dtype=TYPES[dtype], device="cuda") if both else None
    y8 = torch.full((T, n), -7.0, device="cuda").to(E4M3) if eight else None
    s = torch.full((T, m), -7.0, device="cuda") if eight else None
    binding.treewy_add_norm(binding.make_norm(x=x, residual=res, residual_out=out, weight=w, eps=eps, y=y, y8=y8, y8_scale=s,
                                              group=group))
    torch.cuda.synchronize()
    check(x, res, w, eps, out, y, y8, s, group)
    return out, y, y8, s


def check(x, res, w, eps, out, y, y8, s, group):
    """f32 sums of n squares: n 2^-24 of the mean, half of that of its root, and a few roundings."""
    n = x.shape[1]
    z, ref = orc.add_norm(f64(x), f64(res) if res is not None else None, f64(w) if w is not None else None, eps)
    rel = n * 2.0 ** -25 + 8 * 2.0 ** -24
    if out is not None:
        assert (np.abs(f64(out) - z) <= (HALF[out.dtype] + 2.0 ** -24) * np.abs(z)).all()
    # z itself is rounded to f32: that of a sum that cancels is no more than its terms' 2^-24
    if y is not None:
        assert (np.abs(f64(y) - ref) <= (HALF[y.dtype] + rel) * np.abs(ref)).all()
    if y8 is not None:
        scale = orc.group_scales(ref, group)
        assert (np.abs(f64(s) - scale) <= (rel + 2.0 ** -23) * scale).all()
        wide = np.repeat(f64(s), group or n, axis=1)[:, :n]
        # half a step of e4m3: 2^-4 of the value, 2^-10 units below its normal range
        tol = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * wide) + (rel + 2.0 ** -22) * np.abs(ref)
        assert (np.abs(f64(y8) * wide - ref) <= tol).all()


@pytest.mark.parametrize("n", [1, 7, 8, 64, 200, 256, 264, 1000, 1024, 1032, 2048, 4096, 4104, 8192, 16384, 16392, 32768])
@pytest.mark.parametrize("group", [0, 128])
def test_widths(cuda_lib, n, group):
    run(5, n, group=group, seed=n)


@pytest.mark.parametrize("n", [72, 1000, 4096, 5001])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("dtype,residual", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16"), ("bf16", None),
                                            ("f32", None)])
def test_types_and_groups(cuda_lib, dtype, residual, group, n):
    run(9, n, dtype=dtype, residual=residual, group=group, seed=n)


@pytest.mark.parametrize("pad,shift", [(8, 0), (24, 8), (1, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("n", [256, 1000, 2048])
def test_strided_and_unaligned_rows(cuda_lib, n, pad, shift):
    run(6, n, pad=pad, shift=shift, seed=pad)


@pytest.mark.parametrize("both,eight,weight", [(True, False, True), (False, True, False), (False, False, True), (True, True, False)])
@pytest.mark.parametrize("n", [512, 513])
def test_outputs_left_out(cuda_lib, n, both, eight, weight):
    run(4, n, both=both, eight=eight, weight=weight)


@pytest.mark.parametrize("T", [1, 2, 3, 5, 151, 1000])
@pytest.mark.parametrize("n", [128, 2048])
def test_numbers_of_rows(cuda_lib, T, n):
    run(T, n, group=64)


@pytest.mark.parametrize("size,eps", [(1e-12, 1e-6), (1e-12, 0.0), (1e12, 1e-5), (1.0, 10.0)])
def test_small_and_large_rows(cuda_lib, size, eps):
    run(3, 1024, dtype="f32", residual="f32", size=size, eps=eps)
    run(3, 1023, dtype="f32", residual="f32", size=size, eps=eps)


@pytest.mark.parametrize("n", [256, 1024, 1023, 8192])
@pytest.mark.parametrize("group", [0, 64])
def test_rows_and_groups_of_zeros(cuda_lib, n, group):
    x = torch.zeros(3, n, device="cuda", dtype=torch.bfloat16)
    x[1, -1] = 2.0
    y8, s = torch.ones(3, n, device="cuda").to(E4M3), torch.zeros(3, -(-n // group) if group else 1, device="cuda")
    binding.treewy_add_norm(binding.make_norm(x=x, y8=y8, y8_scale=s, group=group))
    assert (y8.float()[[0, 2]] == 0).all() and (y8.float()[1, :-1] == 0).all() and float(y8.float()[1, -1]) == 448.0
    assert (s[[0, 2]] == 1).all() and (s[1, :-1] == 1).all()


@pytest.mark.parametrize("n", [512, 511])
def test_no_numbers_stay_in_their_rows(cuda_lib, n):
    x = torch.randn(4, n, device="cuda").bfloat16()
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    y, y8, s = torch.empty_like(x), torch.empty(4, n, device="cuda", dtype=E4M3), torch.empty(4, 1, device="cuda")
    binding.treewy_add_norm(binding.make_norm(x=x, y=y, y8=y8, y8_scale=s))
    assert torch.isnan(y[1]).all() and torch.isnan(y8.float()[1]).all() and torch.isnan(y[2, 5])
    assert torch.isfinite(y[[0, 3]]).all() and torch.isfinite(y8.float()[[0, 3]]).all() and torch.isfinite(s[[0, 3]]).all()


@pytest.mark.parametrize("n", [1024, 1001])
def test_in_place(cuda_lib, n):
    """The residual and x overwritten by the sum and the normed rows."""
    g = torch.Generator().manual_seed(1)
    x, res = (torch.randn(7, n, generator=g).bfloat16().cuda() for _ in range(2))
    out, y = torch.empty_like(res), torch.empty_like(x)
    binding.treewy_add_norm(binding.make_norm(x=x, residual=res, residual_out=out, y=y))
    binding.treewy_add_norm(binding.make_norm(x=x, residual=res, residual_out=res, y=x))
    assert torch.equal(res, out) and torch.equal(x, y)


def test_same_bits_in_a_graph_on_another_stream(cuda_lib):
    out, y, y8, s = run(300, 2048, seed=3)
    g = torch.Generator().manual_seed(3)
    x, res = strided(300, 2048, torch.bfloat16, 0, 0, g), strided(300, 2048, torch.bfloat16, 0, 0, g, 3.0)
    w = 1 + 0.3 * torch.randn(2048, generator=g).cuda()
    o2, y2, z2, s2 = torch.empty_like(out), torch.empty_like(y), torch.empty_like(y8), torch.empty_like(s)
    call = binding.make_norm(x=x, residual=res, residual_out=o2, weight=w, y=y2, y8=z2, y8_scale=s2, group=128)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        binding.treewy_add_norm(call)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in ((out, o2), (y, y2), (y8, z2), (s, s2)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("n", [64, 61])
def test_zeros_beside_the_smallest_numbers(cuda_lib, n, group):
    """One over a scale below 2^-128 would be infinite, and zeros times it no numbers."""
    x = torch.zeros(5, n)
    x[:, ::2] = torch.arange(1, (n + 1) // 2 + 1) * 2.0 ** -149 * torch.tensor([[1.0], [5.0], [100.0], [-3.0], [0.0]])
    x = x.cuda()
    m = -(-n // group) if group else 1
    y8, s = torch.full((5, n), -7.0, device="cuda").to(E4M3), torch.full((5, m), -7.0, device="cuda")
    binding.treewy_add_norm(binding.make_norm(x=x, y8=y8, y8_scale=s, group=group))
    ref = orc.add_norm(f64(x), None, None, 1e-6)[1]
    scale = np.repeat(f64(s), group or n, axis=1)[:, :n]
    assert (f64(s)[:4] == 2.0 ** -126).all() and (f64(s)[4] == 1).all()
    # y in f32 is off by a step of 2^-149 or 2^-21 of it, its code by half a step of e4m3
    assert (np.abs(f64(y8) * scale - ref) <= 2.0 ** -148 + 2.0 ** -21 * np.abs(ref) + np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * scale)).all()
