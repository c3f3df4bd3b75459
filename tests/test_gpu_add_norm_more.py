"""treewy_add_norm where it writes over what it reads, and its codes against the quotient that they stand for."""
import pytest
import torch

from gdn_speculative_tree_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,n", [(1, 1), (300, 7), (2000, 61), (700, 1001), (152, 4001), (40, 32767)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_at_widths_whose_rows_share_cache_lines(cuda_lib, T, n, dtype):
    g = torch.Generator().manual_seed(n)
    x, res = (torch.randn(T, n, generator=g).to(dtype).cuda() for _ in range(2))
    out, y = torch.empty_like(res), torch.empty_like(x)
    binding.treewy_add_norm(binding.make_norm(x=x, residual=res, residual_out=out, y=y))
    binding.treewy_add_norm(binding.make_norm(x=x, residual=res, residual_out=res, y=x))
    assert torch.equal(res, out) and torch.equal(x, y)


def codes_of_the_quotient(y8, y, s, group):
    """Each code is that of y / scale or of a neighbour within 2^-22 of it: y times 1 / scale has two roundings of 2^-24."""
    q = y.double() / s.double().repeat_interleave(group or y.shape[1], dim=1)[:, :y.shape[1]]
    ends = [(q * (1 + e)).float().to(torch.float8_e4m3fn).float() for e in (-2.0 ** -22, 2.0 ** -22)]
    got = y8.float()
    return bool(((got >= torch.minimum(*ends)) & (got <= torch.maximum(*ends))).all())


@pytest.mark.parametrize("n,group,T", [(4096, 0, 8192), (4096, 128, 8192), (2048, 32, 16384), (200, 64, 100000), (4001, 0, 4000),
                                       (4001, 64, 4000)])
def test_codes_are_those_of_the_quotient(cuda_lib, n, group, T):
    """For every one of tens of millions of values: f32 outputs are what the codes are made of."""
    torch.manual_seed(n)
    x = torch.randn(T, n, device="cuda")
    x[:4] *= torch.tensor([[1e-30], [1e-12], [1e15], [0.0]], device="cuda")
    y, y8 = torch.empty_like(x), torch.empty(T, n, device="cuda", dtype=torch.float8_e4m3fn)
    s = torch.empty(T, -(-n // group) if group else 1, device="cuda")
    binding.treewy_add_norm(binding.make_norm(x=x, y=y, y8=y8, y8_scale=s, group=group))
    assert codes_of_the_quotient(y8, y, s, group)


@pytest.mark.parametrize("n", [512, 511])
@pytest.mark.parametrize("group", [0, 64])
def test_scales_at_the_ends_of_f32(cuda_lib, n, group):
    """Weights that make rows of next to nothing, as large as f32 goes, and infinite ones."""
    torch.manual_seed(n)
    x = torch.randn(6, n, device="cuda")
    for size in (1e-38, 2e-36, 1e-33, 3e-31, 1e-28, 1e37, 8e37):
        w = torch.full((n,), size, device="cuda")
        y, y8 = torch.empty_like(x), torch.empty(6, n, device="cuda", dtype=torch.float8_e4m3fn)
        s = torch.empty(6, -(-n // group) if group else 1, device="cuda")
        binding.treewy_add_norm(binding.make_norm(x=x, weight=w, y=y, y8=y8, y8_scale=s, group=group))
        assert codes_of_the_quotient(y8, y, s, group)
    w = torch.ones(n, device="cuda")
    w[3] = float("inf")
    binding.treewy_add_norm(binding.make_norm(x=x, weight=w, y=y, y8=y8, y8_scale=s, group=group))
    first = y8.float()[:, :group or n]
    assert torch.isinf(y[:, 3]).all() and torch.isinf(s[:, 0]).all() and torch.isnan(first[:, 3]).all()
    assert (first[:, torch.arange(first.shape[1], device="cuda") != 3] == 0).all()
