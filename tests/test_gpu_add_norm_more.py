"""treewy_add_norm where it writes over what it reads."""
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
