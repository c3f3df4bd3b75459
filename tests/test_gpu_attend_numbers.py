"""treewy_attend where rows hold infinities and no numbers, and where scores pass f32."""
import pytest
import torch

from gdn_speculative_tree_gb300 import binding
from tests.cache_helpers import Attend

pytestmark = pytest.mark.gpu

GENERIC = binding.FLAG_FORCE_GENERIC


@pytest.mark.parametrize("flags", [0, GENERIC])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("Hq", [4, 40])
def test_infinite_keys_and_values_count_as_no_numbers(cuda_lib, flags, dtype, out, sign, Hq):
    """Whatever the sign of what they are multiplied by."""
    a = Attend([100, 0], [3, 2], Hq=Hq, Hkv=2, d=64, page=32, kind="star", dtype=dtype, out=out, flags=flags, seed=31)
    half = Hq // 2
    a.q[:, :, 0] = torch.tensor([1.5, -1.5], device="cuda").to(a.q.dtype).repeat(half)   # both signs at every key head
    a.k[1, 0, 0] = sign * float("inf")
    a.v[2, 1, 5] = sign * float("inf")
    a.v[a.off[1] + 1, 0, 7] = -sign * float("inf")
    a.run()
    want = torch.zeros_like(a.o, dtype=torch.bool)
    want[1, :half] = True
    want[2, half:, 5] = True
    want[a.off[1] + 1, :half, 7] = True
    assert torch.equal(torch.isnan(a.o.float()), want) and torch.isfinite(a.o.float()[~want]).all()


@pytest.mark.parametrize("flags", [0, GENERIC])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("Hq", [4, 40])
def test_a_query_that_is_no_number_is_its_own_rows(cuda_lib, flags, value, Hq):
    a = Attend([100, 40], [2, 2], Hq=Hq, Hkv=2, d=64, page=32, flags=flags, seed=32)
    a.q[1, 1, 3] = value
    a.run()
    want = torch.zeros_like(a.o, dtype=torch.bool)
    want[1, 1] = True
    assert torch.equal(torch.isnan(a.o.float()), want)


def test_scores_that_pass_f32(cuda_lib):
    """f32 rows whose products overflow, both ways: no numbers, not a score that counts for nothing."""
    a = Attend([0, 0], [1, 1], Hq=2, Hkv=1, d=8, dtype="f32", out="f32", seed=34)
    a.q.zero_(), a.k.zero_()
    a.q[..., 0], a.k[..., 0] = 1e25, torch.tensor([-1e25, 1e25], device="cuda")[:, None]
    a.run()
    assert torch.isnan(a.o).all()


def test_two_tokens_of_which_one_score_passes_f32(cuda_lib):
    a = Attend([0], [2], Hq=1, Hkv=1, d=8, kind="chain", dtype="f32", out="f32", seed=35)
    a.q.zero_(), a.k.zero_()
    a.q[..., 0], a.k[0, 0, 0] = 1e25, -1e25
    a.run()
    assert torch.isnan(a.o).all()


@pytest.mark.parametrize("flags", [0, GENERIC])
@pytest.mark.parametrize("Hq", [4, 40])
@pytest.mark.parametrize("token", [5, 64, 200])
def test_a_value_that_is_no_number_beside_far_larger_weights(cuda_lib, flags, Hq, token):
    """It reaches its column, however little its token weighs: that of a tile far below the others', and none at all in f32."""
    a = Attend([256], [1], Hq=Hq, Hkv=1, d=64, page=16, flags=flags, seed=33)
    a.cache.k.view(torch.uint8).zero_()
    a.cache.k.view(torch.uint8)[:, :, :, 0] = 0x38           # 1
    a.q.zero_()
    a.q[..., 0] = 100.0
    a.k.zero_()
    a.cache.ks.fill_(1.0)
    a.scale = 1.0
    for p in range(16):                                       # scores of 1,600 down to 100, and of 0 for the draft's own
        a.cache.ks[int(a.cache.table_np[0, p])] = float((p + 5) % 16 + 1)
    a.cache.v.view(torch.uint8)[int(a.cache.table_np[0, token // 16]), 0, token % 16, 9] = 127
    a.run()
    want = torch.zeros_like(a.o, dtype=torch.bool)
    want[..., 9] = True
    assert torch.equal(torch.isnan(a.o.float()), want)
