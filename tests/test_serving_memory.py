"""What the binding refuses because a kernel would reach memory that is not the tensor's (host only, nothing runs)."""
import pytest
import torch

from gdn_speculative_tree_gb300 import binding


def moves(n=1):
    return {f: torch.zeros(n, dtype=torch.int32) for f in ("src", "dst", "status")}


@pytest.mark.parametrize("layers", [2, 3])
def test_slots_of_layers_that_share_memory_are_refused(layers):
    """An expanded pool's layer stride is 0, which the library takes for dense layers."""
    pool = torch.zeros(4, 2, 8)
    with pytest.raises(ValueError):
        binding.make_slots(state=pool.expand(layers, 4, 2, 8), layers=layers, **moves())
    with pytest.raises(ValueError):
        binding.make_slots(state=torch.zeros(200).as_strided((layers, 4, 2, 8), (16, 16, 8, 1)), layers=layers, **moves())


def test_slots_of_layers_of_their_own_are_described():
    for layers, pad in ((1, 0), (3, 0), (3, 5)):
        pool = torch.zeros(layers, 4 + pad, 2, 8)[:, :4]
        a = binding.make_slots(state=pool, layers=layers, **moves())
        assert a.layer_stride == (0 if layers == 1 else (4 + pad) * 64) and a.slot_bytes == 64
    one = binding.make_slots(state=torch.zeros(4, 2, 8).expand(1, 4, 2, 8), layers=1, **moves())
    assert (one.layers, one.layer_stride) == (1, 0)
