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


class NoLibrary:
    """In the place of the CUDA library: counts the calls that would have been made."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return binding.TREEWY_OK
        return call


def arguments():
    """The three calls and their arguments, described from CPU tensors."""
    T, H, d = 3, 2, 8
    x, gate, i32 = torch.zeros(T, H, d), torch.zeros(T, H), torch.zeros(1, dtype=torch.int32)
    return ((binding.treewy_extend,
             binding.make_seqs(seq_offset=torch.zeros(2, dtype=torch.int32), q=x, k=x, v=x, alpha=gate, beta=gate,
                               state=torch.zeros(2, H, d, d), state_slot=i32, o=torch.zeros(T, H, d), status=i32,
                               max_len=3)),
            (binding.treewy_qk_norm, binding.make_qk(q=x, q_out=torch.zeros(T, H, d))),
            (binding.treewy_copy_slots, binding.make_slots(state=torch.zeros(4, 2, 8), **moves())))


@pytest.mark.parametrize("which", [0, 1, 2])
def test_calls_refuse_tensors_that_the_current_device_cannot_reach(monkeypatch, which):
    lib = NoLibrary()
    monkeypatch.setattr(binding, "_lib", lib)
    call, args = arguments()[which]
    with pytest.raises(ValueError, match="CPU"):
        call(args, 0)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    args._device = 1
    with pytest.raises(ValueError, match="device 1"):
        call(args, 0)
    assert lib.calls == 0
    args._device = 0
    call(args, 0)
    call(type(args)(), 0)  # filled by hand: its pointers are the caller's business
    assert lib.calls == 2
