"""Arguments of the three calls around verification that are refused before any launch (host only)."""
import ctypes

import pytest

from gdn_speculative_tree_gb300 import binding
from tests.test_serving_host import FAKE, INVALID, lib, qk, seqs  # noqa: F401


def slots():
    a = binding.TreewySlots()
    a.n, a.layers, a.num_slots, a.slot_bytes = 2, 3, 8, 64
    a.state = a.src = a.dst = a.status = FAKE
    return a


@pytest.mark.parametrize("make,call,fields", [
    (seqs, "treewy_extend", ("seq_offset", "state_slot", "status")),
    (qk, "treewy_qk_norm", ("position", "status")),
    (slots, "treewy_copy_slots", ("src", "dst", "status")),
])
def test_whole_numbers_are_aligned_to_their_elements(lib, make, call, fields):  # noqa: F811
    for field in fields:
        for off in (1, 2):
            a = make()
            setattr(a, field, FAKE + off)
            assert getattr(lib, call)(ctypes.byref(a), None) == INVALID, (field, off)
            assert "aligned" in binding.treewy_last_error()


@pytest.mark.parametrize("n,layers,slot_bytes", [((1 << 31) - 1, (1 << 31) - 1, 1 << 20), (1 << 16, 1 << 16, 1 << 31),
                                                 (1 << 15, 1 << 16, 1 << 10)])
def test_more_moves_than_a_launch_holds(lib, n, layers, slot_bytes):  # noqa: F811
    """Their number passes 2^31, and 2^63 in the first case: none of them may wrap to a smaller one."""
    a = slots()
    a.n, a.layers, a.num_slots, a.slot_bytes = n, layers, 2, slot_bytes
    assert lib.treewy_copy_slots(ctypes.byref(a), None) == binding.TREEWY_ERR_UNSUPPORTED
    assert "moves" in binding.treewy_last_error()
