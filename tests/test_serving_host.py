"""Host-side checks of the operators around verification: structure layouts,
refusals before any CUDA call, and the 64-bit definitions against one another."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from gdn_speculative_tree_gb300 import binding, build
from oracle import gdn_tree_oracle
from oracle import serving_oracle as orc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = binding.TREEWY_ERR_INVALID_ARG, binding.TREEWY_ERR_UNSUPPORTED
FAKE = 0x10000  # never dereferenced: these calls fail validation first


@pytest.fixture(scope="module")
def lib():
    try:
        build.nvcc_path()
    except RuntimeError:
        pytest.skip("no CUDA toolkit")
    return binding.load(build.build())


def test_struct_layouts_match_c(tmp_path):
    """Sizes and offsets as the C compiler sees them."""
    structs = {"treewy_seqs": binding.TreewySeqs, "treewy_qk": binding.TreewyQk, "treewy_slots": binding.TreewySlots}
    lines = []
    for name, cls in structs.items():
        lines.append(f'printf("%zu", sizeof({name}));')
        lines += [f'printf(" %zu", offsetof({name}, {f}));' for f, _ in cls._fields_]
        lines.append('printf("\\n");')
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"treewy.h\"\nint main(void) {" +
                   "\n".join(lines) + "return 0; }\n")
    cuda = os.path.dirname(os.path.dirname(build.nvcc_path()))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-I", os.path.join(cuda, "include"), str(src), "-o",
                    str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout
    for line, cls in zip(out.splitlines(), structs.values()):
        got = [int(x) for x in line.split()]
        assert got == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]


def seqs():
    s = binding.TreewySeqs()
    s.R, s.H, s.Hk, s.dk, s.dv, s.max_len = 2, 4, 2, 128, 128, 100
    s.T, s.num_slots = 10, 3
    for f in ("seq_offset", "q", "k", "v", "alpha", "beta", "state", "state_slot", "o", "status"):
        setattr(s, f, FAKE)
    return s


@pytest.mark.parametrize("field,value,code", [
    ("R", -1, INVALID), ("H", 0, INVALID), ("Hk", 0, INVALID), ("Hk", 3, INVALID), ("Hk", 8, INVALID),
    ("dk", 0, INVALID), ("dv", -1, INVALID), ("dk", 129, UNSUPPORTED), ("dv", 256, UNSUPPORTED),
    ("max_len", -1, INVALID), ("qkv_dtype", 2, INVALID), ("o_dtype", -1, INVALID), ("flags", 4, INVALID),
    ("T", -1, INVALID), ("T", 1 << 31, INVALID), ("num_slots", 0, INVALID), ("num_slots", 1 << 30, UNSUPPORTED),
    ("R", 1 << 30, UNSUPPORTED), ("q_stride", 255, INVALID), ("k_stride", -1, INVALID), ("v_stride", 511, INVALID),
    ("v_stride", 1 << 40, UNSUPPORTED), ("q", None, INVALID), ("o", None, INVALID), ("beta", None, INVALID),
    ("seq_offset", None, INVALID), ("state", None, INVALID), ("status", None, INVALID), ("state_slot", None, INVALID),
    ("state", FAKE + 8, INVALID), ("q", FAKE + 1, INVALID), ("alpha", FAKE + 2, INVALID),
])
def test_extend_refuses(lib, field, value, code):
    s = seqs()
    setattr(s, field, value)
    assert lib.treewy_extend(ctypes.byref(s), None) == code
    assert binding.treewy_last_error()


def test_extend_of_no_sequence_is_fine(lib):
    s = binding.TreewySeqs()
    s.H = s.Hk = s.dk = s.dv = s.num_slots = 1
    assert lib.treewy_extend(ctypes.byref(s), None) == binding.TREEWY_OK
    assert lib.treewy_extend(None, None) == INVALID


def qk():
    a = binding.TreewyQk()
    a.T, a.Hq, a.Hk, a.d, a.q_repeat, a.k_repeat, a.rope_dims, a.rope_rows = 4, 2, 1, 128, 1, 1, 64, 10
    for f in ("q", "k", "rope", "position", "status"):
        setattr(a, f, FAKE)
    a.q_out = a.k_out = 2 * FAKE
    return a


@pytest.mark.parametrize("field,value,code", [
    ("T", -1, INVALID), ("T", 1 << 31, INVALID), ("Hq", -1, INVALID), ("d", 0, INVALID), ("d", 257, UNSUPPORTED),
    ("dtype", 2, INVALID), ("norm", 2, INVALID), ("eps", -1.0, INVALID), ("eps", float("nan"), INVALID),
    ("rope_dims", 63, INVALID), ("rope_dims", 130, INVALID), ("rope_dims", -2, INVALID), ("q_repeat", 0, INVALID),
    ("k_repeat", -1, INVALID), ("q_stride", 255, INVALID), ("k_stride", 1 << 40, UNSUPPORTED), ("q", None, INVALID),
    ("k_out", None, INVALID), ("rope", None, INVALID), ("position", None, INVALID), ("status", None, INVALID),
    ("rope_rows", 0, INVALID), ("q", FAKE + 1, INVALID), ("Hq", 1 << 21, UNSUPPORTED),
])
def test_qk_norm_refuses(lib, field, value, code):
    a = qk()
    setattr(a, field, value)
    assert lib.treewy_qk_norm(ctypes.byref(a), None) == code


def test_qk_norm_refuses_in_place_where_rows_move(lib):
    a = qk()
    a.q_out, a.q_repeat = FAKE, 2
    assert lib.treewy_qk_norm(ctypes.byref(a), None) == INVALID
    a.q_repeat, a.q_stride = 1, 300
    assert lib.treewy_qk_norm(ctypes.byref(a), None) == INVALID
    a = qk()
    a.Hq = a.Hk = 0
    assert lib.treewy_qk_norm(ctypes.byref(a), None) == INVALID
    assert lib.treewy_qk_norm(None, None) == INVALID
    a = qk()
    a.T = 0
    assert lib.treewy_qk_norm(ctypes.byref(a), None) == binding.TREEWY_OK


@pytest.mark.parametrize("field,value,code", [
    ("n", -1, INVALID), ("layers", -1, INVALID), ("num_slots", 0, INVALID), ("slot_bytes", 0, INVALID),
    ("slot_bytes", 1 << 40, UNSUPPORTED), ("layer_stride", 100, INVALID), ("layer_stride", -1, INVALID),
    ("state", None, INVALID), ("src", None, INVALID), ("dst", None, INVALID), ("status", None, INVALID),
])
def test_copy_slots_refuses(lib, field, value, code):
    a = binding.TreewySlots()
    a.n, a.layers, a.num_slots, a.slot_bytes = 2, 3, 8, 64
    a.state = a.src = a.dst = a.status = FAKE
    setattr(a, field, value)
    assert lib.treewy_copy_slots(ctypes.byref(a), None) == code
    assert lib.treewy_copy_slots(None, None) == INVALID


def test_binding_refuses_what_it_cannot_describe():
    T, H, d = 3, 2, 8
    x = torch.zeros(T, H, d)
    i32 = torch.zeros(1, dtype=torch.int32)
    ok = dict(seq_offset=torch.zeros(2, dtype=torch.int32), q=x, k=x, v=x, alpha=torch.zeros(T, H),
              beta=torch.zeros(T, H), state=torch.zeros(2, H, d, d), state_slot=i32, o=x, status=i32, max_len=3)
    binding.make_seqs(**ok)
    for name, bad, err in (("q", x.transpose(0, 1), ValueError), ("q", x.half(), TypeError),
                           ("k", x[:, :1], ValueError), ("alpha", torch.zeros(T, H + 1), ValueError),
                           ("alpha", torch.zeros(T, H).double(), TypeError),
                           ("state", torch.zeros(2, H, d, d).half(), TypeError),
                           ("state", torch.zeros(2, H, d, d + 1), ValueError), ("o", x.double(), TypeError),
                           ("state_slot", torch.zeros(1, dtype=torch.int64), TypeError),
                           ("fresh", torch.zeros(1, dtype=torch.int32), TypeError),
                           ("v", x.permute(0, 2, 1), ValueError)):
        with pytest.raises(err):
            binding.make_seqs(**{**ok, name: bad})
    with pytest.raises(ValueError):
        binding.make_qk()
    with pytest.raises(ValueError):
        binding.make_qk(q=x)
    with pytest.raises(ValueError):
        binding.make_qk(q=x, q_out=x, norm="l1")
    with pytest.raises(ValueError):
        binding.make_qk(q=x, q_out=torch.zeros(T, 3, d))
    with pytest.raises(ValueError):
        binding.make_qk(q=x, q_out=x, rope=torch.zeros(4, 4))
    with pytest.raises(ValueError):
        binding.make_slots(state=torch.zeros(4), src=i32, dst=i32, status=i32)
    with pytest.raises(TypeError):
        binding.make_slots(state=torch.zeros(4, 2), src=i32.long(), dst=i32, status=i32)
    with pytest.raises(ValueError):
        binding.make_slots(state=torch.zeros(4, 2), src=i32, dst=torch.zeros(2, dtype=torch.int32), status=i32)


def test_definition_agrees_with_the_tree_oracle():
    """Extending over a chain equals the tree oracle's chain of nodes."""
    rng = np.random.default_rng(0)
    n, dk, dv = 6, 5, 7
    S0 = rng.normal(size=(1, dv, dk))
    q, k, v = rng.normal(size=(n, 1, dk)), rng.normal(size=(n, 1, dk)), rng.normal(size=(n, 1, dv))
    a, b = rng.uniform(0.5, 1, (n, 1)), rng.uniform(0, 1, (n, 1))
    o, S = orc.extend(S0, q, k, v, a, b)
    ref = gdn_tree_oracle.verify_request(S0, np.arange(-1, n - 1, dtype=np.int32), q, k, v, a, b)
    np.testing.assert_allclose(o, ref.o, rtol=0, atol=1e-12)
    np.testing.assert_allclose(S, gdn_tree_oracle.commit_request(S0, ref, n - 1), rtol=0, atol=1e-12)


def test_moves_by_hand():
    pool = np.arange(4.0).reshape(1, 4, 1)
    out, status = orc.move_slots(pool, [0, -1], [2, 3])
    assert out.ravel().tolist() == [0, 1, 0, 0] and status.tolist() == [0, 0]
    out, status = orc.move_slots(pool, [0, 1], [1, 2])
    assert out.ravel().tolist() == [0, 0, 2, 3] and status.tolist() == [0, 128]
