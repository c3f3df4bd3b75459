"""Host-side checks of the softmax layers' operators: structure layouts, refusals before any CUDA call, what the
binding refuses, and the 64-bit definitions against torch and one another."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from gdn_speculative_tree_gb300 import binding, build
from oracle import attend_oracle as orc
from tests.test_serving_host import FAKE, INVALID, ROOT, UNSUPPORTED, lib  # noqa: F401


def test_struct_layouts_match_c(tmp_path):
    structs = {"treewy_cache": binding.TreewyCache, "treewy_attn": binding.TreewyAttn,
               "treewy_append_args": binding.TreewyAppendArgs, "treewy_norm": binding.TreewyNorm}
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


def fill(a, fields):
    for f in fields:
        setattr(a, f, FAKE)
    return a


def cache(c):
    c.Hkv, c.d, c.page_len, c.max_pages, c.num_pages = 2, 128, 64, 4, 16
    fill(c, ("k", "v", "k_scale", "v_scale", "page_table", "length"))


def attn():
    a = binding.TreewyAttn()
    a.R, a.Hq, a.max_nodes, a.max_context, a.T, a.scale = 2, 4, 8, 200, 10, 0.1
    cache(a.cache)
    fill(a, ("node_offset", "parent", "q", "k", "v", "o", "status", "workspace"))
    a.workspace_bytes = 1 << 40
    return a


def append():
    a = binding.TreewyAppendArgs()
    a.R, a.max_new, a.T = 2, 64, 10
    cache(a.cache)
    fill(a, ("node_offset", "parent", "accepted", "k", "v", "status"))
    a.new_length = 2 * FAKE
    return a


def norm():
    a = binding.TreewyNorm()
    a.T, a.n, a.group = 4, 256, 128
    fill(a, ("x", "residual", "weight", "y8", "y8_scale"))
    a.residual_out = a.y = 2 * FAKE
    return a


def put(a, field, value):
    for name in field.split(".")[:-1]:
        a = getattr(a, name)
    setattr(a, field.split(".")[-1], value)


CACHE = [("cache.Hkv", 0, INVALID), ("cache.d", 0, INVALID), ("cache.d", 257, UNSUPPORTED), ("cache.page_len", 48, UNSUPPORTED),
         ("cache.page_len", 0, UNSUPPORTED), ("cache.max_pages", -1, INVALID), ("cache.num_pages", -1, INVALID),
         ("cache.num_pages", 1 << 30, UNSUPPORTED), ("cache.k", None, INVALID), ("cache.v", FAKE + 8, INVALID),
         ("cache.k_scale", None, INVALID), ("cache.v_scale", FAKE + 2, INVALID), ("cache.page_table", None, INVALID),
         ("cache.page_table", FAKE + 1, INVALID), ("cache.length", None, INVALID), ("cache.length", FAKE + 2, INVALID)]


@pytest.mark.parametrize("field,value,code", CACHE + [
    ("R", -1, INVALID), ("Hq", 0, INVALID), ("Hq", 3, INVALID), ("Hq", 1 << 21, UNSUPPORTED), ("max_nodes", 0, INVALID),
    ("max_nodes", 65, UNSUPPORTED), ("max_context", -1, INVALID), ("qkv_dtype", 2, INVALID), ("o_dtype", -1, INVALID),
    ("flags", 2, INVALID), ("T", -1, INVALID), ("T", 1 << 31, INVALID), ("scale", 0.0, INVALID), ("scale", -1.0, INVALID),
    ("scale", float("nan"), INVALID), ("scale", float("inf"), INVALID), ("q_stride", 511, INVALID),
    ("k_stride", -1, INVALID), ("v_stride", 1 << 40, UNSUPPORTED), ("q", None, INVALID), ("v", None, INVALID),
    ("o", None, INVALID), ("node_offset", None, INVALID), ("status", None, INVALID), ("q", FAKE + 1, INVALID),
    ("o", FAKE + 1, INVALID), ("parent", FAKE + 2, INVALID), ("node_offset", FAKE + 2, INVALID), ("status", FAKE + 1, INVALID),
    ("workspace", None, INVALID), ("workspace", FAKE + 8, INVALID), ("workspace_bytes", 0, INVALID),
])
def test_attend_refuses(lib, field, value, code):  # noqa: F811
    a = attn()
    put(a, field, value)
    assert lib.treewy_attend(ctypes.byref(a), None) == code
    assert binding.treewy_last_error()


def test_attend_refuses_more_than_a_launch_holds(lib):  # noqa: F811
    a = attn()
    a.R = (1 << 31) - 1
    assert lib.treewy_attend(ctypes.byref(a), None) == UNSUPPORTED
    a.flags = binding.FLAG_FORCE_GENERIC
    assert lib.treewy_attend(ctypes.byref(a), None) == UNSUPPORTED


def test_attend_of_no_request_is_fine(lib):  # noqa: F811
    a = attn()
    a.R = 0
    assert lib.treewy_attend(ctypes.byref(a), None) == binding.TREEWY_OK
    assert lib.treewy_attend(None, None) == INVALID
    assert lib.treewy_attend_workspace(None, None) == INVALID
    assert lib.treewy_attend_workspace(ctypes.byref(a), None) == INVALID


@pytest.mark.parametrize("field,value,code", CACHE + [
    ("R", -1, INVALID), ("max_new", -1, INVALID), ("max_new", 65, UNSUPPORTED), ("kv_dtype", 2, INVALID), ("T", -1, INVALID),
    ("T", 1 << 31, INVALID), ("k_stride", 255, INVALID), ("v_stride", 1 << 40, UNSUPPORTED), ("k", None, INVALID),
    ("v", FAKE + 1, INVALID), ("node_offset", None, INVALID), ("status", None, INVALID), ("accepted", FAKE + 2, INVALID),
    ("new_length", FAKE, INVALID), ("new_length", FAKE + 2, INVALID), ("R", (1 << 31) - 1, UNSUPPORTED),
])
def test_append_refuses(lib, field, value, code):  # noqa: F811
    a = append()
    put(a, field, value)
    assert lib.treewy_append(ctypes.byref(a), None) == code
    assert binding.treewy_last_error()


def test_append_of_no_request_is_fine(lib):  # noqa: F811
    a = append()
    a.R = 0
    assert lib.treewy_append(ctypes.byref(a), None) == binding.TREEWY_OK
    assert lib.treewy_append(None, None) == INVALID


@pytest.mark.parametrize("field,value,code", [
    ("T", -1, INVALID), ("T", 1 << 31, INVALID), ("n", 0, INVALID), ("n", 32769, UNSUPPORTED), ("x_dtype", 2, INVALID),
    ("residual_dtype", -1, INVALID), ("group", 16, UNSUPPORTED), ("group", -1, UNSUPPORTED), ("group", 256, UNSUPPORTED),
    ("eps", -1.0, INVALID), ("eps", float("nan"), INVALID), ("x_stride", 255, INVALID), ("residual_stride", 1, INVALID),
    ("x_stride", 1 << 40, UNSUPPORTED), ("x", None, INVALID), ("residual", None, INVALID), ("residual_out", None, INVALID),
    ("y8_scale", None, INVALID), ("x", FAKE + 1, INVALID), ("weight", FAKE + 2, INVALID), ("y8_scale", FAKE + 1, INVALID),
    ("residual_out", FAKE + 1, INVALID), ("y", FAKE + 1, INVALID),
])
def test_add_norm_refuses(lib, field, value, code):  # noqa: F811
    a = norm()
    put(a, field, value)
    assert lib.treewy_add_norm(ctypes.byref(a), None) == code
    assert binding.treewy_last_error()


def test_add_norm_refuses_in_place_where_rows_are_strided(lib):  # noqa: F811
    a = norm()
    a.residual_out, a.residual_stride = FAKE, 300
    assert lib.treewy_add_norm(ctypes.byref(a), None) == INVALID
    a = norm()
    a.y, a.x_stride = FAKE, 300
    assert lib.treewy_add_norm(ctypes.byref(a), None) == INVALID
    a = norm()
    a.residual = a.residual_out = a.y = a.y8 = None
    assert lib.treewy_add_norm(ctypes.byref(a), None) == INVALID
    assert lib.treewy_add_norm(None, None) == INVALID
    a = norm()
    a.T = 0
    assert lib.treewy_add_norm(ctypes.byref(a), None) == binding.TREEWY_OK


def tensors(R=2, T=5, Hq=4, Hkv=2, d=32, P=16, pages=6, width=3):
    e4m3, i32 = torch.float8_e4m3fn, torch.int32
    codes = torch.zeros(pages, Hkv, P, d, dtype=torch.uint8)
    c = dict(k=codes.view(e4m3), v=codes.clone().view(e4m3), k_scale=torch.ones(pages, Hkv), v_scale=torch.ones(pages, Hkv),
             page_table=torch.zeros(R, width, dtype=i32), length=torch.zeros(R, dtype=i32))
    rows = dict(node_offset=torch.zeros(R + 1, dtype=i32), status=torch.zeros(R, dtype=i32),
                k=torch.zeros(T, Hkv, d, dtype=torch.bfloat16), v=torch.zeros(T, Hkv, d, dtype=torch.bfloat16))
    query = dict(q=torch.zeros(T, Hq, d, dtype=torch.bfloat16), o=torch.zeros(T, Hq, d, dtype=torch.bfloat16), scale=1.0,
                 max_nodes=4, max_context=40)
    return c, rows, query


@pytest.mark.parametrize("name,change,error", [
    ("k", lambda x: x.view(torch.uint8), TypeError), ("v", lambda x: x[:-1], ValueError), ("k", lambda x: x[0], ValueError),
    ("k_scale", lambda x: x.double(), TypeError), ("v_scale", lambda x: x[:, :1], ValueError),
    ("page_table", lambda x: x.long(), TypeError), ("page_table", lambda x: x[0], ValueError),
    ("length", lambda x: x[:1], ValueError), ("k", lambda x: x.transpose(1, 2), ValueError),
])
def test_make_cache_refuses(name, change, error):
    c, _, _ = tensors()
    c[name] = change(c[name])
    with pytest.raises(error):
        binding.make_cache(**c)


@pytest.mark.parametrize("name,change,error", [
    ("q", lambda x: x.half(), TypeError), ("q", lambda x: x[:-1], ValueError), ("q", lambda x: x.float(), TypeError),
    ("k", lambda x: x[:, :1], ValueError), ("v", lambda x: x[:, :, :16], ValueError), ("o", lambda x: x[:-1], ValueError),
    ("o", lambda x: x.half(), TypeError), ("node_offset", lambda x: x[:-1], ValueError),
    ("status", lambda x: x.long(), TypeError), ("q", lambda x: x.transpose(1, 2), ValueError),
])
def test_make_attn_refuses(lib, name, change, error):  # noqa: F811
    c, rows, query = tensors()
    args = {**rows, **query}
    args[name] = change(args[name])
    with pytest.raises(error):
        binding.make_attn(cache=binding.make_cache(**c), **args)


def test_calls_refuse_tensors_on_the_cpu(lib):  # noqa: F811
    c, rows, query = tensors()
    made = binding.make_cache(**c)
    with pytest.raises(ValueError, match="CPU"):
        binding.treewy_attend(binding.make_attn(cache=made, **rows, **query))
    with pytest.raises(ValueError, match="CPU"):
        binding.treewy_append(binding.make_append(cache=made, max_new=4, **rows))
    with pytest.raises(ValueError, match="CPU"):
        binding.treewy_add_norm(binding.make_norm(x=torch.zeros(2, 64), y=torch.zeros(2, 64)))


@pytest.mark.parametrize("change,error", [
    (dict(x=torch.zeros(2, 64).half()), TypeError), (dict(residual=torch.zeros(2, 32)), ValueError),
    (dict(residual=torch.zeros(2, 64)), ValueError), (dict(residual_out=torch.zeros(2, 64)), ValueError),
    (dict(y=torch.zeros(2, 64).bfloat16()), TypeError), (dict(y8=torch.zeros(2, 64).to(torch.float8_e4m3fn)), ValueError),
    (dict(y8=torch.zeros(2, 64).to(torch.float8_e4m3fn), y8_scale=torch.zeros(2, 2), group=64), ValueError),
    (dict(weight=torch.zeros(63)), ValueError), (dict(x=torch.zeros(64, 2).T), ValueError),
    (dict(x=torch.zeros(1, 64).expand(2, 64)), ValueError),
])
def test_make_norm_refuses(change, error):
    with pytest.raises(error):
        binding.make_norm(**{**dict(x=torch.zeros(2, 64), y=torch.zeros(2, 64)), **change})


def test_the_codes_are_torchs():
    """Every code's value, and the rounding of values on, between and beyond the steps."""
    code = torch.arange(256, dtype=torch.uint8)
    ours, theirs = orc.from_e4m3(code.numpy()), code.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ours, theirs, equal_nan=True)
    values = np.sort(ours[np.isfinite(ours)])
    middle = (values[1:] + values[:-1]) / 2
    x = np.concatenate([values, middle, middle * (1 + 1e-7), middle * (1 - 1e-7),
                        np.random.RandomState(0).randn(5000) * 100]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    assert np.array_equal(orc.to_e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert orc.from_e4m3(orc.to_e4m3(np.array([1e9, -460.0]))).tolist() == [448.0, -448.0]
    assert np.isnan(orc.from_e4m3(orc.to_e4m3(np.array([np.inf, -np.inf, np.nan])))).all()


def test_scales_are_the_least_that_hold():
    for x in (1e-30, 0.0, 2.0 ** -40 * 448, 2.0 ** -31, 0.9, 447.9, 448.0, 448.1, 1e5, 3e38):
        s = orc.page_scale(x)
        assert x <= 448 * s and (s == 2.0 ** -40 or x > 448 * s / 2)


def test_definitions_by_hand():
    """One node sees the context and itself; its sibling's child does not see it."""
    one = np.ones((1, 1, 1))
    k = np.zeros((3, 1, 1))
    v = np.array([1.0, 10.0, 100.0]).reshape(3, 1, 1)
    q = np.zeros((3, 1, 1))
    o = orc.attend(q, k, v, [-1, 0, 0], np.zeros((1, 2, 1)), 4 * np.ones((1, 2, 1)), 1.0)
    assert np.allclose(o[:, 0, 0], [(8 + 1) / 3, (8 + 1 + 10) / 4, (8 + 1 + 100) / 4])
    o = orc.attend(np.log(3) * one, one, 5 * one, [-1], 0 * np.ones((1, 1, 1)), one, 1.0)
    assert np.allclose(o, (1 * 1 + 3 * 5) / 4)


def test_append_grows_a_page():
    """A larger token raises the page's scale: the older codes stand for the same values."""
    codes, scale = np.full((2, 1, 16, 2), 127, np.uint8), np.full((2, 1), 99.0)
    rows = np.array([[[1.0, -0.5]], [[0.25, 448.0]], [[500.0, 3.0]]])
    orc.append(codes, scale, [1], 0, rows[:1])
    assert scale[1, 0] == 2.0 ** -8
    orc.append(codes, scale, [1], 1, rows[1:])
    assert scale[1, 0] == 2.0
    got = orc.gather(codes, scale, [1], 3)[0]
    assert np.allclose(got, [[1.0, -0.5], [0.25, 448.0], [512.0, 3.0]])
    assert (codes[1, 0, 3:] == 127).all() and (codes[0] == 127).all()
