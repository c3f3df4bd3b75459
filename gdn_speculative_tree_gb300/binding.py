"""Thin Python binding of the TreeWY C ABI (include/treewy.h).

Argument marshalling only: every step of verification and commit runs in the
CUDA library.  There is no CPU fallback; if the library is missing this
module raises instead of computing anything.

Entry points keep the C names: ``treewy_verify``, ``treewy_commit``,
``treewy_storeall_verify``, ``treewy_storeall_commit``, ``treewy_extend``,
``treewy_qk_norm``, ``treewy_copy_slots``, ``treewy_attend``,
``treewy_append``, ``treewy_add_norm``, ``treewy_last_error`` and
``treewy_version``.  ``TreewyBatch`` mirrors ``struct treewy_batch``;
``make_batch`` fills one from torch tensors (device memory and streams are
PyTorch's; the library only receives raw pointers), as ``make_seqs``,
``make_qk`` and ``make_slots`` fill the arguments of the three calls around
verification, and ``make_cache``, ``make_attn``, ``make_append`` and
``make_norm`` those of the softmax layers' calls.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtreewy.so")

TREEWY_OK = 0
TREEWY_ERR_INVALID_ARG = 1
TREEWY_ERR_UNSUPPORTED = 3
TREEWY_ERR_CUDA = 4

STATUS_BAD_TREE = 1
STATUS_TOO_MANY_NODES = 2
STATUS_BAD_ACCEPTED = 4
STATUS_BAD_SLOT = 8
STATUS_TIMEOUT = 16
STATUS_COMMIT_REFUSED = 32
STATUS_BAD_POSITION = 64
STATUS_SLOT_CLASH = 128
STATUS_BAD_PAGE = 256

DTYPE_BF16 = 0
DTYPE_F32 = 1
FLAG_FORCE_GENERIC = 1
FLAG_STATE_BF16 = 2
NORM_L2 = 0
NORM_RMS = 1
MAX_NODES = 64


class TreewyError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"treewy error {code}: {message}")
        self.code = code


class TreewyBatch(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int32),
        ("H", ctypes.c_int32),
        ("dk", ctypes.c_int32),
        ("dv", ctypes.c_int32),
        ("max_nodes", ctypes.c_int32),
        ("qkv_dtype", ctypes.c_int32),
        ("T", ctypes.c_int64),
        ("num_slots", ctypes.c_int64),
        ("node_offset", ctypes.c_void_p),
        ("parent", ctypes.c_void_p),
        ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("alpha", ctypes.c_void_p),
        ("beta", ctypes.c_void_p),
        ("state", ctypes.c_void_p),
        ("state_slot", ctypes.c_void_p),
        ("o", ctypes.c_void_p),
        ("U", ctypes.c_void_p),
        ("gamma", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
        ("flags", ctypes.c_uint32),
        ("reserved", ctypes.c_uint32),
    ]


class TreewySeqs(ctypes.Structure):
    _device = None  # of the tensors it was made from
    _fields_ = [(f, ctypes.c_int32) for f in
                ("R", "H", "Hk", "dk", "dv", "max_len", "qkv_dtype", "o_dtype")] + [
        (f, ctypes.c_int64) for f in ("T", "num_slots", "q_stride", "k_stride", "v_stride")] + [
        (f, ctypes.c_void_p) for f in
        ("seq_offset", "q", "k", "v", "alpha", "beta", "state", "state_slot", "fresh", "o", "status")] + [
        ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class TreewyQk(ctypes.Structure):
    _device = None  # of the tensors it was made from
    _fields_ = [("T", ctypes.c_int64)] + [(f, ctypes.c_int32) for f in
                ("Hq", "Hk", "d", "dtype", "norm", "rope_dims", "interleaved", "q_repeat", "k_repeat")] + [
        (f, ctypes.c_float) for f in ("eps", "q_scale", "k_scale")] + [
        (f, ctypes.c_int64) for f in ("q_stride", "k_stride", "rope_rows")] + [
        (f, ctypes.c_void_p) for f in
        ("q", "k", "q_weight", "k_weight", "rope", "position", "q_out", "k_out", "status")]


class TreewySlots(ctypes.Structure):
    _device = None  # of the tensors it was made from
    _fields_ = [("n", ctypes.c_int32), ("layers", ctypes.c_int32)] + [
        (f, ctypes.c_int64) for f in ("num_slots", "slot_bytes", "layer_stride")] + [
        (f, ctypes.c_void_p) for f in ("state", "src", "dst", "status")]


class TreewyCache(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("Hkv", "d", "page_len", "max_pages")] + [
        ("num_pages", ctypes.c_int64)] + [
        (f, ctypes.c_void_p) for f in ("k", "v", "k_scale", "v_scale", "page_table", "length")]


class TreewyAttn(ctypes.Structure):
    _device = None  # of the tensors it was made from
    _own = None     # workspaces that the binding made, by the stream whose memory each is
    _stream = None  # of the one in the fields
    _fields_ = [(f, ctypes.c_int32) for f in ("R", "Hq", "max_nodes", "max_context", "qkv_dtype", "o_dtype")] + [
        (f, ctypes.c_int64) for f in ("T", "q_stride", "k_stride", "v_stride")] + [
        (f, ctypes.c_void_p) for f in ("node_offset", "parent", "q", "k", "v", "o", "status", "workspace")] + [
        ("workspace_bytes", ctypes.c_uint64), ("scale", ctypes.c_float), ("flags", ctypes.c_uint32),
        ("cache", TreewyCache)]


class TreewyAppendArgs(ctypes.Structure):
    _device = None  # of the tensors it was made from
    _fields_ = [("R", ctypes.c_int32), ("max_new", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_uint32)] + [
        (f, ctypes.c_int64) for f in ("T", "k_stride", "v_stride")] + [
        (f, ctypes.c_void_p) for f in ("node_offset", "parent", "accepted", "k", "v", "new_length", "status")] + [
        ("cache", TreewyCache)]


class TreewyNorm(ctypes.Structure):
    _device = None  # of the tensors it was made from
    _fields_ = [(f, ctypes.c_int64) for f in ("T", "x_stride", "residual_stride")] + [
        (f, ctypes.c_int32) for f in ("n", "x_dtype", "residual_dtype", "group")] + [
        ("eps", ctypes.c_float), ("reserved", ctypes.c_uint32)] + [
        (f, ctypes.c_void_p) for f in ("x", "residual", "residual_out", "weight", "y", "y8", "y8_scale")]


_lib: Optional[ctypes.CDLL] = None

ENTRY_POINTS = ("treewy_verify", "treewy_commit", "treewy_commit_verify", "treewy_storeall_verify",
                "treewy_storeall_commit", "treewy_extend", "treewy_qk_norm", "treewy_copy_slots",
                "treewy_attend", "treewy_attend_workspace", "treewy_append", "treewy_add_norm",
                "treewy_selftest_wait_timeout", "treewy_last_error", "treewy_version")


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libtreewy.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"TreeWY CUDA library not found at {p}; build it with "
            "gdn_speculative_tree_gb300.build.build() (there is no CPU fallback)")
    lib = ctypes.CDLL(p)
    bp = ctypes.POINTER(TreewyBatch)
    vp = ctypes.c_void_p
    lib.treewy_verify.argtypes = [bp, vp]
    lib.treewy_commit.argtypes = [bp, vp, vp]
    lib.treewy_commit_verify.argtypes = [bp, vp, bp, vp]
    lib.treewy_storeall_verify.argtypes = [bp, vp, vp]
    lib.treewy_storeall_commit.argtypes = [bp, vp, vp, vp]
    lib.treewy_extend.argtypes = [ctypes.POINTER(TreewySeqs), vp]
    lib.treewy_qk_norm.argtypes = [ctypes.POINTER(TreewyQk), vp]
    lib.treewy_copy_slots.argtypes = [ctypes.POINTER(TreewySlots), vp]
    lib.treewy_attend.argtypes = [ctypes.POINTER(TreewyAttn), vp]
    lib.treewy_attend_workspace.argtypes = [ctypes.POINTER(TreewyAttn), ctypes.POINTER(ctypes.c_uint64)]
    lib.treewy_append.argtypes = [ctypes.POINTER(TreewyAppendArgs), vp]
    lib.treewy_add_norm.argtypes = [ctypes.POINTER(TreewyNorm), vp]
    lib.treewy_selftest_wait_timeout.argtypes = [vp, ctypes.c_uint32, vp]
    for name in ("treewy_verify", "treewy_commit", "treewy_commit_verify", "treewy_storeall_verify",
                 "treewy_storeall_commit", "treewy_extend", "treewy_qk_norm", "treewy_copy_slots",
                 "treewy_attend", "treewy_attend_workspace", "treewy_append", "treewy_add_norm",
                 "treewy_selftest_wait_timeout"):
        getattr(lib, name).restype = ctypes.c_int
    lib.treewy_last_error.argtypes = []
    lib.treewy_last_error.restype = ctypes.c_char_p
    lib.treewy_version.argtypes = []
    lib.treewy_version.restype = ctypes.c_char_p
    if path is None:
        _lib = lib
    return lib


def _check(code: int) -> None:
    if code != TREEWY_OK:
        raise TreewyError(code, treewy_last_error())


_current_raw_stream = None


def _current_stream_handle() -> int:
    """The current stream's handle, by the call that makes no Stream object
    where this PyTorch has it (a small call's time is mostly the host's)."""
    global _current_raw_stream
    if _current_raw_stream is None:
        import torch
        torch.cuda.current_stream()  # initialises CUDA
        raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        _current_raw_stream = ((lambda: raw(device())) if raw is not None and device is not None
                               else (lambda: torch.cuda.current_stream().cuda_stream))
    return _current_raw_stream()


_get_device = None


def _current_device() -> int:
    global _get_device
    if _get_device is None:
        import torch
        # without the checks of torch.cuda.current_device, where this PyTorch has it
        _get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _get_device()


def _reachable(args) -> None:
    """Refuses arguments described from tensors that a kernel on the current device cannot reach."""
    device = args._device
    if device is None:
        return
    if device < 0:
        raise ValueError("the tensors are on the CPU")
    if device != _current_device():
        raise ValueError(f"the tensors are on device {device}, the current device is {_current_device()}")


def _stream_handle(stream) -> int:
    if stream is None:
        return _current_stream_handle()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _own_workspace(attn, handle: int) -> None:
    """The structure's own workspace for calls on this stream, from this stream's memory: when it is given back, nobody gets
    it before what the stream has been told until then is done."""
    import torch
    if handle not in attn._own:
        made = next(iter(attn._own.values()))
        stream = (torch.cuda.default_stream(made.device) if handle == 0
                  else torch.cuda.ExternalStream(handle, device=made.device))
        with torch.cuda.stream(stream):
            attn._own[handle] = torch.empty_like(made)
    attn._stream, attn.workspace = handle, attn._own[handle].data_ptr()


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def treewy_last_error() -> str:
    return load().treewy_last_error().decode()


def treewy_version() -> str:
    return load().treewy_version().decode()


def treewy_selftest_wait_timeout(status, limit_us: int, stream=None) -> None:
    """Diagnostic of the bounded barrier wait: ``status`` is a device int32
    tensor of 3 words (status[0] gets TREEWY_STATUS_TIMEOUT, status[1:3] the
    wait in nanoseconds, low and high word)."""
    _check(load().treewy_selftest_wait_timeout(_ptr(status), int(limit_us), _stream_handle(stream)))


def treewy_verify(batch: TreewyBatch, stream=None) -> None:
    """Verify every draft node (asynchronous on ``stream``)."""
    _check(load().treewy_verify(ctypes.byref(batch), _stream_handle(stream)))


def treewy_commit(batch: TreewyBatch, accepted, stream=None) -> None:
    """Rebuild the accepted state in place; ``accepted`` int32 [R] on the device."""
    _check(load().treewy_commit(ctypes.byref(batch), _ptr(accepted), _stream_handle(stream)))


def treewy_commit_verify(prev: TreewyBatch, prev_accepted, next_batch: TreewyBatch,
                         stream=None) -> None:
    """Apply the previous round's commit inside this round's verification."""
    _check(load().treewy_commit_verify(ctypes.byref(prev), _ptr(prev_accepted), ctypes.byref(next_batch),
                                       _stream_handle(stream)))


def treewy_storeall_verify(batch: TreewyBatch, snapshots, stream=None) -> None:
    """Snapshot-per-node comparator: writes every node's state to ``snapshots``."""
    _check(load().treewy_storeall_verify(ctypes.byref(batch), _ptr(snapshots), _stream_handle(stream)))


def treewy_storeall_commit(batch: TreewyBatch, snapshots, accepted, stream=None) -> None:
    """Snapshot rollback: copy the accepted node's snapshot into the state pool."""
    _check(load().treewy_storeall_commit(ctypes.byref(batch), _ptr(snapshots), _ptr(accepted),
                                         _stream_handle(stream)))


def treewy_extend(seqs: TreewySeqs, stream=None) -> None:
    """The gated delta rule over every sequence's new tokens, from and into its state slot."""
    _reachable(seqs)
    _check(load().treewy_extend(ctypes.byref(seqs), _stream_handle(stream)))


def treewy_qk_norm(qk: TreewyQk, stream=None) -> None:
    """Norm, weight, scale and rotation of every query and key head."""
    _reachable(qk)
    _check(load().treewy_qk_norm(ctypes.byref(qk), _stream_handle(stream)))


def treewy_copy_slots(slots: TreewySlots, stream=None) -> None:
    """Copy, fork, compact and clear slots of the state pools of all layers."""
    _reachable(slots)
    _check(load().treewy_copy_slots(ctypes.byref(slots), _stream_handle(stream)))


def treewy_attend(attn: TreewyAttn, stream=None) -> None:
    """Softmax attention of every draft node over its context in 8 bits and its path in the draft."""
    _reachable(attn)
    handle = _stream_handle(stream)
    if attn._own is not None and handle != attn._stream:
        _own_workspace(attn, handle)
    _check(load().treewy_attend(ctypes.byref(attn), handle))


def treewy_append(args: TreewyAppendArgs, stream=None) -> None:
    """Accepted (or all) rows of keys and values into the 8-bit pages."""
    _reachable(args)
    _check(load().treewy_append(ctypes.byref(args), _stream_handle(stream)))


def treewy_add_norm(norm: TreewyNorm, stream=None) -> None:
    """The residual's addition and the RMS norm, in 8 bits with scales where wanted."""
    _reachable(norm)
    _check(load().treewy_add_norm(ctypes.byref(norm), _stream_handle(stream)))


def treewy_attend_workspace(attn: TreewyAttn) -> int:
    """Bytes of workspace that a call with these sizes needs."""
    n = ctypes.c_uint64(0)
    _check(load().treewy_attend_workspace(ctypes.byref(attn), ctypes.byref(n)))
    return n.value


def make_batch(*, node_offset, parent, q, k, v, alpha, beta, state, state_slot, o, U, status,
               gamma=None, max_nodes: int = MAX_NODES, T: Optional[int] = None,
               flags: int = 0) -> TreewyBatch:
    """Fill a TreewyBatch from torch tensors (shapes as in include/treewy.h).

    The tensors must stay alive while the library uses them; the returned
    structure keeps references to them in ``_keep``.
    """
    import torch
    R = int(node_offset.numel()) - 1
    Tn = int(q.shape[0]) if T is None else int(T)
    H = int(q.shape[1])
    dk = int(q.shape[2])
    dv = int(v.shape[2])
    if q.dtype == torch.bfloat16:
        dt = DTYPE_BF16
    elif q.dtype == torch.float32:
        dt = DTYPE_F32
    else:
        raise TypeError(f"q/k/v dtype {q.dtype} is not bf16 or fp32")
    for name, x in (("q", q), ("k", k), ("v", v), ("alpha", alpha), ("beta", beta), ("state", state),
                    ("o", o), ("U", U), ("status", status), ("node_offset", node_offset),
                    ("parent", parent), ("state_slot", state_slot)):
        if x is not None and not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if state.dtype == torch.bfloat16:
        flags |= FLAG_STATE_BF16
    elif state.dtype != torch.float32:
        raise TypeError(f"state dtype {state.dtype} is not fp32 or bf16")
    b = TreewyBatch()
    b.R, b.H, b.dk, b.dv = R, H, dk, dv
    b.max_nodes = int(max_nodes)
    b.qkv_dtype = dt
    b.T = Tn
    b.num_slots = int(state.shape[0])
    b.node_offset = _ptr(node_offset)
    b.parent = _ptr(parent)
    b.q, b.k, b.v = _ptr(q), _ptr(k), _ptr(v)
    b.alpha, b.beta = _ptr(alpha), _ptr(beta)
    b.state = _ptr(state)
    b.state_slot = _ptr(state_slot)
    b.o, b.U = _ptr(o), _ptr(U)
    b.gamma = _ptr(gamma)
    b.status = _ptr(status)
    b.flags = int(flags)
    b._keep = (node_offset, parent, q, k, v, alpha, beta, state, state_slot, o, U, gamma, status)
    return b


def _dtype_code(x, name: str) -> int:
    import torch
    if x.dtype == torch.bfloat16:
        return DTYPE_BF16
    if x.dtype == torch.float32:
        return DTYPE_F32
    raise TypeError(f"{name} dtype {x.dtype} is not bf16 or fp32")


def _need(x, name: str, dtype, shape=None) -> None:
    """``x`` is contiguous, of this type and, where given, of this shape; None passes."""
    if x is None:
        return
    if x.dtype != dtype:
        raise TypeError(f"{name} dtype {x.dtype} is not {dtype}")
    if shape is not None and x.shape != shape:
        raise ValueError(f"{name} has shape {tuple(x.shape)}, not {tuple(shape)}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _one_device(tensors) -> int:
    """The device that all of the tensors are on (-1: the CPU)."""
    found = {x.get_device() for x in tensors if x is not None}
    if len(found) > 1:
        raise ValueError(f"tensors on several devices: {sorted(found)} (-1: the CPU)")
    return found.pop()


def _token_stride(x, name: str) -> int:
    """Elements between the token rows of ``x`` [T][heads][d], whose heads are
    contiguous within a row (a slice of a fused projection has longer rows)."""
    if x.dim() != 3:
        raise ValueError(f"{name} must be [T][heads][d]")
    T, heads, d = x.shape
    st, sh, sd = x.stride()
    if (d > 1 and sd != 1) or (heads > 1 and sh != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if T <= 1 or heads * d == 0:
        return heads * d
    if st < heads * d:
        raise ValueError(f"{name}: token rows overlap")
    return st


def make_seqs(*, seq_offset, q, k, v, alpha, beta, state, state_slot, o, status, max_len: int, fresh=None,
              flags: int = 0) -> TreewySeqs:
    """Fill a TreewySeqs from torch tensors (shapes as in include/treewy.h; the
    token rows of q, k and v may be strided).  ``max_len`` bounds every
    sequence's number of new tokens.  The structure keeps the tensors alive.
    """
    import torch
    strides = [_token_stride(x, n) for n, x in (("q", q), ("k", k), ("v", v))]
    T, Hk, dk = q.shape
    Tv, H, dv = v.shape
    R = seq_offset.numel() - 1
    if k.shape != q.shape or Tv != T:
        raise ValueError("k must have q's shape, and v as many tokens")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must have one dtype")
    i32, f32 = torch.int32, torch.float32
    num_slots = state.shape[0]
    _need(seq_offset, "seq_offset", i32, (R + 1,))
    _need(state_slot, "state_slot", i32, (R,))
    _need(status, "status", i32, (R,))
    _need(fresh, "fresh", torch.uint8, (R,))
    _need(alpha, "alpha", f32, (T, H))
    _need(beta, "beta", f32, (T, H))
    _need(o, "o", o.dtype, (T, H, dv))
    _need(state, "state", state.dtype, (num_slots, H, dv, dk))
    keep = (seq_offset, q, k, v, alpha, beta, state, state_slot, fresh, o, status)
    device = _one_device(keep)
    if _dtype_code(state, "state") == DTYPE_BF16:
        flags |= FLAG_STATE_BF16
    s = TreewySeqs(R, H, Hk, dk, dv, int(max_len), _dtype_code(q, "q/k/v"), _dtype_code(o, "o"), T, num_slots,
                   *strides, *map(_ptr, keep), int(flags), 0)
    s._keep, s._device = keep, device
    return s


def make_qk(*, q=None, k=None, q_out=None, k_out=None, norm: str = "l2", eps: float = 1e-6, q_weight=None,
            k_weight=None, q_scale: float = 1.0, k_scale: float = 1.0, rope=None, position=None,
            interleaved: bool = False, status=None) -> TreewyQk:
    """Fill a TreewyQk from torch tensors: q [T][Hq][d], k [T][Hk][d] (strided
    token rows allowed; either may be left out), outputs with a multiple of
    their heads, ``norm`` "l2" or "rms", ``rope`` f32 [rows][rotated dims].
    """
    import torch
    if q is None and k is None:
        raise ValueError("q or k is needed")
    if norm not in ("l2", "rms"):
        raise ValueError(f"norm {norm!r} is not 'l2' or 'rms'")
    x = q if q is not None else k
    T, d = int(x.shape[0]), int(x.shape[2])
    a = TreewyQk()
    a.T, a.d, a.dtype = T, d, _dtype_code(x, "q/k")
    a.norm = NORM_L2 if norm == "l2" else NORM_RMS
    a.q_repeat = a.k_repeat = 1
    for name, src, out, w in (("q", q, q_out, q_weight), ("k", k, k_out, k_weight)):
        if src is None:
            continue
        stride = _token_stride(src, name)
        heads = int(src.shape[1])
        if (int(src.shape[0]), int(src.shape[2]), src.dtype) != (T, d, x.dtype):
            raise ValueError("q and k must agree on tokens, head size and dtype")
        if out is None:
            raise ValueError(f"{name}_out is needed")
        repeat = int(out.shape[1]) // heads if heads else 1
        _need(out, f"{name}_out", x.dtype, (T, heads * repeat, d))
        _need(w, f"{name}_weight", torch.float32, (d,))
        if repeat < 1 and heads:
            raise ValueError(f"{name}_out has fewer heads than {name}")
        setattr(a, "Hq" if name == "q" else "Hk", heads)
        setattr(a, f"{name}_repeat", max(repeat, 1))
        setattr(a, f"{name}_stride", stride)
        setattr(a, name, _ptr(src))
        setattr(a, f"{name}_out", _ptr(out))
        setattr(a, f"{name}_weight", _ptr(w))
    if rope is not None:
        _need(rope, "rope", torch.float32, (rope.shape[0], rope.shape[1]))
        if position is None or status is None:
            raise ValueError("position and status are needed with rope")
        _need(position, "position", torch.int32, (T,))
        a.rope_rows, a.rope_dims = int(rope.shape[0]), int(rope.shape[1])
    if status is not None:
        _need(status, "status", torch.int32)
    keep = (q, k, q_out, k_out, q_weight, k_weight, rope, position, status)
    a._device = _one_device(keep)
    a.eps, a.q_scale, a.k_scale, a.interleaved = float(eps), float(q_scale), float(k_scale), int(interleaved)
    a.rope, a.position, a.status = _ptr(rope), _ptr(position), _ptr(status)
    a._keep = keep
    return a


def make_slots(*, state, src, dst, status, layers: Optional[int] = None) -> TreewySlots:
    """Fill a TreewySlots: ``state`` is one pool [num_slots][...] or, with
    ``layers`` given, [layers][num_slots][...] (each layer's pool contiguous);
    src, dst and status are int32 of one length, src -1 clears a slot.
    """
    import torch
    for name, x in (("src", src), ("dst", dst), ("status", status)):
        _need(x, name, torch.int32, (int(src.numel()),))
    pool = state if layers is None else state[0] if layers else None
    if layers is not None and int(state.shape[0]) != layers:
        raise ValueError(f"state has {int(state.shape[0])} layers, not {layers}")
    if pool is not None and not pool.is_contiguous():
        raise ValueError("a layer's pool must be contiguous")
    shape = state.shape[1:] if layers is not None else state.shape
    if len(shape) < 2:
        raise ValueError("state must be [num_slots][...] or [layers][num_slots][...]")
    per = 1
    for n in shape[1:]:
        per *= int(n)
    if layers is not None and layers > 1 and state.stride(0) < int(shape[0]) * per:
        raise ValueError("state: layers overlap")  # a stride of 0 would pass for dense layers
    device = _one_device((state, src, dst, status))
    a = TreewySlots()
    a.n, a.layers = int(src.numel()), 1 if layers is None else int(layers)
    a.num_slots, a.slot_bytes = int(shape[0]), per * state.element_size()
    a.layer_stride = int(state.stride(0)) * state.element_size() if layers is not None and layers > 1 else 0
    a.state, a.src, a.dst, a.status = _ptr(state), _ptr(src), _ptr(dst), _ptr(status)
    a._keep, a._device = (state, src, dst, status), device
    return a


def make_cache(*, k, v, k_scale, v_scale, page_table, length) -> TreewyCache:
    """Fill a TreewyCache: k and v float8_e4m3fn [num_pages][Hkv][page_len][d],
    scales f32 [num_pages][Hkv], page_table int32 [R][max_pages], length int32 [R].
    """
    import torch
    if k.dim() != 4 or page_table.dim() != 2:
        raise ValueError("k must be [num_pages][Hkv][page_len][d], page_table [R][max_pages]")
    num_pages, Hkv, page_len, d = k.shape
    _need(k, "k", torch.float8_e4m3fn)
    _need(v, "v", torch.float8_e4m3fn, k.shape)
    _need(k_scale, "k_scale", torch.float32, (num_pages, Hkv))
    _need(v_scale, "v_scale", torch.float32, (num_pages, Hkv))
    _need(page_table, "page_table", torch.int32)
    _need(length, "length", torch.int32, (page_table.shape[0],))
    keep = (k, v, k_scale, v_scale, page_table, length)
    c = TreewyCache(Hkv, d, page_len, page_table.shape[1], num_pages, *map(_ptr, keep))
    c._keep, c._device, c._R = keep, _one_device(keep), int(page_table.shape[0])
    return c


def _rows_of_cache(cache: TreewyCache, tensors, node_offset, status, others) -> tuple:
    """What make_attn and make_append check alike; the tensors' strides and the device."""
    import torch
    strides = [_token_stride(x, n) for n, x in tensors]
    T = tensors[0][1].shape[0]
    for n, x in tensors:
        if x.dtype != tensors[0][1].dtype:
            raise TypeError(f"{n} must have the other rows' dtype, {tensors[0][1].dtype}")
        if x.shape[0] != T or x.shape[2] != cache.d:
            raise ValueError(f"{n} must have {T} rows of the cache's head size {cache.d}")
        if n != "q" and x.shape[1] != cache.Hkv:
            raise ValueError(f"{n} must have the cache's {cache.Hkv} heads")
    _need(node_offset, "node_offset", torch.int32, (cache._R + 1,))
    _need(status, "status", torch.int32, (cache._R,))
    device = _one_device([x for _, x in tensors] + [node_offset, status, *others])
    if device != cache._device:
        raise ValueError(f"the cache is on device {cache._device}, the rows on {device} (-1: the CPU)")
    return T, strides, device


def make_attn(*, cache: TreewyCache, node_offset, q, k, v, o, status, scale: float, max_nodes: int, max_context: int,
              parent=None, workspace=None, flags: int = 0) -> TreewyAttn:
    """Fill a TreewyAttn: q [T][Hq][d], k and v [T][Hkv][d] (strided token rows
    allowed), o [T][Hq][d]; ``parent`` None: chains.  ``workspace`` is a uint8
    tensor; without one, the structure gets its own, as large as it needs, and
    another for each further stream that it is called on.  A captured call needs
    the structure for as long as the graph is replayed, and one replay at a time
    uses its workspace.
    """
    import torch
    T, strides, device = _rows_of_cache(cache, (("q", q), ("k", k), ("v", v)), node_offset, status,
                                        (o, parent, workspace))
    Hq = int(q.shape[1])
    _need(o, "o", o.dtype, (T, Hq, cache.d))
    _need(parent, "parent", torch.int32, (T,))
    _need(workspace, "workspace", torch.uint8)
    a = TreewyAttn()
    a.R, a.Hq, a.max_nodes, a.max_context = cache._R, Hq, int(max_nodes), int(max_context)
    a.qkv_dtype, a.o_dtype, a.T = _dtype_code(q, "q/k/v"), _dtype_code(o, "o"), T
    a.q_stride, a.k_stride, a.v_stride = strides
    a.scale, a.flags, a.cache = float(scale), int(flags), cache
    if workspace is None:
        workspace = torch.empty(treewy_attend_workspace(a), dtype=torch.uint8, device=q.device)
        if q.is_cuda and workspace.numel() > 0:
            a._stream = torch.cuda.current_stream(q.device).cuda_stream
            a._own = {a._stream: workspace}
    a.node_offset, a.parent, a.q, a.k, a.v, a.o, a.status = map(_ptr, (node_offset, parent, q, k, v, o, status))
    a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel()
    a._keep, a._device = (cache._keep, node_offset, parent, q, k, v, o, status, workspace), device
    return a


def make_append(*, cache: TreewyCache, node_offset, k, v, status, max_new: int, parent=None, accepted=None,
                new_length=None) -> TreewyAppendArgs:
    """Fill a TreewyAppendArgs: k and v [T][Hkv][d] (strided token rows allowed);
    ``accepted`` None: every row; ``new_length`` int32 [R], not the cache's own.
    """
    import torch
    T, strides, device = _rows_of_cache(cache, (("k", k), ("v", v)), node_offset, status, (parent, accepted, new_length))
    _need(parent, "parent", torch.int32, (T,))
    _need(accepted, "accepted", torch.int32, (cache._R,))
    _need(new_length, "new_length", torch.int32, (cache._R,))
    a = TreewyAppendArgs()
    a.R, a.max_new, a.kv_dtype, a.T = cache._R, int(max_new), _dtype_code(k, "k/v"), T
    a.k_stride, a.v_stride = strides
    a.cache = cache
    a.node_offset, a.parent, a.accepted, a.k, a.v, a.new_length, a.status = map(
        _ptr, (node_offset, parent, accepted, k, v, new_length, status))
    a._keep, a._device = (cache._keep, node_offset, parent, accepted, k, v, new_length, status), device
    return a


def _row_stride(x, name: str) -> int:
    """Elements between the rows of ``x`` [T][n], contiguous within a row."""
    T, n = x.shape
    if n > 1 and x.stride(1) != 1:
        raise ValueError(f"{name}: a row must be contiguous")
    if T <= 1:
        return n
    if x.stride(0) < n:
        raise ValueError(f"{name}: rows overlap")
    return x.stride(0)


def make_norm(*, x, residual=None, residual_out=None, weight=None, eps: float = 1e-6, y=None, y8=None, y8_scale=None,
              group: int = 0) -> TreewyNorm:
    """Fill a TreewyNorm: x [T][n] and residual [T][n] (strided rows allowed),
    residual_out of the residual's type, y of x's, y8 float8_e4m3fn with
    y8_scale [T][groups]; ``group`` columns to a scale, 0: the row.
    """
    import torch
    if x.dim() != 2 or (residual is not None and residual.shape != x.shape):
        raise ValueError("x and residual must be [T][n]")
    T, n = x.shape
    if residual is None and residual_out is not None:
        raise ValueError("residual_out without a residual")
    if y8 is not None and y8_scale is None:
        raise ValueError("y8_scale is needed with y8")
    a = TreewyNorm()
    a.T, a.n, a.group, a.eps = T, n, int(group), float(eps)
    a.x_dtype, a.x_stride = _dtype_code(x, "x"), _row_stride(x, "x")
    if residual is not None:
        a.residual_dtype, a.residual_stride = _dtype_code(residual, "residual"), _row_stride(residual, "residual")
        if residual_out is None:
            raise ValueError("residual_out is needed with a residual")
        _need(residual_out, "residual_out", residual.dtype, (T, n))
    _need(weight, "weight", torch.float32, (n,))
    _need(y, "y", x.dtype, (T, n))
    _need(y8, "y8", torch.float8_e4m3fn, (T, n))
    if y8 is not None:
        _need(y8_scale, "y8_scale", torch.float32, (T, -(-n // group) if group else 1))
    keep = (x, residual, residual_out, weight, y, y8, y8_scale)
    a._device = _one_device(keep)
    a.x, a.residual, a.residual_out, a.weight, a.y, a.y8, a.y8_scale = map(_ptr, keep)
    a._keep = keep
    return a


class TreeVerifier:
    """Convenience holder: one layer's device tensors, outputs and batch struct.

    ``wl`` is a workloads.Workload already on the device.  Outputs o, U,
    gamma and status are allocated once (torch) and reused across calls.
    """

    def __init__(self, wl, flags: int = 0, max_nodes: Optional[int] = None):
        import torch
        dev = wl.q.device
        self.wl = wl
        self.o = torch.empty(wl.T, wl.H, wl.dv, device=dev, dtype=torch.float32)
        self.U = torch.empty_like(self.o)
        self.gamma = torch.empty(wl.T, wl.H, device=dev, dtype=torch.float32)
        self.status = torch.zeros(wl.R, device=dev, dtype=torch.int32)
        self.batch = make_batch(node_offset=wl.node_offset, parent=wl.parent, q=wl.q, k=wl.k,
                                v=wl.v, alpha=wl.alpha, beta=wl.beta, state=wl.state,
                                state_slot=wl.state_slot, o=self.o, U=self.U, status=self.status,
                                gamma=self.gamma, max_nodes=max_nodes or wl.max_nodes, flags=flags)

    def verify(self, stream=None) -> None:
        treewy_verify(self.batch, stream)

    def commit(self, accepted=None, stream=None) -> None:
        treewy_commit(self.batch, self.wl.accepted if accepted is None else accepted, stream)
