"""Thin ctypes binding of libmoe_ep.so (include/moe_ep.h).

Argument marshalling only: every function passes torch tensors' device
pointers and the current CUDA stream to the C entry point of the same name and
raises MoeError on a negative return code. No step of the path runs here.
If the library has not been built, loading it raises immediately: there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

from . import build as _build

MOE_BF16 = 0
MOE_FP8_E4M3 = 1
MOE_INT8 = 2
MOE_STATUS_BAD_EXPERT_ID = 0x1
MOE_STATUS_TIMEOUT = 0x2
MOE_STATUS_SLOT_OVERFLOW = 0x4
MOE_STATUS_BOUNDS = 0x8
MOE_FORM_ROWS = 0
MOE_FORM_TILES = 1
MOE_FORM_WIDENED = 2
MOE_MAX_EXPERTS = 1024
MOE_MAX_TOPK = 32
MOE_MAX_RANKS = 1024

_c_void_p = ctypes.c_void_p

#: Every symbol include/moe_ep.h declares.
EXPORTED_SYMBOLS = (
    "moe_workspace_bytes", "moe_recv_rows_max", "moe_handle_create", "moe_handle_destroy",
    "moe_route_topk", "moe_dispatch_layout", "moe_route_dispatch_layout", "moe_get_layout",
    "moe_dispatch", "moe_expert_standin", "moe_combine", "moe_read_status", "moe_error_string",
    "moe_dispatch_layout_noalloc", "moe_copy_h2d_async", "moe_copy_d2h_async",
    "moe_dispatch_two_stage", "moe_layout_dispatch_fused", "moe_set_wait_limit",
    "moe_dispatch_tokens", "moe_expert_standin_tokens", "moe_combine_tokens",
    "moe_dispatch_allgather", "moe_layout_tables", "moe_dispatch_fixed_slots",
    "moe_fixed_slot_rows", "moe_debug_bounds", "moe_expert_workspace_bytes", "moe_expert_create",
    "moe_expert_destroy", "moe_expert_gated", "moe_expert_down", "moe_expert_backward",
    "moe_expert_set_wait_limit", "moe_expert_read_status", "moe_combine_backward",
    "moe_expert_form",
)


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed: {msg} ({code})")
        self.code = code


class moe_config_t(ctypes.Structure):
    _fields_ = [("num_ranks", ctypes.c_int32), ("tokens_per_rank", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("dispatch_dtype", ctypes.c_int32),
                ("combine_dtype", ctypes.c_int32), ("expert_capacity", ctypes.c_int32)]


class moe_layout_view_t(ctypes.Structure):
    _fields_ = [(n, _c_void_p) for n in (
        "expert_count", "expert_count_raw", "expert_offset", "src_expert_count",
        "src_expert_kept", "count_matrix", "send_offset", "recv_offset", "rank_base", "inv",
        "totals")]


class moe_recv_meta_t(ctypes.Structure):
    _fields_ = [(n, _c_void_p) for n in (
        "local_expert", "src_rank", "src_token", "slot", "weight")]


class moe_expert_config_t(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("inter", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("rows_max", ctypes.c_int64), ("train", ctypes.c_int32)]


class moe_expert_form_t(ctypes.Structure):
    _fields_ = [("kernels", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("split", ctypes.c_int32)]


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    """The release library; with MOE_EP_DEBUG_BOUNDS=1 in the environment the
    build with device bounds checks (MOE_STATUS_BOUNDS); with MOE_EP_LIBRARY
    set, that file (another build of the same sources)."""
    if os.environ.get("MOE_EP_LIBRARY"):
        return os.environ["MOE_EP_LIBRARY"]
    if os.environ.get("MOE_EP_DEBUG_BOUNDS", "") == "1":
        return _build.DEBUG_LIB_PATH
    return _build.LIB_PATH


def load_library():
    """Loads the built library; raises if it is missing (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise ImportError(
                f"libmoe_ep.so is not built ({path}); run __graft_entry__.build() first")
        lib = ctypes.CDLL(path)
        i32, sz, vp = ctypes.c_int, ctypes.c_size_t, _c_void_p
        cfgp = ctypes.POINTER(moe_config_t)
        lib.moe_workspace_bytes.restype = sz
        lib.moe_workspace_bytes.argtypes = [cfgp]
        lib.moe_recv_rows_max.restype = ctypes.c_int64
        lib.moe_recv_rows_max.argtypes = [cfgp]
        lib.moe_handle_create.restype = i32
        lib.moe_handle_create.argtypes = [cfgp, vp, sz, ctypes.POINTER(vp)]
        lib.moe_handle_destroy.restype = i32
        lib.moe_handle_destroy.argtypes = [vp]
        lib.moe_route_topk.restype = i32
        lib.moe_route_topk.argtypes = [vp, vp, vp, vp, vp]
        lib.moe_dispatch_layout.restype = i32
        lib.moe_dispatch_layout.argtypes = [vp, vp, vp]
        lib.moe_route_dispatch_layout.restype = i32
        lib.moe_route_dispatch_layout.argtypes = [vp, vp, vp, vp, vp]
        lib.moe_dispatch_fixed_slots.restype = i32
        lib.moe_dispatch_fixed_slots.argtypes = [vp, vp, vp, vp, vp, ctypes.POINTER(moe_recv_meta_t), vp]
        lib.moe_fixed_slot_rows.restype = ctypes.c_int64
        lib.moe_fixed_slot_rows.argtypes = [cfgp]
        lib.moe_layout_tables.restype = i32
        lib.moe_layout_tables.argtypes = [vp, vp]
        lib.moe_get_layout.restype = i32
        lib.moe_get_layout.argtypes = [vp, ctypes.POINTER(moe_layout_view_t)]
        lib.moe_dispatch.restype = i32
        lib.moe_dispatch.argtypes = [vp, vp, vp, vp, vp, ctypes.POINTER(moe_recv_meta_t), vp]
        lib.moe_dispatch_two_stage.restype = i32
        lib.moe_dispatch_two_stage.argtypes = [vp, vp, vp, vp, vp, vp, vp,
                                               ctypes.POINTER(moe_recv_meta_t), vp]
        lib.moe_layout_dispatch_fused.restype = i32
        lib.moe_layout_dispatch_fused.argtypes = [vp, vp, vp, vp, vp, vp, vp,
                                                  ctypes.POINTER(moe_recv_meta_t), vp]
        lib.moe_set_wait_limit.restype = i32
        lib.moe_set_wait_limit.argtypes = [vp, ctypes.c_int64]
        i64 = ctypes.c_int64
        lib.moe_dispatch_tokens.restype = i32
        lib.moe_dispatch_tokens.argtypes = [vp, i64, i64, vp, vp, vp, vp,
                                            ctypes.POINTER(moe_recv_meta_t), vp]
        lib.moe_expert_standin_tokens.restype = i32
        lib.moe_expert_standin_tokens.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp]
        lib.moe_combine_tokens.restype = i32
        lib.moe_combine_tokens.argtypes = [vp, i64, i64, vp, vp, vp, vp]
        lib.moe_dispatch_allgather.restype = i32
        lib.moe_dispatch_allgather.argtypes = [vp, vp, vp, vp, vp, vp, vp,
                                               ctypes.POINTER(moe_recv_meta_t), vp]
        lib.moe_expert_standin.restype = i32
        lib.moe_expert_standin.argtypes = [vp, vp, vp, vp, vp, vp]
        lib.moe_combine.restype = i32
        lib.moe_combine.argtypes = [vp, vp, vp, vp, vp]
        lib.moe_read_status.restype = i32
        lib.moe_read_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), vp]
        lib.moe_dispatch_layout_noalloc.restype = i32
        lib.moe_dispatch_layout_noalloc.argtypes = [cfgp, vp, ctypes.POINTER(moe_layout_view_t), vp]
        lib.moe_copy_h2d_async.restype = i32
        lib.moe_copy_h2d_async.argtypes = [vp, vp, sz, vp]
        lib.moe_copy_d2h_async.restype = i32
        lib.moe_copy_d2h_async.argtypes = [vp, vp, sz, vp]
        lib.moe_error_string.restype = ctypes.c_char_p
        lib.moe_error_string.argtypes = [i32]
        xcfgp = ctypes.POINTER(moe_expert_config_t)
        lib.moe_expert_workspace_bytes.restype = sz
        lib.moe_expert_workspace_bytes.argtypes = [xcfgp]
        lib.moe_expert_form.restype = i32
        lib.moe_expert_form.argtypes = [xcfgp, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.POINTER(moe_expert_form_t)]
        lib.moe_expert_create.restype = i32
        lib.moe_expert_create.argtypes = [xcfgp, vp, sz, ctypes.POINTER(vp)]
        lib.moe_expert_destroy.restype = i32
        lib.moe_expert_destroy.argtypes = [vp]
        lib.moe_expert_gated.restype = i32
        lib.moe_expert_gated.argtypes = [vp] * 10
        lib.moe_expert_down.restype = i32
        lib.moe_expert_down.argtypes = [vp] * 8
        lib.moe_expert_backward.restype = i32
        lib.moe_expert_backward.argtypes = [vp] * 12
        lib.moe_expert_set_wait_limit.restype = i32
        lib.moe_expert_set_wait_limit.argtypes = [vp, i64]
        lib.moe_expert_read_status.restype = i32
        lib.moe_expert_read_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), vp]
        lib.moe_combine_backward.restype = i32
        lib.moe_combine_backward.argtypes = [vp] * 7
        lib.moe_debug_bounds.restype = i32
        lib.moe_debug_bounds.argtypes = []
        _lib = lib
        return lib


def _check(fn: str, rc: int) -> None:
    if rc < 0:
        raise MoeError(fn, rc, load_library().moe_error_string(rc).decode())


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_raw_stream = None


def _current_stream() -> int:
    """The current device's current stream, without a Stream object where torch can give its
    handle alone (3 us less a call)."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        dev = getattr(torch._C, "_cuda_getDevice", None)
        torch.cuda.current_stream()  # initialises CUDA, or raises
        _raw_stream = ((lambda: get(dev())) if get and dev else
                       (lambda: torch.cuda.current_stream().cuda_stream))
    return _raw_stream()


def make_config(P: int, Tr: int, E: int, k: int, H: int, dispatch_dtype: int = MOE_BF16,
                cap: int = 0) -> moe_config_t:
    return moe_config_t(P, Tr, E, k, H, dispatch_dtype, MOE_BF16, cap)


def moe_workspace_bytes(cfg: moe_config_t) -> int:
    return int(load_library().moe_workspace_bytes(ctypes.byref(cfg)))


def moe_recv_rows_max(cfg: moe_config_t) -> int:
    return int(load_library().moe_recv_rows_max(ctypes.byref(cfg)))


class Handle:
    """Owns the C handle and keeps its workspace tensor alive."""

    def __init__(self, cfg: moe_config_t, workspace):
        self.cfg = cfg
        self.workspace = workspace
        #: rows that the last dispatch's inv can name (the receive rows, or the fixed slots)
        self.recv_rows = self.rows = moe_recv_rows_max(cfg)
        h = _c_void_p()
        _check("moe_handle_create", load_library().moe_handle_create(
            ctypes.byref(cfg), _ptr(workspace), workspace.numel() * workspace.element_size(),
            ctypes.byref(h)))
        self._h = h

    @property
    def ptr(self):
        return self._h

    def close(self):
        if self._h:
            load_library().moe_handle_destroy(self._h)
            self._h = _c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def moe_handle_create(cfg: moe_config_t, workspace=None, device=None) -> Handle:
    """Creates a handle; allocates the workspace with torch when none is given."""
    import torch
    if workspace is None:
        nbytes = moe_workspace_bytes(cfg)
        if nbytes == 0:
            _check("moe_workspace_bytes", -1)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
    return Handle(cfg, workspace)


def moe_route_topk(h: Handle, logits, ids, w, stream=None) -> None:
    _check("moe_route_topk", load_library().moe_route_topk(
        h.ptr, _ptr(logits), _ptr(ids), _ptr(w), _stream(stream)))


def moe_dispatch_layout(h: Handle, ids, stream=None) -> None:
    _check("moe_dispatch_layout", load_library().moe_dispatch_layout(
        h.ptr, _ptr(ids), _stream(stream)))


def moe_route_dispatch_layout(h: Handle, logits, ids, w, stream=None) -> None:
    _check("moe_route_dispatch_layout", load_library().moe_route_dispatch_layout(
        h.ptr, _ptr(logits), _ptr(ids), _ptr(w), _stream(stream)))


def moe_fixed_slot_rows(cfg) -> int:
    return int(load_library().moe_fixed_slot_rows(ctypes.byref(cfg)))


def moe_dispatch_fixed_slots(h: Handle, x, w, slot_x, slot_scale, meta: dict, stream=None) -> None:
    """Dispatch into fixed per-(source, expert) slot regions (see the header)."""
    m = moe_recv_meta_t(*(_ptr(meta[n]) for n in (
        "local_expert", "src_rank", "src_token", "slot", "weight")))
    _check("moe_dispatch_fixed_slots", load_library().moe_dispatch_fixed_slots(
        h.ptr, _ptr(x), _ptr(w), _ptr(slot_x), _ptr(slot_scale), ctypes.byref(m),
        _stream(stream)))
    h.rows = moe_fixed_slot_rows(h.cfg)


def moe_layout_tables(h: Handle, stream=None) -> None:
    """Completes the per-source tables of the last layout without dispatching."""
    _check("moe_layout_tables", load_library().moe_layout_tables(h.ptr, _stream(stream)))


def moe_get_layout(h: Handle) -> dict:
    """Views (int32 tensors on the workspace) of every layout array."""
    import torch
    v = moe_layout_view_t()
    _check("moe_get_layout", load_library().moe_get_layout(h.ptr, ctypes.byref(v)))
    cfg = h.cfg
    P, E = cfg.num_ranks, cfg.num_experts
    Na = P * cfg.tokens_per_rank * cfg.top_k
    sizes = dict(expert_count=(E,), expert_count_raw=(E,), expert_offset=(E + 1,),
                 src_expert_count=(P, E), src_expert_kept=(P, E), count_matrix=(P, P),
                 send_offset=(P, P), recv_offset=(P, E), rank_base=(P + 1,), inv=(Na,),
                 totals=(4,))
    ws = h.workspace
    base = ws.data_ptr()
    out = {}
    for name, shape in sizes.items():
        off = getattr(v, name) - base
        n = 1
        for s in shape:
            n *= s
        out[name] = ws[off: off + 4 * n].view(torch.int32).view(*shape)
    return out


def moe_dispatch(h: Handle, x, w, recv_x, recv_scale, meta: dict, stream=None) -> None:
    m = moe_recv_meta_t(*(_ptr(meta[n]) for n in (
        "local_expert", "src_rank", "src_token", "slot", "weight")))
    _check("moe_dispatch", load_library().moe_dispatch(
        h.ptr, _ptr(x), _ptr(w), _ptr(recv_x), _ptr(recv_scale), ctypes.byref(m),
        _stream(stream)))
    h.rows = h.recv_rows


def moe_dispatch_two_stage(h: Handle, x, w, send_x, send_scale, recv_x, recv_scale, meta: dict,
                           stream=None) -> None:
    m = moe_recv_meta_t(*(_ptr(meta[n]) for n in (
        "local_expert", "src_rank", "src_token", "slot", "weight")))
    _check("moe_dispatch_two_stage", load_library().moe_dispatch_two_stage(
        h.ptr, _ptr(x), _ptr(w), _ptr(send_x), _ptr(send_scale), _ptr(recv_x), _ptr(recv_scale),
        ctypes.byref(m), _stream(stream)))
    h.rows = h.recv_rows


def moe_layout_dispatch_fused(h: Handle, logits, ids, w, x, recv_x, recv_scale, meta: dict,
                              stream=None) -> None:
    """Route (logits given) or take ids/w, lay out and dispatch in one launch."""
    m = moe_recv_meta_t(*(_ptr(meta[n]) for n in (
        "local_expert", "src_rank", "src_token", "slot", "weight")))
    _check("moe_layout_dispatch_fused", load_library().moe_layout_dispatch_fused(
        h.ptr, _ptr(logits), _ptr(ids), _ptr(w), _ptr(x), _ptr(recv_x), _ptr(recv_scale),
        ctypes.byref(m), _stream(stream)))
    h.rows = h.recv_rows


def moe_set_wait_limit(h: Handle, polls: int) -> None:
    _check("moe_set_wait_limit", load_library().moe_set_wait_limit(h.ptr, int(polls)))


def moe_dispatch_tokens(h: Handle, begin: int, end: int, x, w, recv_x, recv_scale, meta: dict,
                        stream=None) -> None:
    m = moe_recv_meta_t(*(_ptr(meta[n]) for n in (
        "local_expert", "src_rank", "src_token", "slot", "weight")))
    _check("moe_dispatch_tokens", load_library().moe_dispatch_tokens(
        h.ptr, int(begin), int(end), _ptr(x), _ptr(w), _ptr(recv_x), _ptr(recv_scale),
        ctypes.byref(m), _stream(stream)))
    h.rows = h.recv_rows


def moe_expert_standin_tokens(h: Handle, begin: int, end: int, recv_x, recv_scale, expert_scale,
                              y, stream=None) -> None:
    _check("moe_expert_standin_tokens", load_library().moe_expert_standin_tokens(
        h.ptr, int(begin), int(end), _ptr(recv_x), _ptr(recv_scale), _ptr(expert_scale),
        _ptr(y), _stream(stream)))


def moe_combine_tokens(h: Handle, begin: int, end: int, y, w, out, stream=None) -> None:
    _check("moe_combine_tokens", load_library().moe_combine_tokens(
        h.ptr, int(begin), int(end), _ptr(y), _ptr(w), _ptr(out), _stream(stream)))


def moe_dispatch_allgather(h: Handle, x, w, gathered_x, gathered_scale, recv_x, recv_scale,
                           meta: dict, stream=None) -> None:
    m = moe_recv_meta_t(*(_ptr(meta[n]) for n in (
        "local_expert", "src_rank", "src_token", "slot", "weight")))
    _check("moe_dispatch_allgather", load_library().moe_dispatch_allgather(
        h.ptr, _ptr(x), _ptr(w), _ptr(gathered_x), _ptr(gathered_scale), _ptr(recv_x),
        _ptr(recv_scale), ctypes.byref(m), _stream(stream)))
    h.rows = h.recv_rows


def moe_expert_standin(h: Handle, recv_x, recv_scale, expert_scale, y, stream=None) -> None:
    _check("moe_expert_standin", load_library().moe_expert_standin(
        h.ptr, _ptr(recv_x), _ptr(recv_scale), _ptr(expert_scale), _ptr(y), _stream(stream)))


def moe_combine(h: Handle, y, w, out, stream=None) -> None:
    _check("moe_combine", load_library().moe_combine(
        h.ptr, _ptr(y), _ptr(w), _ptr(out), _stream(stream)))


_types = None


def _element_types():
    """The tensor types of bf16 values, e4m3 codes (as bytes, or as torch's own type), fp32
    values, int32 offsets and int8 codes."""
    global _types
    if _types is None:
        import torch
        _types = ((torch.bfloat16,), (torch.uint8, torch.float8_e4m3fn), (torch.float32,),
                  (torch.int32,), (torch.int8,))
    return _types


def _buf(name: str, t, count: int, types: tuple, optional: bool = False) -> Optional[int]:
    """Device pointer of a tensor that must hold `count` elements of one of the types."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name}: a tensor is needed")
    if t.dtype not in types or t.numel() < count:
        raise ValueError(f"{name}: expected at least {count} elements of {types[0]}, "
                         f"got {t.numel()} of {t.dtype}")
    return _ptr(t)


def moe_combine_backward(h: Handle, dout, y, w, dy, dw, stream=None) -> None:
    """Gradients of moe_combine on the last dispatch's layout (see the header); y and dy hold
    every row that it can name."""
    c = h.cfg
    T, rows_h = c.num_ranks * c.tokens_per_rank, h.rows * c.hidden
    bf16, _, fp32, _, _ = _element_types()
    _check("moe_combine_backward", load_library().moe_combine_backward(
        h.ptr, _buf("dout", dout, T * c.hidden, bf16), _buf("y", y, rows_h, bf16),
        _buf("w", w, T * c.top_k, fp32), _buf("dy", dy, rows_h, bf16),
        _buf("dw", dw, T * c.top_k, fp32), _stream(stream)))


def make_expert_config(E: int, H: int, F: int, rows_max: int, dtype: int = MOE_BF16,
                       train: bool = False) -> moe_expert_config_t:
    """E experts of hidden width H and inner width F over up to rows_max rows."""
    return moe_expert_config_t(E, H, F, dtype, rows_max, int(train))


def moe_expert_workspace_bytes(cfg: moe_expert_config_t) -> int:
    return int(load_library().moe_expert_workspace_bytes(ctypes.byref(cfg)))


def moe_expert_form(cfg: moe_expert_config_t, down: bool, num_sms: int) -> tuple:
    """(kernels, tokens, split) of a handle's gated or down product (see the header)."""
    out = moe_expert_form_t()
    _check("moe_expert_form", load_library().moe_expert_form(
        ctypes.byref(cfg), int(down), num_sms, ctypes.byref(out)))
    return out.kernels, out.tokens, out.split


class ExpertHandle:
    """Owns the C handle of an expert block and keeps its workspace tensor alive."""

    def __init__(self, cfg: moe_expert_config_t, workspace):
        self.cfg = cfg
        self.workspace = workspace
        self.fp8, self.int8 = cfg.dtype == MOE_FP8_E4M3, cfg.dtype == MOE_INT8
        E, H, F, R = cfg.num_experts, cfg.hidden, cfg.inter, cfg.rows_max
        #: elements that each tensor must hold, and their types
        self.offsets, self.rows_h, self.rows_f = E + 1, R * H, R * F
        self.w13, self.w2 = E * 2 * F * H, E * H * F
        #: scales: of a row's 128 channels and a weight's 128 x 128 blocks, or of a row and a
        #: weight's output channel
        self.s_h, self.s_f = (R, R) if self.int8 else (R * H // 128, R * F // 128)
        self.s13, self.s2 = ((E * 2 * F, E * H) if self.int8 else
                             (self.w13 // 128 // 128, self.w2 // 128 // 128))
        self.bf16, e4m3, self.fp32, self.int32, int8 = _element_types()
        self.elt = e4m3 if self.fp8 else int8 if self.int8 else self.bf16
        h = _c_void_p()
        _check("moe_expert_create", load_library().moe_expert_create(
            ctypes.byref(cfg), _ptr(workspace), workspace.numel() * workspace.element_size(),
            ctypes.byref(h)))
        self._h = h

    @property
    def ptr(self):
        return self._h

    def close(self):
        if self._h:
            load_library().moe_expert_destroy(self._h)
            self._h = _c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def moe_expert_create(cfg: moe_expert_config_t, workspace=None, device=None) -> ExpertHandle:
    """Creates a handle; allocates the workspace with torch when none is given."""
    import torch
    if workspace is None:
        nbytes = moe_expert_workspace_bytes(cfg)
        if nbytes == 0:
            _check("moe_expert_workspace_bytes", -1)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
    return ExpertHandle(cfg, workspace)


def _scale(name: str, x: ExpertHandle, t, count: int) -> Optional[int]:
    if t is None and not (x.fp8 or x.int8):
        return None
    return _buf(name, t, count, x.fp32)


def moe_expert_gated(x: ExpertHandle, expert_offset, inp, inp_scale, w13, w13_scale, hid,
                     hid_scale=None, gate_up=None, stream=None) -> None:
    """hid = silu(inp Wg^T) * (inp Wu^T) over the experts' segments (see the header)."""
    elt = x.elt
    _check("moe_expert_gated", load_library().moe_expert_gated(
        x.ptr, _buf("expert_offset", expert_offset, x.offsets, x.int32),
        _buf("inp", inp, x.rows_h, elt), _scale("inp_scale", x, inp_scale, x.s_h),
        _buf("w13", w13, x.w13, elt), _scale("w13_scale", x, w13_scale, x.s13),
        _buf("hid", hid, x.rows_f, elt), _scale("hid_scale", x, hid_scale, x.s_f),
        _buf("gate_up", gate_up, 2 * x.rows_f, x.bf16, optional=True), _stream(stream)))


def moe_expert_down(x: ExpertHandle, expert_offset, hid, hid_scale, w2, w2_scale, y,
                    stream=None) -> None:
    """y = hid W2^T over the experts' segments (see the header)."""
    elt = x.elt
    _check("moe_expert_down", load_library().moe_expert_down(
        x.ptr, _buf("expert_offset", expert_offset, x.offsets, x.int32),
        _buf("hid", hid, x.rows_f, elt), _scale("hid_scale", x, hid_scale, x.s_f),
        _buf("w2", w2, x.w2, elt), _scale("w2_scale", x, w2_scale, x.s2),
        _buf("y", y, x.rows_h, x.bf16), _stream(stream)))


def moe_expert_backward(x: ExpertHandle, expert_offset, inp, gate_up, hid, dy, w13, w2, dx=None,
                        dw13=None, dw2=None, stream=None) -> None:
    """Gradients of the gated block; dx, or dw13 and dw2 together, may be left out."""
    bf16 = x.bf16
    _check("moe_expert_backward", load_library().moe_expert_backward(
        x.ptr, _buf("expert_offset", expert_offset, x.offsets, x.int32),
        _buf("inp", inp, x.rows_h, bf16), _buf("gate_up", gate_up, 2 * x.rows_f, bf16),
        _buf("hid", hid, x.rows_f, bf16), _buf("dy", dy, x.rows_h, bf16),
        _buf("w13", w13, x.w13, bf16), _buf("w2", w2, x.w2, bf16),
        _buf("dx", dx, x.rows_h, bf16, optional=True),
        _buf("dw13", dw13, x.w13, bf16, optional=True),
        _buf("dw2", dw2, x.w2, bf16, optional=True), _stream(stream)))


def moe_expert_set_wait_limit(x: ExpertHandle, cycles: int) -> None:
    _check("moe_expert_set_wait_limit",
           load_library().moe_expert_set_wait_limit(x.ptr, int(cycles)))


def moe_expert_read_status(x: ExpertHandle, stream=None) -> int:
    flags = ctypes.c_uint32(0)
    _check("moe_expert_read_status", load_library().moe_expert_read_status(
        x.ptr, ctypes.byref(flags), _stream(stream)))
    return int(flags.value)


def moe_read_status(h: Handle, stream=None) -> int:
    flags = ctypes.c_uint32(0)
    _check("moe_read_status", load_library().moe_read_status(
        h.ptr, ctypes.byref(flags), _stream(stream)))
    return int(flags.value)


def moe_dispatch_layout_noalloc(cfg: moe_config_t, ids, out: dict, stream=None) -> None:
    """Layout + inverse permutation into caller tensors (int32, sized as in
    moe_get_layout's views), with no device allocation by the library. For
    callers that cannot allocate (graph capture, fixed-pool runtimes); the
    first call on a device must precede any stream capture; overlapping calls
    race on the library's static scratch."""
    v = moe_layout_view_t(*(_ptr(out[n]) for n, _ in moe_layout_view_t._fields_))
    _check("moe_dispatch_layout_noalloc", load_library().moe_dispatch_layout_noalloc(
        ctypes.byref(cfg), _ptr(ids), ctypes.byref(v), _stream(stream)))


def _host_ptr(t) -> int:
    if t.is_cuda:
        raise ValueError("expected a host tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def moe_copy_h2d_async(dst, src_host, stream=None) -> None:
    """Stream-ordered copy of a (pinned) host tensor into a device tensor."""
    n = src_host.numel() * src_host.element_size()
    if n != dst.numel() * dst.element_size():
        raise ValueError("size mismatch")
    _check("moe_copy_h2d_async", load_library().moe_copy_h2d_async(
        _ptr(dst), _host_ptr(src_host), n, _stream(stream)))


def moe_copy_d2h_async(dst_host, src, stream=None) -> None:
    """Stream-ordered copy of a device tensor into a (pinned) host tensor."""
    n = src.numel() * src.element_size()
    if n != dst_host.numel() * dst_host.element_size():
        raise ValueError("size mismatch")
    _check("moe_copy_d2h_async", load_library().moe_copy_d2h_async(
        _host_ptr(dst_host), _ptr(src), n, _stream(stream)))


def moe_error_string(code: int) -> str:
    return load_library().moe_error_string(code).decode()


def moe_debug_bounds() -> bool:
    """True if the loaded library checks every computed row index on the device."""
    return bool(load_library().moe_debug_bounds())
