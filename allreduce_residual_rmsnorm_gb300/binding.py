"""Thin ctypes binding of libarfusion (include/ar_fusion.h).

Argument marshalling only: every function has the name of the C entry point,
turns torch tensors into device pointers / sizes, calls the library, and raises
:class:`ArFusionError` on a non-zero status.  No compute happens here and
there is no fallback: if the library is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from .build import marshal_path

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libarfusion.so")

# enum ar_dtype
AR_DT_BF16 = 0
AR_DT_FP16 = 1
AR_DT_FP32 = 2
AR_DT_E4M3 = 3
# enum ar_pattern
AR_RESIDUAL_OUT = 1
AR_NORM_OUT = 2
AR_QUANT_FP8 = 4
AR_QUANT_NVFP4 = 8
# enum ar_status
AR_OK = 0
AR_ERR_INVALID = -1
AR_ERR_UNSUPPORTED = -2
AR_ERR_CUDA = -3
AR_ERR_TIMEOUT = -4
AR_ERR_CAPACITY = -5
# enum ar_mode
AR_MODE_AUTO = 0
AR_MODE_LAMPORT = 1
AR_MODE_BUFFER = 2
# enum ar_variant
AR_VARIANT_AUTO = 0
AR_VARIANT_WARP_ROW = 1
AR_VARIANT_CTA_ROW = 2
AR_VARIANT_BULK_PIPE = 3

# enum ar_scale_layout
AR_SF_LINEAR = 0
AR_SF_SWIZZLED = 1
# enum ar_accumulate
AR_ACC_FP32 = 0
AR_ACC_ELEMENT = 1

# enum ar_score
AR_SCORE_SOFTMAX = 0
AR_SCORE_SIGMOID = 1
# enum ar_group_score
AR_GROUP_MAX = 0
AR_GROUP_TOP2 = 1
# enum ar_activation
AR_ACT_NONE = 0
AR_ACT_SILU_MUL = 1

AR_MAX_RANKS = 16
AR_ONESHOT_MAX_TOKENS = 128
AR_BARRIER_FLAG_COUNT = 256
AR_MAX_HIDDEN = 32768
AR_NOALLOC_SLOT_BYTES = 4 << 20
AR_MAX_EXPERTS = 1024
AR_MAX_TOPK = 32
AR_MAX_GROUPS = 32
AR_QUANT_BLOCK = 128
AR_MAX_SEQUENCES = 2048
AR_MAX_HEAD_GROUP = 128
AR_MAX_HEAD_DIM = 128
AR_MAX_AXES = 4
AR_ATTENTION_WORKSPACE_BYTES = 32 << 20

PATTERNS = {
    "res_norm": AR_RESIDUAL_OUT | AR_NORM_OUT,
    "norm": AR_NORM_OUT,
    "res_fp8": AR_RESIDUAL_OUT | AR_QUANT_FP8,
    "res_nvfp4": AR_RESIDUAL_OUT | AR_QUANT_NVFP4,
    "res_norm_fp8": AR_RESIDUAL_OUT | AR_NORM_OUT | AR_QUANT_FP8,
    "res_norm_nvfp4": AR_RESIDUAL_OUT | AR_NORM_OUT | AR_QUANT_NVFP4,
}


class ArFusionError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"ar_fusion error {code}: {msg}")
        self.code = code


class WsInfo(ctypes.Structure):
    _fields_ = [
        ("tp_size", ctypes.c_int32), ("max_token_num", ctypes.c_int32),
        ("hidden_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("elem_bytes", ctypes.c_int32), ("oneshot_max_tokens", ctypes.c_int32),
        ("total_bytes", ctypes.c_uint64), ("buffer_bytes", ctypes.c_uint64),
        ("flag_bytes", ctypes.c_uint64), ("lamport_comm_bytes", ctypes.c_uint64),
        ("lamport_buffer_bytes", ctypes.c_uint64), ("state_bytes", ctypes.c_uint64),
        ("base", ctypes.c_void_p), ("buffer", ctypes.c_void_p), ("flags", ctypes.c_void_p),
        ("lamport", ctypes.c_void_p), ("state", ctypes.c_void_p),
        ("last_variant", ctypes.c_int32), ("last_cluster", ctypes.c_int32),
    ]


class State(ctypes.Structure):
    _fields_ = [
        ("counter", ctypes.c_uint32), ("flag", ctypes.c_uint32),
        ("lamport_flag", ctypes.c_uint32), ("clear_elem_bytes", ctypes.c_uint32),
        ("comm_size", ctypes.c_uint64), ("clear_size", ctypes.c_uint64),
        ("status", ctypes.c_int32), ("detail", ctypes.c_int32), ("calls", ctypes.c_uint64),
    ]


class _HeadRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row", ctypes.c_int64), ("head", ctypes.c_int64)]


class _KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [
        (f"{x}_{s}", ctypes.c_int64) for x in "kv" for s in ("page", "row", "head")] + [
        (n, ctypes.c_int32) for n in ("dtype", "pages", "page_size", "heads", "head_dim",
                                      "sequences", "max_pages")] + [
        ("scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("lengths", ctypes.c_void_p)]


_lib = None
_native = None      # _marshal, once the library is loaded and if it was built
_vp = ctypes.c_void_p
_i = ctypes.c_int


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libarfusion.so (built in-tree by ``build.py``) and declare its
    signatures.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    L = ctypes.CDLL(path)
    L.ar_fusion_version.restype = _i
    L.ar_fusion_version.argtypes = []
    L.ar_fusion_last_error.restype = ctypes.c_char_p
    L.ar_fusion_last_error.argtypes = []
    L.ar_fusion_workspace_bytes.argtypes = [_i, _i, _i, _i, ctypes.POINTER(ctypes.c_size_t)]
    L.ar_fusion_workspace_create.argtypes = [_i, _i, _i, _i, _vp, ctypes.c_size_t, _vp,
                                             ctypes.POINTER(_vp)]
    L.ar_fusion_workspace_destroy.argtypes = [_vp]
    L.ar_fusion_workspace_info.argtypes = [_vp, ctypes.POINTER(WsInfo)]
    L.ar_fusion_workspace_copy_state.argtypes = [_vp, _vp, ctypes.POINTER(State)]
    L.ar_fusion_workspace_status.argtypes = [_vp, _vp, ctypes.POINTER(_i)]
    L.ar_fusion_workspace_reset.argtypes = [_vp, _vp]
    L.ar_fusion_workspace_set_timeout_ns.argtypes = [_vp, ctypes.c_uint64]
    L.ar_fusion_workspace_set_variant.argtypes = [_vp, _i]
    L.ar_fusion_workspace_set_mode.argtypes = [_vp, _i]
    L.ar_fusion_workspace_set_launch.argtypes = [_vp, _i, _i]
    L.ar_fusion_workspace_set_accumulate.argtypes = [_vp, _i]
    L.ar_fusion_workspace_set_scale_layout.argtypes = [_vp, _i]
    L.ar_fusion_sum_ex.argtypes = [ctypes.POINTER(_vp), _i, ctypes.c_size_t, _i, _i, _vp, _vp]
    L.ar_fusion_workspace_stage.argtypes = [_vp, _i, _vp, _i, _i, _vp]
    L.ar_fusion_workspace_partial_ptr.argtypes = [_vp, _i, _i, _i, _vp, ctypes.POINTER(_vp)]
    L.ar_fusion_run.argtypes = [_vp, ctypes.POINTER(_vp), _i, _i, _i, _i, _vp, _vp,
                                ctypes.c_float, _i, _vp, _vp, _vp, _vp, _vp, _vp]
    L.ar_fusion_norm_amax.argtypes = [_vp, ctypes.POINTER(_vp), _i, _i, _i, _i, _vp, _vp,
                                      ctypes.c_float, _vp, _vp]
    L.ar_fusion_sum.argtypes = [ctypes.POINTER(_vp), _i, ctypes.c_size_t, _i, _vp, _vp]
    L.ar_fusion_run_noalloc.argtypes = [ctypes.POINTER(_vp), _i, _i, _i, _i, _vp, _vp,
                                        ctypes.c_float, _i, _vp, _vp, _vp, _vp, _vp, _vp]
    L.ar_fusion_noalloc_status.argtypes = [_vp, ctypes.POINTER(_i)]
    L.ar_fusion_route.argtypes = [_vp, _i, _i, _i, _vp, _i, _i, _i, _i, _i, _i, ctypes.c_float,
                                  _vp, _vp, _vp]
    L.ar_fusion_expert_plan.argtypes = [_vp, _i, _i, _i, _i, _vp, _vp, _vp]
    L.ar_fusion_quant_blocks.argtypes = [_vp, _i, _i, _i, _i, _vp, _i, _vp, _i, _vp, _vp, _vp]
    L.ar_fusion_matmul_fp8.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp]
    L.ar_fusion_expert_matmul_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp,
                                              _vp]
    L.ar_fusion_combine.argtypes = [_vp, _i, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp]
    L.ar_fusion_matmul_status.argtypes = [_vp, ctypes.POINTER(_i)]
    cache, rows = ctypes.POINTER(_KvCache), ctypes.POINTER(_HeadRows)
    L.ar_fusion_rope_append.argtypes = [cache, rows, rows, rows, rows, _i, _i, _i, _vp, _vp, _vp, _i,
                                        ctypes.POINTER(_i), _i, _i, _vp]
    L.ar_fusion_decode_attention.argtypes = [cache, rows, rows, _vp, _i, _i, ctypes.c_float, _i, _i,
                                             _vp, ctypes.c_size_t, _vp]
    L.ar_fusion_prompt_attention.argtypes = [cache, rows, rows, _vp, _vp, _i, _i, _i, ctypes.c_float,
                                             _i, _i, _vp, ctypes.c_size_t, _vp]
    L.ar_fusion_attention_status.argtypes = [_vp, ctypes.POINTER(_i)]
    for name in ("ar_fusion_workspace_bytes", "ar_fusion_workspace_create",
                 "ar_fusion_workspace_destroy", "ar_fusion_workspace_info",
                 "ar_fusion_workspace_copy_state", "ar_fusion_workspace_status",
                 "ar_fusion_workspace_reset", "ar_fusion_workspace_set_timeout_ns",
                 "ar_fusion_workspace_set_variant", "ar_fusion_workspace_set_mode",
                 "ar_fusion_workspace_set_launch", "ar_fusion_workspace_set_accumulate",
                 "ar_fusion_workspace_set_scale_layout",
                 "ar_fusion_sum_ex",
                 "ar_fusion_workspace_stage", "ar_fusion_workspace_partial_ptr",
                 "ar_fusion_run", "ar_fusion_norm_amax",
                 "ar_fusion_sum", "ar_fusion_run_noalloc", "ar_fusion_noalloc_status",
                 "ar_fusion_route", "ar_fusion_expert_plan", "ar_fusion_quant_blocks",
                 "ar_fusion_matmul_fp8", "ar_fusion_expert_matmul_fp8", "ar_fusion_combine",
                 "ar_fusion_matmul_status", "ar_fusion_rope_append",
                 "ar_fusion_decode_attention", "ar_fusion_prompt_attention",
                 "ar_fusion_attention_status"):
        getattr(L, name).restype = _i
    _lib = L
    _load_native(L)
    return L


def _load_native(L: ctypes.CDLL) -> None:
    """The expert-layer and attention-layer calls' marshalling in C++ (csrc/marshal.cpp).  The calls
    work without it, through ctypes, some microseconds slower each."""
    global _native
    path = marshal_path()
    if not os.path.exists(path):
        return
    spec = importlib.util.spec_from_file_location("_marshal", path)
    try:
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
    except ImportError:
        return
    m.bind(*(ctypes.cast(getattr(L, f), _vp).value
             for f in ("ar_fusion_route", "ar_fusion_expert_plan", "ar_fusion_quant_blocks",
                       "ar_fusion_matmul_fp8", "ar_fusion_expert_matmul_fp8",
                       "ar_fusion_combine", "ar_fusion_rope_append",
                       "ar_fusion_decode_attention", "ar_fusion_prompt_attention")))
    _native = m


def lib() -> ctypes.CDLL:
    return load()


def _check(rc: int) -> int:
    if rc != AR_OK:
        raise ArFusionError(rc, ar_fusion_last_error())
    return rc


def _dtype_id(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return AR_DT_BF16
    if t.dtype == torch.float16:
        return AR_DT_FP16
    if t.dtype == torch.float32:
        return AR_DT_FP32
    raise TypeError(f"unsupported element type {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        return int(t)
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        # the handle alone: building the Stream object takes 2.8 us, most of a launch
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr_array(ts):
    arr = (_vp * len(ts))()
    for i, t in enumerate(ts):
        arr[i] = _ptr(t)
    return arr


class Workspace:
    """Handle of an ``ar_fusion_ws``; keeps caller-supplied memory alive."""

    def __init__(self, handle: int, mem, tp_size, max_token_num, hidden_dim, dtype):
        self.handle = handle
        self.mem = mem
        self.tp_size = tp_size
        self.max_token_num = max_token_num
        self.hidden_dim = hidden_dim
        self.dtype = dtype

    def __del__(self):
        try:
            if self.handle:
                ar_fusion_workspace_destroy(self)
        except Exception:
            pass


# ------------------------------------------------------------------- calls

def ar_fusion_version() -> int:
    return lib().ar_fusion_version()


def ar_fusion_last_error() -> str:
    return lib().ar_fusion_last_error().decode()


def ar_fusion_workspace_bytes(tp_size: int, max_token_num: int, hidden_dim: int,
                              dtype: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ar_fusion_workspace_bytes(tp_size, max_token_num, hidden_dim, dtype,
                                           ctypes.byref(n)))
    return n.value


def ar_fusion_workspace_create(tp_size: int, max_token_num: int, hidden_dim: int, dtype: int,
                               device_mem: torch.Tensor | None = None, stream=None) -> Workspace:
    h = _vp()
    mem_ptr = _ptr(device_mem) if device_mem is not None else None
    mem_bytes = device_mem.numel() * device_mem.element_size() if device_mem is not None else 0
    _check(lib().ar_fusion_workspace_create(tp_size, max_token_num, hidden_dim, dtype, mem_ptr,
                                            mem_bytes, _stream(stream), ctypes.byref(h)))
    return Workspace(h.value, device_mem, tp_size, max_token_num, hidden_dim, dtype)


def ar_fusion_workspace_destroy(ws: Workspace) -> None:
    if ws.handle:
        h, ws.handle = ws.handle, None
        _check(lib().ar_fusion_workspace_destroy(h))


def ar_fusion_workspace_info(ws: Workspace) -> dict:
    info = WsInfo()
    _check(lib().ar_fusion_workspace_info(ws.handle, ctypes.byref(info)))
    return {name: getattr(info, name) for name, _ in WsInfo._fields_}


def ar_fusion_workspace_copy_state(ws: Workspace, stream=None) -> dict:
    st = State()
    _check(lib().ar_fusion_workspace_copy_state(ws.handle, _stream(stream), ctypes.byref(st)))
    return {name: getattr(st, name) for name, _ in State._fields_}


def ar_fusion_workspace_status(ws: Workspace, stream=None):
    """Returns (status code, detail); does not raise on a device error."""
    d = _i(-1)
    rc = lib().ar_fusion_workspace_status(ws.handle, _stream(stream), ctypes.byref(d))
    return rc, d.value


def ar_fusion_workspace_reset(ws: Workspace, stream=None) -> None:
    _check(lib().ar_fusion_workspace_reset(ws.handle, _stream(stream)))


def ar_fusion_workspace_set_timeout_ns(ws: Workspace, ns: int) -> None:
    _check(lib().ar_fusion_workspace_set_timeout_ns(ws.handle, int(ns)))


def ar_fusion_workspace_set_variant(ws: Workspace, variant: int) -> None:
    _check(lib().ar_fusion_workspace_set_variant(ws.handle, int(variant)))


def ar_fusion_workspace_set_mode(ws: Workspace, mode: int) -> None:
    _check(lib().ar_fusion_workspace_set_mode(ws.handle, int(mode)))


def ar_fusion_workspace_set_launch(ws: Workspace, cluster_size: int = 0, pdl: int = 0) -> None:
    _check(lib().ar_fusion_workspace_set_launch(ws.handle, int(cluster_size), int(pdl)))


def ar_fusion_workspace_set_accumulate(ws: Workspace, accumulate: int) -> None:
    _check(lib().ar_fusion_workspace_set_accumulate(ws.handle, int(accumulate)))


def ar_fusion_workspace_set_scale_layout(ws: Workspace, layout: int) -> None:
    _check(lib().ar_fusion_workspace_set_scale_layout(ws.handle, int(layout)))


def swizzled_scale_bytes(tokens: int, hidden: int) -> int:
    """Size of an AR_SF_SWIZZLED scale buffer (whole 128 x 4 tiles)."""
    kb = hidden // 16
    return (tokens + 127) // 128 * 128 * ((kb + 3) // 4) * 4


def ar_fusion_workspace_stage(ws: Workspace, rank: int, src: torch.Tensor, tokens: int | None = None,
                              mode: int = AR_MODE_AUTO, stream=None) -> None:
    if tokens is None:
        tokens = src.shape[0] if src.dim() >= 2 else src.numel() // ws.hidden_dim
    _check(lib().ar_fusion_workspace_stage(ws.handle, rank, _ptr(src), tokens, mode,
                                           _stream(stream)))


def ar_fusion_workspace_partial_ptr(ws: Workspace, rank: int, tokens: int,
                                    mode: int = AR_MODE_AUTO, stream=None) -> int:
    """Device address where rank `rank`'s [tokens, hidden] partial is staged."""
    out = ctypes.c_void_p()
    _check(lib().ar_fusion_workspace_partial_ptr(ws.handle, rank, tokens, mode, _stream(stream),
                                                 ctypes.byref(out)))
    return out.value


def ar_fusion_run(ws: Workspace, partials, residual_in: torch.Tensor, gamma: torch.Tensor,
                  eps: float, pattern: int, residual_out=None, norm_out=None, quant_out=None,
                  scale_out=None, scale_factor=None, stream=None, nranks: int | None = None) -> None:
    """partials: list of R [tokens, hidden] CUDA tensors, or None for the
    partials staged in ``ws``."""
    tokens, hidden = residual_in.shape[0], residual_in.shape[-1]
    if partials is None:
        parr = None
        R = ws.tp_size if nranks is None else nranks
    else:
        parr = _ptr_array(partials)
        R = len(partials) if nranks is None else nranks
    _check(lib().ar_fusion_run(ws.handle, parr, R, tokens, hidden, _dtype_id(residual_in),
                               _ptr(residual_in), _ptr(gamma), ctypes.c_float(eps), pattern,
                               _ptr(residual_out), _ptr(norm_out), _ptr(quant_out),
                               _ptr(scale_out), _ptr(scale_factor), _stream(stream)))


def bound_run(ws: Workspace, partials, residual_in: torch.Tensor, gamma: torch.Tensor,
              eps: float, pattern: int, residual_out=None, norm_out=None, quant_out=None,
              scale_out=None, scale_factor=None, stream=None, nranks: int | None = None):
    """ar_fusion_run with every argument marshalled once: returns a callable
    that launches the call (same tensors, same stream) with no per-call
    Python work beyond the C call itself, for loops that repeat one call.
    The tensors must stay alive while the callable is used."""
    tokens, hidden = residual_in.shape[0], residual_in.shape[-1]
    if partials is None:
        parr = None
        R = ws.tp_size if nranks is None else nranks
    else:
        parr = _ptr_array(partials)
        R = len(partials) if nranks is None else nranks
    fn = lib().ar_fusion_run
    args = (ws.handle, parr, R, tokens, hidden, _dtype_id(residual_in), _ptr(residual_in),
            _ptr(gamma), ctypes.c_float(eps), pattern, _ptr(residual_out), _ptr(norm_out),
            _ptr(quant_out), _ptr(scale_out), _ptr(scale_factor), _stream(stream))

    def call():
        rc = fn(*args)
        if rc != AR_OK:
            _check(rc)

    return call


def ar_fusion_norm_amax(ws: Workspace, partials, residual_in: torch.Tensor, gamma: torch.Tensor,
                        eps: float, amax_out: torch.Tensor, stream=None,
                        nranks: int | None = None) -> None:
    tokens, hidden = residual_in.shape[0], residual_in.shape[-1]
    if partials is None:
        parr = None
        R = ws.tp_size if nranks is None else nranks
    else:
        parr = _ptr_array(partials)
        R = len(partials) if nranks is None else nranks
    _check(lib().ar_fusion_norm_amax(ws.handle, parr, R, tokens, hidden, _dtype_id(residual_in),
                                     _ptr(residual_in), _ptr(gamma), ctypes.c_float(eps),
                                     _ptr(amax_out), _stream(stream)))


def ar_fusion_sum_ex(bufs, out: torch.Tensor, accumulate: int, n: int | None = None,
                     stream=None) -> None:
    if n is None:
        n = out.numel()
    _check(lib().ar_fusion_sum_ex(_ptr_array(bufs), len(bufs), n, _dtype_id(out), int(accumulate),
                                  _ptr(out), _stream(stream)))


def ar_fusion_sum(bufs, out: torch.Tensor, n: int | None = None, stream=None) -> None:
    if n is None:
        n = out.numel()
    _check(lib().ar_fusion_sum(_ptr_array(bufs), len(bufs), n, _dtype_id(out), _ptr(out),
                               _stream(stream)))


def ar_fusion_run_noalloc(partials, residual_in: torch.Tensor, gamma: torch.Tensor, eps: float,
                          pattern: int, residual_out=None, norm_out=None, quant_out=None,
                          scale_out=None, scale_factor=None, stream=None) -> None:
    """The one-shot fused call without a workspace (no device allocation):
    scratch lives in a fixed device array inside the library."""
    tokens, hidden = residual_in.shape[0], residual_in.shape[-1]
    _check(lib().ar_fusion_run_noalloc(_ptr_array(partials), len(partials), tokens, hidden,
                                       _dtype_id(residual_in), _ptr(residual_in), _ptr(gamma),
                                       ctypes.c_float(eps), pattern, _ptr(residual_out),
                                       _ptr(norm_out), _ptr(quant_out), _ptr(scale_out),
                                       _ptr(scale_factor), _stream(stream)))


def ar_fusion_noalloc_status(stream=None):
    """(status, detail) of the no-allocation call on the current device: the
    first device-side error since the previous query (AR_OK if none), which
    the query clears.  Synchronises the stream."""
    d = ctypes.c_int(-1)
    rc = lib().ar_fusion_noalloc_status(_stream(stream), ctypes.byref(d))
    if rc not in (AR_OK, AR_ERR_TIMEOUT):
        _check(rc)
    return rc, d.value


# ----------------------------------------------------------- expert layers

class _Refused(Exception):
    """An operand failed the quick check; the caller's slow check names it."""


def _operand(t: torch.Tensor, dtypes, shape, dev: int):
    if (t.dtype in dtypes and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr()
    raise _Refused


def _handle(stream):
    """None for the current stream, else the stream's address."""
    return None if stream is None else _stream(stream)


def _call(name: str, args) -> None:
    f = getattr(_lib or load(), name)
    for a, kind in zip(args, f.argtypes):       # ctypes would drop the upper bits
        if kind is _i and not -1 << 31 <= a < 1 << 31:
            raise ValueError(f"{name}: {a} does not fit a 32-bit integer")
    rc = f(*args)
    if rc:
        _check(rc)


def _device_of(t: torch.Tensor) -> int:
    """The operands' device, which is the current one: the library launches there."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise _Refused
    return dev


def _explain(*operands) -> None:
    """Names what is wrong with (name, tensor or None, types, shape or None): types
    and shapes of all of them first, then where they are and how they lie."""
    for name, t, dtypes, shape in operands:
        if t is None:
            continue
        if t.dtype not in dtypes:
            raise TypeError(f"{name}: unsupported type {t.dtype}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    for name, t, _, _ in operands:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name}: expected a CUDA tensor")
        if t.get_device() != torch.cuda.current_device():
            raise ValueError(f"{name}: on {t.device}, and the current device is "
                             f"cuda:{torch.cuda.current_device()}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous tensor")
    raise ValueError("operands do not fit together")


def _shapes(*named) -> None:
    """Raises for the first (name, tensor, n) that has not n dimensions."""
    for name, t, n in named:
        if t.dim() != n:
            raise ValueError(f"{name}: {t.dim()} dimensions, expected {n}")


_ELEM = {torch.bfloat16: AR_DT_BF16, torch.float16: AR_DT_FP16, torch.float32: AR_DT_FP32}
_FP8 = (torch.uint8, torch.float8_e4m3fn)
_I32 = (torch.int32,)
_F32 = (torch.float32,)


def ar_fusion_route(logits: torch.Tensor, bias: torch.Tensor | None, ids_out: torch.Tensor,
                    weights_out: torch.Tensor, score: int = AR_SCORE_SIGMOID, groups: int = 1,
                    groups_kept: int = 1, group_score: int = AR_GROUP_TOP2,
                    renormalize: bool = True, scale: float = 1.0, stream=None) -> None:
    """logits [tokens, experts]; bias [experts] fp32 or None; ids_out (int32)
    and weights_out (fp32) [tokens, topk]."""
    if _native is not None:
        rc = _native.route(logits, bias, ids_out, weights_out, score, groups, groups_kept,
                           group_score, renormalize, scale, _handle(stream))
        if rc is not None:
            if rc:
                _check(rc)
            return
    if logits.dim() != 2 or ids_out.dim() != 2:
        _shapes(("logits", logits, 2), ("ids_out", ids_out, 2))
    tokens, experts = logits.shape
    topk = ids_out.shape[1]
    slots = (tokens, topk)
    try:
        dev = _device_of(logits)
        args = (_operand(logits, _ELEM, (tokens, experts), dev), tokens, experts,
                _ELEM[logits.dtype],
                None if bias is None else _operand(bias, _F32, (experts,), dev), score, groups,
                groups_kept, group_score, topk, 1 if renormalize else 0, scale,
                _operand(ids_out, _I32, slots, dev), _operand(weights_out, _F32, slots, dev),
                _stream(stream))
    except _Refused:
        _explain(("logits", logits, _ELEM, None), ("ids_out", ids_out, _I32, slots),
                 ("weights_out", weights_out, _F32, slots), ("bias", bias, _F32, (experts,)))
    _call("ar_fusion_route", args)


def ar_fusion_expert_plan(ids: torch.Tensor, experts: int, offsets_out: torch.Tensor,
                          position_out: torch.Tensor, first_expert: int = 0,
                          stream=None) -> None:
    """ids [tokens, topk] int32; offsets_out [experts + 1] and position_out
    [tokens, topk] int32, for the experts first_expert .. first_expert + experts - 1."""
    if _native is not None:
        rc = _native.expert_plan(ids, experts, offsets_out, position_out, first_expert,
                                 _handle(stream))
        if rc is not None:
            if rc:
                _check(rc)
            return
    if ids.dim() != 2:
        _shapes(("ids", ids, 2))
    slots = ids.shape
    try:
        dev = _device_of(ids)
        args = (_operand(ids, _I32, slots, dev), slots[0], slots[1], first_expert, experts,
                _operand(offsets_out, _I32, (experts + 1,), dev),
                _operand(position_out, _I32, slots, dev), _stream(stream))
    except _Refused:
        _explain(("ids", ids, _I32, None), ("offsets_out", offsets_out, _I32, (experts + 1,)),
                 ("position_out", position_out, _I32, slots))
    _call("ar_fusion_expert_plan", args)


def ar_fusion_quant_blocks(x: torch.Tensor, quant_out: torch.Tensor, scale_out: torch.Tensor,
                           position: torch.Tensor | None = None,
                           activation: int = AR_ACT_NONE,
                           row_count: torch.Tensor | None = None, stream=None) -> None:
    """x [rows, hidden] ([rows, 2 * hidden] with AR_ACT_SILU_MUL); quant_out
    [out_rows, hidden] (uint8 or float8_e4m3fn); scale_out [out_rows,
    ceil(hidden / 128)] fp32; position [rows, copies] int32 or None; row_count: a
    one-element int32 tensor or None (a view of the plan's last offset)."""
    if _native is not None:
        rc = _native.quant_blocks(x, quant_out, scale_out, position, activation, row_count,
                                  _handle(stream))
        if rc is not None:
            if rc:
                _check(rc)
            return
    if x.dim() != 2 or quant_out.dim() != 2:
        _shapes(("x", x, 2), ("quant_out", quant_out, 2))
    rows = x.shape[0]
    out_rows, hidden = quant_out.shape
    copies = 1
    if position is not None:
        if position.dim() != 2:
            _shapes(("position", position, 2))
        copies = position.shape[1]
    shape = (rows, 2 * hidden if activation == AR_ACT_SILU_MUL else hidden)
    scales = (out_rows, (hidden + AR_QUANT_BLOCK - 1) // AR_QUANT_BLOCK)
    try:
        dev = _device_of(x)
        args = (_operand(x, _ELEM, shape, dev), rows, hidden, _ELEM[x.dtype], activation,
                None if position is None else _operand(position, _I32, (rows, copies), dev),
                copies, None if row_count is None else _operand(row_count, _I32, (1,), dev),
                out_rows, _operand(quant_out, _FP8, (out_rows, hidden), dev),
                _operand(scale_out, _F32, scales, dev), _stream(stream))
    except _Refused:
        _explain(("x", x, _ELEM, shape), ("quant_out", quant_out, _FP8, None),
                 ("scale_out", scale_out, _F32, scales),
                 ("position", position, _I32, (rows, copies)),
                 ("row_count", row_count, _I32, (1,)))
    _call("ar_fusion_quant_blocks", args)


def ar_fusion_matmul_fp8(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor,
                         b_scale: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """a [rows, depth], b [cols, depth] (uint8 or float8_e4m3fn); a_scale [rows,
    ceil(depth / 128)], b_scale [ceil(cols / 128), ceil(depth / 128)] fp32; out [rows, cols]."""
    if _native is not None:
        rc = _native.matmul_fp8(a, a_scale, b, b_scale, out, _handle(stream))
        if rc is not None:
            if rc:
                _check(rc)
            return
    if a.dim() != 2 or b.dim() != 2:
        _shapes(("a", a, 2), ("b", b, 2))
    rows, depth = a.shape
    cols = b.shape[0]
    blocks = (depth + AR_QUANT_BLOCK - 1) // AR_QUANT_BLOCK
    col_blocks = (cols + AR_QUANT_BLOCK - 1) // AR_QUANT_BLOCK
    try:
        dev = _device_of(a)
        args = (_operand(a, _FP8, (rows, depth), dev), _operand(a_scale, _F32, (rows, blocks), dev),
                _operand(b, _FP8, (cols, depth), dev),
                _operand(b_scale, _F32, (col_blocks, blocks), dev), rows, cols, depth,
                _ELEM.get(out.dtype), _operand(out, _ELEM, (rows, cols), dev), _stream(stream))
    except _Refused:
        _explain(("a", a, _FP8, None), ("b", b, _FP8, (cols, depth)),
                 ("a_scale", a_scale, _F32, (rows, blocks)),
                 ("b_scale", b_scale, _F32, (col_blocks, blocks)),
                 ("out", out, _ELEM, (rows, cols)))
    _call("ar_fusion_matmul_fp8", args)


def ar_fusion_expert_matmul_fp8(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor,
                                b_scale: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor,
                                stream=None) -> None:
    """ar_fusion_matmul_fp8 by experts: b [experts, cols, depth], b_scale
    [experts, ceil(cols / 128), ceil(depth / 128)], offsets [experts + 1] int32."""
    if _native is not None:
        rc = _native.expert_matmul_fp8(a, a_scale, b, b_scale, offsets, out,
                                       _handle(stream))
        if rc is not None:
            if rc:
                _check(rc)
            return
    if a.dim() != 2 or b.dim() != 3:
        _shapes(("a", a, 2), ("b", b, 3))
    rows, depth = a.shape
    experts, cols, _ = b.shape
    blocks = (depth + AR_QUANT_BLOCK - 1) // AR_QUANT_BLOCK
    col_blocks = (cols + AR_QUANT_BLOCK - 1) // AR_QUANT_BLOCK
    try:
        dev = _device_of(a)
        args = (_operand(a, _FP8, (rows, depth), dev), _operand(a_scale, _F32, (rows, blocks), dev),
                _operand(b, _FP8, (experts, cols, depth), dev),
                _operand(b_scale, _F32, (experts, col_blocks, blocks), dev),
                _operand(offsets, _I32, (experts + 1,), dev), experts, rows, cols, depth,
                _ELEM.get(out.dtype), _operand(out, _ELEM, (rows, cols), dev), _stream(stream))
    except _Refused:
        _explain(("a", a, _FP8, None), ("b", b, _FP8, (experts, cols, depth)),
                 ("a_scale", a_scale, _F32, (rows, blocks)),
                 ("b_scale", b_scale, _F32, (experts, col_blocks, blocks)),
                 ("offsets", offsets, _I32, (experts + 1,)), ("out", out, _ELEM, (rows, cols)))
    _call("ar_fusion_expert_matmul_fp8", args)


def ar_fusion_matmul_status(stream=None):
    """(status, detail) of the products on the current device: the first
    device-side error since the previous query (AR_OK if none), which the query
    clears.  Synchronises the stream."""
    d = ctypes.c_int(-1)
    rc = lib().ar_fusion_matmul_status(_stream(stream), ctypes.byref(d))
    if rc not in (AR_OK, AR_ERR_TIMEOUT):
        _check(rc)
    return rc, d.value


def ar_fusion_combine(rows_in: torch.Tensor, position: torch.Tensor, weights: torch.Tensor,
                      out: torch.Tensor, add: torch.Tensor | None = None, stream=None) -> None:
    """rows_in [in_rows, hidden]; position (int32) and weights (fp32) [tokens,
    topk]; out and add [tokens, hidden], of rows_in's type."""
    if _native is not None:
        rc = _native.combine(rows_in, position, weights, out, add, _handle(stream))
        if rc is not None:
            if rc:
                _check(rc)
            return
    if rows_in.dim() != 2 or position.dim() != 2:
        _shapes(("rows_in", rows_in, 2), ("position", position, 2))
    in_rows, hidden = rows_in.shape
    slots = tokens, topk = position.shape
    same, shape = (rows_in.dtype,), (tokens, hidden)
    try:
        dev = _device_of(rows_in)
        args = (_operand(rows_in, _ELEM, (in_rows, hidden), dev), in_rows,
                _operand(position, _I32, slots, dev), _operand(weights, _F32, slots, dev), tokens,
                topk, hidden, _ELEM[rows_in.dtype],
                None if add is None else _operand(add, same, shape, dev),
                _operand(out, same, shape, dev), _stream(stream))
    except _Refused:
        _explain(("rows_in", rows_in, _ELEM, None), ("position", position, _I32, None),
                 ("weights", weights, _F32, slots), ("out", out, same, shape),
                 ("add", add, same, shape))
    _call("ar_fusion_combine", args)


# -------------------------------------------------------- attention layers

_CACHE = {torch.bfloat16: AR_DT_BF16, torch.float16: AR_DT_FP16, torch.float8_e4m3fn: AR_DT_E4M3}
_ROWS = (torch.bfloat16, torch.float16)


def _fits(name: str, value: int) -> int:
    if not -1 << 31 <= value < 1 << 31:
        raise ValueError(f"{name}: {value} does not fit a 32-bit integer")
    return value


def _head_rows(name: str, t: torch.Tensor, rows: int, dtype, dim: int, heads: int | None = None):
    """A [rows, heads, dim] tensor whose last dimension is contiguous."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: type {t.dtype}, expected {dtype}")
    if t.dim() != 3 or t.shape[0] != rows or t.shape[2] != dim or heads not in (None, t.shape[1]):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected "
                         f"({rows}, {'heads' if heads is None else heads}, {dim})")
    _placed(name, t)
    if dim > 1 and t.stride(2) != 1 and t.numel():
        raise ValueError(f"{name}: expected a contiguous last dimension")
    return _HeadRows(t.data_ptr(), t.stride(0), t.stride(1))


def _placed(name: str, t: torch.Tensor) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name}: on {t.device}, and the current device is "
                         f"cuda:{torch.cuda.current_device()}")


def _array(name: str, t: torch.Tensor, dtype, shape) -> int:
    if t.dtype != dtype:
        raise TypeError(f"{name}: type {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    _placed(name, t)
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _kv_cache(k_cache, v_cache, page_table, lengths, kv_scale) -> _KvCache:
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype not in _CACHE:
            raise TypeError(f"{name}: unsupported type {t.dtype}")
        if t.dim() != 4:
            raise ValueError(f"{name}: {t.dim()} dimensions, expected 4")
    if v_cache.dtype != k_cache.dtype:
        raise TypeError(f"v_cache: type {v_cache.dtype}, expected {k_cache.dtype}")
    if v_cache.shape != k_cache.shape:
        raise ValueError(f"v_cache: shape {tuple(v_cache.shape)}, expected {tuple(k_cache.shape)}")
    if page_table.dim() != 2:
        raise ValueError(f"page_table: {page_table.dim()} dimensions, expected 2")
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _placed(name, t)
        if t.shape[3] > 1 and t.stride(3) != 1 and t.numel():
            raise ValueError(f"{name}: expected a contiguous last dimension")
    pages, page_size, heads, dim = (_fits("k_cache", n) for n in k_cache.shape)
    S, most = (_fits("page_table", n) for n in page_table.shape)
    return _KvCache(
        k_cache.data_ptr(), v_cache.data_ptr(), *k_cache.stride()[:3], *v_cache.stride()[:3],
        _CACHE[k_cache.dtype], pages, page_size, heads, dim, S, most,
        None if kv_scale is None else _array("kv_scale", kv_scale, torch.float32, (2,)),
        _array("page_table", page_table, torch.int32, (S, most)),
        _array("lengths", lengths, torch.int32, (S,)))


def ar_fusion_rope_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
                          k_cache: torch.Tensor, v_cache: torch.Tensor,
                          page_table: torch.Tensor, lengths: torch.Tensor,
                          inv_freq: torch.Tensor | None, q_out: torch.Tensor | None = None,
                          starts: torch.Tensor | None = None,
                          positions: torch.Tensor | None = None, sections=None,
                          interleaved: bool = False, kv_scale: torch.Tensor | None = None,
                          stream=None) -> None:
    """Rotates q [tokens, q_heads, dim] into q_out (q itself if None) and k [tokens, heads, dim],
    and writes k and v into the caches [pages, page_size, heads, dim] (bf16 / fp16 as the
    rows, or float8_e4m3fn with kv_scale [2] fp32 or None).  Any strides with a
    contiguous last dimension.  page_table [sequences, max_pages], lengths [sequences] (the
    new tokens included), starts [sequences + 1] (None: a row for each sequence),
    positions [tokens] or [axes, tokens] (None: the index in the sequence) int32; inv_freq
    [rot / 2] fp32 (None: no rotation); sections: pairs of each axis (None: one axis)."""
    if sections is not None:
        sections = tuple(sections)
    if _native is not None:
        rc = _native.rope_append(q, k, v, k_cache, v_cache, page_table, lengths, inv_freq, q_out,
                                 starts, positions, sections, interleaved, kv_scale,
                                 _handle(stream))
        if rc is not None:
            if rc:
                _check(rc)
            return
    if k.dim() != 3:
        raise ValueError(f"k: {k.dim()} dimensions, expected 3")
    if k.dtype not in _ROWS:
        raise TypeError(f"k: unsupported type {k.dtype}")
    cache = _kv_cache(k_cache, v_cache, page_table, lengths, kv_scale)
    tokens, dt, dim, heads = _fits("k", k.shape[0]), k.dtype, cache.head_dim, cache.heads
    if cache.dtype != AR_DT_E4M3 and k_cache.dtype != dt:
        raise TypeError(f"k_cache: type {k_cache.dtype}, expected {dt} or {torch.float8_e4m3fn}")
    kr, vr = _head_rows("k", k, tokens, dt, dim, heads), _head_rows("v", v, tokens, dt, dim, heads)
    qr = qo = None
    q_heads = 0
    if q is not None:
        qr = _head_rows("q", q, tokens, dt, dim)
        q_heads = _fits("q", q.shape[1])
        qo = qr if q_out is None else _head_rows("q_out", q_out, tokens, dt, dim, q_heads)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rot = 0 if inv_freq is None else _fits("inv_freq", 2 * inv_freq.numel())
    axes = 1 if sections is None else len(sections)
    shape = (axes, tokens) if positions is not None and positions.dim() == 2 else (tokens,)
    if sections is not None and axes > 1:
        shape = (axes, tokens)
    table = None if sections is None else (_i * max(axes, 1))(*(_fits("sections", n) for n in sections))
    rc = lib().ar_fusion_rope_append(
        ctypes.byref(cache), None if qr is None else ctypes.byref(qr),
        None if qo is None else ctypes.byref(qo), ctypes.byref(kr), ctypes.byref(vr), tokens,
        q_heads, _ELEM[dt],
        None if starts is None else _array("starts", starts, torch.int32, (cache.sequences + 1,)),
        None if positions is None else _array("positions", positions, torch.int32, shape),
        None if inv_freq is None else _array("inv_freq", inv_freq, torch.float32, (rot // 2,)),
        rot, table, axes, 1 if interleaved else 0, _stream(stream))
    if rc:
        _check(rc)


def _attention(name, q, k_cache, v_cache, page_table, lengths, out, workspace, scale, window,
               sinks, lse, kv_scale, starts, stream):
    if scale is None:
        scale = max(1, k_cache.shape[-1] if k_cache.dim() else 1) ** -0.5
    if _native is not None:
        rc = _native.attention(q, k_cache, v_cache, page_table, lengths, starts, out, workspace,
                               float(scale), window, sinks, lse, kv_scale, _handle(stream))
        if rc is not None:
            if rc:
                _check(rc)
            return
    if q.dim() != 3:
        raise ValueError(f"q: {q.dim()} dimensions, expected 3")
    if q.dtype not in _ROWS:
        raise TypeError(f"q: unsupported type {q.dtype}")
    cache = _kv_cache(k_cache, v_cache, page_table, lengths, kv_scale)
    tokens, q_heads = (_fits("q", n) for n in q.shape[:2])
    if cache.dtype != AR_DT_E4M3 and k_cache.dtype != q.dtype:
        raise TypeError(f"k_cache: type {k_cache.dtype}, expected {q.dtype} or {torch.float8_e4m3fn}")
    if name == "ar_fusion_decode_attention" and tokens != cache.sequences:
        raise ValueError(f"q: {tokens} rows for {cache.sequences} sequences")
    qr = _head_rows("q", q, tokens, q.dtype, cache.head_dim)
    to = _head_rows("out", out, tokens, q.dtype, cache.head_dim, q_heads)
    work, size = None, 0
    if workspace is not None:
        size = workspace.numel() * workspace.element_size()
        work = _array("workspace", workspace, workspace.dtype, workspace.shape)
    args = [ctypes.byref(cache), ctypes.byref(qr), ctypes.byref(to),
            None if lse is None else _array("lse", lse, torch.float32, (tokens, q_heads))]
    if name == "ar_fusion_prompt_attention":
        args += [_array("starts", starts, torch.int32, (cache.sequences + 1,)), tokens]
    args += [q_heads, _ELEM[q.dtype], scale, _fits("window", window), _fits("sinks", sinks), work,
             size, _stream(stream)]
    rc = getattr(lib(), name)(*args)
    if rc:
        _check(rc)


def ar_fusion_decode_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               page_table: torch.Tensor, lengths: torch.Tensor,
                               out: torch.Tensor, workspace: torch.Tensor | None = None,
                               scale: float | None = None, window: int = 0, sinks: int = 0,
                               lse: torch.Tensor | None = None,
                               kv_scale: torch.Tensor | None = None, stream=None) -> None:
    """One new token per sequence: q and out [sequences, q_heads, dim], lse [sequences, q_heads]
    fp32; caches and sequences as ar_fusion_rope_append takes them.  scale None:
    1 / sqrt(dim).  workspace: AR_ATTENTION_WORKSPACE_BYTES of one call at a time (None: a
    sequence's keys are not split over the GPU)."""
    _attention("ar_fusion_decode_attention", q, k_cache, v_cache, page_table, lengths, out,
               workspace, scale, window, sinks, lse, kv_scale, None, stream)


def ar_fusion_prompt_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               page_table: torch.Tensor, lengths: torch.Tensor,
                               starts: torch.Tensor, out: torch.Tensor,
                               workspace: torch.Tensor | None = None,
                               scale: float | None = None, window: int = 0, sinks: int = 0,
                               lse: torch.Tensor | None = None,
                               kv_scale: torch.Tensor | None = None, stream=None) -> None:
    """Any number of new tokens per sequence: q and out [tokens, q_heads, dim], lse [tokens,
    q_heads] fp32, starts [sequences + 1] int32; the rest as ar_fusion_decode_attention."""
    if starts is None:
        raise ValueError("starts: expected a tensor")
    _attention("ar_fusion_prompt_attention", q, k_cache, v_cache, page_table, lengths, out,
               workspace, scale, window, sinks, lse, kv_scale, starts, stream)


def ar_fusion_attention_status(stream=None):
    """ar_fusion_matmul_status of ar_fusion_prompt_attention."""
    d = ctypes.c_int(-1)
    rc = lib().ar_fusion_attention_status(_stream(stream), ctypes.byref(d))
    if rc not in (AR_OK, AR_ERR_TIMEOUT):
        _check(rc)
    return rc, d.value
