"""Thin ctypes binding of libarfusion (include/ar_fusion.h).

Argument marshalling only: every function has the name of the C entry point,
turns torch tensors into device pointers / sizes, calls the library, and raises
:class:`ArFusionError` on a non-zero status.  No compute happens here and
there is no fallback: if the library is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libarfusion.so")

# enum ar_dtype
AR_DT_BF16 = 0
AR_DT_FP16 = 1
AR_DT_FP32 = 2
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


_lib = None
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
                 "ar_fusion_matmul_status"):
        getattr(L, name).restype = _i
    _lib = L
    return L


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
        return torch.cuda.current_stream().cuda_stream
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

def _expect(cond: bool, what: str) -> None:
    if not cond:
        raise ValueError(what)


def _typed(name: str, t: torch.Tensor, dtypes, shape=None) -> None:
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported type {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _on_current(*ts) -> None:
    """The library launches on the current device: operands of another one are refused."""
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("expected a CUDA tensor")
        if dev is None:
            dev = torch.cuda.current_device()
        if t.device.index != dev:
            raise ValueError(f"expected tensors of the current device cuda:{dev}, got {t.device}")


_ELEM = (torch.bfloat16, torch.float16, torch.float32)
_FP8 = (torch.uint8, torch.float8_e4m3fn)
_I32 = (torch.int32,)
_F32 = (torch.float32,)


def _quant_blocks(depth: int) -> int:
    return (depth + AR_QUANT_BLOCK - 1) // AR_QUANT_BLOCK


def ar_fusion_route(logits: torch.Tensor, bias: torch.Tensor | None, ids_out: torch.Tensor,
                    weights_out: torch.Tensor, score: int = AR_SCORE_SIGMOID, groups: int = 1,
                    groups_kept: int = 1, group_score: int = AR_GROUP_TOP2,
                    renormalize: bool = True, scale: float = 1.0, stream=None) -> None:
    """logits [tokens, experts]; bias [experts] fp32 or None; ids_out (int32)
    and weights_out (fp32) [tokens, topk]."""
    _typed("logits", logits, _ELEM)
    _expect(logits.dim() == 2 and ids_out.dim() == 2, "logits and ids_out have two dimensions")
    tokens, experts = logits.shape
    topk = ids_out.shape[1]
    _typed("ids_out", ids_out, _I32, (tokens, topk))
    _typed("weights_out", weights_out, _F32, (tokens, topk))
    if bias is not None:
        _typed("bias", bias, _F32, (experts,))
    _on_current(logits, bias, ids_out, weights_out)
    _check(lib().ar_fusion_route(_ptr(logits), tokens, experts, _dtype_id(logits), _ptr(bias),
                                 int(score), int(groups), int(groups_kept), int(group_score),
                                 topk, int(renormalize), ctypes.c_float(scale), _ptr(ids_out),
                                 _ptr(weights_out), _stream(stream)))


def ar_fusion_expert_plan(ids: torch.Tensor, experts: int, offsets_out: torch.Tensor,
                          position_out: torch.Tensor, first_expert: int = 0,
                          stream=None) -> None:
    """ids [tokens, topk] int32; offsets_out [experts + 1] and position_out
    [tokens, topk] int32, for the experts first_expert .. first_expert + experts - 1."""
    _expect(ids.dim() == 2, "ids has two dimensions")
    _typed("ids", ids, _I32)
    _typed("offsets_out", offsets_out, _I32, (experts + 1,))
    _typed("position_out", position_out, _I32, ids.shape)
    _on_current(ids, offsets_out, position_out)
    _check(lib().ar_fusion_expert_plan(_ptr(ids), ids.shape[0], ids.shape[1], int(first_expert),
                                       int(experts), _ptr(offsets_out), _ptr(position_out),
                                       _stream(stream)))


def ar_fusion_quant_blocks(x: torch.Tensor, quant_out: torch.Tensor, scale_out: torch.Tensor,
                           position: torch.Tensor | None = None,
                           activation: int = AR_ACT_NONE,
                           row_count: torch.Tensor | None = None, stream=None) -> None:
    """x [rows, hidden] ([rows, 2 * hidden] with AR_ACT_SILU_MUL); quant_out
    [out_rows, hidden] (uint8 or float8_e4m3fn); scale_out [out_rows,
    ceil(hidden / 128)] fp32; position [rows, copies] int32 or None; row_count: a
    one-element int32 tensor or None (a view of the plan's last offset)."""
    _typed("x", x, _ELEM)
    _expect(x.dim() == 2 and quant_out.dim() == 2, "x and quant_out have two dimensions")
    rows = x.shape[0]
    out_rows, hidden = quant_out.shape
    _typed("x", x, _ELEM, (rows, hidden * (2 if activation == AR_ACT_SILU_MUL else 1)))
    _typed("quant_out", quant_out, _FP8)
    _typed("scale_out", scale_out, _F32, (out_rows, _quant_blocks(hidden)))
    copies = 1
    if position is not None:
        _expect(position.dim() == 2 and position.shape[0] == rows, "position is [rows, copies]")
        _typed("position", position, _I32)
        copies = position.shape[1]
    if row_count is not None:
        _typed("row_count", row_count, _I32)
        _expect(row_count.numel() == 1, "row_count has one element")
    _on_current(x, quant_out, scale_out, position, row_count)
    _check(lib().ar_fusion_quant_blocks(_ptr(x), rows, hidden, _dtype_id(x), int(activation),
                                        _ptr(position), copies, _ptr(row_count), out_rows,
                                        _ptr(quant_out), _ptr(scale_out), _stream(stream)))


def ar_fusion_matmul_fp8(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor,
                         b_scale: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """a [rows, depth], b [cols, depth] (uint8 or float8_e4m3fn); a_scale [rows,
    ceil(depth / 128)], b_scale [ceil(cols / 128), ceil(depth / 128)] fp32; out [rows, cols]."""
    _expect(a.dim() == 2 and b.dim() == 2, "a and b have two dimensions")
    (rows, depth), cols = a.shape, b.shape[0]
    blocks = _quant_blocks(depth)
    _typed("a", a, _FP8)
    _typed("b", b, _FP8, (cols, depth))
    _typed("a_scale", a_scale, _F32, (rows, blocks))
    _typed("b_scale", b_scale, _F32, (_quant_blocks(cols), blocks))
    _typed("out", out, _ELEM, (rows, cols))
    _on_current(a, a_scale, b, b_scale, out)
    _check(lib().ar_fusion_matmul_fp8(_ptr(a), _ptr(a_scale), _ptr(b), _ptr(b_scale), rows, cols,
                                      depth, _dtype_id(out), _ptr(out), _stream(stream)))


def ar_fusion_expert_matmul_fp8(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor,
                                b_scale: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor,
                                stream=None) -> None:
    """ar_fusion_matmul_fp8 by experts: b [experts, cols, depth], b_scale
    [experts, ceil(cols / 128), ceil(depth / 128)], offsets [experts + 1] int32."""
    _expect(a.dim() == 2 and b.dim() == 3, "a has two dimensions, b three")
    (rows, depth), (experts, cols) = a.shape, b.shape[:2]
    blocks = _quant_blocks(depth)
    _typed("a", a, _FP8)
    _typed("b", b, _FP8, (experts, cols, depth))
    _typed("a_scale", a_scale, _F32, (rows, blocks))
    _typed("b_scale", b_scale, _F32, (experts, _quant_blocks(cols), blocks))
    _typed("offsets", offsets, _I32, (experts + 1,))
    _typed("out", out, _ELEM, (rows, cols))
    _on_current(a, a_scale, b, b_scale, offsets, out)
    _check(lib().ar_fusion_expert_matmul_fp8(_ptr(a), _ptr(a_scale), _ptr(b), _ptr(b_scale),
                                             _ptr(offsets), experts, rows, cols, depth,
                                             _dtype_id(out), _ptr(out), _stream(stream)))


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
    _typed("rows_in", rows_in, _ELEM)
    _expect(rows_in.dim() == 2 and position.dim() == 2, "rows_in and position have two dimensions")
    in_rows, hidden = rows_in.shape
    tokens, topk = position.shape
    _typed("position", position, _I32)
    _typed("weights", weights, _F32, (tokens, topk))
    _typed("out", out, (rows_in.dtype,), (tokens, hidden))
    if add is not None:
        _typed("add", add, (rows_in.dtype,), (tokens, hidden))
    _on_current(rows_in, position, weights, out, add)
    _check(lib().ar_fusion_combine(_ptr(rows_in), in_rows, _ptr(position), _ptr(weights), tokens,
                                   topk, hidden, _dtype_id(rows_in), _ptr(add), _ptr(out),
                                   _stream(stream)))
