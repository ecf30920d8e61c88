"""Python binding of the GB300 MoE FFN layer's C ABI (include/moe.h).

Argument marshalling only: every function below hands pointers and sizes to ``libmoe.so`` and
every step of the layer runs in its CUDA kernels.  PyTorch is used for device memory and streams.
There is no fallback: if the library is missing or fails to load, ``load()`` raises.

Tensors are passed as torch tensors (their ``data_ptr()``), ``None`` for optional ones.  bf16
tensors may be ``torch.bfloat16`` or any 16-bit dtype holding bf16 bits.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK = 0
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
          4: "MOE_ERR_CUDA", 5: "MOE_ERR_BAD_INDEX", 6: "MOE_ERR_TIMEOUT"}

# Every entry point declared in include/moe.h.
EXPORTS = ("moe_workspace_size", "moe_perm_rows", "moe_workspace_init", "moe_route", "moe_dispatch",
           "moe_dispatch_noalloc",
           "moe_expert_ffn_fwd", "moe_combine", "moe_expert_ffn_bwd", "moe_router_bwd",
           "moe_combine_bwd", "moe_layer_fwd", "moe_layer_bwd", "moe_check_error",
           "moe_debug_inject", "moe_profile_enable", "moe_profile_read", "moe_status_string",
           "moe_quantize_rows_e4m3", "moe_gate_up_fp8", "moe_down_fp8", "moe_layer_fwd_fp8",
           "moe_keep_rows_for_budget", "moe_keep_rows_for_free_memory", "moe_quantize_cols_e4m3",
           "moe_layer_bwd_fp8", "moe_saved_layout", "moe_profile_sm_clock", "moe_grouped_workspace_size",
           "moe_grouped_workspace_init", "moe_segments", "moe_grouped_mm", "moe_grouped_mm_dx", "moe_grouped_mm_dw",
           "moe_quantize_rows_i8", "moe_grouped_mm_i8", "moe_select", "moe_select_bwd", "moe_router_wgrad",
           "moe_mx_scale_stride", "moe_quantize_rows_mxf4", "moe_grouped_mm_mxf4")


class moe_config_t(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("capacity_factor", ctypes.c_float),
                ("keep_rows", ctypes.c_int32), ("gather_in_gemm", ctypes.c_int32)]


class moe_grouped_t(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("n_in", ctypes.c_int32), ("n_out", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("dtype", ctypes.c_int32), ("dw_dtype", ctypes.c_int32),
                ("accumulate", ctypes.c_int32), ("in_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64)]


class moe_select_t(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("score", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


# moe_score_t
SCORES = {"softmax": 0, "sigmoid": 1}

# moe_dtype_t
BF16, FP16, FP32 = 0, 1, 2


class MoEError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)}")


_lib = None
_P = ctypes.c_void_p


def load(path: str | None = None):
    """Load libmoe.so (building it first if it is missing and nvcc is available)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        from . import _build
        _build.build()
    lib = ctypes.CDLL(path)
    cfgp = ctypes.POINTER(moe_config_t)
    grpp = ctypes.POINTER(moe_grouped_t)
    selp = ctypes.POINTER(moe_select_t)
    sig = {
        "moe_workspace_size": [cfgp, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)],
        "moe_perm_rows": [cfgp, ctypes.POINTER(ctypes.c_int64)],
        "moe_saved_layout": [cfgp] + [ctypes.POINTER(ctypes.c_size_t)] * 4,
        "moe_keep_rows_for_budget": [cfgp, ctypes.c_uint64, ctypes.POINTER(ctypes.c_int32),
                                     ctypes.POINTER(ctypes.c_uint64)],
        "moe_keep_rows_for_free_memory": [cfgp, ctypes.c_uint64, ctypes.POINTER(ctypes.c_int32),
                                          ctypes.POINTER(ctypes.c_uint64)],
        "moe_workspace_init": [cfgp, _P, ctypes.c_size_t, _P],
        "moe_route": [cfgp, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_dispatch": [cfgp, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_dispatch_noalloc": [cfgp, _P, _P, _P, _P, _P, _P, _P, _P, _P],
        "moe_expert_ffn_fwd": [cfgp, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_combine": [cfgp, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_expert_ffn_bwd": [cfgp, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_router_bwd": [cfgp, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_combine_bwd": [cfgp, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_quantize_rows_e4m3": [_P, ctypes.c_int64, ctypes.c_int32, _P, _P, _P],
        "moe_gate_up_fp8": [cfgp, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_down_fp8": [cfgp, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_layer_fwd_fp8": [cfgp, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_quantize_cols_e4m3": [_P, _P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P,
                                   _P],
        "moe_layer_bwd_fp8": [cfgp] + [_P] * 20 + [ctypes.c_size_t, _P],
        "moe_layer_fwd": [cfgp, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_layer_bwd": [cfgp, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                          ctypes.c_size_t, _P],
        "moe_check_error": [_P, _P],
        "moe_debug_inject": [_P, ctypes.c_int32, ctypes.c_int32, ctypes.c_uint64, _P],
        "moe_profile_enable": [ctypes.c_int32],
        "moe_profile_sm_clock": [ctypes.c_int32, ctypes.POINTER(ctypes.c_double)],
        "moe_profile_read": [ctypes.c_int32, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_double),
                             ctypes.POINTER(ctypes.c_int32)],
        "moe_grouped_workspace_size": [grpp, ctypes.POINTER(ctypes.c_size_t)],
        "moe_grouped_workspace_init": [grpp, _P, ctypes.c_size_t, _P],
        "moe_segments": [cfgp, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_grouped_mm": [grpp, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_grouped_mm_dx": [grpp, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_grouped_mm_dw": [grpp, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_quantize_rows_i8": [_P, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, _P, _P, _P],
        "moe_grouped_mm_i8": [grpp, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_mx_scale_stride": [ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)],
        "moe_quantize_rows_mxf4": [_P, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, _P, _P, _P],
        "moe_grouped_mm_mxf4": [grpp, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_select": [selp, _P, _P, _P, _P, _P],
        "moe_select_bwd": [selp, _P, _P, _P, _P, _P],
        "moe_router_wgrad": [cfgp, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
        "moe_status_string": [ctypes.c_int],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_char_p if name == "moe_status_string" else ctypes.c_int
    _lib = lib
    return lib


# ------------------------------------------------------------------------------------------------
# marshalling helpers
# ------------------------------------------------------------------------------------------------

def config(T: int, d: int, f: int, E: int, k: int, S: int = 0, renorm: int = 0, cf: float = 0.0,
           keep_rows: int = 0, gather_in_gemm: int = 0):
    return moe_config_t(int(T), int(d), int(f), int(E), int(k), int(S), int(renorm), float(cf), int(keep_rows),
                        int(gather_in_gemm))


def dtype_code(t) -> int:
    """moe_dtype_t of a torch dtype (or the code itself)."""
    if isinstance(t, int):
        return t
    code = {"torch.bfloat16": BF16, "torch.float16": FP16, "torch.float32": FP32}.get(str(t))
    if code is None:
        raise ValueError(f"no grouped product of {t}")
    return code


def grouped_config(rows: int, n_in: int, n_out: int, groups: int, dtype=BF16, dw_dtype=None, accumulate: int = 0,
                   in_stride: int = 0, out_stride: int = 0) -> moe_grouped_t:
    """Description of the grouped products of [rows, n_in] rows with weights [groups, n_out, n_in]; the
    types are torch dtypes or moe_dtype_t codes, dW's the operands' unless given."""
    code = dtype_code(dtype)
    return moe_grouped_t(int(rows), int(n_in), int(n_out), int(groups), code,
                         code if dw_dtype is None else dtype_code(dw_dtype), int(accumulate), int(in_stride),
                         int(out_stride))


def select_config(T: int, E: int, k: int, score="softmax", groups: int = 1, top_groups: int | None = None,
                  group_top: int = 1, renorm: int = 0, scale: float = 1.0, dtype=FP32) -> moe_select_t:
    """Description of a selection of k of E experts for T tokens; score is "softmax" or "sigmoid" (or a moe_score_t
    code), dtype that of the logits (a torch dtype or a moe_dtype_t code); all groups stay unless top_groups
    says how many."""
    code = SCORES.get(score, score)
    if not isinstance(code, int):
        raise ValueError(f"no score {score!r}")
    return moe_select_t(int(T), int(E), int(k), code, int(groups), int(groups if top_groups is None else top_groups),
                        int(group_top), int(renorm), float(scale), dtype_code(dtype))


def grouped_workspace(cfg: moe_grouped_t, device="cuda", stream=None):
    """A device workspace for the grouped products of cfg, its header initialised."""
    import torch
    ws = torch.empty(moe_grouped_workspace_size(cfg), dtype=torch.uint8, device=device)
    moe_grouped_workspace_init(cfg, ws, stream)
    return ws


def config_from(c: dict) -> moe_config_t:
    """From a workload dict with keys T, d, f, E, k, S, renorm, cf (and keep_rows, gather_in_gemm,
    default 0)."""
    return config(c["T"], c["d"], c["f"], c["E"], c["k"], c.get("S", 0), c.get("renorm", 0), c.get("cf", 0.0),
                  c.get("keep_rows", 0), c.get("gather_in_gemm", 0))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to the MoE library must be contiguous")
    return t.data_ptr()


_holds = None            # kind -> the torch dtypes that hold it
_current_device = None   # () -> index of the device that calls run on
_current_stream = None   # index of a device -> handle of its current stream


def _bind_torch():
    """The names above, each after those that its users take with it: another thread may look at any time."""
    global _holds, _current_device, _current_stream
    import torch
    if _current_device is None:
        _current_device = torch._C._cuda_getDevice
    _current_stream = torch._C._cuda_getCurrentRawStream
    _holds = {BF16: (torch.bfloat16, torch.int16, torch.uint16), FP16: (torch.float16, torch.int16, torch.uint16),
              "f32": (torch.float32,), "i32": (torch.int32,), "i8": (torch.int8,),
              "u8": (torch.uint8,)}


def _grouped_ptr(t, shape, kind, what, on, stride=0):
    """Pointer of an operand of the grouped products: a CUDA tensor of this shape and type on the device `on`
    of the workspace (which is checked for itself), contiguous but for the rows of a matrix, which may be
    `stride` elements apart.  None and integers pass."""
    if t is None or isinstance(t, int):
        return t
    if _holds is None:
        _bind_torch()
    at = t.get_device()   # -1: the host
    holds = _holds.get(kind)   # None: a type that is none, the library's to refuse
    if t.shape != shape or at < 0 or (holds and t.dtype not in holds):
        raise ValueError(f"{what}: CUDA tensor {shape} of {holds[0] if holds else 'any type'} expected, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    if at != on and on >= 0:
        raise ValueError(f"{what}: tensors on one device expected, got one on {t.device}, others on cuda:{on}")
    if stride and stride != shape[1]:
        if t.numel() and (t.stride(1) != 1 or (shape[0] > 1 and t.stride(0) != stride)):
            raise ValueError(f"{what}: rows {stride} elements apart expected, got strides {t.stride()}")
    elif not t.is_contiguous():
        raise ValueError(f"{what}: contiguous tensor expected, got strides {t.stride()}")
    return t.data_ptr()


def _on_current(on, t, what):
    """t's device `on` is the one that the call runs on (an address of another may be none there)."""
    if _holds is None:
        _bind_torch()
    if on < 0 or on != _current_device():
        raise ValueError(f"{what}: a tensor on the current device expected, got one on {t.device}")


def _grouped_ws(ws, on, stream):
    """Pointer and size of a workspace on device `on`, and the stream of the call."""
    _on_current(on, ws, "ws")
    return _ptr(ws), ws.nbytes, _current_stream(on) if stream is None else _stream(stream)


def _stream(stream):
    if stream is None:
        if _current_stream is None:
            _bind_torch()
        # (the raw handle: a Stream object costs more than the rest of a call's marshalling)
        return _current_stream(_current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(code: int, where: str):
    if code != MOE_OK:
        raise MoEError(code, where)


def _call(name, *args):
    _check(getattr(load(), name)(*args), name)


# ------------------------------------------------------------------------------------------------
# the C entry points, one to one
# ------------------------------------------------------------------------------------------------

def moe_workspace_size(cfg: moe_config_t):
    ws, saved = ctypes.c_size_t(), ctypes.c_size_t()
    _call("moe_workspace_size", ctypes.byref(cfg), ctypes.byref(ws), ctypes.byref(saved))
    return ws.value, saved.value


def moe_saved_layout(cfg: moe_config_t):
    """(logits_off, logits_bytes, kept_off, kept_bytes) of the `saved` buffer."""
    v = [ctypes.c_size_t() for _ in range(4)]
    _call("moe_saved_layout", ctypes.byref(cfg), *(ctypes.byref(x) for x in v))
    return tuple(x.value for x in v)


def moe_perm_rows(cfg: moe_config_t) -> int:
    r = ctypes.c_int64()
    _call("moe_perm_rows", ctypes.byref(cfg), ctypes.byref(r))
    return r.value


def moe_keep_rows_for_budget(cfg: moe_config_t, budget_bytes: int):
    """(keep_rows, kept bytes) for a byte budget of kept activations."""
    r, b = ctypes.c_int32(), ctypes.c_uint64()
    _call("moe_keep_rows_for_budget", ctypes.byref(cfg), int(budget_bytes), ctypes.byref(r), ctypes.byref(b))
    return r.value, b.value


def moe_keep_rows_for_free_memory(cfg: moe_config_t, reserve_bytes: int):
    """(keep_rows, kept bytes) for the current device's free memory less ``reserve_bytes``."""
    r, b = ctypes.c_int32(), ctypes.c_uint64()
    _call("moe_keep_rows_for_free_memory", ctypes.byref(cfg), int(reserve_bytes), ctypes.byref(r),
          ctypes.byref(b))
    return r.value, b.value


def moe_workspace_init(cfg, ws, stream=None):
    _call("moe_workspace_init", ctypes.byref(cfg), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))


def moe_route(cfg, x, W_r, b_r, idx, gates, logits, ws, stream=None):
    _call("moe_route", ctypes.byref(cfg), _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(idx), _ptr(gates),
          _ptr(logits), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))


def moe_dispatch(cfg, idx, x, counts, offsets, row_of_slot, token_of_row, x_perm, ws, stream=None):
    _call("moe_dispatch", ctypes.byref(cfg), _ptr(idx), _ptr(x), _ptr(counts), _ptr(offsets),
          _ptr(row_of_slot), _ptr(token_of_row), _ptr(x_perm), _ptr(ws), ws.numel(), _stream(stream))


def moe_dispatch_noalloc(cfg, idx, x, counts, offsets, row_of_slot, token_of_row, x_perm, status=None,
                         stream=None):
    """moe_dispatch without a workspace (scratch in a fixed array inside the library); ``status``
    (optional int32 device tensor of one element) receives the call's device-side status."""
    _call("moe_dispatch_noalloc", ctypes.byref(cfg), _ptr(idx), _ptr(x), _ptr(counts), _ptr(offsets),
          _ptr(row_of_slot), _ptr(token_of_row), _ptr(x_perm), _ptr(status), _stream(stream))


def moe_expert_ffn_fwd(cfg, x_perm, W_gate, W_up, W_down, o_perm, ws, stream=None):
    _call("moe_expert_ffn_fwd", ctypes.byref(cfg), _ptr(x_perm), _ptr(W_gate), _ptr(W_up), _ptr(W_down),
          _ptr(o_perm), _ptr(ws), ws.numel(), _stream(stream))


def moe_combine(cfg, o_perm, gates, y, ws, stream=None):
    _call("moe_combine", ctypes.byref(cfg), _ptr(o_perm), _ptr(gates), _ptr(y), _ptr(ws), ws.numel(),
          _stream(stream))


def moe_expert_ffn_bwd(cfg, x_perm, dy, gates, W_gate, W_up, W_down, dx_perm, dgates,
                       dW_gate, dW_up, dW_down, ws, stream=None):
    _call("moe_expert_ffn_bwd", ctypes.byref(cfg), _ptr(x_perm), _ptr(dy), _ptr(gates), _ptr(W_gate),
          _ptr(W_up), _ptr(W_down), _ptr(dx_perm), _ptr(dgates), _ptr(dW_gate), _ptr(dW_up),
          _ptr(dW_down), _ptr(ws), ws.numel(), _stream(stream))


def moe_router_bwd(cfg, x, W_r, b_r, idx, gates, dgates, dlogits, dW_r, db_r, ws, stream=None):
    _call("moe_router_bwd", ctypes.byref(cfg), _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(idx), _ptr(gates),
          _ptr(dgates), _ptr(dlogits), _ptr(dW_r), _ptr(db_r), _ptr(ws), ws.numel(), _stream(stream))


def moe_combine_bwd(cfg, dx_perm, dlogits, W_r, dx, ws, stream=None):
    _call("moe_combine_bwd", ctypes.byref(cfg), _ptr(dx_perm), _ptr(dlogits), _ptr(W_r), _ptr(dx),
          _ptr(ws), ws.numel(), _stream(stream))


def _select_ptrs(c, logits, what):
    """Device of a selection's logits, on which the call has to run, and the kind of their type."""
    on = logits.get_device()
    _on_current(on, logits, what)
    return on, "f32" if c.dtype == FP32 else c.dtype


def moe_select(cfg, logits, bias, idx, weights, stream=None):
    """logits [T, E], bias [E] fp32 or None -> idx [T, k] int32, weights [T, k] fp32."""
    c = cfg
    on, kind = _select_ptrs(c, logits, "logits")
    _call("moe_select", ctypes.byref(c), _grouped_ptr(logits, (c.T, c.E), kind, "logits", on),
          _grouped_ptr(bias, (c.E,), "f32", "bias", on), _grouped_ptr(idx, (c.T, c.k), "i32", "idx", on),
          _grouped_ptr(weights, (c.T, c.k), "f32", "weights", on), _current_stream(on) if stream is None else _stream(stream))


def moe_select_bwd(cfg, logits, idx, dweights, dlogits, stream=None):
    """dlogits [T, E] of dweights [T, k], the selection held."""
    c = cfg
    on, kind = _select_ptrs(c, logits, "logits")
    _call("moe_select_bwd", ctypes.byref(c), _grouped_ptr(logits, (c.T, c.E), kind, "logits", on),
          _grouped_ptr(idx, (c.T, c.k), "i32", "idx", on), _grouped_ptr(dweights, (c.T, c.k), "f32", "dweights", on),
          _grouped_ptr(dlogits, (c.T, c.E), kind, "dlogits", on), _current_stream(on) if stream is None else _stream(stream))


def moe_router_wgrad(cfg, x, dlogits, dW_r, db_r, ws, stream=None):
    """dW_r [d, E] = x^T dlogits and db_r [E] (or None), the sum of dlogits over the tokens."""
    c, on = cfg, ws.get_device()
    _call("moe_router_wgrad", ctypes.byref(c), _grouped_ptr(x, (c.T, c.d_model), BF16, "x", on),
          _grouped_ptr(dlogits, (c.T, c.E), "f32", "dlogits", on), _grouped_ptr(dW_r, (c.d_model, c.E), "f32", "dW_r", on),
          _grouped_ptr(db_r, (c.E,), "f32", "db_r", on), *_grouped_ws(ws, on, stream))


def moe_quantize_rows_e4m3(src, codes, scales, stream=None):
    """src [rows, cols] bf16 -> codes [rows, cols] uint8, scales [rows] fp32."""
    rows, cols = src.shape[0], src.shape[-1]
    _call("moe_quantize_rows_e4m3", _ptr(src), int(src.numel() // cols) if rows else 0, int(cols), _ptr(codes),
          _ptr(scales), _stream(stream))


def moe_gate_up_fp8(cfg, x8, x_scale, wg8, wg_scale, wu8, wu_scale, h, ws, stream=None):
    _call("moe_gate_up_fp8", ctypes.byref(cfg), _ptr(x8), _ptr(x_scale), _ptr(wg8), _ptr(wg_scale), _ptr(wu8),
          _ptr(wu_scale), _ptr(h), _ptr(ws), ws.numel(), _stream(stream))


def moe_down_fp8(cfg, h8, h_scale, wd8, wd_scale, o_perm, ws, stream=None):
    _call("moe_down_fp8", ctypes.byref(cfg), _ptr(h8), _ptr(h_scale), _ptr(wd8), _ptr(wd_scale), _ptr(o_perm),
          _ptr(ws), ws.numel(), _stream(stream))


def moe_layer_fwd_fp8(cfg, x, W_r, b_r, wg8, wg_scale, wu8, wu_scale, wd8, wd_scale, y, saved, ws, stream=None):
    _call("moe_layer_fwd_fp8", ctypes.byref(cfg), _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(wg8), _ptr(wg_scale),
          _ptr(wu8), _ptr(wu_scale), _ptr(wd8), _ptr(wd_scale), _ptr(y), _ptr(saved), _ptr(ws), ws.numel(),
          _stream(stream))


def moe_quantize_cols_e4m3(top, bottom, codes, scales, stream=None):
    """top [G, r1, cols] (and bottom [G, r2, cols] or None) bf16 -> codes [G, cols, r1 + r2] uint8 and
    scales [G, cols] fp32: per-column codes of the stacked source, transposed."""
    G, r1, cols = top.shape
    r2 = 0 if bottom is None else bottom.shape[1]
    _call("moe_quantize_cols_e4m3", _ptr(top), _ptr(bottom), int(G), int(r1), int(r2), int(cols), _ptr(codes),
          _ptr(scales), _stream(stream))


def moe_layer_bwd_fp8(cfg, x, W_r, b_r, wg8, wg_scale, wu8, wu_scale, wdt8, wdt_scale, wgut8, wgut_scale, saved, dy,
                      dx, dW_r, db_r, dW_gate, dW_up, dW_down, ws, stream=None):
    _call("moe_layer_bwd_fp8", ctypes.byref(cfg), _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(wg8), _ptr(wg_scale),
          _ptr(wu8), _ptr(wu_scale), _ptr(wdt8), _ptr(wdt_scale), _ptr(wgut8), _ptr(wgut_scale), _ptr(saved),
          _ptr(dy), _ptr(dx), _ptr(dW_r), _ptr(db_r), _ptr(dW_gate), _ptr(dW_up), _ptr(dW_down), _ptr(ws),
          ws.numel(), _stream(stream))


def moe_layer_fwd(cfg, x, W_r, b_r, W_gate, W_up, W_down, y, saved, ws, stream=None):
    _call("moe_layer_fwd", ctypes.byref(cfg), _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(W_gate), _ptr(W_up),
          _ptr(W_down), _ptr(y), _ptr(saved), _ptr(ws), ws.numel(), _stream(stream))


def moe_layer_bwd(cfg, x, W_r, b_r, W_gate, W_up, W_down, saved, dy, dx, dW_r, db_r,
                  dW_gate, dW_up, dW_down, ws, stream=None):
    _call("moe_layer_bwd", ctypes.byref(cfg), _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(W_gate), _ptr(W_up),
          _ptr(W_down), _ptr(saved), _ptr(dy), _ptr(dx), _ptr(dW_r), _ptr(db_r), _ptr(dW_gate),
          _ptr(dW_up), _ptr(dW_down), _ptr(ws), ws.numel(), _stream(stream))


def moe_segments(cfg, row_begin, row_end, ws, stream=None):
    """begin and end [E + S] int32 of the padded segments of the last moe_dispatch on ws."""
    n, on = (cfg.E + cfg.n_shared,), ws.get_device()
    _call("moe_segments", ctypes.byref(cfg), _grouped_ptr(row_begin, n, "i32", "row_begin", on),
          _grouped_ptr(row_end, n, "i32", "row_end", on), *_grouped_ws(ws, on, stream))


def moe_grouped_workspace_size(cfg: moe_grouped_t) -> int:
    n = ctypes.c_size_t()
    _call("moe_grouped_workspace_size", ctypes.byref(cfg), ctypes.byref(n))
    return n.value


def moe_grouped_workspace_init(cfg, ws, stream=None):
    _call("moe_grouped_workspace_init", ctypes.byref(cfg), *_grouped_ws(ws, ws.get_device(), stream))


def moe_grouped_mm(cfg, row_begin, row_end, x, W, y, ws, stream=None):
    """y = x W[g]^T for the rows of every group g."""
    c, n, on = cfg, (cfg.groups,), ws.get_device()
    _call("moe_grouped_mm", ctypes.byref(c), _grouped_ptr(row_begin, n, "i32", "row_begin", on),
          _grouped_ptr(row_end, n, "i32", "row_end", on),
          _grouped_ptr(x, (c.rows, c.n_in), c.dtype, "x", on, c.in_stride),
          _grouped_ptr(W, (c.groups, c.n_out, c.n_in), c.dtype, "W", on),
          _grouped_ptr(y, (c.rows, c.n_out), c.dtype, "y", on, c.out_stride), *_grouped_ws(ws, on, stream))


def moe_grouped_mm_dx(cfg, row_begin, row_end, dy, W, dx, ws, stream=None):
    """dx = dy W[g] for the rows of every group g."""
    c, n, on = cfg, (cfg.groups,), ws.get_device()
    _call("moe_grouped_mm_dx", ctypes.byref(c), _grouped_ptr(row_begin, n, "i32", "row_begin", on),
          _grouped_ptr(row_end, n, "i32", "row_end", on),
          _grouped_ptr(dy, (c.rows, c.n_out), c.dtype, "dy", on, c.out_stride),
          _grouped_ptr(W, (c.groups, c.n_out, c.n_in), c.dtype, "W", on),
          _grouped_ptr(dx, (c.rows, c.n_in), c.dtype, "dx", on, c.in_stride), *_grouped_ws(ws, on, stream))


def moe_grouped_mm_dw(cfg, row_begin, row_end, dy, x, dW, ws, stream=None):
    """dW[g] = dy^T x over the rows of group g; with cfg.accumulate added to dW."""
    c, n, on = cfg, (cfg.groups,), ws.get_device()
    kind = "f32" if c.dw_dtype == FP32 and c.dtype != FP32 else c.dw_dtype
    _call("moe_grouped_mm_dw", ctypes.byref(c), _grouped_ptr(row_begin, n, "i32", "row_begin", on),
          _grouped_ptr(row_end, n, "i32", "row_end", on),
          _grouped_ptr(dy, (c.rows, c.n_out), c.dtype, "dy", on, c.out_stride),
          _grouped_ptr(x, (c.rows, c.n_in), c.dtype, "x", on, c.in_stride),
          _grouped_ptr(dW, (c.groups, c.n_out, c.n_in), kind, "dW", on), *_grouped_ws(ws, on, stream))


def moe_quantize_rows_i8(src, codes, scales, stream=None):
    """src [.., rows, cols] bf16 or fp16 -> codes of the same shape int8, scales [.., rows] fp32."""
    cols = src.shape[-1]
    rows = src.numel() // cols if cols else 0
    code, on = dtype_code(src.dtype), src.get_device()
    _on_current(on, src, "src")
    _call("moe_quantize_rows_i8", _grouped_ptr(src, tuple(src.shape), code, "src", on), code, int(rows), int(cols),
          _grouped_ptr(codes, tuple(src.shape), "i8", "codes", on),
          _grouped_ptr(scales, tuple(src.shape[:-1]), "f32", "scales", on), _stream(stream))


def moe_grouped_mm_i8(cfg, row_begin, row_end, codes, scales, Wq, W_scale, y, ws, stream=None):
    """y = (codes Wq[g]^T) scaled by the rows' and the output channels' scales."""
    c, n, on = cfg, (cfg.groups,), ws.get_device()
    _call("moe_grouped_mm_i8", ctypes.byref(c), _grouped_ptr(row_begin, n, "i32", "row_begin", on),
          _grouped_ptr(row_end, n, "i32", "row_end", on),
          _grouped_ptr(codes, (c.rows, c.n_in), "i8", "codes", on, c.in_stride),
          _grouped_ptr(scales, (c.rows,), "f32", "scales", on),
          _grouped_ptr(Wq, (c.groups, c.n_out, c.n_in), "i8", "Wq", on),
          _grouped_ptr(W_scale, (c.groups, c.n_out), "f32", "W_scale", on),
          _grouped_ptr(y, (c.rows, c.n_out), c.dtype, "y", on, c.out_stride), *_grouped_ws(ws, on, stream))


def moe_mx_scale_stride(cols: int) -> int:
    """Bytes from one row of 4-bit values' scales to the next: cols / 32 rounded up to 16."""
    n = ctypes.c_int32()
    _call("moe_mx_scale_stride", int(cols), ctypes.byref(n))
    return n.value


def moe_quantize_rows_mxf4(src, codes, scales, stream=None):
    """src [.., rows, cols] bf16, fp16 or fp32 -> codes [.., rows, cols / 2] and scales [.., rows,
    moe_mx_scale_stride(cols)], both uint8."""
    cols = src.shape[-1]
    rows = src.numel() // cols if cols else 0
    code, on = dtype_code(src.dtype), src.get_device()
    _on_current(on, src, "src")
    lead = tuple(src.shape[:-1])
    _call("moe_quantize_rows_mxf4", _grouped_ptr(src, tuple(src.shape), "f32" if code == FP32 else code, "src", on), code,
          int(rows), int(cols), _grouped_ptr(codes, (*lead, cols // 2), "u8", "codes", on),
          _grouped_ptr(scales, (*lead, (cols // 32 + 15) // 16 * 16), "u8", "scales", on),
          _current_stream(on) if stream is None else _stream(stream))


def moe_grouped_mm_mxf4(cfg, row_begin, row_end, codes, scales, Wq, W_scale, y, ws, stream=None):
    """y = x W[g]^T of 4-bit values with their scales, as moe_quantize_rows_mxf4 gives them."""
    c, n, on = cfg, (cfg.groups,), ws.get_device()
    lds = (c.n_in // 32 + 15) // 16 * 16
    _call("moe_grouped_mm_mxf4", ctypes.byref(c), _grouped_ptr(row_begin, n, "i32", "row_begin", on),
          _grouped_ptr(row_end, n, "i32", "row_end", on),
          _grouped_ptr(codes, (c.rows, c.n_in // 2), "u8", "codes", on, c.in_stride // 2),
          _grouped_ptr(scales, (c.rows, lds), "u8", "scales", on),
          _grouped_ptr(Wq, (c.groups, c.n_out, c.n_in // 2), "u8", "Wq", on),
          _grouped_ptr(W_scale, (c.groups, c.n_out, lds), "u8", "W_scale", on),
          _grouped_ptr(y, (c.rows, c.n_out), c.dtype, "y", on, c.out_stride), *_grouped_ws(ws, on, stream))


def moe_check_error(ws, stream=None) -> int:
    """Synchronise and return (and clear) the first device-side status recorded in ws."""
    return load().moe_check_error(_ptr(ws), _stream(stream))


def moe_debug_inject(ws, stall_block: int, timeout_ns: int, stream=None, stall_fill: int = -1):
    _call("moe_debug_inject", _ptr(ws), int(stall_block), int(stall_fill), int(timeout_ns), _stream(stream))


def moe_profile_enable(on: bool):
    _call("moe_profile_enable", int(bool(on)))


def moe_profile_read() -> dict:
    """{kernel name: (total ms, launches)} for every kernel of the library (waits for the events)."""
    out, i = {}, 0
    name, ms, n = ctypes.c_char_p(), ctypes.c_double(), ctypes.c_int32()
    while True:
        code = load().moe_profile_read(i, ctypes.byref(name), ctypes.byref(ms), ctypes.byref(n))
        if code == 1:
            return out
        _check(code, "moe_profile_read")
        out[name.value.decode()] = (ms.value, n.value)
        i += 1


def moe_profile_sm_clock() -> dict:
    """{kernel name: mean SM MHz} of the tensor-core GEMM kernels that ran since
    moe_profile_enable (in-kernel clock64 over globaltimer; synchronises the device)."""
    names = moe_profile_read()
    out = {}
    mhz = ctypes.c_double()
    for i, name in enumerate(names):
        _call("moe_profile_sm_clock", i, ctypes.byref(mhz))
        if mhz.value > 0:
            out[name] = mhz.value
    return out


def moe_status_string(code: int) -> str:
    return load().moe_status_string(int(code)).decode()


# ------------------------------------------------------------------------------------------------
# buffers of one layer instance
# ------------------------------------------------------------------------------------------------

@dataclass
class Buffers:
    """Device buffers a layer instance needs: the workspace (header initialised) and `saved`."""
    cfg: moe_config_t
    ws: object
    saved: object
    rows: int

    @classmethod
    def allocate(cls, cfg: moe_config_t, device="cuda", stream=None):
        import torch
        ws_bytes, saved_bytes = moe_workspace_size(cfg)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=device)
        saved = torch.empty(saved_bytes, dtype=torch.uint8, device=device)
        moe_workspace_init(cfg, ws, stream)
        return cls(cfg, ws, saved, moe_perm_rows(cfg))

    def saved_views(self):
        """Views of `saved`: idx int32 [T,k], gates fp32 [T,k], logits fp32 [T,E] (None with
        renormalised gates, which keep none)."""
        import torch
        T, k, E = self.cfg.T, self.cfg.k, self.cfg.E
        idx = self.saved[:4 * T * k].view(torch.int32).view(T, k)
        gates = self.saved[4 * T * k:8 * T * k].view(torch.float32).view(T, k)
        off, nbytes, _, _ = moe_saved_layout(self.cfg)
        logits = self.saved[off:off + nbytes].view(torch.float32).view(T, E) if nbytes else None
        return idx, gates, logits
