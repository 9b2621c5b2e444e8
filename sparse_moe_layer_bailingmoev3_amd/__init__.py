"""Python binding of libmoe, the HIP (gfx950) forward pass of one BailingMoeV3 sparse MoE
layer (Ling-3.0-flash / Ling-3.0-flash-VL).

Argument marshalling only: every step of the layer runs in the library's kernels.  The
functions carry the C-ABI names of include/moe.h and take torch tensors that already live on
the GPU (torch provides device memory and streams).  The library must be built first:

    python -m sparse_moe_layer_bailingmoev3_amd.build

There is no fallback: if libmoe.so is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

__all__ = ["MoEConfig", "MoEExpertWeights", "MoEError", "lib_path", "load_library", "moe_workspace_size",
           "moe_route", "moe_dispatch", "moe_expert_ffn", "moe_combine", "moe_forward", "moe_forward_traced",
           "moe_forward_timed", "moe_update_expert_bias", "moe_dense_ffn_workspace_size", "moe_dense_ffn",
           "moe_forward_noalloc", "moe_quantise_mxfp8", "moe_pack_mxfp4", "moe_pack_mxfp8", "moe_status_string",
           "MOE_WEIGHTS_BF16", "MOE_WEIGHTS_MXFP4", "MOE_WEIGHTS_MXFP8", "MOE_WEIGHTS_MXFP4_TILED",
           "MOE_WEIGHTS_MXFP8_TILED",
           "MOE_ACT_BF16", "MOE_ACT_MXFP8",
           "MOE_DTYPE_BF16", "MOE_DTYPE_FP32", "MOE_STATE_FP32", "MOE_STATE_8BIT",
           "moe_grouped_gemm", "moe_grouped_gemm_dgrad", "moe_grouped_gemm_wgrad", "moe_swiglu", "moe_swiglu_backward",
           "MoEAdamWPlan", "moe_adamw_step", "moe_adamw_dequantise",
           "EXPORTED_SYMBOLS"]

MOE_WEIGHTS_BF16 = 0
MOE_WEIGHTS_MXFP4 = 1
MOE_WEIGHTS_MXFP8 = 2
MOE_WEIGHTS_MXFP4_TILED = 3
MOE_WEIGHTS_MXFP8_TILED = 4
MOE_ACT_BF16 = 0
MOE_ACT_MXFP8 = 1
MOE_DTYPE_BF16 = 0
MOE_DTYPE_FP32 = 1
MOE_STATE_FP32 = 0
MOE_STATE_8BIT = 1

EXPORTED_SYMBOLS = ("moe_workspace_size", "moe_route", "moe_dispatch", "moe_expert_ffn", "moe_combine",
                    "moe_forward", "moe_forward_traced", "moe_forward_timed", "moe_update_expert_bias",
                    "moe_dense_ffn_workspace_size", "moe_dense_ffn", "moe_forward_noalloc", "moe_quantise_mxfp8",
                    "moe_pack_mxfp4", "moe_pack_mxfp8", "moe_grouped_gemm", "moe_grouped_gemm_dgrad",
                    "moe_grouped_gemm_wgrad", "moe_swiglu", "moe_swiglu_backward", "moe_adamw_plan", "moe_adamw_step",
                    "moe_adamw_dequantise", "moe_status_string", "moe_last_error")

_HERE = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_HERE, "libmoe.so")


class MoEConfig(ctypes.Structure):
    """moe_config_t; field names follow the model's text_config."""
    _fields_ = [("hidden_size", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("num_experts_per_tok", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("moe_intermediate_size", ctypes.c_int32),
                ("num_shared_experts", ctypes.c_int32), ("shared_intermediate_size", ctypes.c_int32),
                ("norm_topk_prob", ctypes.c_int32), ("routed_scaling_factor", ctypes.c_float),
                ("swiglu_limit", ctypes.c_float), ("shared_swiglu_limit", ctypes.c_float),
                ("expert_weight_format", ctypes.c_int32), ("expert_act_format", ctypes.c_int32)]


class _Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("gate", "up", "down", "gate_scale", "up_scale", "down_scale",
                                                "shared_gate", "shared_up", "shared_down")]


class _Groups(ctypes.Structure):
    _fields_ = [("groups", ctypes.c_int32), ("out_features", ctypes.c_int32), ("in_features", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("offsets", ctypes.c_void_p)]


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_int64), ("ld", ctypes.c_int64), ("row_map", ctypes.c_void_p)]


class _AdamWTensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "master", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale",
                                                "exp_avg_sq_scale")] + [
        ("numel", ctypes.c_int64), ("weight_decay", ctypes.c_float), ("reserved", ctypes.c_int32)]


class _AdamWPlan(ctypes.Structure):
    _fields_ = [("n_tensors", ctypes.c_int64), ("n_chunks", ctypes.c_int64), ("flags", ctypes.c_uint64),
                ("image_bytes", ctypes.c_size_t)]


class _AdamWConfig(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("step", ctypes.c_int64), ("seed", ctypes.c_uint32), ("lr_ptr", ctypes.c_void_p),
                ("step_ptr", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p)]


class MoEExpertWeights:
    """moe_expert_weights_t built from device tensors (references are kept alive here)."""

    def __init__(self, gate, up, down, gate_scale=None, up_scale=None, down_scale=None,
                 shared_gate=None, shared_up=None, shared_down=None):
        self._keep = (gate, up, down, gate_scale, up_scale, down_scale, shared_gate, shared_up, shared_down)
        self.struct = _Weights(*[_ptr(t) for t in self._keep])


class MoEError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{moe_status_string(status)}: {message}")
        self.status = status


_lib = None


def load_library():
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run: python -m sparse_moe_layer_bailingmoev3_amd.build")
    lib = ctypes.CDLL(path)
    P, I64, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    C = ctypes.POINTER(MoEConfig)
    W = ctypes.POINTER(_Weights)
    I32, GR, RW = ctypes.c_int32, ctypes.POINTER(_Groups), ctypes.POINTER(_Rows)
    sigs = {
        "moe_workspace_size": [C, I64, ctypes.POINTER(SZ)],
        "moe_route": [C, I64, P, P, P, P, P, P, SZ, P],
        "moe_dispatch": [C, I64, P, P, P, P, P, P, SZ, P],
        "moe_expert_ffn": [C, I64, P, P, P, W, P, P, SZ, P],
        "moe_combine": [C, I64, P, P, P, P, P],
        "moe_forward": [C, I64, P, P, P, W, P, P, P, P, P, SZ, P],
        "moe_forward_traced": [C, I64, P, P, P, W, P, P, SZ, P, ctypes.POINTER(P), ctypes.c_int32,
                               ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_int32)],
        "moe_forward_timed": [C, I64, P, P, P, W, P, P, SZ, P, ctypes.c_int32, P, P],
        "moe_update_expert_bias": [C, P, P, ctypes.c_float, P],
        "moe_dense_ffn_workspace_size": [ctypes.c_int32, ctypes.c_int32, I64, ctypes.POINTER(SZ)],
        "moe_dense_ffn": [ctypes.c_int32, ctypes.c_int32, ctypes.c_float, I64, P, P, P, P, P, P, SZ, P],
        "moe_forward_noalloc": [C, I64, P, P, P, W, P, P, P, P, P],
        "moe_quantise_mxfp8": [P, I64, ctypes.c_int32, P, P, P],
        "moe_pack_mxfp4": [P, P, I64, ctypes.c_int32, ctypes.c_int32, P, P, P],
        "moe_pack_mxfp8": [P, P, I64, ctypes.c_int32, ctypes.c_int32, P, P, P],
        "moe_grouped_gemm": [GR, RW, P, P, I64, I32, I32, P],
        "moe_grouped_gemm_dgrad": [GR, RW, P, RW, P, P, I64, I32, I32, P],
        "moe_grouped_gemm_wgrad": [GR, RW, RW, P, I32, I32, P],
        "moe_swiglu": [I64, I64, I32, ctypes.c_float, P, P, I64, P, P, P, I64, P],
        "moe_swiglu_backward": [I64, I64, I32, ctypes.c_float, P, P, I64, P, I64, P, P, P, P, I64, P, P],
        "moe_adamw_plan": [I64, P, I32, I32, I32, ctypes.POINTER(_AdamWPlan), P, SZ],
        "moe_adamw_step": [ctypes.POINTER(_AdamWConfig), ctypes.POINTER(_AdamWPlan), P, P],
        "moe_adamw_dequantise": [P, P, I64, I32, P, P],
    }
    for name, args in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.moe_status_string.argtypes = [ctypes.c_int]
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_last_error.argtypes = []
    lib.moe_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def moe_status_string(status: int) -> str:
    return load_library().moe_status_string(status).decode()


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int):
    if status != 0:
        raise MoEError(status, load_library().moe_last_error().decode())


def _ws(ws):
    if ws is None:
        return None, 0
    return ws.data_ptr(), ws.numel() * ws.element_size()


def moe_workspace_size(cfg: MoEConfig, T: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().moe_workspace_size(ctypes.byref(cfg), T, ctypes.byref(n)))
    return n.value


def moe_route(cfg, T, x, router_w, expert_bias, topk_idx, topk_w, ws, stream=None):
    p, n = _ws(ws)
    _check(load_library().moe_route(ctypes.byref(cfg), T, _ptr(x), _ptr(router_w), _ptr(expert_bias),
                                    _ptr(topk_idx), _ptr(topk_w), p, n, _stream(stream)))


def moe_dispatch(cfg, T, topk_idx, expert_counts, expert_offsets, sorted_token, inv_perm, ws, stream=None):
    p, n = _ws(ws)
    _check(load_library().moe_dispatch(ctypes.byref(cfg), T, _ptr(topk_idx), _ptr(expert_counts),
                                       _ptr(expert_offsets), _ptr(sorted_token), _ptr(inv_perm), p, n,
                                       _stream(stream)))


def moe_expert_ffn(cfg, T, x, expert_offsets, sorted_token, weights: MoEExpertWeights, y_sorted, ws, stream=None):
    p, n = _ws(ws)
    _check(load_library().moe_expert_ffn(ctypes.byref(cfg), T, _ptr(x), _ptr(expert_offsets), _ptr(sorted_token),
                                         ctypes.byref(weights.struct), _ptr(y_sorted), p, n, _stream(stream)))


def moe_combine(cfg, T, y_sorted, inv_perm, topk_w, out, stream=None):
    _check(load_library().moe_combine(ctypes.byref(cfg), T, _ptr(y_sorted), _ptr(inv_perm), _ptr(topk_w),
                                      _ptr(out), _stream(stream)))


def moe_forward(cfg, T, x, router_w, expert_bias, weights: MoEExpertWeights, out, topk_idx_out=None,
                topk_w_out=None, expert_counts_out=None, ws=None, stream=None):
    p, n = _ws(ws)
    _check(load_library().moe_forward(ctypes.byref(cfg), T, _ptr(x), _ptr(router_w), _ptr(expert_bias),
                                      ctypes.byref(weights.struct), _ptr(out), _ptr(topk_idx_out),
                                      _ptr(topk_w_out), _ptr(expert_counts_out), p, n, _stream(stream)))


def moe_forward_traced(cfg, T, x, router_w, expert_bias, weights: MoEExpertWeights, out, ws, events, stream=None):
    """moe_forward recording events[0] before and events[i+1] after the i-th kernel.  `events`
    are raw hipEvent_t handles (ints).  Returns the list of kernel names in launch order."""
    p, n = _ws(ws)
    ev = (ctypes.c_void_p * len(events))(*events)
    names = (ctypes.c_char_p * max(1, len(events) - 1))()
    nk = ctypes.c_int32()
    _check(load_library().moe_forward_traced(ctypes.byref(cfg), T, _ptr(x), _ptr(router_w), _ptr(expert_bias),
                                             ctypes.byref(weights.struct), _ptr(out), p, n, _stream(stream), ev,
                                             len(events), names, ctypes.byref(nk)))
    return [names[i].decode() for i in range(nk.value)]


def moe_forward_timed(cfg, T, x, router_w, expert_bias, weights: MoEExpertWeights, out, ws, kernel_index,
                      start_event, stop_event, stream=None):
    """moe_forward with kernel `kernel_index` (its position in moe_forward_traced's list) timed
    by two raw hipEvent_t handles bound to its dispatch; adds nothing else to the queue."""
    p, n = _ws(ws)
    _check(load_library().moe_forward_timed(ctypes.byref(cfg), T, _ptr(x), _ptr(router_w), _ptr(expert_bias),
                                            ctypes.byref(weights.struct), _ptr(out), p, n, _stream(stream),
                                            kernel_index, start_event, stop_event))


def moe_update_expert_bias(cfg, expert_counts, expert_bias, gamma, stream=None):
    """In-place sign-rule update of the routed experts' selection bias from a step's counts."""
    _check(load_library().moe_update_expert_bias(ctypes.byref(cfg), _ptr(expert_counts), _ptr(expert_bias),
                                                 float(gamma), _stream(stream)))


def moe_dense_ffn_workspace_size(hidden_size, intermediate_size, T) -> int:
    n = ctypes.c_size_t()
    _check(load_library().moe_dense_ffn_workspace_size(hidden_size, intermediate_size, T, ctypes.byref(n)))
    return n.value


def moe_dense_ffn(hidden_size, intermediate_size, swiglu_limit, T, x, gate, up, down, out, ws, stream=None):
    """Dense SwiGLU FFN out = (silu(x gate^T) * (x up^T)) down^T (bf16 in and out)."""
    p, n = _ws(ws)
    _check(load_library().moe_dense_ffn(hidden_size, intermediate_size, float(swiglu_limit), T, _ptr(x), _ptr(gate),
                                        _ptr(up), _ptr(down), _ptr(out), p, n, _stream(stream)))


def moe_forward_noalloc(cfg, T, x, router_w, expert_bias, weights: MoEExpertWeights, out, topk_idx_out=None,
                        topk_w_out=None, expert_counts_out=None, stream=None):
    """moe_forward on the library's static 64 MiB device scratch instead of a caller workspace
    (for callers that cannot allocate); rejects T whose workspace does not fit."""
    _check(load_library().moe_forward_noalloc(ctypes.byref(cfg), T, _ptr(x), _ptr(router_w), _ptr(expert_bias),
                                              ctypes.byref(weights.struct), _ptr(out), _ptr(topk_idx_out),
                                              _ptr(topk_w_out), _ptr(expert_counts_out), _stream(stream)))


def moe_pack_mxfp4(codes, scales, mats, N, Kd, codes_out, scales_out, stream=None):
    """Row-major MXFP4 codes [mats, N, Kd/2] and scales [mats, N, Kd/32] -> the tiled order of
    MOE_WEIGHTS_MXFP4_TILED (same sizes)."""
    _check(load_library().moe_pack_mxfp4(_ptr(codes), _ptr(scales), mats, N, Kd, _ptr(codes_out), _ptr(scales_out),
                                         _stream(stream)))


def moe_pack_mxfp8(codes, scales, mats, N, Kd, codes_out, scales_out, stream=None):
    """Row-major MXFP8 codes [mats, N, Kd] and scales [mats, N, Kd/32] -> the tiled order of
    MOE_WEIGHTS_MXFP8_TILED (same sizes)."""
    _check(load_library().moe_pack_mxfp8(_ptr(codes), _ptr(scales), mats, N, Kd, _ptr(codes_out), _ptr(scales_out),
                                         _stream(stream)))


def moe_quantise_mxfp8(x, rows, cols, codes, scales, stream=None):
    """bf16 [rows, cols] -> MXFP8 E4M3 codes [rows, cols] and e8m0 scales [rows, cols/32] (the
    rounding the MXFP8-activation path applies to x)."""
    _check(load_library().moe_quantise_mxfp8(_ptr(x), rows, cols, _ptr(codes), _ptr(scales), _stream(stream)))


# ---- training the experts ------------------------------------------------------------------------
# These take their sizes from the tensors, so what a wrong tensor would make a kernel read is found
# here: types, shapes, unit strides, one device.  A refused argument raises MoEError like one that
# the library refuses.

_ERR_INVALID, _ERR_UNSUPPORTED = -1, -2


def _refuse(message, status=_ERR_INVALID):
    raise MoEError(status, message)


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _enqueue(fn, dev, stream, *args):
    """fn(*args, stream) with device `dev`, which holds the tensors, current; its current stream
    unless one is given (which must belong to it)."""
    if dev < 0:
        _refuse("tensors must lie on a GPU")
    torch = _torch()
    if stream is not None:
        given = getattr(stream, "device", None)
        if given is not None and given.index != dev:
            _refuse(f"stream belongs to {given}, tensors lie on cuda:{dev}")
        stream = _stream(stream)
    else:
        stream = _raw_stream(dev)
    if torch.cuda.current_device() == dev:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        _check(status)


def _raw_stream(dev):
    """Handle of the device's current stream."""
    torch = _torch()
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(dev) if get is not None else torch.cuda.current_stream(dev).cuda_stream


def _device_of(t, name):
    """Index of the GPU that holds t (-1: none; refused once everything else is in order)."""
    if not isinstance(t, _torch().Tensor):
        _refuse(f"{name} must be a tensor")
    return t.get_device()


def _explain(t, name, dtype, dim, dev):
    """Refuses t: why it is not a tensor of that type and dimension on that device."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        _refuse(f"{name} must be a tensor")
    if dtype is not None and t.dtype is not dtype:
        _refuse(f"{name} must be {dtype}, not {t.dtype}")
    if t.dim() != dim:
        _refuse(f"{name} must have {dim} dimension(s), not {t.dim()}")
    _refuse(f"{name} lies on {t.device}, the others on {f'cuda:{dev}' if dev >= 0 else 'the CPU'}")


def _matrix(t, name, dtype, dev):
    """(rows, columns, row stride) of a matrix whose columns lie side by side."""
    try:
        wrong = dtype is not None and t.dtype is not dtype or t.dim() != 2 or t.get_device() != dev
    except AttributeError:  # no tensor
        wrong = True
    if wrong:
        _explain(t, name, dtype, 2, dev)
    rows, cols = t.shape
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        _refuse(f"{name}: the values of a row must lie side by side")
    return rows, cols, ld if rows > 1 else (cols + 7) // 8 * 8


def _vector(t, name, dtype, n, dev):
    try:
        wrong = t.dtype is not dtype or t.dim() != 1 or t.get_device() != dev
    except AttributeError:  # no tensor
        wrong = True
    if wrong:
        _explain(t, name, dtype, 1, dev)
    size = t.shape[0]
    if n is not None and size != n:
        _refuse(f"{name} has {size} entries, {n} needed")
    if size > 1 and t.stride(0) != 1:
        _refuse(f"{name} must be contiguous")
    return size


def _weights3(t, name, dtype, dev):
    try:
        wrong = dtype is not None and t.dtype is not dtype or t.dim() != 3 or t.get_device() != dev
    except AttributeError:  # no tensor
        wrong = True
    if wrong:
        _explain(t, name, dtype, 3, dev)
    if not t.is_contiguous():
        _refuse(f"{name} must be contiguous")
    return t.shape


def _dtype_code(t, name):
    torch = _torch()
    if t.dtype is torch.bfloat16:
        return MOE_DTYPE_BF16
    if t.dtype is not torch.float32:
        _refuse(f"{name} must be bfloat16 or float32, not {t.dtype}", _ERR_UNSUPPORTED)
    return MOE_DTYPE_FP32


def _operand(t, name, cols, row_map, positions, dev):
    torch = _torch()
    rows, c, ld = _matrix(t, name, torch.bfloat16, dev)
    if c != cols:
        _refuse(f"{name} has {c} columns, {cols} needed")
    at = None
    if row_map is not None:
        _vector(row_map, f"the row map of {name}", torch.int32, positions, dev)
        at = row_map.data_ptr()
    return _Rows(t.data_ptr() if rows else None, rows, ld, at)


def _positions(t, row_map, name, dev):
    """Positions that an operand covers: the entries of its row map, or its rows."""
    t, name, dim = (t, name, 2) if row_map is None else (row_map, f"the row map of {name}", 1)
    if not isinstance(t, _torch().Tensor) or t.dim() != dim:
        _explain(t, name, None, dim, dev)
    return t.shape[0]


def moe_grouped_gemm(x, w, offsets, y, row_map=None, accumulate=False, stream=None):
    """y[p] = w[g] x[row_map[p]] for the positions offsets[g] <= p < offsets[g+1] of every group g:
    x bf16 [.., in], w bf16 [G, out, in], offsets int32 [G+1], y bf16 or fp32 [P, out] (added to
    with accumulate, fp32 only), row_map int32 [P] (None: position p is row p)."""
    torch, dev = _torch(), _device_of(w, "w")
    G, N, K = _weights3(w, "w", torch.bfloat16, dev)
    P, cols, ldy = _matrix(y, "y", None, dev)
    if cols != N:
        _refuse(f"y has {cols} columns, w makes {N}")
    _vector(offsets, "offsets", torch.int32, G + 1, dev)
    _enqueue(load_library().moe_grouped_gemm, dev, stream, _Groups(G, N, K, P, offsets.data_ptr()),
             _operand(x, "x", K, row_map, P, dev), w.data_ptr(), y.data_ptr(), ldy, _dtype_code(y, "y"), 1 if accumulate else 0)


def moe_grouped_gemm_dgrad(dy, w, offsets, dx, row_map=None, dy2=None, w2=None, accumulate=False, stream=None):
    """dx[p] = dy[row_map[p]] w[g] (+ dy2[row_map[p]] w2[g]): dy bf16 [.., out], w bf16 [G, out, in],
    dx bf16 or fp32 [P, in]; dy2 has dy's rows and row stride."""
    torch, dev = _torch(), _device_of(w, "w")
    G, N, K = shape = _weights3(w, "w", torch.bfloat16, dev)
    P, cols, lddx = _matrix(dx, "dx", None, dev)
    if cols != K:
        _refuse(f"dx has {cols} columns, w makes {K}")
    if (dy2 is None) != (w2 is None):
        _refuse("dy2 and w2 must be given together")
    _vector(offsets, "offsets", torch.int32, G + 1, dev)
    b, pw2 = None, None
    if w2 is not None:
        if _weights3(w2, "w2", torch.bfloat16, dev) != shape:
            _refuse(f"w2 is {tuple(w2.shape)}, w is {tuple(shape)}")
        b, pw2 = _operand(dy2, "dy2", N, row_map, P, dev), w2.data_ptr()
    _enqueue(load_library().moe_grouped_gemm_dgrad, dev, stream, _Groups(G, N, K, P, offsets.data_ptr()),
             _operand(dy, "dy", N, row_map, P, dev), w.data_ptr(), b, pw2, dx.data_ptr(), lddx, _dtype_code(dx, "dx"),
             1 if accumulate else 0)


def moe_grouped_gemm_wgrad(dy, x, offsets, dw, dy_map=None, x_map=None, accumulate=False, stream=None):
    """dw[g] = sum over group g's positions of dy[dy_map[p]]^T x[x_map[p]]: dy bf16 [.., out], x bf16
    [.., in], dw bf16 or fp32 [G, out, in] (added to with accumulate, fp32 only)."""
    torch, dev = _torch(), _device_of(dw, "dw")
    G, N, K = _weights3(dw, "dw", None, dev)
    P, px = _positions(dy, dy_map, "dy", dev), _positions(x, x_map, "x", dev)
    if P != px:
        _refuse(f"dy and x cover different numbers of positions: {P} and {px}")
    _vector(offsets, "offsets", torch.int32, G + 1, dev)
    _enqueue(load_library().moe_grouped_gemm_wgrad, dev, stream, _Groups(G, N, K, P, offsets.data_ptr()),
             _operand(dy, "dy", N, dy_map, P, dev), _operand(x, "x", K, x_map, P, dev), dw.data_ptr(), _dtype_code(dw, "dw"),
             1 if accumulate else 0)


def _like(first, t, name, dev):
    """Row stride of a bf16 matrix with the rows and columns of gate (`first`)."""
    rows, cols, ld = _matrix(t, name, _torch().bfloat16, dev)
    if rows != first[0] or cols != first[1]:
        _refuse(f"{name} is [{rows}, {cols}], gate is [{first[0]}, {first[1]}]")
    return ld


def _pairs(row_w, pos, rows, dev):
    """Rows handled (those of the positions or weights given, else all), the two addresses."""
    torch = _torch()
    n, pw, pp = None, None, None
    if pos is not None:
        n, pp = _vector(pos, "pos", torch.int32, None, dev), pos.data_ptr()
    if row_w is not None:
        n, pw = _vector(row_w, "row_w", torch.float32, n, dev), row_w.data_ptr()
    return rows if n is None else n, pw, pp


def moe_swiglu(gate, up, h, limit=0.0, row_w=None, pos=None, stream=None):
    """h[pos[i]] = row_w[i] * clamp(silu(gate[pos[i]]) * up[pos[i]], -limit, limit): gate, up, h bf16
    [R, C]; row_w fp32 [n] (None: 1), pos int32 [n], distinct (None: row i), entries outside [0, R)
    skipped; limit <= 0: no clamp."""
    dev = _device_of(gate, "gate")
    R, C, ld = first = _matrix(gate, "gate", _torch().bfloat16, dev)
    if _like(first, up, "up", dev) != ld:
        _refuse("gate and up must have the same row stride")
    ldh, (n, pw, pp) = _like(first, h, "h", dev), _pairs(row_w, pos, R, dev)
    _enqueue(load_library().moe_swiglu, dev, stream, n, R, C, float(limit), gate.data_ptr(), up.data_ptr(), ld, pw, pp, h.data_ptr(), ldh)


def moe_swiglu_backward(gate, up, dh, dgate, dup, limit=0.0, row_w=None, pos=None, drow_w=None, stream=None):
    """Gradients of moe_swiglu from dh: dgate, dup bf16 [R, C], drow_w fp32 [n] (None: not wanted)."""
    torch, dev = _torch(), _device_of(gate, "gate")
    R, C, ld = first = _matrix(gate, "gate", torch.bfloat16, dev)
    if _like(first, up, "up", dev) != ld:
        _refuse("gate and up must have the same row stride")
    lddh, ldd = _like(first, dh, "dh", dev), _like(first, dgate, "dgate", dev)
    if _like(first, dup, "dup", dev) != ldd:
        _refuse("dgate and dup must have the same row stride")
    (n, pw, pp), pd = _pairs(row_w, pos, R, dev), None
    if drow_w is not None:
        _vector(drow_w, "drow_w", torch.float32, n, dev)
        pd = drow_w.data_ptr()
    _enqueue(load_library().moe_swiglu_backward, dev, stream, n, R, C, float(limit), gate.data_ptr(), up.data_ptr(), ld, dh.data_ptr(),
             lddh, pw, pp, dgate.data_ptr(), dup.data_ptr(), ldd, pd)


class MoEAdamWPlan:
    """The table of an AdamW step over many tensors (moe_adamw_plan): built once, kept with its
    tensors, which must stay where they are.  All arguments are equally long lists of contiguous
    tensors on one device: params and grads bf16 or fp32 (one type each), exp_avg and exp_avg_sq
    fp32, or uint8 codes with their fp32 scales ([ceil(numel / 128)]), master fp32 copies of bf16
    params; weight_decay a number or one for each tensor."""

    def __init__(self, params, grads, exp_avg, exp_avg_sq, master=None, exp_avg_scale=None, exp_avg_sq_scale=None,
                 weight_decay=0.0):
        torch = _torch()
        cols = {}
        for name, ts, must in (("params", params, True), ("grads", grads, True), ("exp_avg", exp_avg, True),
                               ("exp_avg_sq", exp_avg_sq, True), ("master", master, False),
                               ("exp_avg_scale", exp_avg_scale, False), ("exp_avg_sq_scale", exp_avg_sq_scale, False)):
            if must or ts is not None:
                try:
                    cols[name] = list(ts)
                except TypeError:
                    _refuse(f"{name} must be a list of tensors")
        n = len(cols["params"])
        if n == 0:
            _refuse("params must not be empty")
        for name, ts in cols.items():
            for i, t in enumerate(ts):
                if not isinstance(t, torch.Tensor):
                    _refuse(f"{name}[{i}] must be a tensor")
        eight = len(cols["exp_avg"]) > 0 and cols["exp_avg"][0].dtype == torch.uint8
        if (exp_avg_scale is not None) != eight or (exp_avg_sq_scale is not None) != eight:
            _refuse("scales belong to uint8 states, and both must be given")
        state = torch.uint8 if eight else torch.float32
        types = {"params": cols["params"][0].dtype, "grads": cols["grads"][0].dtype if cols["grads"] else None,
                 "exp_avg": state, "exp_avg_sq": state, "master": torch.float32, "exp_avg_scale": torch.float32,
                 "exp_avg_sq_scale": torch.float32}
        sizes = [t.numel() for t in cols["params"]]
        blocks = [-(-k // 128) for k in sizes]
        for name, ts in cols.items():
            if len(ts) != n:
                _refuse(f"{name} has {len(ts)} tensors, params {n}")
            dtype, wanted = types[name], blocks if name.endswith("scale") else sizes
            for i, (t, want) in enumerate(zip(ts, wanted)):
                if t.dtype is not dtype:
                    _refuse(f"{name}[{i}] must be {dtype}, not {t.dtype}")
                if not t.is_contiguous():
                    _refuse(f"{name}[{i}] must be contiguous")
                if t.numel() != want:
                    _refuse(f"{name}[{i}] has {t.numel()} values, {want} needed")
        one = isinstance(weight_decay, torch.Tensor) and weight_decay.dim() == 0 or not hasattr(weight_decay, "__len__")
        try:
            decay = [float(weight_decay)] * n if one else [float(d) for d in weight_decay]
        except (TypeError, ValueError):
            _refuse("weight_decay must be a number or one for each tensor")
        if len(decay) != n:
            _refuse(f"weight_decay has {len(decay)} entries, params {n}")
        device, dev = cols["params"][0].device, cols["params"][0].get_device()
        for name, ts in cols.items():
            for i, t in enumerate(ts):
                if t.get_device() != dev or dev < 0:
                    _refuse(f"{name}[{i}] lies on {t.device}; one GPU must hold them all")
        self._keep, self.device = cols, device
        none = [None] * n
        at = {name: [t.data_ptr() or None for t in ts] for name, ts in cols.items()}
        table = (_AdamWTensor * n)(*zip(at["params"], at.get("master", none), at["grads"], at["exp_avg"], at["exp_avg_sq"],
                                        at.get("exp_avg_scale", none), at.get("exp_avg_sq_scale", none), sizes, decay))
        self.struct = _AdamWPlan()
        args = (n, ctypes.byref(table), _dtype_code(cols["params"][0], "params"), _dtype_code(cols["grads"][0], "grads"),
                MOE_STATE_8BIT if eight else MOE_STATE_FP32, ctypes.byref(self.struct))
        lib = load_library()
        _check(lib.moe_adamw_plan(*args, None, 0))
        host = torch.empty(self.struct.image_bytes, dtype=torch.uint8)
        _check(lib.moe_adamw_plan(*args, host.data_ptr(), host.numel()))
        self.image = host.to(device)
        self.at, self.home = self.image.data_ptr(), _raw_stream(dev)

    def _used_on(self, stream):
        """The table is the plan's own: its memory stays until the work on `stream` (None: the device's
        current one) is done, also where the plan goes before that."""
        raw = _raw_stream(self.device.index) if stream is None else _stream(stream)
        if raw != self.home:
            cuda = _torch().cuda
            self.image.record_stream(cuda.ExternalStream(raw, device=self.device) if raw else cuda.default_stream(self.device))


def moe_adamw_step(plan: MoEAdamWPlan, lr, step, betas=(0.9, 0.999), eps=1e-8, seed=0, grad_scale=None, stream=None):
    """One AdamW step over the plan's tensors, in place.  lr and step (1 for the first) are numbers,
    or device tensors (fp32, int64) read when the step runs (which writes nothing if it then finds a
    step below 1); grad_scale an fp32 device tensor that
    multiplies every gradient; seed that of the 8-bit states' stochastic rounding."""
    if not isinstance(plan, MoEAdamWPlan):
        _refuse("plan must be a MoEAdamWPlan")
    Tensor, dev = _torch().Tensor, plan.device.index
    lr_at = step_at = scale_at = None
    if isinstance(lr, Tensor):
        lr, lr_at = 0.0, _scalar_at(lr, "lr", _torch().float32, dev)
    if isinstance(step, Tensor):
        step, step_at = 0, _scalar_at(step, "step", _torch().int64, dev)
    if grad_scale is not None:
        scale_at = _scalar_at(grad_scale, "grad_scale", _torch().float32, dev)
    _enqueue(load_library().moe_adamw_step, dev, stream,
             _AdamWConfig(lr, betas[0], betas[1], eps, step, seed & 0xFFFFFFFF, lr_at, step_at, scale_at), plan.struct, plan.at)
    plan._used_on(stream)


def _scalar_at(t, name, dtype, dev):
    """Address of a device tensor that holds one value."""
    if not isinstance(t, _torch().Tensor) or t.dtype is not dtype or t.numel() != 1 or t.get_device() != dev:
        _refuse(f"{name} must hold one {dtype} value on cuda:{dev}")
    return t.data_ptr()


def moe_adamw_dequantise(codes, scales, out, signed, stream=None):
    """Values of an 8-bit state array: codes uint8 [n], scales fp32 [ceil(n / 128)] -> out fp32 [n];
    signed: exp_avg's codes, else exp_avg_sq's."""
    torch, dev = _torch(), _device_of(codes, "codes")
    n = _vector(codes, "codes", torch.uint8, None, dev)
    _vector(scales, "scales", torch.float32, -(-n // 128), dev)
    _vector(out, "out", torch.float32, n, dev)
    _enqueue(load_library().moe_adamw_dequantise, dev, stream, codes.data_ptr(), scales.data_ptr(), n, 1 if signed else 0,
             out.data_ptr())
