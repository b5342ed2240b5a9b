"""ctypes binding of libmoe.so: the five layer calls plus helpers, same names as the C ABI.

Argument marshalling only.  Tensor arguments are torch tensors on the GPU (or
raw integer device addresses, or None for NULL); the stream defaults to torch's
current stream.  Every call raises MoeError on a non-zero status.  There is no
fallback: if libmoe.so is missing the import of the library raises.
"""
from __future__ import annotations

import ctypes
import os
import re

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "moe.h")

MOE_OK, MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_LAUNCH = 0, -1, -2, -3, -4, -5
MOE_ERR_SCRATCH = -6
MOE_F32, MOE_BF16, MOE_FP8_E4M3, MOE_MXFP4, MOE_INT8 = 0, 1, 2, 3, 4
MOE_SCORES_IN, MOE_SOFTMAX, MOE_GATES_RAW = 1, 2, 4
MOE_FFN_ALL, MOE_FFN_GATE_UP, MOE_FFN_DOWN = 0, 1, 2
MOE_WS_DISPATCH, MOE_WS_FFN, MOE_WS_FFN_BWD, MOE_WS_ROUTE_BWD, MOE_WS_ROUTE = 1, 2, 3, 4, 5
MOE_WS_NORM_BWD, MOE_WS_ROUTE_BWD_SOFTMAX = 6, 7
MOE_WSP_H, MOE_WSP_H_SCALE, MOE_WSP_H_SHARED, MOE_WSP_H_SHARED_SCALE = 0, 1, 2, 3
_DTYPES = {"f32": MOE_F32, "bf16": MOE_BF16, "fp8_e4m3": MOE_FP8_E4M3, "mxfp4": MOE_MXFP4, "int8": MOE_INT8}


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status} ({status_string(status)})")
        self.status = status


class MoeCfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "E", "G", "M", "k", "S", "I", "group_topr")] + [
        ("route_scale", ctypes.c_float), ("act", ctypes.c_int32), ("wgt", ctypes.c_int32),
        ("bias_eq_mode", ctypes.c_int32)]


class MoeExpertWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "w_gate_up", "w_down", "w_gate_up_scale", "w_down_scale",
        "ws_gate_up", "ws_down", "ws_gate_up_scale", "ws_down_scale")]


class MoeExpertGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w_gate_up", "w_down", "ws_gate_up", "ws_down")]


class MoeFfnSaved(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("g", "u", "gs", "us")]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmoe.so (built by biased_top_routing_amd.build); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run python -m biased_top_routing_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, u32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_float, ctypes.c_size_t
        cfgp = ctypes.POINTER(MoeCfg)
        sig = {
            "moe_route": [cfgp, vp, vp, vp, vp, vp, u32, vp, vp, vp, sz, vp],
            "moe_dispatch": [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_dispatch_noalloc": [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp],
            "moe_expert_ffn": [cfgp, vp, vp, vp, ctypes.POINTER(MoeExpertWeights), vp, vp, vp, vp, sz,
                               ctypes.c_int, vp],
            "moe_expert_ffn_gather": [cfgp, vp, vp, vp, ctypes.POINTER(MoeExpertWeights), vp, vp, vp, sz,
                                      ctypes.c_int, vp],
            "moe_expert_ffn_save": [cfgp, vp, vp, vp, ctypes.POINTER(MoeExpertWeights), vp, vp, vp,
                                    ctypes.POINTER(MoeFfnSaved), vp, sz, ctypes.c_int, vp],
            "moe_combine": [cfgp, vp, vp, vp, vp, vp, vp],
            "moe_combine_backward": [cfgp, vp, vp, vp, vp, vp, vp, vp],
            "moe_expert_ffn_backward": [cfgp, vp, vp, vp, ctypes.POINTER(MoeExpertWeights), vp, vp, vp, vp,
                                        ctypes.POINTER(MoeExpertGrads), vp, sz, vp],
            "moe_expert_ffn_backward_saved": [cfgp, vp, vp, vp, ctypes.POINTER(MoeExpertWeights),
                                              ctypes.POINTER(MoeFfnSaved), vp, vp, vp, vp,
                                              ctypes.POINTER(MoeExpertGrads), vp, sz, vp],
            "moe_route_backward": [cfgp, vp, vp, vp, vp, vp, f32, i32, vp, vp, vp, vp, sz, vp],
            "moe_dispatch_backward": [cfgp, vp, vp, vp, vp, vp, vp],
            "moe_update_bias": [cfgp, vp, vp, f32, vp],
            "moe_quantize_fp8": [vp, i32, i32, i32, i32, vp, vp, vp],
            "moe_dispatch_local": [cfgp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_combine_local": [cfgp, vp, vp, vp, vp, vp, vp],
            "moe_combine_local_backward": [cfgp, vp, vp, vp, vp, vp, vp, vp],
            "moe_dispatch_local_backward": [cfgp, vp, vp, vp, vp, vp, vp],
            "moe_expert_ffn_codes": [cfgp, vp, vp, vp, vp, ctypes.POINTER(MoeExpertWeights), vp, vp, vp, sz,
                                     ctypes.c_int, vp],
            "moe_quantize_int8": [vp, i32, i32, i32, i32, vp, vp, vp],
            "moe_norm": [cfgp, vp, vp, vp, vp, f32, vp, vp, vp, vp, vp],
            "moe_norm_backward": [cfgp, vp, vp, vp, f32, vp, vp, vp, vp, vp, sz, vp],
            "moe_route_backward_flags": [cfgp, u32, vp, vp, vp, vp, vp, f32, i32, vp, vp, vp, vp, sz, vp],
            "moe_quantize_fp4": [vp, i32, i32, i32, vp, vp, vp],
            "moe_dequantize_fp4": [vp, vp, i32, i32, i32, vp, vp],
            "moe_ffn_workspace_part": [cfgp, ctypes.c_int, ctypes.POINTER(sz), ctypes.POINTER(sz)],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.moe_workspace_bytes.argtypes = [cfgp, ctypes.c_int]
        L.moe_workspace_bytes.restype = sz
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_abi_version.argtypes = []
        L.moe_abi_version.restype = ctypes.c_int
        _lib = L
    return _lib


def header_functions() -> list:
    """Names of the functions include/moe.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:moe_status|size_t|const char\*|int)\s+(moe_\w+)\s*\(", text, re.M)))


def make_cfg(T, H, E, G, M, k, S, I, group_topr=2, route_scale=1.0, act="bf16", wgt="bf16",
             bias_eq_mode=0) -> MoeCfg:
    a = _DTYPES[act] if isinstance(act, str) else act
    w = _DTYPES[wgt] if isinstance(wgt, str) else wgt
    return MoeCfg(T, H, E, G, M, k, S, I, group_topr, route_scale, a, w, bias_eq_mode)


def cfg_from(c, **over) -> MoeCfg:
    """MoeCfg from any object with the layer attributes (T H E G M k S I group_topr
    route_scale act wgt bias_eq_mode)."""
    d = {n: getattr(c, n) for n in ("T", "H", "E", "G", "M", "k", "S", "I", "group_topr", "route_scale",
                                     "act", "wgt")}
    d["bias_eq_mode"] = getattr(c, "bias_eq_mode", 0)
    d.update(over)
    return make_cfg(**d)


def _p(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _c(t) -> int | None:
    """_p for the entry points that check what they are given: a tensor has to be dense, and on the
    current device (its stream and kernels are there) or in pinned host memory, unless it is empty."""
    if t is None or isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError(f"tensor of shape {tuple(t.shape)} with strides {t.stride()} is not contiguous")
    d = t.get_device()                       # -1 on the host
    if d < 0:
        if t.numel() and not t.is_pinned():
            raise ValueError(f"tensor of shape {tuple(t.shape)} on {t.device}: no GPU can read it")
    elif d != _device():
        raise ValueError(f"tensor on {t.device}, but the current device is cuda:{_device()}")
    return t.data_ptr()


_device_fn = _stream_fn = None


def _bind_torch() -> None:
    """Torch's own current-device and current-stream queries, without the objects that torch.cuda wraps
    them in (a call of a small kernel costs 4 us; torch.cuda.current_stream() took 2.8 of the binding's 5.5).
    They are no public names: where a torch lacks one, the public calls serve."""
    global _device_fn, _stream_fn
    import torch
    torch.cuda.init()
    _device_fn = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _stream_fn = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                  or (lambda device: torch.cuda.current_stream(device).cuda_stream))


def _device() -> int:
    if _device_fn is None:
        _bind_torch()
    return _device_fn()


def _s(stream) -> int | None:
    if stream is None:
        return _stream_fn(_device_fn()) if _stream_fn is not None else _first_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _first_stream() -> int:
    _bind_torch()
    return _stream_fn(_device_fn())


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _check(name: str, st: int) -> None:
    if st != MOE_OK:
        raise MoeError(name, st)


def moe_route(cfg, x, w_router, logit_offset, bias, scores, flags, topk_idx, topk_w, ws=None, stream=None):
    _check("moe_route", lib().moe_route(ctypes.byref(cfg), _p(x), _p(w_router), _p(logit_offset), _p(bias),
                                        _p(scores), flags, _p(topk_idx), _p(topk_w), _p(ws), _nbytes(ws),
                                        _s(stream)))


def moe_dispatch(cfg, topk_idx, x, counts, offsets, perm, inv, x_perm, x_perm_scale, ws, stream=None):
    _check("moe_dispatch", lib().moe_dispatch(ctypes.byref(cfg), _p(topk_idx), _p(x), _p(counts), _p(offsets),
                                              _p(perm), _p(inv), _p(x_perm), _p(x_perm_scale), _p(ws),
                                              _nbytes(ws), _s(stream)))


def moe_dispatch_noalloc(cfg, topk_idx, x, counts, offsets, perm, inv, x_perm, x_perm_scale, stream=None):
    _check("moe_dispatch_noalloc", lib().moe_dispatch_noalloc(
        ctypes.byref(cfg), _p(topk_idx), _p(x), _p(counts), _p(offsets), _p(perm), _p(inv), _p(x_perm),
        _p(x_perm_scale), _s(stream)))


def expert_weights(w_gate_up, w_down, ws_gate_up=None, ws_down=None, w_gate_up_scale=None,
                   w_down_scale=None, ws_gate_up_scale=None, ws_down_scale=None) -> MoeExpertWeights:
    return MoeExpertWeights(_p(w_gate_up), _p(w_down), _p(w_gate_up_scale), _p(w_down_scale),
                            _p(ws_gate_up), _p(ws_down), _p(ws_gate_up_scale), _p(ws_down_scale))


def moe_expert_ffn(cfg, x_perm, x_perm_scale, offsets, weights: MoeExpertWeights, x, y_perm, y_shared, ws,
                   phase=MOE_FFN_ALL, stream=None):
    _check("moe_expert_ffn", lib().moe_expert_ffn(ctypes.byref(cfg), _p(x_perm), _p(x_perm_scale), _p(offsets),
                                                  ctypes.byref(weights), _p(x), _p(y_perm), _p(y_shared),
                                                  _p(ws), _nbytes(ws), phase, _s(stream)))


def moe_expert_ffn_gather(cfg, x, perm, offsets, weights: MoeExpertWeights, y_perm, y_shared, ws,
                          phase=MOE_FFN_ALL, stream=None):
    _check("moe_expert_ffn_gather", lib().moe_expert_ffn_gather(
        ctypes.byref(cfg), _p(x), _p(perm), _p(offsets), ctypes.byref(weights), _p(y_perm), _p(y_shared),
        _p(ws), _nbytes(ws), phase, _s(stream)))


def ffn_saved(g, u, gs=None, us=None) -> MoeFfnSaved:
    return MoeFfnSaved(_p(g), _p(u), _p(gs), _p(us))


def moe_expert_ffn_save(cfg, x_perm, perm, offsets, weights: MoeExpertWeights, x, y_perm, y_shared,
                        saved: MoeFfnSaved, ws, phase=MOE_FFN_ALL, stream=None):
    _check("moe_expert_ffn_save", lib().moe_expert_ffn_save(
        ctypes.byref(cfg), _p(x_perm), _p(perm), _p(offsets), ctypes.byref(weights), _p(x), _p(y_perm),
        _p(y_shared), ctypes.byref(saved), _p(ws), _nbytes(ws), phase, _s(stream)))


def moe_combine(cfg, y_perm, y_shared, inv, topk_w, y, stream=None):
    _check("moe_combine", lib().moe_combine(ctypes.byref(cfg), _p(y_perm), _p(y_shared), _p(inv), _p(topk_w),
                                            _p(y), _s(stream)))


def expert_grads(w_gate_up, w_down, ws_gate_up=None, ws_down=None) -> MoeExpertGrads:
    return MoeExpertGrads(_p(w_gate_up), _p(w_down), _p(ws_gate_up), _p(ws_down))


def moe_combine_backward(cfg, dy, y_perm, inv, topk_w, dy_perm, d_topk_w, stream=None):
    _check("moe_combine_backward", lib().moe_combine_backward(
        ctypes.byref(cfg), _p(dy), _p(y_perm), _p(inv), _p(topk_w), _p(dy_perm), _p(d_topk_w), _s(stream)))


def moe_expert_ffn_backward(cfg, x_perm, x, offsets, weights: MoeExpertWeights, dy_perm, dy, dx_perm, dx_shared,
                            grads: MoeExpertGrads, ws, stream=None):
    _check("moe_expert_ffn_backward", lib().moe_expert_ffn_backward(
        ctypes.byref(cfg), _p(x_perm), _p(x), _p(offsets), ctypes.byref(weights), _p(dy_perm), _p(dy), _p(dx_perm),
        _p(dx_shared), ctypes.byref(grads), _p(ws), _nbytes(ws), _s(stream)))


def moe_expert_ffn_backward_saved(cfg, x_perm, x, offsets, weights: MoeExpertWeights, saved: MoeFfnSaved, dy_perm,
                                  dy, dx_perm, dx_shared, grads: MoeExpertGrads, ws, stream=None):
    _check("moe_expert_ffn_backward_saved", lib().moe_expert_ffn_backward_saved(
        ctypes.byref(cfg), _p(x_perm), _p(x), _p(offsets), ctypes.byref(weights), ctypes.byref(saved), _p(dy_perm),
        _p(dy), _p(dx_perm), _p(dx_shared), ctypes.byref(grads), _p(ws), _nbytes(ws), _s(stream)))


def moe_route_backward(cfg, x, w_router, scores, topk_idx, d_topk_w, alpha, seq_len, dx_router, dw_router, loss, ws,
                       stream=None):
    _check("moe_route_backward", lib().moe_route_backward(
        ctypes.byref(cfg), _p(x), _p(w_router), _p(scores), _p(topk_idx), _p(d_topk_w), float(alpha), int(seq_len),
        _p(dx_router), _p(dw_router), _p(loss), _p(ws), _nbytes(ws), _s(stream)))


def moe_dispatch_backward(cfg, dx_perm, dx_shared, dx_router, inv, dx, stream=None):
    _check("moe_dispatch_backward", lib().moe_dispatch_backward(
        ctypes.byref(cfg), _p(dx_perm), _p(dx_shared), _p(dx_router), _p(inv), _p(dx), _s(stream)))


def moe_update_bias(cfg, counts, bias, gamma, stream=None):
    _check("moe_update_bias", lib().moe_update_bias(ctypes.byref(cfg), _p(counts), _p(bias), float(gamma),
                                                    _s(stream)))


def moe_quantize_fp8(src, n_mat, rows, cols, block_rows, dst, scales, stream=None):
    _check("moe_quantize_fp8", lib().moe_quantize_fp8(_p(src), n_mat, rows, cols, block_rows, _p(dst),
                                                      _p(scales), _s(stream)))


def live_count(n_tokens) -> int | None:
    """Address of the live count of a padded batch: None (every token), or an int32 tensor of one element, which the
    kernels read on the device.  A Python number is refused, as it would be taken for an address."""
    import torch
    if n_tokens is None:
        return None
    if not isinstance(n_tokens, torch.Tensor):
        raise TypeError(f"n_tokens is an int32 tensor of one element on the device, not {n_tokens!r}")
    if n_tokens.dtype != torch.int32 or n_tokens.numel() != 1:
        raise ValueError(f"n_tokens is an int32 tensor of one element, not {n_tokens.numel()} of {n_tokens.dtype}")
    return _c(n_tokens)


def moe_dispatch_local(cfg, first_expert, n_tokens, topk_idx, x, counts, offsets, perm, inv, x_perm, x_perm_scale, ws,
                       stream=None):
    _check("moe_dispatch_local", lib().moe_dispatch_local(
        ctypes.byref(cfg), int(first_expert), live_count(n_tokens), _c(topk_idx), _c(x), _c(counts), _c(offsets),
        _c(perm), _c(inv), _c(x_perm), _c(x_perm_scale), _c(ws), _nbytes(ws), _s(stream)))


def moe_combine_local(cfg, y_perm, y_shared, inv, topk_w, y, stream=None):
    _check("moe_combine_local", lib().moe_combine_local(ctypes.byref(cfg), _c(y_perm), _c(y_shared), _c(inv),
                                                        _c(topk_w), _c(y), _s(stream)))


def moe_combine_local_backward(cfg, dy, y_perm, inv, topk_w, dy_perm, d_topk_w, stream=None):
    _check("moe_combine_local_backward", lib().moe_combine_local_backward(
        ctypes.byref(cfg), _c(dy), _c(y_perm), _c(inv), _c(topk_w), _c(dy_perm), _c(d_topk_w), _s(stream)))


def moe_dispatch_local_backward(cfg, dx_perm, dx_shared, dx_router, inv, dx, stream=None):
    _check("moe_dispatch_local_backward", lib().moe_dispatch_local_backward(
        ctypes.byref(cfg), _c(dx_perm), _c(dx_shared), _c(dx_router), _c(inv), _c(dx), _s(stream)))


def moe_quantize_fp4(src, n_mat, rows, cols, dst, scales, stream=None):
    """bf16 [n_mat, rows, cols] -> MXFP4 codes [n_mat, rows, cols/2] and scale bytes [n_mat, cols/128, rows, 4]."""
    _check("moe_quantize_fp4", lib().moe_quantize_fp4(_c(src), n_mat, rows, cols, _c(dst), _c(scales), _s(stream)))


def moe_dequantize_fp4(codes, scales, n_mat, rows, cols, dst, stream=None):
    """The bf16 values [n_mat, rows, cols] of MXFP4 codes and scale bytes."""
    _check("moe_dequantize_fp4", lib().moe_dequantize_fp4(_c(codes), _c(scales), n_mat, rows, cols, _c(dst),
                                                          _s(stream)))


def moe_expert_ffn_codes(cfg, x_codes, x_scale, perm, offsets, weights: MoeExpertWeights, y_perm, y_shared, ws,
                         phase=MOE_FFN_ALL, stream=None):
    """moe_expert_ffn_gather on int8 or E4M3 codes [T, H] with their scales."""
    _check("moe_expert_ffn_codes", lib().moe_expert_ffn_codes(
        ctypes.byref(cfg), _c(x_codes), _c(x_scale), _c(perm), _c(offsets), ctypes.byref(weights), _c(y_perm),
        _c(y_shared), _c(ws), _nbytes(ws), phase, _s(stream)))


def moe_quantize_int8(src, n_mat, rows, cols, group, dst, scales, stream=None):
    """bf16 [n_mat, rows, cols] -> int8 codes of the same shape and fp32 scales [n_mat / group, rows]."""
    _check("moe_quantize_int8", lib().moe_quantize_int8(_c(src), n_mat, rows, cols, group, _c(dst), _c(scales),
                                                        _s(stream)))


def moe_norm(cfg, n_tokens, x, residual, weight, eps, h, y, codes=None, code_scale=None, stream=None):
    """h = x + residual, y = h * weight / rms(h), and y as int8 or E4M3 codes."""
    _check("moe_norm", lib().moe_norm(ctypes.byref(cfg), live_count(n_tokens), _c(x), _c(residual), _c(weight),
                                      float(eps), _c(h), _c(y), _c(codes), _c(code_scale), _s(stream)))


def moe_norm_backward(cfg, n_tokens, h, weight, eps, dy, dh, dx, dweight, ws, stream=None):
    _check("moe_norm_backward", lib().moe_norm_backward(
        ctypes.byref(cfg), live_count(n_tokens), _c(h), _c(weight), float(eps), _c(dy), _c(dh), _c(dx), _c(dweight),
        _c(ws), _nbytes(ws), _s(stream)))


def moe_route_backward_flags(cfg, flags, x, w_router, scores, topk_idx, d_topk_w, alpha, seq_len, dx_router, dw_router,
                             loss, ws, stream=None):
    _check("moe_route_backward_flags", lib().moe_route_backward_flags(
        ctypes.byref(cfg), flags, _c(x), _c(w_router), _c(scores), _c(topk_idx), _c(d_topk_w), float(alpha),
        int(seq_len), _c(dx_router), _c(dw_router), _c(loss), _c(ws), _nbytes(ws), _s(stream)))


def moe_ffn_workspace_part(cfg, part) -> tuple:
    """(byte offset, byte size) of an intermediate inside the moe_expert_ffn workspace."""
    off, nb = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check("moe_ffn_workspace_part", lib().moe_ffn_workspace_part(ctypes.byref(cfg), part, ctypes.byref(off),
                                                                  ctypes.byref(nb)))
    return int(off.value), int(nb.value)


def moe_workspace_bytes(cfg, which) -> int:
    return int(lib().moe_workspace_bytes(ctypes.byref(cfg), which))


def status_string(st: int) -> str:
    try:
        return lib().moe_status_string(st).decode()
    except Exception:  # pragma: no cover
        return "?"


moe_status_string = status_string


def moe_abi_version() -> int:
    return int(lib().moe_abi_version())
