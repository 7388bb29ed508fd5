"""Thin ctypes binding of the operators on microscaled numbers
(include/q4_mx.h), the same names as the C ABI, in the manner of ``block``:
argument marshalling only, outputs allocated when the caller passes none,
Q4Error on a non-zero status.

An MX tensor [R, K] is the tuple of its planes (codes, scales): uint8 codes
[R, K / 2] (4 bits) or [R, K] (8 bits), uint8 scales [R, K / 32].  Weights are
4-bit ones.  Planes may also be one-byte views (torch.float8_e4m3fn codes).
"""
from __future__ import annotations

import ctypes

import torch

from .binding import Q4_BF16, _DT, _check, _dt, lib as _base_lib
from .block import (Q4_ACT_NONE, Q4_ACT_SILU, Q4_NORM_NONE, Q4_NORM_RMS, _code, _gate_rows, _handle, _like, _new, _out, _ptr,
                    _summed, _vectors, _workspace)

Q4_MXFP4, Q4_MXFP8 = 8, 9

_P, _I64, _INT, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
SIGNATURES = {
    "mx_quantize": (_INT, [_P, _INT, _INT, _P, _P, _I64, _I64, _P]),
    "mx_dequantize": (_INT, [_INT, _P, _P, _P, _INT, _I64, _I64, _P]),
    "mx_linear_workspace_size": (_I64, [_INT, _I64, _I64, _I64]),
    "mx_linear": (_INT, [_P, _P, _P, _INT, _P, _INT, _P, _P, _INT, _P, _P, _I64, _I64, _I64, _P, _I64, _P]),
    "mx_linear_backward_workspace_size": (_I64, [_I64, _I64, _I64]),
    "mx_linear_backward": (_INT, [_P, _P, _INT, _P, _P, _INT, _P, _P, _P, _I64, _I64, _I64, _P, _I64, _P]),
    "mx_gated_workspace_size": (_I64, [_INT, _I64, _I64, _I64]),
    "mx_gated": (_INT, [_P, _P, _P, _P, _P, _P, _INT, _INT, _P, _P, _INT, _P, _P, _P, _I64, _I64, _I64, _P, _I64, _P]),
    "mx_gated_backward_workspace_size": (_I64, [_I64, _I64, _I64]),
    "mx_gated_backward": (_INT, [_P, _P, _P, _P, _INT, _P, _P, _P, _INT, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _I64,
                                 _P]),
    "block_norm_mx": (_INT, [_P, _P, _INT, _INT, _I64, _I64, _INT, _P, _P, _P, _I64, _F, _INT, _P, _P, _F, _P, _INT, _P,
                             _P, _P, _P]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libq4.so with these entry points' signatures."""
    global _lib
    if _lib is None:
        l = _base_lib()
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run(name, args, like, stream, *tensors):
    """The call, on the GPU of `like`, where every other tensor has to be too."""
    at = like.get_device()
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.get_device() != at:
            raise ValueError(f"{name}: tensors on different devices")
    if at == _device():
        _check(name, getattr(_lib, name)(*args, _handle(stream, like)))
    else:
        with torch.cuda.device(at):
            _check(name, getattr(_lib, name)(*args, _handle(stream, like)))


def _mx(t, name):
    """(type, rows, K) of an MX tensor's planes."""
    if len(t) != 2:
        raise ValueError(f"{name} must be (codes, scales)")
    q, s = t
    R, groups = s.shape
    if q.element_size() != 1 or s.element_size() != 1 or q.dim() != 2 or q.shape[0] != R:
        raise ValueError(f"the planes of {name} do not fit each other")
    width = q.shape[1]
    if width == groups * 16:
        return Q4_MXFP4, R, groups * 32
    if width != groups * 32:
        raise ValueError(f"the planes of {name} do not fit each other")
    return Q4_MXFP8, R, width


def _weight(w, name="w"):
    kind, N, K = _mx(w, name)
    if kind != Q4_MXFP4:
        raise ValueError(f"{name} must have 4-bit codes")
    return N, K


def _pair(gate, up):
    shape = _weight(gate, "gate")
    if _weight(up, "up") != shape:
        raise ValueError("gate and up must have the same shape")
    return shape


def _x(x, K, dtype):
    """(type, rows, planes, the tensor itself or its codes, output dtype) of an activation."""
    if isinstance(x, torch.Tensor):
        M = x.shape[0]
        _like(x, "x", (M, K), x.dtype)
        if dtype is not None and dtype != x.dtype:
            raise ValueError(f"dtype must be x's, {x.dtype}")
        return _dt(x), M, (x, None), x, x.dtype
    kind, M, width = _mx(x, "x")
    if width != K:
        raise ValueError(f"x must have {K} values a row, not {width}")
    dtype = dtype or torch.bfloat16
    _code(dtype)
    return kind, M, x, x[0], dtype


# ---- planes ---------------------------------------------------------------------

def mx_quantize(v, type=Q4_MXFP8, codes=None, scales=None, stream=None):
    """The planes (codes, scales) of v [M, K] as Q4_MXFP8 or Q4_MXFP4."""
    lib()
    M, K = v.shape
    if K % 32:
        raise ValueError(f"{K} values a row: not whole blocks of 32")
    codes = _out(codes, "codes", (M, K // 2 if type == Q4_MXFP4 else K), torch.uint8, v, stream)
    scales = _out(scales, "scales", (M, K // 32), torch.uint8, v, stream)
    _run("mx_quantize", (_ptr(v), _dt(v), type, _ptr(codes), _ptr(scales), M, K), v, stream, codes, scales)
    return codes, scales


def mx_dequantize(planes, dtype=torch.bfloat16, v=None, stream=None):
    """The values [M, K] that planes stand for."""
    lib()
    kind, M, K = _mx(planes, "planes")
    v = _out(v, "v", (M, K), dtype, planes[0], stream)
    _run("mx_dequantize", (kind, _ptr(planes[0]), _ptr(planes[1]), _ptr(v), _code(dtype), M, K), planes[0], stream,
         planes[1], v)
    return v


# ---- linear ---------------------------------------------------------------------

def mx_linear_workspace_size(M, N, K, x_type=Q4_MXFP8) -> int:
    return int(lib().mx_linear_workspace_size(x_type, M, N, K))


def mx_linear(w, x, bias=None, act=Q4_ACT_NONE, residual=None, save_pre=False, dtype=None, y=None, pre=None,
              workspace="auto", stream=None):
    """y [M, N] = act(x . W^T + bias) + residual of `dtype` (x's; for MX x
    bfloat16 unless given); with save_pre (or a `pre` tensor) also the values
    before the activation: (y, pre)."""
    N, K = _weight(w)
    xt, M, (xq, xs), like, dtype = _x(x, K, dtype)
    _like(bias, "bias", (N,), dtype)
    _like(residual, "residual", (M, N), dtype)
    y = _out(y, "y", (M, N), dtype, like, stream)
    if pre is None and save_pre:
        pre = _new((M, N), dtype, like, stream)
    _like(pre, "pre", (M, N), dtype)
    ws, n = _workspace(workspace, mx_linear_workspace_size(M, N, K, xt), like, stream)
    _run("mx_linear", (_ptr(w[0]), _ptr(w[1]), _ptr(bias), act, _ptr(residual), xt, _ptr(xq), _ptr(xs), _code(dtype), _ptr(y),
                       _ptr(pre), M, N, K, _ptr(ws), n), like, stream, w[0], w[1], xs, bias, residual, y, pre, ws)
    return y if pre is None else (y, pre)


def mx_linear_backward_workspace_size(M, N, K) -> int:
    return int(lib().mx_linear_backward_workspace_size(M, N, K))


def mx_linear_backward(w, dy, act=Q4_ACT_NONE, pre=None, bias_grad=False, dx=None, dz=None, dbias=None,
                       workspace="auto", stream=None):
    """Gradients {"dx", "dz" (with an activation), "dbias" (with bias_grad)}
    of mx_linear; the residual's gradient is dy itself."""
    N, K = _weight(w)
    M = dy.shape[0]
    _like(dy, "dy", (M, N), dy.dtype)
    _like(pre, "pre", (M, N), dy.dtype)
    out = {"dx": _summed(dx, "dx", (M, K), dy.dtype, N, dy, stream)}
    if act != Q4_ACT_NONE or dz is not None:              # the library refuses a dz that would be dy
        out["dz"] = _out(dz, "dz", (M, N), dy.dtype, dy, stream)
    if bias_grad or dbias is not None:
        out["dbias"] = _summed(dbias, "dbias", (N,), torch.float32, M, dy, stream)
    ws, n = _workspace(workspace, mx_linear_backward_workspace_size(M, N, K), dy, stream)
    _run("mx_linear_backward", (_ptr(w[0]), _ptr(w[1]), act, _ptr(pre), _ptr(dy), _dt(dy), _ptr(out["dx"]),
                                _ptr(out.get("dz")), _ptr(out.get("dbias")), M, N, K, _ptr(ws), n), dy, stream, w[0], w[1],
         pre, ws, *out.values())
    return out


# ---- gated ----------------------------------------------------------------------

def mx_gated_workspace_size(M, N, K, x_type=Q4_MXFP8) -> int:
    return int(lib().mx_gated_workspace_size(x_type, M, N, K))


def mx_gated(gate, up, x, act=Q4_ACT_SILU, gate_bias=None, up_bias=None, save_pre=False, dtype=None, h=None,
             gate_pre=None, up_pre=None, workspace="auto", stream=None):
    """h [M, N] = act(x . Wgate^T + gate_bias) * (x . Wup^T + up_bias); with
    save_pre (or both tensors) also the two projections: (h, gate_pre, up_pre)."""
    N, K = _pair(gate, up)
    xt, M, (xq, xs), like, dtype = _x(x, K, dtype)
    _like(gate_bias, "gate_bias", (N,), dtype)
    _like(up_bias, "up_bias", (N,), dtype)
    h = _out(h, "h", (M, N), dtype, like, stream)
    if save_pre:
        gate_pre = _new((M, N), dtype, like, stream) if gate_pre is None else gate_pre
        up_pre = _new((M, N), dtype, like, stream) if up_pre is None else up_pre
    _like(gate_pre, "gate_pre", (M, N), dtype)
    _like(up_pre, "up_pre", (M, N), dtype)
    ws, n = _workspace(workspace, mx_gated_workspace_size(M, N, K, xt), like, stream)
    _run("mx_gated", (_ptr(gate[0]), _ptr(gate[1]), _ptr(up[0]), _ptr(up[1]), _ptr(gate_bias), _ptr(up_bias), act, xt, _ptr(xq),
                      _ptr(xs), _code(dtype), _ptr(h), _ptr(gate_pre), _ptr(up_pre), M, N, K, _ptr(ws), n), like, stream,
         gate[0], gate[1], up[0], up[1], gate_bias, up_bias, xs, h, gate_pre, up_pre, ws)
    return h if gate_pre is None else (h, gate_pre, up_pre)


def mx_gated_backward_workspace_size(M, N, K) -> int:
    return int(lib().mx_gated_backward_workspace_size(M, N, K))


def mx_gated_backward(gate, up, dh, gate_pre, up_pre, act=Q4_ACT_SILU, bias_grad=False, dx=None, dgate=None, dup=None,
                      dgate_bias=None, dup_bias=None, workspace="auto", stream=None):
    """Gradients {"dx", "dgate", "dup", and with bias_grad "dgate_bias", "dup_bias"} of mx_gated."""
    N, K = _pair(gate, up)
    M = dh.shape[0]
    for t, name in ((dh, "dh"), (gate_pre, "gate_pre"), (up_pre, "up_pre"), (dgate, "dgate"), (dup, "dup")):
        _like(t, name, (M, N), dh.dtype)
    out = {"dx": _summed(dx, "dx", (M, K), dh.dtype, N, dh, stream),
           "dgate": _new((M, N), dh.dtype, dh, stream) if dgate is None else dgate,
           "dup": _new((M, N), dh.dtype, dh, stream) if dup is None else dup}
    for name, t in (("dgate_bias", dgate_bias), ("dup_bias", dup_bias)):
        if bias_grad or t is not None:
            out[name] = _summed(t, name, (N,), torch.float32, M, dh, stream)
    ws, n = _workspace(workspace, mx_gated_backward_workspace_size(M, N, K), dh, stream)
    _run("mx_gated_backward", (_ptr(gate[0]), _ptr(gate[1]), _ptr(up[0]), _ptr(up[1]), act, _ptr(gate_pre), _ptr(up_pre),
                               _ptr(dh), _dt(dh), _ptr(out["dx"]), _ptr(out["dgate"]), _ptr(out["dup"]),
                               _ptr(out.get("dgate_bias")), _ptr(out.get("dup_bias")), M, N, K, _ptr(ws), n), dh, stream,
         gate[0], gate[1], up[0], up[1], gate_pre, up_pre, ws, *out.values())
    return out


# ---- norm -----------------------------------------------------------------------

def block_norm_mx(r, y=None, pre_norm=Q4_NORM_RMS, pre_weight=None, pre_bias=None, post_norm=Q4_NORM_NONE,
                  post_weight=None, post_bias=None, gate=None, gate_rows=None, scale=1.0, eps=1e-5, n_type=Q4_MXFP8,
                  save_stats=False, dtype=None, r_out=None, n=None, stats=None, stream=None):
    """block_norm with n = pre(r') as MX planes: (r', (codes, scales), stats).

    stats (float32 [M, 4], for block_norm_backward) is None unless asked for;
    without y, r' is r itself and `dtype` the type of the weights (r's)."""
    lib()
    M, D = r.shape
    if D % 32:
        raise ValueError(f"{D} values a row: not whole blocks of 32")
    dt = y.dtype if y is not None else (dtype or r.dtype)
    if y is not None:
        _like(y, "y", (M, D), dt)
        r_out = _out(r_out, "r_out", (M, D), r.dtype, r, stream)
    _vectors(D, dt, pre_weight=pre_weight, pre_bias=pre_bias, post_weight=post_weight, post_bias=post_bias)
    rows = _gate_rows(gate, gate_rows, M)
    if gate is not None:
        _like(gate, "gate", (gate.shape[0], D), dt)
    codes, scales = n if n is not None else (None, None)
    codes = _out(codes, "codes", (M, D // 2 if n_type == Q4_MXFP4 else D), torch.uint8, r, stream)
    scales = _out(scales, "scales", (M, D // 32), torch.uint8, r, stream)
    if stats is None and save_stats:
        stats = _new((M, 4), torch.float32, r, stream)
    _like(stats, "stats", (M, 4), torch.float32)
    _run("block_norm_mx", (_ptr(y), _ptr(r), _code(dt), _dt(r), M, D, post_norm, _ptr(post_weight), _ptr(post_bias), _ptr(gate),
                           rows, scale, pre_norm, _ptr(pre_weight), _ptr(pre_bias), eps, _ptr(r_out), n_type, _ptr(codes),
                           _ptr(scales), _ptr(stats)), r, stream, y, post_weight, post_bias, gate, pre_weight, pre_bias,
         r_out, codes, scales, stats)
    return r if y is None else r_out, (codes, scales), stats
