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
import functools

import torch

from .binding import Q4_BF16, _DT, _check, _dt, lib as _base_lib
from .block import (Q4_ACT_NONE, Q4_ACT_SILU, Q4_NORM_NONE, Q4_NORM_RMS, _code, _gate_rows, _handle, _like, _new, _out,
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


# A token's calls are host-bound (a launch is 4 us, its kernel 3 to 12), so the
# marshalling asks a tensor for little: its device, contiguity and address once.
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _there(fn):
    """Runs an operator on the GPU of its tensors: `fn` raises _Elsewhere where that is not the current one."""
    @functools.wraps(fn)
    def call(*args, **kw):
        try:
            return fn(*args, **kw)
        except _Elsewhere as e:
            with torch.cuda.device(e.args[0]):
                return fn(*args, **kw)
    return call


class _Elsewhere(Exception):
    pass


def _here(like):
    at = like.get_device()
    if at < 0:
        raise ValueError("tensors must live on the GPU")
    if at != _device():
        raise _Elsewhere(at)
    return at


def _p(t, at):
    """A tensor's address (raw pointers pass through), on GPU `at`."""
    if t is None or t.__class__ is int:
        return t
    if t.get_device() != at:
        raise ValueError("tensors must live on the GPU, all on the same one")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _mx(t, name):
    """(type, rows, K) of an MX tensor's planes."""
    if len(t) != 2:
        raise ValueError(f"{name} must be (codes, scales)")
    q, s = t
    (rows, width), (R, groups) = q.shape, s.shape
    if rows == R and q.element_size() == 1 and s.element_size() == 1:
        if width == groups * 16:
            return Q4_MXFP4, R, groups * 32
        if width == groups * 32:
            return Q4_MXFP8, R, width
    raise ValueError(f"the planes of {name} do not fit each other")


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
        M, width = x.shape
        if width != K:
            raise ValueError(f"x must have {K} values a row, not {width}")
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

@_there
def mx_quantize(v, type=Q4_MXFP8, codes=None, scales=None, stream=None):
    """The planes (codes, scales) of v [M, K] as Q4_MXFP8 or Q4_MXFP4."""
    M, K = v.shape
    if K % 32:
        raise ValueError(f"{K} values a row: not whole blocks of 32")
    at = _here(v)
    codes = _out(codes, "codes", (M, K // 2 if type == Q4_MXFP4 else K), torch.uint8, v, stream)
    scales = _out(scales, "scales", (M, K // 32), torch.uint8, v, stream)
    _check("mx_quantize", lib().mx_quantize(_p(v, at), _dt(v), type, _p(codes, at), _p(scales, at), M, K, _handle(stream, v)))
    return codes, scales


@_there
def mx_dequantize(planes, dtype=torch.bfloat16, v=None, stream=None):
    """The values [M, K] that planes stand for."""
    kind, M, K = _mx(planes, "planes")
    at = _here(planes[0])
    v = _out(v, "v", (M, K), dtype, planes[0], stream)
    _check("mx_dequantize", lib().mx_dequantize(kind, _p(planes[0], at), _p(planes[1], at), _p(v, at), _code(dtype), M, K,
                                                _handle(stream, planes[0])))
    return v


# ---- linear ---------------------------------------------------------------------

def mx_linear_workspace_size(M, N, K, x_type=Q4_MXFP8) -> int:
    return int(lib().mx_linear_workspace_size(x_type, M, N, K))


@_there
def mx_linear(w, x, bias=None, act=Q4_ACT_NONE, residual=None, save_pre=False, dtype=None, y=None, pre=None,
              workspace="auto", stream=None):
    """y [M, N] = act(x . W^T + bias) + residual of `dtype` (x's; for MX x
    bfloat16 unless given); with save_pre (or a `pre` tensor) also the values
    before the activation: (y, pre)."""
    N, K = _weight(w)
    xt, M, (xq, xs), like, dtype = _x(x, K, dtype)
    at = _here(like)
    _like(bias, "bias", (N,), dtype)
    _like(residual, "residual", (M, N), dtype)
    y = _out(y, "y", (M, N), dtype, like, stream)
    if pre is None and save_pre:
        pre = _new((M, N), dtype, like, stream)
    _like(pre, "pre", (M, N), dtype)
    ws, n = _workspace(workspace, mx_linear_workspace_size(M, N, K, xt), like, stream)
    _check("mx_linear", lib().mx_linear(_p(w[0], at), _p(w[1], at), _p(bias, at), act, _p(residual, at), xt, _p(xq, at),
                                        _p(xs, at), _code(dtype), _p(y, at), _p(pre, at), M, N, K, _p(ws, at), n,
                                        _handle(stream, like)))
    return y if pre is None else (y, pre)


def mx_linear_backward_workspace_size(M, N, K) -> int:
    return int(lib().mx_linear_backward_workspace_size(M, N, K))


@_there
def mx_linear_backward(w, dy, act=Q4_ACT_NONE, pre=None, bias_grad=False, dx=None, dz=None, dbias=None,
                       workspace="auto", stream=None):
    """Gradients {"dx", "dz" (with an activation), "dbias" (with bias_grad)}
    of mx_linear; the residual's gradient is dy itself."""
    N, K = _weight(w)
    M, at = dy.shape[0], _here(dy)
    _like(dy, "dy", (M, N), dy.dtype)
    _like(pre, "pre", (M, N), dy.dtype)
    out = {"dx": _summed(dx, "dx", (M, K), dy.dtype, N, dy, stream)}
    if act != Q4_ACT_NONE or dz is not None:              # the library refuses a dz that would be dy
        out["dz"] = _out(dz, "dz", (M, N), dy.dtype, dy, stream)
    if bias_grad or dbias is not None:
        out["dbias"] = _summed(dbias, "dbias", (N,), torch.float32, M, dy, stream)
    ws, n = _workspace(workspace, mx_linear_backward_workspace_size(M, N, K), dy, stream)
    _check("mx_linear_backward",
           lib().mx_linear_backward(_p(w[0], at), _p(w[1], at), act, _p(pre, at), _p(dy, at), _dt(dy), _p(out["dx"], at),
                                    _p(out.get("dz"), at), _p(out.get("dbias"), at), M, N, K, _p(ws, at), n,
                                    _handle(stream, dy)))
    return out


# ---- gated ----------------------------------------------------------------------

def mx_gated_workspace_size(M, N, K, x_type=Q4_MXFP8) -> int:
    return int(lib().mx_gated_workspace_size(x_type, M, N, K))


@_there
def mx_gated(gate, up, x, act=Q4_ACT_SILU, gate_bias=None, up_bias=None, save_pre=False, dtype=None, h=None,
             gate_pre=None, up_pre=None, workspace="auto", stream=None):
    """h [M, N] = act(x . Wgate^T + gate_bias) * (x . Wup^T + up_bias); with
    save_pre (or both tensors) also the two projections: (h, gate_pre, up_pre)."""
    N, K = _pair(gate, up)
    xt, M, (xq, xs), like, dtype = _x(x, K, dtype)
    at = _here(like)
    _like(gate_bias, "gate_bias", (N,), dtype)
    _like(up_bias, "up_bias", (N,), dtype)
    h = _out(h, "h", (M, N), dtype, like, stream)
    if save_pre:
        gate_pre = _new((M, N), dtype, like, stream) if gate_pre is None else gate_pre
        up_pre = _new((M, N), dtype, like, stream) if up_pre is None else up_pre
    _like(gate_pre, "gate_pre", (M, N), dtype)
    _like(up_pre, "up_pre", (M, N), dtype)
    ws, n = _workspace(workspace, mx_gated_workspace_size(M, N, K, xt), like, stream)
    _check("mx_gated", lib().mx_gated(_p(gate[0], at), _p(gate[1], at), _p(up[0], at), _p(up[1], at), _p(gate_bias, at),
                                      _p(up_bias, at), act, xt, _p(xq, at), _p(xs, at), _code(dtype), _p(h, at),
                                      _p(gate_pre, at), _p(up_pre, at), M, N, K, _p(ws, at), n, _handle(stream, like)))
    return h if gate_pre is None else (h, gate_pre, up_pre)


def mx_gated_backward_workspace_size(M, N, K) -> int:
    return int(lib().mx_gated_backward_workspace_size(M, N, K))


@_there
def mx_gated_backward(gate, up, dh, gate_pre, up_pre, act=Q4_ACT_SILU, bias_grad=False, dx=None, dgate=None, dup=None,
                      dgate_bias=None, dup_bias=None, workspace="auto", stream=None):
    """Gradients {"dx", "dgate", "dup", and with bias_grad "dgate_bias", "dup_bias"} of mx_gated."""
    N, K = _pair(gate, up)
    M, at = dh.shape[0], _here(dh)
    for t, name in ((dh, "dh"), (gate_pre, "gate_pre"), (up_pre, "up_pre"), (dgate, "dgate"), (dup, "dup")):
        _like(t, name, (M, N), dh.dtype)
    out = {"dx": _summed(dx, "dx", (M, K), dh.dtype, N, dh, stream),
           "dgate": _new((M, N), dh.dtype, dh, stream) if dgate is None else dgate,
           "dup": _new((M, N), dh.dtype, dh, stream) if dup is None else dup}
    for name, t in (("dgate_bias", dgate_bias), ("dup_bias", dup_bias)):
        if bias_grad or t is not None:
            out[name] = _summed(t, name, (N,), torch.float32, M, dh, stream)
    ws, n = _workspace(workspace, mx_gated_backward_workspace_size(M, N, K), dh, stream)
    _check("mx_gated_backward",
           lib().mx_gated_backward(_p(gate[0], at), _p(gate[1], at), _p(up[0], at), _p(up[1], at), act, _p(gate_pre, at),
                                   _p(up_pre, at), _p(dh, at), _dt(dh), _p(out["dx"], at), _p(out["dgate"], at),
                                   _p(out["dup"], at), _p(out.get("dgate_bias"), at), _p(out.get("dup_bias"), at), M, N, K,
                                   _p(ws, at), n, _handle(stream, dh)))
    return out


# ---- norm -----------------------------------------------------------------------

@_there
def block_norm_mx(r, y=None, pre_norm=Q4_NORM_RMS, pre_weight=None, pre_bias=None, post_norm=Q4_NORM_NONE,
                  post_weight=None, post_bias=None, gate=None, gate_rows=None, scale=1.0, eps=1e-5, n_type=Q4_MXFP8,
                  save_stats=False, dtype=None, r_out=None, n=None, stats=None, stream=None):
    """block_norm with n = pre(r') as MX planes: (r', (codes, scales), stats).

    stats (float32 [M, 4], for block_norm_backward) is None unless asked for;
    without y, r' is r itself and `dtype` the type of the weights (r's)."""
    M, D = r.shape
    if D % 32:
        raise ValueError(f"{D} values a row: not whole blocks of 32")
    at, shape = _here(r), (M, D)
    dt = y.dtype if y is not None else (dtype or r.dtype)
    if y is not None:
        _like(y, "y", shape, dt)
        r_out = _out(r_out, "r_out", shape, r.dtype, r, stream)
    if pre_weight is not None:
        _like(pre_weight, "pre_weight", (D,), dt)
    if pre_bias is not None or post_weight is not None or post_bias is not None:
        _vectors(D, dt, pre_bias=pre_bias, post_weight=post_weight, post_bias=post_bias)
    rows = 1
    if gate is not None:
        rows = _gate_rows(gate, gate_rows, M)
        _like(gate, "gate", (gate.shape[0], D), dt)
    codes, scales = n if n is not None else (None, None)
    width = D // 2 if n_type == Q4_MXFP4 else D
    if codes is None and scales is None and stream is None:
        codes, scales = r.new_empty((M, width), dtype=torch.uint8), r.new_empty((M, D // 32), dtype=torch.uint8)
    else:
        codes = _out(codes, "codes", (M, width), torch.uint8, r, stream)
        scales = _out(scales, "scales", (M, D // 32), torch.uint8, r, stream)
    if stats is not None:
        _like(stats, "stats", (M, 4), torch.float32)
    elif save_stats:
        stats = _new((M, 4), torch.float32, r, stream)
    _check("block_norm_mx",
           lib().block_norm_mx(_p(y, at), _p(r, at), _code(dt), _dt(r), M, D, post_norm, _p(post_weight, at), _p(post_bias, at),
                               _p(gate, at), rows, scale, pre_norm, _p(pre_weight, at), _p(pre_bias, at), eps, _p(r_out, at),
                               n_type, _p(codes, at), _p(scales, at), _p(stats, at), _handle(stream, r)))
    return r if y is None else r_out, (codes, scales), stats
