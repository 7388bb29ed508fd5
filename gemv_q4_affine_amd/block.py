"""Thin ctypes binding of the feed-forward operators (include/q4_block.h), the
same names as the C ABI, in the manner of ``binding``: argument marshalling
only, outputs allocated when the caller passes none, Q4Error on a non-zero
status.

A weight matrix is the tuple of its planes, as the quantisers return them:
(qs, d) for Q4_0, (codes, scales, biases) for the affine formats.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import Q4_BF16, Q4_FMT_AFFINE4, Q4_FMT_AFFINE8, Q4_FMT_Q4_0, _DT, _alloc_stream, _check, _dt, _stream, lib as _base_lib

Q4_ACT_NONE, Q4_ACT_SILU, Q4_ACT_GELU, Q4_ACT_GELU_TANH, Q4_ACT_RELU = 0, 1, 2, 3, 4
Q4_NORM_NONE, Q4_NORM_RMS, Q4_NORM_LAYER = 0, 1, 2
Q4_NORM_MAX_D = 32768

_P, _I64, _INT, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
SIGNATURES = {
    "q4_linear_workspace_size": (_I64, [_INT, _INT, _I64, _I64, _I64]),
    "q4_linear": (_INT, [_INT, _P, _P, _P, _P, _INT, _P, _P, _INT, _P, _P, _I64, _I64, _I64, _P, _I64, _P]),
    "q4_linear_backward_workspace_size": (_I64, [_INT, _I64, _I64, _I64]),
    "q4_linear_backward": (_INT, [_INT, _P, _P, _P, _INT, _P, _P, _INT, _P, _P, _P, _I64, _I64, _I64, _P, _I64, _P]),
    "q4_gated_workspace_size": (_I64, [_INT, _INT, _I64, _I64, _I64]),
    "q4_gated": (_INT, [_INT, _P, _P, _P, _P, _P, _P, _P, _P, _INT, _P, _INT, _P, _P, _P, _I64, _I64, _I64, _P, _I64,
                        _P]),
    "q4_gated_backward_workspace_size": (_I64, [_INT, _I64, _I64, _I64]),
    "q4_gated_backward": (_INT, [_INT, _P, _P, _P, _P, _P, _P, _INT, _P, _P, _P, _INT, _P, _P, _P, _P, _P, _I64, _I64,
                                 _I64, _P, _I64, _P]),
    "block_norm": (_INT, [_P, _P, _INT, _INT, _I64, _I64, _INT, _P, _P, _P, _I64, _F, _INT, _P, _P, _F, _P, _P, _P,
                          _P]),
    "block_norm_backward_workspace_size": (_I64, [_I64, _I64, _I64]),
    "block_norm_backward": (_INT, [_P, _P, _P, _P, _P, _INT, _INT, _I64, _I64, _INT, _P, _P, _P, _I64, _F, _INT, _P,
                                   _P, _P, _P, _P, _P, _P, _P, _P, _I64, _P]),
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


# The marshalling is on the clock of a call on one token (its kernels take 3 to
# 20 us), so it is kept short: pointers as plain ints, the stream's handle
# without a Stream object, outputs like their inputs where the shape is theirs.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _handle(stream, like):
    """The hipStream_t of a call: the caller's stream, or the current one of the tensor's GPU."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(like.get_device())
    return _stream(stream)


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        return t                       # raw pointer (int) passed through
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _new(shape, dtype, like, stream):
    """An output, owned by the call's stream."""
    if stream is None:
        if shape == like.shape and dtype == like.dtype:
            return torch.empty_like(like)
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(_alloc_stream(stream)):
        return like.new_empty(shape, dtype=dtype)


def _planes(w):
    """(format, N, K, three plane pointers) of a weight tuple."""
    n = len(w)
    if n not in (2, 3):
        raise ValueError("a weight is (qs, d) or (codes, scales, biases)")
    q, s = w[0], w[1]
    N, groups = s.shape
    if n == 2:
        fmt, K, want = Q4_FMT_Q4_0, groups * 32, groups * 16
    elif q.shape[-1] == groups * 64:
        fmt, K, want = Q4_FMT_AFFINE8, groups * 64, groups * 64
    else:
        fmt, K, want = Q4_FMT_AFFINE4, groups * 64, groups * 32
    if q.numel() != N * want or q.element_size() != 1 or s.element_size() != 2 or (n == 3 and w[2].shape != s.shape):
        raise ValueError("the planes of a weight do not fit each other")
    return fmt, N, K, (_ptr(q), _ptr(s), _ptr(w[2]) if n == 3 else None)


def _like(t, name, shape, dtype):
    """An optional tensor of the given shape and dtype (raw pointers pass through)."""
    if t is not None and isinstance(t, torch.Tensor) and (t.shape != shape or t.dtype != dtype):
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, not {t.dtype} {tuple(t.shape)}")
    return t


def _out(t, name, shape, dtype, like, stream):
    return _new(shape, dtype, like, stream) if t is None else _like(t, name, shape, dtype)


def _workspace(workspace, n, like, stream):
    """"auto": n bytes owned by the call's stream (None if n is 0); else the caller's tensor or None."""
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace must be 'auto', None or a tensor, not {workspace!r}")
        return (_new((n,), torch.uint8, like, stream), n) if n > 0 else (None, 0)
    return workspace, workspace.numel() * workspace.element_size() if workspace is not None else 0


def _summed(t, name, shape, dtype, terms, like, stream):
    """An output that sums over `terms` rows or columns: allocated if None,
    and zero where there are none (the library writes nothing then)."""
    t = _out(t, name, shape, dtype, like, stream)
    if terms == 0 and t.numel():
        with torch.cuda.stream(_alloc_stream(stream)):
            t.zero_()
    return t


# ---- linear ---------------------------------------------------------------------

def q4_linear_workspace_size(M, N, K, fmt=Q4_FMT_Q4_0, dtype=Q4_BF16) -> int:
    return int(lib().q4_linear_workspace_size(fmt, dtype, M, N, K))


def q4_linear(w, x, bias=None, act=Q4_ACT_NONE, residual=None, save_pre=False, y=None, pre=None, workspace="auto",
              stream=None):
    """y [M, N] = act(x . W^T + bias) + residual; with save_pre (or a `pre`
    tensor) also the values before the activation: (y, pre)."""
    fmt, N, K, wp = _planes(w)
    M = x.shape[0]
    _like(x, "x", (M, K), x.dtype)
    _like(bias, "bias", (N,), x.dtype)
    _like(residual, "residual", (M, N), x.dtype)
    y = _out(y, "y", (M, N), x.dtype, x, stream)
    if pre is None and save_pre:
        pre = _new((M, N), x.dtype, x, stream)
    _like(pre, "pre", (M, N), x.dtype)
    ws, n = _workspace(workspace, q4_linear_workspace_size(M, N, K, fmt, _dt(x)), x, stream)
    _check("q4_linear", lib().q4_linear(fmt, *wp, _ptr(bias), act, _ptr(residual), _ptr(x), _dt(x), _ptr(y), _ptr(pre), M, N, K,
                                        _ptr(ws), n, _handle(stream, x)))
    return y if pre is None else (y, pre)


def q4_linear_backward_workspace_size(M, N, K, fmt=Q4_FMT_Q4_0) -> int:
    return int(lib().q4_linear_backward_workspace_size(fmt, M, N, K))


def q4_linear_backward(w, dy, act=Q4_ACT_NONE, pre=None, bias_grad=False, dx=None, dz=None, dbias=None,
                       workspace="auto", stream=None):
    """Gradients {"dx", "dz" (with an activation), "dbias" (with bias_grad)}
    of q4_linear; the residual's gradient is dy itself."""
    fmt, N, K, wp = _planes(w)
    M = dy.shape[0]
    _like(dy, "dy", (M, N), dy.dtype)
    _like(pre, "pre", (M, N), dy.dtype)
    out = {"dx": _summed(dx, "dx", (M, K), dy.dtype, N, dy, stream)}
    if act != Q4_ACT_NONE or dz is not None:              # the library refuses a dz that would be dy
        out["dz"] = _out(dz, "dz", (M, N), dy.dtype, dy, stream)
    if bias_grad or dbias is not None:
        out["dbias"] = _summed(dbias, "dbias", (N,), torch.float32, M, dy, stream)
    ws, n = _workspace(workspace, q4_linear_backward_workspace_size(M, N, K, fmt), dy, stream)
    _check("q4_linear_backward",
           lib().q4_linear_backward(fmt, *wp, act, _ptr(pre), _ptr(dy), _dt(dy), _ptr(out["dx"]), _ptr(out.get("dz")),
                                    _ptr(out.get("dbias")), M, N, K, _ptr(ws), n, _handle(stream, dy)))
    return out


# ---- gated ----------------------------------------------------------------------

def q4_gated_workspace_size(M, N, K, fmt=Q4_FMT_Q4_0, dtype=Q4_BF16) -> int:
    return int(lib().q4_gated_workspace_size(fmt, dtype, M, N, K))


def _pair(gate, up):
    fmt, N, K, gp = _planes(gate)
    ufmt, uN, uK, up_ = _planes(up)
    if (fmt, N, K) != (ufmt, uN, uK):
        raise ValueError("gate and up must have the same format and shape")
    return fmt, N, K, gp, up_


def q4_gated(gate, up, x, act=Q4_ACT_SILU, gate_bias=None, up_bias=None, save_pre=False, h=None, gate_pre=None,
             up_pre=None, workspace="auto", stream=None):
    """h [M, N] = act(x . Wgate^T + gate_bias) * (x . Wup^T + up_bias); with
    save_pre (or both tensors) also the two projections: (h, gate_pre, up_pre)."""
    fmt, N, K, gp, upp = _pair(gate, up)
    M = x.shape[0]
    _like(x, "x", (M, K), x.dtype)
    _like(gate_bias, "gate_bias", (N,), x.dtype)
    _like(up_bias, "up_bias", (N,), x.dtype)
    h = _out(h, "h", (M, N), x.dtype, x, stream)
    if save_pre:
        gate_pre = _new((M, N), x.dtype, x, stream) if gate_pre is None else gate_pre
        up_pre = _new((M, N), x.dtype, x, stream) if up_pre is None else up_pre
    _like(gate_pre, "gate_pre", (M, N), x.dtype)
    _like(up_pre, "up_pre", (M, N), x.dtype)
    ws, n = _workspace(workspace, q4_gated_workspace_size(M, N, K, fmt, _dt(x)), x, stream)
    _check("q4_gated", lib().q4_gated(fmt, *gp, *upp, _ptr(gate_bias), _ptr(up_bias), act, _ptr(x), _dt(x), _ptr(h),
                                      _ptr(gate_pre), _ptr(up_pre), M, N, K, _ptr(ws), n, _handle(stream, x)))
    return h if gate_pre is None else (h, gate_pre, up_pre)


def q4_gated_backward_workspace_size(M, N, K, fmt=Q4_FMT_Q4_0) -> int:
    return int(lib().q4_gated_backward_workspace_size(fmt, M, N, K))


def q4_gated_backward(gate, up, dh, gate_pre, up_pre, act=Q4_ACT_SILU, bias_grad=False, dx=None, dgate=None, dup=None,
                      dgate_bias=None, dup_bias=None, workspace="auto", stream=None):
    """Gradients {"dx", "dgate", "dup", and with bias_grad "dgate_bias", "dup_bias"} of q4_gated."""
    fmt, N, K, gp, upp = _pair(gate, up)
    M = dh.shape[0]
    for t, name in ((dh, "dh"), (gate_pre, "gate_pre"), (up_pre, "up_pre"), (dgate, "dgate"), (dup, "dup")):
        _like(t, name, (M, N), dh.dtype)
    out = {"dx": _summed(dx, "dx", (M, K), dh.dtype, N, dh, stream),
           "dgate": _new((M, N), dh.dtype, dh, stream) if dgate is None else dgate,
           "dup": _new((M, N), dh.dtype, dh, stream) if dup is None else dup}
    for name, t in (("dgate_bias", dgate_bias), ("dup_bias", dup_bias)):
        if bias_grad or t is not None:
            out[name] = _summed(t, name, (N,), torch.float32, M, dh, stream)
    ws, n = _workspace(workspace, q4_gated_backward_workspace_size(M, N, K, fmt), dh, stream)
    _check("q4_gated_backward",
           lib().q4_gated_backward(fmt, *gp, *upp, act, _ptr(gate_pre), _ptr(up_pre), _ptr(dh), _dt(dh), _ptr(out["dx"]),
                                   _ptr(out["dgate"]), _ptr(out["dup"]), _ptr(out.get("dgate_bias")), _ptr(out.get("dup_bias")),
                                   M, N, K, _ptr(ws), n, _handle(stream, dh)))
    return out


# ---- norms ----------------------------------------------------------------------

def _gate_rows(gate, gate_rows, M):
    """Rows of the activations that share one gate row (the rows of a gate of
    G rows when the caller does not say: M / G)."""
    if gate is None:
        return 1
    G = gate.shape[0]
    if gate_rows is None:
        if M == 0:
            return 1
        if G < 1 or M % G:
            raise ValueError(f"a gate of {G} rows does not divide {M} rows: pass gate_rows")
        gate_rows = M // G
    if gate_rows < 1 or G != -(-M // gate_rows):
        raise ValueError(f"a gate of {G} rows does not fit {M} rows, {gate_rows} to each")
    return gate_rows


def _code(dtype):
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    return _DT[dtype]


def _vectors(D, dtype, **named):
    for name, t in named.items():
        _like(t, name, (D,), dtype)


def block_norm(r, y=None, pre_norm=Q4_NORM_RMS, pre_weight=None, pre_bias=None, post_norm=Q4_NORM_NONE,
               post_weight=None, post_bias=None, gate=None, gate_rows=None, scale=1.0, eps=1e-5, save_stats=False,
               dtype=None, r_out=None, n=None, stats=None, stream=None):
    """r' = r + scale * gate * post(y), n = pre(r').

    Returns (r', n, stats): n is None with pre_norm Q4_NORM_NONE, stats
    (float32 [M, 4]) is None unless asked for; without y, r' is r itself.
    The type of n is y's; without y `dtype` (by default r's)."""
    M, D = r.shape
    dt = y.dtype if y is not None else (dtype or r.dtype)
    if y is not None:
        _like(y, "y", (M, D), dt)
        r_out = _out(r_out, "r_out", (M, D), r.dtype, r, stream)
    _vectors(D, dt, pre_weight=pre_weight, pre_bias=pre_bias, post_weight=post_weight, post_bias=post_bias)
    rows = _gate_rows(gate, gate_rows, M)
    if gate is not None:
        _like(gate, "gate", (gate.shape[0], D), dt)
    if pre_norm != Q4_NORM_NONE:
        n = _out(n, "n", (M, D), dt, r, stream)
    if stats is None and save_stats:
        stats = _new((M, 4), torch.float32, r, stream)
    _like(stats, "stats", (M, 4), torch.float32)
    _check("block_norm",
           lib().block_norm(_ptr(y), _ptr(r), _code(dt), _dt(r), M, D, post_norm, _ptr(post_weight), _ptr(post_bias), _ptr(gate),
                            rows, scale, pre_norm, _ptr(pre_weight), _ptr(pre_bias), eps, _ptr(r_out), _ptr(n), _ptr(stats),
                            _handle(stream, r)))
    return r if y is None else r_out, n, stats


def block_norm_backward_workspace_size(M, D, gate_rows=1) -> int:
    return int(lib().block_norm_backward_workspace_size(M, D, gate_rows))


def block_norm_backward(r_out, y, stats, dn=None, dr_out=None, pre_norm=Q4_NORM_RMS, pre_weight=None, pre_bias=None,
                        post_norm=Q4_NORM_NONE, post_weight=None, post_bias=None, gate=None, gate_rows=None, scale=1.0,
                        dtype=None, workspace="auto", stream=None):
    """Gradients of block_norm from r' (as stored), y, the statistics and the
    gradients of n and r': a dict of "dr", "dy" (with y), "dgate" (with a
    gate), and float32 "pre_dw", "post_dw" (where there is a weight), "pre_db",
    "post_db" (where there is a bias)."""
    M, D = r_out.shape
    dt = y.dtype if y is not None else dn.dtype if dn is not None else (dtype or r_out.dtype)
    for t, name, d in ((y, "y", dt), (dn, "dn", dt), (dr_out, "dr_out", r_out.dtype)):
        _like(t, name, (M, D), d)
    _like(stats, "stats", (M, 4), torch.float32)
    _vectors(D, dt, pre_weight=pre_weight, pre_bias=pre_bias, post_weight=post_weight, post_bias=post_bias)
    rows = _gate_rows(gate, gate_rows, M)
    out = {"dr": _new((M, D), r_out.dtype, r_out, stream)}
    if y is not None:
        out["dy"] = _new((M, D), dt, r_out, stream)
    if gate is not None:
        _like(gate, "gate", (gate.shape[0], D), dt)
        out["dgate"] = _summed(None, "dgate", gate.shape, dt, M, r_out, stream)
    for name, t in (("pre_dw", pre_weight), ("pre_db", pre_bias), ("post_dw", post_weight), ("post_db", post_bias)):
        if t is not None:
            out[name] = _summed(None, name, (D,), torch.float32, M, r_out, stream)
    ws, n = _workspace(workspace, block_norm_backward_workspace_size(M, D, rows), r_out, stream)
    _check("block_norm_backward",
           lib().block_norm_backward(_ptr(y), _ptr(r_out), _ptr(stats), _ptr(dn), _ptr(dr_out), _code(dt), _dt(r_out), M, D,
                                     post_norm, _ptr(post_weight), _ptr(post_bias), _ptr(gate), rows, scale, pre_norm,
                                     _ptr(pre_weight), _ptr(out["dr"]), _ptr(out.get("dy")), _ptr(out.get("dgate")),
                                     _ptr(out.get("pre_dw")), _ptr(out.get("pre_db")), _ptr(out.get("post_dw")),
                                     _ptr(out.get("post_db")), _ptr(ws), n, _handle(stream, r_out)))
    return out
