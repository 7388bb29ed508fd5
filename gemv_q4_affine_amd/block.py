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

from .binding import (Q4_FMT_AFFINE4, Q4_FMT_AFFINE8, Q4_FMT_Q4_0, _alloc_stream, _check, _dt, _empty, _p, _stream, lib as _base_lib)

Q4_ACT_NONE, Q4_ACT_SILU, Q4_ACT_GELU, Q4_ACT_GELU_TANH, Q4_ACT_RELU = 0, 1, 2, 3, 4
Q4_NORM_NONE, Q4_NORM_RMS, Q4_NORM_LAYER = 0, 1, 2
Q4_NORM_MAX_D = 32768

_P, _I64, _INT, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
SIGNATURES = {
    "q4_linear_workspace_size": (_I64, [_INT, _I64, _I64, _I64]),
    "q4_linear": (_INT, [_INT, _P, _P, _P, _P, _INT, _P, _P, _INT, _P, _P, _I64, _I64, _I64, _P, _I64, _P]),
    "q4_linear_backward_workspace_size": (_I64, [_INT, _I64, _I64, _I64]),
    "q4_linear_backward": (_INT, [_INT, _P, _P, _P, _INT, _P, _P, _INT, _P, _P, _P, _I64, _I64, _I64, _P, _I64, _P]),
    "q4_gated_workspace_size": (_I64, [_INT, _I64, _I64, _I64]),
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


def _planes(w, fmt=None):
    """(format, N, K, three plane pointers) of a weight tuple."""
    if len(w) not in (2, 3):
        raise ValueError("a weight is (qs, d) or (codes, scales, biases)")
    q, s = w[0], w[1]
    if fmt is None:
        fmt = Q4_FMT_Q4_0 if len(w) == 2 else Q4_FMT_AFFINE8 if q.shape[-1] == s.shape[1] * 64 else Q4_FMT_AFFINE4
    N, K = s.shape[0], s.shape[1] * (32 if fmt == Q4_FMT_Q4_0 else 64)
    want = {Q4_FMT_Q4_0: N * K // 2, Q4_FMT_AFFINE4: N * K // 2, Q4_FMT_AFFINE8: N * K}[fmt]
    if q.numel() * q.element_size() != want or any(t.shape != s.shape for t in w[2:]):
        raise ValueError("the planes of a weight do not fit each other")
    return fmt, N, K, (_p(q), _p(s), _p(w[2]) if len(w) == 3 else None)


def _like(t, name, shape, dtype):
    """An optional tensor of the given shape and dtype (raw pointers pass through)."""
    if isinstance(t, torch.Tensor) and (tuple(t.shape) != tuple(shape) or t.dtype != dtype):
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, not {t.dtype} {tuple(t.shape)}")
    return t


def _workspace(workspace, n, like, stream):
    """"auto": n bytes owned by the call's stream (None if n is 0); else the caller's tensor or None."""
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace must be 'auto', None or a tensor, not {workspace!r}")
        workspace = _empty((n,), torch.uint8, like, stream) if n > 0 else None
    return workspace, workspace.numel() * workspace.element_size() if workspace is not None else 0


def _summed(t, name, shape, dtype, terms, like, stream):
    """An output that sums over `terms` rows or columns: allocated if None,
    and zero where there are none (the library writes nothing then)."""
    t = _empty(shape, dtype, like, stream) if t is None else _like(t, name, shape, dtype)
    if terms == 0 and t.numel():
        with torch.cuda.stream(_alloc_stream(stream)):
            t.zero_()
    return t


# ---- linear ---------------------------------------------------------------------

def q4_linear_workspace_size(M, N, K, fmt=Q4_FMT_Q4_0) -> int:
    return int(lib().q4_linear_workspace_size(fmt, M, N, K))


def q4_linear(w, x, bias=None, act=Q4_ACT_NONE, residual=None, save_pre=False, y=None, pre=None, workspace="auto",
              stream=None):
    """y [M, N] = act(x . W^T + bias) + residual; with save_pre (or a `pre`
    tensor) also the values before the activation: (y, pre)."""
    fmt, N, K, wp = _planes(w)
    M = x.shape[0]
    _like(x, "x", (M, K), x.dtype)
    _like(bias, "bias", (N,), x.dtype)
    _like(residual, "residual", (M, N), x.dtype)
    y = _empty((M, N), x.dtype, x, stream) if y is None else _like(y, "y", (M, N), x.dtype)
    if pre is None and save_pre:
        pre = _empty((M, N), x.dtype, x, stream)
    _like(pre, "pre", (M, N), x.dtype)
    ws, n = _workspace(workspace, q4_linear_workspace_size(M, N, K, fmt), x, stream)
    _check("q4_linear", lib().q4_linear(fmt, *wp, _p(bias), act, _p(residual), _p(x), _dt(x), _p(y), _p(pre), M, N, K,
                                        _p(ws), n, _stream(stream)))
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
    if act != Q4_ACT_NONE:
        out["dz"] = _empty((M, N), dy.dtype, dy, stream) if dz is None else _like(dz, "dz", (M, N), dy.dtype)
    if bias_grad or dbias is not None:
        out["dbias"] = _summed(dbias, "dbias", (N,), torch.float32, M, dy, stream)
    ws, n = _workspace(workspace, q4_linear_backward_workspace_size(M, N, K, fmt), dy, stream)
    _check("q4_linear_backward",
           lib().q4_linear_backward(fmt, *wp, act, _p(pre), _p(dy), _dt(dy), _p(out["dx"]), _p(out.get("dz")),
                                    _p(out.get("dbias")), M, N, K, _p(ws), n, _stream(stream)))
    return out


# ---- gated ----------------------------------------------------------------------

def q4_gated_workspace_size(M, N, K, fmt=Q4_FMT_Q4_0) -> int:
    return int(lib().q4_gated_workspace_size(fmt, M, N, K))


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
    h = _empty((M, N), x.dtype, x, stream) if h is None else _like(h, "h", (M, N), x.dtype)
    if save_pre:
        gate_pre = _empty((M, N), x.dtype, x, stream) if gate_pre is None else gate_pre
        up_pre = _empty((M, N), x.dtype, x, stream) if up_pre is None else up_pre
    _like(gate_pre, "gate_pre", (M, N), x.dtype)
    _like(up_pre, "up_pre", (M, N), x.dtype)
    ws, n = _workspace(workspace, q4_gated_workspace_size(M, N, K, fmt), x, stream)
    _check("q4_gated", lib().q4_gated(fmt, *gp, *upp, _p(gate_bias), _p(up_bias), act, _p(x), _dt(x), _p(h),
                                      _p(gate_pre), _p(up_pre), M, N, K, _p(ws), n, _stream(stream)))
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
           "dgate": _empty((M, N), dh.dtype, dh, stream) if dgate is None else dgate,
           "dup": _empty((M, N), dh.dtype, dh, stream) if dup is None else dup}
    for name, t in (("dgate_bias", dgate_bias), ("dup_bias", dup_bias)):
        if bias_grad or t is not None:
            out[name] = _summed(t, name, (N,), torch.float32, M, dh, stream)
    ws, n = _workspace(workspace, q4_gated_backward_workspace_size(M, N, K, fmt), dh, stream)
    _check("q4_gated_backward",
           lib().q4_gated_backward(fmt, *gp, *upp, act, _p(gate_pre), _p(up_pre), _p(dh), _dt(dh), _p(out["dx"]),
                                   _p(out["dgate"]), _p(out["dup"]), _p(out.get("dgate_bias")), _p(out.get("dup_bias")),
                                   M, N, K, _p(ws), n, _stream(stream)))
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
        r_out = _empty((M, D), r.dtype, r, stream) if r_out is None else _like(r_out, "r_out", (M, D), r.dtype)
    _vectors(D, dt, pre_weight=pre_weight, pre_bias=pre_bias, post_weight=post_weight, post_bias=post_bias)
    rows = _gate_rows(gate, gate_rows, M)
    if gate is not None:
        _like(gate, "gate", (gate.shape[0], D), dt)
    if pre_norm != Q4_NORM_NONE:
        n = _empty((M, D), dt, r, stream) if n is None else _like(n, "n", (M, D), dt)
    if stats is None and save_stats:
        stats = _empty((M, 4), torch.float32, r, stream)
    _like(stats, "stats", (M, 4), torch.float32)
    _check("block_norm",
           lib().block_norm(_p(y), _p(r), _code(dt), _dt(r), M, D, post_norm, _p(post_weight), _p(post_bias), _p(gate),
                            rows, scale, pre_norm, _p(pre_weight), _p(pre_bias), eps, _p(r_out), _p(n), _p(stats),
                            _stream(stream)))
    return r if y is None else r_out, n, stats


def _code(dtype):
    return _dt(torch.empty(0, dtype=dtype))


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
    out = {"dr": _empty((M, D), r_out.dtype, r_out, stream)}
    if y is not None:
        out["dy"] = _empty((M, D), dt, r_out, stream)
    if gate is not None:
        out["dgate"] = _empty(_like(gate, "gate", (gate.shape[0], D), dt).shape, dt, r_out, stream)
    for name, t in (("pre_dw", pre_weight), ("pre_db", pre_bias), ("post_dw", post_weight), ("post_db", post_bias)):
        if t is not None:
            out[name] = _summed(None, name, (D,), torch.float32, M, r_out, stream)
    ws, n = _workspace(workspace, block_norm_backward_workspace_size(M, D, rows), r_out, stream)
    _check("block_norm_backward",
           lib().block_norm_backward(_p(y), _p(r_out), _p(stats), _p(dn), _p(dr_out), _code(dt), _dt(r_out), M, D,
                                     post_norm, _p(post_weight), _p(post_bias), _p(gate), rows, scale, pre_norm,
                                     _p(pre_weight), _p(out["dr"]), _p(out.get("dy")), _p(out.get("dgate")),
                                     _p(out.get("pre_dw")), _p(out.get("pre_db")), _p(out.get("post_dw")),
                                     _p(out.get("post_db")), _p(ws), n, _stream(stream)))
    return out
