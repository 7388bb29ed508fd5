"""Host-only checks of the operators on microscaled numbers (include/q4_mx.h):
exports, every refusal before any HIP call (fake, never dereferenced pointers
are enough to reach them), and the binary64 quantiser against its definition."""
import os
import re

import numpy as np
import pytest
import torch

import mx_reference as X
from gemv_q4_affine_amd import binding as B
from gemv_q4_affine_amd import mx as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, MIS = 0x10000, 0x10008
BIG = 1 << 42
FP4, FP8 = K.Q4_MXFP4, K.Q4_MXFP8


def test_every_declared_function_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "q4_mx.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|int64_t)\s+([a-z_0-9]+)\s*\(", text, flags=re.M))
    assert len(names) == 11 and names == set(K.SIGNATURES)
    assert all(hasattr(K.lib(), n) for n in names)


def quantize(v=P, dt=B.Q4_BF16, kind=FP8, q=P, s=P, M=4, K_=64):
    return K.lib().mx_quantize(v, dt, kind, q, s, M, K_, None)


def dequantize(v=P, dt=B.Q4_BF16, kind=FP8, q=P, s=P, M=4, K_=64):
    return K.lib().mx_dequantize(kind, q, s, v, dt, M, K_, None)


def linear(q=P, s=P, bias=None, act=0, res=None, xt=FP8, x=P, xs=P, dt=B.Q4_BF16, y=P, pre=None, M=4, N=64, K_=64, ws=P, n=BIG):
    return K.lib().mx_linear(q, s, bias, act, res, xt, x, xs, dt, y, pre, M, N, K_, ws, n, None)


def gated(q=P, s=P, uq=P, us=P, bias=None, ubias=None, act=1, xt=FP8, x=P, xs=P, dt=B.Q4_BF16, y=P, gp=None, up=None, M=4, N=64,
          K_=64, ws=P, n=BIG):
    return K.lib().mx_gated(q, s, uq, us, bias, ubias, act, xt, x, xs, dt, y, gp, up, M, N, K_, ws, n, None)


def linear_backward(q=P, s=P, act=1, pre=P, dy=P, dt=B.Q4_BF16, dx=P, dz=None, db=None, M=4, N=64, K_=64, ws=P, n=BIG):
    return K.lib().mx_linear_backward(q, s, act, pre, dy, dt, dx, dz, db, M, N, K_, ws, n, None)


def gated_backward(q=P, s=P, uq=P, us=P, act=1, gp=P, up=P, dh=P, dt=B.Q4_BF16, dx=P, dg=None, du=None, M=4, N=64, K_=64, ws=P,
                   n=BIG):
    return K.lib().mx_gated_backward(q, s, uq, us, act, gp, up, dh, dt, dx, dg, du, None, None, M, N, K_, ws, n, None)


def norm(y=P, r=P, dt=B.Q4_BF16, rdt=B.Q4_BF16, M=4, D=64, post=0, pw=None, pb=None, gate=None, rows=1, scale=1.0, pre=1, w=None,
         b=None, eps=1e-5, ro=P, kind=FP8, q=P, s=P, st=None):
    return K.lib().block_norm_mx(y, r, dt, rdt, M, D, post, pw, pb, gate, rows, scale, pre, w, b, eps, ro, kind, q, s, st, None)


@pytest.mark.parametrize("call", [quantize, dequantize])
def test_plane_refusals(call):
    for bad in (dict(dt=7), dict(dt=-1), dict(kind=0), dict(kind=10), dict(kind=B.Q4_BF16)):
        assert call(**bad) == B.Q4_ERR_DTYPE, bad
    for bad in (dict(M=-1), dict(K_=0), dict(K_=-32), dict(K_=48), dict(M=(1 << 30) + 1), dict(K_=(1 << 30) + 32)):
        assert call(**bad) == B.Q4_ERR_SHAPE, bad
    for name in ("v", "q", "s"):
        assert call(**{name: None}) == B.Q4_ERR_NULL and call(**{name: MIS}) == B.Q4_ERR_ALIGN
    assert call(M=0, v=None, q=None, s=None) == B.Q4_OK


@pytest.mark.parametrize("call", [linear, gated, linear_backward, gated_backward])
def test_product_refusals(call):
    assert call(act=5) == B.Q4_ERR_ARG and call(act=-1) == B.Q4_ERR_ARG
    for dt in (B.Q4_F32, FP8, 7, -1):
        assert call(dt=dt) == B.Q4_ERR_DTYPE
    for bad in (dict(M=-1), dict(N=-1), dict(K_=0), dict(K_=48), dict(K_=-64), dict(M=(1 << 30) + 1), dict(N=(1 << 25) + 1),
                dict(K_=(1 << 25) + 32)):
        assert call(**bad) == B.Q4_ERR_SHAPE, bad
    assert call(M=0, q=None) == B.Q4_OK and call(N=0, q=None) == B.Q4_OK
    for name in ("q", "s"):
        assert call(**{name: None}) == B.Q4_ERR_NULL and call(**{name: MIS}) == B.Q4_ERR_ALIGN


@pytest.mark.parametrize("call", [linear, gated])
def test_forward_pointers_and_types(call):
    for name in ("x", "y"):
        assert call(**{name: None}) == B.Q4_ERR_NULL and call(**{name: MIS}) == B.Q4_ERR_ALIGN
    assert call(xs=None) == B.Q4_ERR_NULL and call(xs=MIS) == B.Q4_ERR_ALIGN          # an MX x has scales,
    assert call(xt=B.Q4_BF16) == B.Q4_ERR_ARG                                           # a 16-bit one none
    assert call(xt=B.Q4_F16, xs=None) == B.Q4_ERR_DTYPE                                 # and its type is the outputs'
    assert call(xt=B.Q4_BF16, xs=None, dt=B.Q4_F16) == B.Q4_ERR_DTYPE
    for xt in (B.Q4_F32, 3, 10):
        assert call(xt=xt) == B.Q4_ERR_DTYPE
    assert call(bias=MIS) == B.Q4_ERR_ALIGN


def test_other_pointers():
    for name in ("res", "pre"):
        assert linear(**{name: MIS}) == B.Q4_ERR_ALIGN
    assert gated(gp=P) == B.Q4_ERR_ARG and gated(up=P) == B.Q4_ERR_ARG and gated(gp=MIS, up=P) == B.Q4_ERR_ALIGN
    for name in ("uq", "us"):
        assert gated(**{name: None}) == B.Q4_ERR_NULL and gated_backward(**{name: MIS}) == B.Q4_ERR_ALIGN
    for name in ("pre", "dy", "dx"):
        assert linear_backward(**{name: None}) == B.Q4_ERR_NULL
    for name in ("gp", "up", "dh", "dx"):
        assert gated_backward(**{name: None}) == B.Q4_ERR_NULL
    assert linear_backward(dt=B.Q4_F16) == gated_backward(dt=B.Q4_F16) == B.Q4_ERR_DTYPE
    assert linear_backward(act=0, pre=None, dz=P) == B.Q4_ERR_ARG
    assert gated_backward(dg=MIS) == B.Q4_ERR_ALIGN


@pytest.mark.parametrize("call,size", [(linear, "mx_linear"), (gated, "mx_gated"), (linear_backward, "mx_linear_backward"),
                                       (gated_backward, "mx_gated_backward")])
def test_workspaces(call, size):
    f = getattr(K, size + "_workspace_size")
    kinds = [dict()] if "backward" in size else [dict(x_type=t) for t in (FP8, FP4, B.Q4_BF16)]
    for kind in kinds:
        more = {} if not kind else dict(xt=kind["x_type"], xs=P if kind["x_type"] in (FP4, FP8) else None)
        for M, N, K_ in ((4, 256, 512), (32, 64, 32768), (64, 256, 8192), (500, 256, 512), (4096, 12288, 4096)):
            n = f(M, N, K_, **kind)
            assert n >= 0
            if n:
                assert call(M=M, N=N, K_=K_, ws=None, n=n, **more) == B.Q4_ERR_WORKSPACE
                assert call(M=M, N=N, K_=K_, n=n - 1, **more) == B.Q4_ERR_WORKSPACE
                assert call(M=M, N=N, K_=K_, ws=MIS, n=n, **more) == B.Q4_ERR_ALIGN
        assert f(0, 256, 512, **kind) == f(4, 256, 100, **kind) == f(-1, 256, 512, **kind) == f(4, 0, 512, **kind) == 0
    if kinds[0]:
        assert f(500, 256, 512, x_type=B.Q4_F32) == f(500, 256, 512, x_type=77) == 0


def test_norm_refusals():
    for bad in (dict(dt=5), dict(rdt=B.Q4_F16), dict(dt=B.Q4_F32), dict(kind=0), dict(kind=B.Q4_F16)):
        assert norm(**bad) == B.Q4_ERR_DTYPE, bad
    for bad in (dict(M=-1), dict(D=-32), dict(D=48), dict(D=32800), dict(M=(1 << 30) + 1)):
        assert norm(**bad) == B.Q4_ERR_SHAPE, bad
    for bad in (dict(pre=0), dict(pre=3), dict(post=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(scale=float("inf")), dict(rows=0), dict(pw=P), dict(pb=P), dict(y=None), dict(y=None, ro=None, gate=P),
                dict(y=None, ro=None, post=1)):
        assert norm(**bad) == B.Q4_ERR_ARG, bad
    for name in ("r", "q", "s", "ro"):
        assert norm(**{name: None}) == B.Q4_ERR_NULL, name
    for name in ("y", "r", "q", "s", "ro", "gate", "w", "b", "st"):
        assert norm(**{name: MIS}) == B.Q4_ERR_ALIGN, name
    assert norm(M=0, r=None) == norm(D=0, r=None) == B.Q4_OK


def test_python_refusals():
    q = lambda R, C: torch.zeros(R, C, dtype=torch.uint8)  # noqa: E731
    w, x8 = (q(8, 32), q(8, 2)), (q(3, 64), q(3, 2))
    for bad in ((q(8, 64), q(8, 2)), (q(8, 33), q(8, 2)), (q(7, 32), q(8, 2)), (q(8, 32).short(), q(8, 2)), (q(8, 32),),
                (q(8, 32), q(8, 2), q(8, 2))):
        with pytest.raises(ValueError):
            K.mx_linear(bad, x8)
    with pytest.raises(ValueError):
        K.mx_linear(w, (q(3, 96), q(3, 3)))                                # another K
    with pytest.raises(ValueError):
        K.mx_linear(w, torch.zeros(3, 64).bfloat16(), dtype=torch.float16)
    with pytest.raises(ValueError):
        K.mx_gated(w, (q(9, 32), q(9, 2)), x8)
    with pytest.raises(ValueError):
        K.mx_quantize(torch.zeros(2, 48))
    with pytest.raises(ValueError):
        K.block_norm_mx(torch.zeros(2, 48))
    with pytest.raises(ValueError):                                           # a tensor of the host
        K.mx_linear(w, x8)
    with pytest.raises(TypeError):
        K.mx_linear(w, x8, dtype=torch.float64)


@pytest.mark.parametrize("kind", ["fp4", "fp8"])
def test_reference_quantiser(kind):
    """Nearest of all codes by search, ties to the even code, at every border of a block whose scale is 1."""
    t = np.unique(X.table(kind)[np.isfinite(X.table(kind))])
    mid = (t[1:] + t[:-1]) / 2
    v = np.concatenate([t, mid, np.nextafter(mid, 9e9), np.nextafter(mid, -9e9), [1.1 * t[-1], 1.12 * t[0]]])
    b = np.zeros((len(v), 32))
    b[:, 0], b[:, 1] = v, t[-1]                            # the largest magnitude sets the scale
    codes, scales = X.quantize(b, kind)
    assert (scales == 127).all()
    got = X.values(codes, scales, kind)[:, 0]
    finite = X.table(kind)[np.isfinite(X.table(kind))]
    for x, g, c in zip(v, got, codes[:, 0]):
        d = np.abs(finite - x)
        assert abs(g - x) == d.min()
        if (np.unique(finite[d == d.min()]).size) == 2:
            assert c % 2 == 0
    assert X.quantize(np.zeros((1, 32)), kind)[1][0, 0] == 0
    bad = np.ones((2, 64))
    bad[0, 3], bad[1, 40] = np.inf, np.nan
    codes, scales = X.quantize(bad, kind)
    assert scales[0, 0] == 255 and scales[1, 1] == 255 and scales[0, 1] != 255 and not codes[0, :32].any()
