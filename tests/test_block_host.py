"""Host-only checks of the feed-forward operators' C ABI (include/q4_block.h):
exports, and every refusal before any HIP call (fake, never dereferenced
pointers are enough to reach them); and the binary64 reference's gradients
against differences."""
import math
import os
import re

import pytest
import torch

import block_reference as R
from gemv_q4_affine_amd import binding as B
from gemv_q4_affine_amd import block as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, MIS = 0x10000, 0x10008
BIG = 1 << 40


def test_every_declared_function_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "q4_block.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|int64_t)\s+([a-z_0-9]+)\s*\(", text, flags=re.M))
    assert len(names) == 11 and names == set(K.SIGNATURES)
    assert all(hasattr(K.lib(), n) for n in names)


def linear(fmt=0, q=P, s=P, b=None, bias=None, act=0, res=None, x=P, dt=B.Q4_BF16, y=P, pre=None, M=4, N=64, K_=64,
           ws=P, n=BIG):
    return K.lib().q4_linear(fmt, q, s, b, bias, act, res, x, dt, y, pre, M, N, K_, ws, n, None)


def linear_backward(fmt=0, q=P, s=P, b=None, act=1, pre=P, dy=P, dt=B.Q4_BF16, dx=P, dz=None, db=None, M=4, N=64, K_=64,
                    ws=P, n=BIG):
    return K.lib().q4_linear_backward(fmt, q, s, b, act, pre, dy, dt, dx, dz, db, M, N, K_, ws, n, None)


def gated(fmt=0, g=(P, P, None), u=(P, P, None), act=1, x=P, dt=B.Q4_BF16, h=P, gp=None, up=None, M=4, N=64, K_=64, ws=P,
          n=BIG, bg=None, bu=None):
    return K.lib().q4_gated(fmt, *g, *u, bg, bu, act, x, dt, h, gp, up, M, N, K_, ws, n, None)


def gated_backward(fmt=0, g=(P, P, None), u=(P, P, None), act=1, gp=P, up=P, dh=P, dt=B.Q4_BF16, dx=P, dg=None, du=None,
                   M=4, N=64, K_=64, ws=P, n=BIG):
    return K.lib().q4_gated_backward(fmt, *g, *u, act, gp, up, dh, dt, dx, dg, du, None, None, M, N, K_, ws, n, None)


@pytest.mark.parametrize("call", [linear, linear_backward, gated, gated_backward])
def test_product_refusals(call):
    assert call(fmt=3) == B.Q4_ERR_ARG and call(fmt=-1) == B.Q4_ERR_ARG
    assert call(act=5) == B.Q4_ERR_ARG and call(act=-1) == B.Q4_ERR_ARG
    for dt in (B.Q4_F32, 7, -1):
        assert call(dt=dt) == B.Q4_ERR_DTYPE
    for bad in (dict(M=-1), dict(N=-1), dict(K_=0), dict(K_=48), dict(K_=-64), dict(M=(1 << 30) + 1), dict(N=1 << 31),
                dict(fmt=1, K_=96)):
        assert call(**bad) == B.Q4_ERR_SHAPE, bad
    assert call(M=0) == B.Q4_OK and call(N=0) == B.Q4_OK


def test_product_pointers():
    for name in ("q", "s", "x", "y"):
        assert linear(**{name: None}) == B.Q4_ERR_NULL
        assert linear(**{name: MIS}) == B.Q4_ERR_ALIGN
    assert linear(fmt=1) == B.Q4_ERR_NULL                    # affine weights need their biases
    for name in ("bias", "res", "pre"):
        assert linear(**{name: MIS}) == B.Q4_ERR_ALIGN
    for name in ("q", "s", "pre", "dy", "dx"):
        assert linear_backward(**{name: None}) == B.Q4_ERR_NULL
    assert linear_backward(dt=B.Q4_F16) == B.Q4_ERR_DTYPE and gated_backward(dt=B.Q4_F16) == B.Q4_ERR_DTYPE
    assert linear_backward(act=0, pre=None, dz=P) == B.Q4_ERR_ARG
    assert gated(gp=P) == B.Q4_ERR_ARG and gated(up=P) == B.Q4_ERR_ARG
    assert gated(g=(P, None, None)) == B.Q4_ERR_NULL and gated(u=(P, MIS, None)) == B.Q4_ERR_ALIGN
    assert gated(fmt=2, g=(P, P, P)) == B.Q4_ERR_NULL
    for name in ("gp", "up", "dh", "dx"):
        assert gated_backward(**{name: None}) == B.Q4_ERR_NULL
    assert gated_backward(dg=MIS) == B.Q4_ERR_ALIGN


@pytest.mark.parametrize("call,size", [(linear, "q4_linear"), (gated, "q4_gated"), (linear_backward, "q4_linear_backward"),
                                       (gated_backward, "q4_gated_backward")])
def test_product_workspaces(call, size):
    for M in (4, 500):
        n = getattr(K, size + "_workspace_size")(M, 256, 512)
        assert n >= 0
        if n:
            assert call(M=M, N=256, K_=512, ws=None, n=n) == B.Q4_ERR_WORKSPACE
            assert call(M=M, N=256, K_=512, n=n - 1) == B.Q4_ERR_WORKSPACE
            assert call(M=M, N=256, K_=512, ws=MIS, n=n) == B.Q4_ERR_ALIGN
    f = getattr(K, size + "_workspace_size")
    assert f(0, 256, 512) == f(4, 256, 100) == f(-1, 256, 512) == f(4, 256, 512, 9) == 0


def norm(y=P, r=P, dt=B.Q4_BF16, rt=B.Q4_BF16, M=4, D=64, post=1, pw=None, pb=None, gate=None, rows=1, scale=1.0, pre=1,
         prew=None, preb=None, eps=1e-5, ro=P, n=P, st=None):
    return K.lib().block_norm(y, r, dt, rt, M, D, post, pw, pb, gate, rows, scale, pre, prew, preb, eps, ro, n, st, None)


def norm_backward(y=P, ro=P, st=P, dn=P, dro=P, dt=B.Q4_BF16, rt=B.Q4_BF16, M=4, D=64, post=1, pw=None, pb=None, gate=None,
                  rows=1, scale=1.0, pre=1, prew=None, dr=P, dy=P, dgate=None, predw=None, predb=None, postdw=None,
                  postdb=None, ws=P, n=BIG):
    return K.lib().block_norm_backward(y, ro, st, dn, dro, dt, rt, M, D, post, pw, pb, gate, rows, scale, pre, prew, dr, dy,
                                       dgate, predw, predb, postdw, postdb, ws, n, None)


@pytest.mark.parametrize("call", [norm, norm_backward])
def test_norm_refusals(call):
    assert call(dt=3) == B.Q4_ERR_DTYPE
    assert call(dt=B.Q4_BF16, rt=B.Q4_F16) == B.Q4_ERR_DTYPE and call(dt=B.Q4_F32, rt=B.Q4_BF16) == B.Q4_ERR_DTYPE
    for bad in (dict(M=-1), dict(D=-1), dict(D=32769), dict(M=1 << 31)):
        assert call(**bad) == B.Q4_ERR_SHAPE
    for bad in (dict(post=3), dict(pre=-1), dict(scale=math.inf), dict(scale=math.nan), dict(rows=0), dict(rows=-2),
                dict(post=0, pw=P), dict(post=0, pb=P) if call is norm else dict(post=0, postdb=P),
                dict(pre=0, prew=P), dict(y=None)):
        assert call(**bad) == B.Q4_ERR_ARG, bad
    assert call(M=0) == B.Q4_OK and call(D=0) == B.Q4_OK


def test_norm_pointers():
    for bad in (dict(r=None), dict(ro=None), dict(n=None)):
        assert norm(**bad) == B.Q4_ERR_NULL
    for bad in (dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(pre=0), dict(y=None, post=0),
                dict(y=None, post=0, ro=None, gate=P)):
        assert norm(**bad) == B.Q4_ERR_ARG, bad
    for name in ("y", "r", "ro", "n", "st", "gate", "pw", "pb", "prew", "preb"):
        assert norm(**{name: MIS}) == B.Q4_ERR_ALIGN, name
    for bad in (dict(ro=None), dict(st=None), dict(dr=None), dict(dy=None), dict(dn=None), dict(pre=0, dn=None, dro=None)):
        assert norm_backward(**bad) == B.Q4_ERR_NULL, bad
    assert norm_backward(dgate=P) == B.Q4_ERR_ARG and norm_backward(pre=0, dn=None, predw=P) == B.Q4_ERR_ARG
    for name in ("y", "ro", "st", "dn", "dro", "dr", "dy", "predw", "postdb"):
        assert norm_backward(**{name: MIS}) == B.Q4_ERR_ALIGN, name
    n = K.block_norm_backward_workspace_size(4, 64, 1)
    if n:
        assert norm_backward(ws=None) == B.Q4_ERR_WORKSPACE and norm_backward(n=n - 1) == B.Q4_ERR_WORKSPACE
        assert norm_backward(ws=MIS) == B.Q4_ERR_ALIGN


def test_binding_refusals():
    q, d = torch.zeros(64, 2, 16, dtype=torch.uint8), torch.zeros(64, 2, dtype=torch.int16)
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        K.q4_linear((q, d, d, d), x)
    with pytest.raises(ValueError):
        K._like(x, "x", (3, 32), torch.bfloat16)
    with pytest.raises(ValueError):
        K._like(x, "x", (3, 64), torch.float16)
    with pytest.raises(ValueError):
        K.q4_linear((q, d), x)                       # not on the GPU
    with pytest.raises(ValueError):
        K._gate_rows(torch.zeros(2, 8), None, 5)
    with pytest.raises(ValueError):
        K._gate_rows(torch.zeros(2, 8), 2, 5)
    assert K._gate_rows(torch.zeros(3, 8), 2, 5) == 2 and K._gate_rows(torch.zeros(5, 8), None, 5) == 1
    with pytest.raises(ValueError):
        K._workspace("none", 4, x, None)


@pytest.mark.parametrize("kind", ["none", "silu", "gelu", "gelu_tanh", "relu"])
def test_reference_slopes_against_differences(kind):
    z = torch.linspace(-9, 9, 1801, dtype=torch.float64) + 1e-3
    eps = 1e-6
    diff = (R.act(z + eps, kind)[0] - R.act(z - eps, kind)[0]) / (2 * eps)
    assert (R.act(z, kind)[1] - diff).abs().max() < 1e-8


@pytest.mark.parametrize("fmt", R.FMTS)
def test_reference_planes_follow_the_formats(fmt):
    """The planes' binary64 values against the oracle's dequantisers."""
    import numpy as np
    import oracle
    p, W = R.planes(fmt, 5, 192, 1)
    p = [t if t.dtype == np.uint8 else t.view(np.uint16) for t in p]
    if fmt == "q4_0":
        want = oracle.q4_0_dequantize(p[0], p[1])
    else:
        want = (oracle.affine4_dequantize if fmt == "affine4" else oracle.affine8_dequantize)(*p)
    assert np.array_equal(W.numpy().astype(np.float32), np.asarray(want, np.float32).reshape(5, 192))
