"""The feed-forward operators (q4_linear, q4_gated, block_norm and their
gradients) on the GPU against the binary64 forms of block_reference.

Tolerances, from the arithmetic:
  * OUT: an output rounded once into its type is within u of its value, u =
    2^-8 (bfloat16), 2^-11 (binary16), 2^-24 (binary32); over many values the
    rounding errors' 2-norm is at most u and about 0.43 u.  Below binary16's
    normal range the spacing is 2^-24: an absolute error of up to 2^-25 each.
  * binary16 operands: weights (and scaled x or dz) rounded to 2^-11 relative,
    independent errors, so at most about 2^-11 of the result's 2-norm each.
  * binary32 sums of n terms: about sqrt(n) 2^-24, below 2^-17 here; the
    binary32 outputs (bias and weight gradients, statistics) are held to 2e-5.
"""
import numpy as np
import pytest
import torch

import block_reference as R
import gemv_q4_affine_amd as Q

pytestmark = pytest.mark.gpu

ACTS = {"none": Q.Q4_ACT_NONE, "silu": Q.Q4_ACT_SILU, "gelu": Q.Q4_ACT_GELU, "gelu_tanh": Q.Q4_ACT_GELU_TANH,
        "relu": Q.Q4_ACT_RELU}
NORMS = {"none": Q.Q4_NORM_NONE, "rms": Q.Q4_NORM_RMS, "layer": Q.Q4_NORM_LAYER}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
F32 = 2e-5


def bar(dtype, operands=2):
    """2-norm bound of an output of `dtype` on `operands` binary16-rounded operands."""
    return U[dtype] + operands * 2.0 ** -11


@pytest.fixture(autouse=True)
def _done():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    yield
    torch.cuda.synchronize()


def say(*a):
    print(*a, flush=True)


def weight(fmt, N, K, seed, scale=0.02):
    p, W = R.planes(fmt, N, K, seed, scale)
    return tuple(torch.from_numpy(np.ascontiguousarray(t)).cuda() for t in p), W


def rand(gen, *shape, dtype=torch.bfloat16, scale=1.0, mean=0.0):
    """A tensor on the GPU, and the same values in binary64 on the CPU."""
    t = (torch.randn(*shape, generator=gen) * scale + mean).to(dtype)
    return t.cuda(), t.double()


def near(got, want, limit, what):
    e = R.rel(got, want)
    if got.dtype == torch.float16 and want.norm() > 0:
        limit += 2.0 ** -25 * want.numel() ** 0.5 / want.norm().item()
    say(f"  {what}: {e:.3g} (limit {limit:.3g})")
    assert tuple(got.shape) == tuple(want.shape), what
    assert e <= limit, f"{what}: {e} > {limit}"


# ---- linear ----------------------------------------------------------------------

SHAPES = [(1, 64, 64), (1, 37, 2048), (2, 300, 320), (3, 1, 64), (7, 129, 4096), (16, 512, 576), (17, 33, 192),
          (32, 260, 1088), (33, 96, 64), (64, 255, 448), (65, 130, 128), (127, 512, 512), (130, 31, 2048), (300, 523, 704),
          (512, 2048, 256), (1000, 136, 1984)]


@pytest.mark.parametrize("fmt", R.FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(fmt, M, N, K):
    gen = torch.Generator().manual_seed(M * 31 + N)
    w, W = weight(fmt, N, K, M + N + K)
    for k, (act, bias, residual, save, dt) in enumerate([("none", False, False, False, torch.bfloat16),
                                                         ("gelu", True, True, True, torch.bfloat16),
                                                         ("silu", True, False, True, torch.float16)]):
        say(f"linear {fmt} M={M} N={N} K={K} {act} {dt}")
        x, x64 = rand(gen, M, K, dtype=dt)
        b, b64 = rand(gen, N, dtype=dt) if bias else (None, None)
        r, r64 = rand(gen, M, N, dtype=dt) if residual else (None, None)
        got = Q.q4_linear(w, x, bias=b, act=ACTS[act], residual=r, save_pre=save)
        y64, z64 = R.linear(x64, W, b64, act, r64)
        near(got[0] if save else got, y64, bar(dt), "y")
        if save:
            near(got[1], z64, bar(dt), "pre")
        again = Q.q4_linear(w, x, bias=b, act=ACTS[act], residual=r, save_pre=save)
        assert torch.equal(again[0] if save else again, got[0] if save else got), "not deterministic"


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("M", [1, 20, 200])
def test_linear_activations(act, M):
    gen = torch.Generator().manual_seed(M)
    N, K = 192, 128
    w, W = weight("affine4", N, K, 5, scale=0.3)          # |z| to about 10: both tails of the activations
    x, x64 = rand(gen, M, K, dtype=torch.float16)
    y, pre = Q.q4_linear(w, x, act=ACTS[act], save_pre=True)
    y64, z64 = R.linear(x64, W, None, act, None)
    near(y, y64, bar(torch.float16), act)
    assert pre.abs().max() > 5


@pytest.mark.parametrize("M", [1, 40, 150])
def test_linear_residual_in_place(M):
    gen = torch.Generator().manual_seed(M)
    N, K = 160, 256
    w, W = weight("q4_0", N, K, 1)
    x, _ = rand(gen, M, K)
    r, _ = rand(gen, M, N)
    want = Q.q4_linear(w, x, residual=r)
    got = Q.q4_linear(w, x, residual=r, y=r)
    assert got.data_ptr() == r.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("M", [4, 33, 200])
@pytest.mark.parametrize("fmt", R.FMTS)
def test_linear_wide_range_and_bad_rows(fmt, M):
    """Rows of very different magnitude keep their own precision, and a row
    with an infinity or a NaN spoils no other row."""
    gen = torch.Generator().manual_seed(M)
    N, K = 128, 256
    w, W = weight(fmt, N, K, 2)
    x, x64 = rand(gen, M, K)
    scale = torch.tensor([1e-30, 1e5, 1.0, 1e30])[torch.arange(M) % 4]
    x = (x.float() * scale[:, None].cuda()).bfloat16()
    x[1, 7] = float("inf")
    x[2, 9] = float("nan")
    y = Q.q4_linear(w, x).double().cpu()
    y64 = x.double().cpu() @ W.T
    for m in range(M):
        if m in (1, 2):
            assert not torch.isfinite(y[m]).any() or fmt == "q4_0" and not torch.isfinite(y[m][W[:, 7 if m == 1 else 9] != 0]).any()
        else:
            e = R.rel(y[m], y64[m])
            assert e <= bar(torch.bfloat16), (m, e)


def test_linear_zero_rows_and_columns():
    w, _ = weight("q4_0", 64, 64, 3)
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    assert Q.q4_linear(w, x).shape == (0, 64)
    out = Q.q4_linear_backward(w, torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), bias_grad=True)
    assert out["dx"].shape == (0, 64) and out["dbias"].abs().max() == 0
    none = tuple(t[:0] for t in w)
    assert Q.q4_linear(none, torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda")).shape == (5, 0)
    dx = Q.q4_linear_backward(none, torch.zeros(5, 0, dtype=torch.bfloat16, device="cuda"))["dx"]
    assert dx.shape == (5, 64) and dx.abs().max() == 0


@pytest.mark.parametrize("fmt", R.FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_backward(fmt, M, N, K):
    gen = torch.Generator().manual_seed(M * 7 + N)
    w, W = weight(fmt, N, K, M + 2 * N + K)
    for act in ("none", "gelu"):
        say(f"linear backward {fmt} M={M} N={N} K={K} {act}")
        dy, dy64 = rand(gen, M, N, scale=1e-3)
        pre, pre64 = rand(gen, M, N)
        out = Q.q4_linear_backward(w, dy, act=ACTS[act], pre=None if act == "none" else pre, bias_grad=True)
        dx, dz, db = R.linear_grad(W, dy64, pre64, act)
        near(out["dx"], dx, bar(torch.bfloat16), "dx")
        near(out["dbias"], db, F32, "dbias")
        if act != "none":
            near(out["dz"], dz, bar(torch.bfloat16, 0), "dz")
        again = Q.q4_linear_backward(w, dy, act=ACTS[act], pre=None if act == "none" else pre, bias_grad=True)
        assert all(torch.equal(out[k], again[k]) for k in out), "not deterministic"


# ---- gated -----------------------------------------------------------------------

@pytest.mark.parametrize("fmt", R.FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gated(fmt, M, N, K):
    gen = torch.Generator().manual_seed(M * 13 + N)
    (gw, Wg), (uw, Wu) = weight(fmt, N, K, M + N), weight(fmt, N, K, M + N + 1)
    for act, bias, save, dt in (("silu", False, False, torch.bfloat16), ("gelu_tanh", True, True, torch.bfloat16),
                                ("gelu", True, True, torch.float16)):
        say(f"gated {fmt} M={M} N={N} K={K} {act} {dt}")
        x, x64 = rand(gen, M, K, dtype=dt)
        (bg, bg64), (bu, bu64) = (rand(gen, N, dtype=dt), rand(gen, N, dtype=dt)) if bias else ((None, None), (None, None))
        got = Q.q4_gated(gw, uw, x, act=ACTS[act], gate_bias=bg, up_bias=bu, save_pre=save)
        h64, g64, u64 = R.gated(x64, Wg, Wu, bg64, bu64, act)
        near(got[0] if save else got, h64, bar(dt, 4), "h")
        if save:
            near(got[1], g64, bar(dt), "gate_pre")
            near(got[2], u64, bar(dt), "up_pre")


@pytest.mark.parametrize("fmt", R.FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gated_backward(fmt, M, N, K):
    gen = torch.Generator().manual_seed(M * 17 + N)
    (gw, Wg), (uw, Wu) = weight(fmt, N, K, M + 3 * N), weight(fmt, N, K, M + 3 * N + 1)
    dh, dh64 = rand(gen, M, N, scale=1e-4)
    (g, g64), (u, u64) = rand(gen, M, N), rand(gen, M, N)
    for act in ("silu", "relu"):
        say(f"gated backward {fmt} M={M} N={N} K={K} {act}")
        out = Q.q4_gated_backward(gw, uw, dh, g, u, act=ACTS[act], bias_grad=True)
        dx, dg, du, dbg, dbu = R.gated_grad(Wg, Wu, dh64, g64, u64, act)
        near(out["dx"], dx, bar(torch.bfloat16), "dx")
        near(out["dgate"], dg, bar(torch.bfloat16, 0), "dgate")
        near(out["dup"], du, bar(torch.bfloat16, 0), "dup")
        near(out["dgate_bias"], dbg, F32, "dgate_bias")
        near(out["dup_bias"], dbu, F32, "dup_bias")


@pytest.mark.parametrize("fmt", R.FMTS)
@pytest.mark.parametrize("M,N,K", [(40, 96, 512), (66, 130, 192), (200, 256, 1024)])
def test_binary16_outputs_are_those_of_exact_weights(fmt, M, N, K):
    """What separates an output from the exact result is its own rounding: binary32
    sums (F32) of weights exact to 2^-22."""
    gen = torch.Generator().manual_seed(M + K)
    (gw, Wg), (uw, Wu) = weight(fmt, N, K, 1, scale=0.05), weight(fmt, N, K, 2, scale=0.05)
    x, x64 = rand(gen, M, K, dtype=torch.float16)
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        say(f"binary16 {fmt} M={M} N={N} K={K} {act}")
        cases = [(Q.q4_gated(gw, uw, x, act=ACTS[act]), R.gated(x64, Wg, Wu, None, None, act)[0])]
        if act != "relu":
            cases.append((Q.q4_linear(gw, x, act=ACTS[act]), R.linear(x64, Wg, None, act, None)[0]))
        for got, want in cases:
            near(got, want, R.rel(want.half().double(), want) + F32, act)


# K of 32 steps and more (256 weights a step at 4 bits, 128 at 8) at 5 to 64 rows:
# a sum in parts, the last of them shorter, with a K that ends inside a step; at 4
# rows and at 31 steps one part.
@pytest.mark.parametrize("fmt", R.FMTS)
@pytest.mark.parametrize("M,N", [(4, 40), (5, 16), (16, 129), (17, 40), (33, 100), (64, 8)])
@pytest.mark.parametrize("steps", [31, 32, 45])
def test_long_sums_of_few_rows(fmt, M, N, steps):
    gen = torch.Generator().manual_seed(M * 17 + N)
    K = steps * (128 if fmt == "affine8" else 256) - 64
    (gw, Wg), (uw, Wu) = weight(fmt, N, K, M + N), weight(fmt, N, K, M + N + 1)
    for dt in (torch.bfloat16, torch.float16):
        say(f"long sums {fmt} M={M} N={N} K={K} {dt}")
        x, x64 = rand(gen, M, K, dtype=dt)
        b, b64 = rand(gen, N, dtype=dt)
        r, r64 = rand(gen, M, N, dtype=dt)
        y, pre = Q.q4_linear(gw, x, bias=b, act=ACTS["gelu"], residual=r, save_pre=True)
        y64, z64 = R.linear(x64, Wg, b64, "gelu", r64)
        near(y, y64, bar(dt), "y")
        near(pre, z64, bar(dt), "pre")
        h, g, u = Q.q4_gated(gw, uw, x, gate_bias=b, save_pre=True)
        for got, want, ops in zip((h, g, u), R.gated(x64, Wg, Wu, b64, None, "silu"), (4, 2, 2)):
            near(got, want, bar(dt, ops), "gated")
        assert torch.equal(Q.q4_gated(gw, uw, x, gate_bias=b), h), "not deterministic"


@pytest.mark.parametrize("M", [3, 40, 300])
def test_gradients_of_very_different_rows(M):
    """Rows of dz far above, far below and at the size of their dy, zero rows, and
    rows with an infinity or a NaN, which spoil no other row."""
    gen = torch.Generator().manual_seed(M)
    N, K = 256, 128
    (gw, Wg), (uw, Wu) = weight("affine4", N, K, 1), weight("affine4", N, K, 2)
    rows = torch.arange(M)
    size = torch.tensor([1.0, 1e-20, 1e12, 1e-30, 0.0])[rows % 5]       # of u, and so of dz against dh
    dh, _ = rand(gen, M, N, scale=1e-3)
    dh = (dh.float() * torch.tensor([1.0, 1e8, 1e-20])[rows % 3][:, None].cuda()).bfloat16()
    g, g64 = rand(gen, M, N)
    u = (torch.randn(M, N, generator=gen) * size[:, None]).bfloat16().cuda()
    g[rows.cuda() % 5 != 0] = 0.0                                      # act(0) = 0: dup is zero there, dgate is dh u / 2
    bad = {1: float("inf"), 2: float("nan")} if M > 2 else {}
    for m, v in bad.items():
        dh[m, 3] = v
    out = Q.q4_gated_backward(gw, uw, dh, g, u)
    dx, dg, du, _, _ = R.gated_grad(Wg, Wu, dh.double().cpu(), g.double().cpu(), u.double().cpu(), "silu")
    got = out["dx"].double().cpu()
    for m in range(M):
        if m in bad:
            assert not torch.isfinite(got[m]).any()
        else:
            # below 2^-126 values keep an absolute spacing only (2^-133), and flush to zero below that
            for a, b, limit in ((got[m], dx[m], bar(torch.bfloat16)), (out["dgate"][m].double().cpu(), dg[m], U[torch.bfloat16])):
                assert (a - b).norm() <= limit * b.norm() + 2.0 ** -132 * b.numel() ** 0.5, m


@pytest.mark.parametrize("M", [1, 5, 70])
def test_product_gradients_against_differences(M):
    """<dx, v> and the bias gradients' <db, v> against central differences of
    the binary64 loss sum(dh * h)."""
    gen = torch.Generator().manual_seed(M)
    N, K, eps = 96, 128, 1e-4
    (gw, Wg), (uw, Wu) = weight("affine8", N, K, 1, 0.1), weight("affine8", N, K, 2, 0.1)
    x, x64 = rand(gen, M, K)
    (bg, bg64), (bu, bu64) = rand(gen, N), rand(gen, N)
    dh, dh64 = rand(gen, M, N)
    _, g, u = Q.q4_gated(gw, uw, x, gate_bias=bg, up_bias=bu, save_pre=True)
    out = Q.q4_gated_backward(gw, uw, dh, g, u, bias_grad=True)

    def loss(x, bg, bu):
        return (dh64 * R.gated(x, Wg, Wu, bg, bu, "silu")[0]).sum().item()

    vx, vg, vu = (torch.randn(t.shape, generator=gen, dtype=torch.float64) for t in (x64, bg64, bu64))
    for name, got, dn in (("dx", (out["dx"].double().cpu() * vx).sum().item(),
                           (loss(x64 + eps * vx, bg64, bu64) - loss(x64 - eps * vx, bg64, bu64)) / (2 * eps)),
                          ("dgate_bias", (out["dgate_bias"].double().cpu() * vg).sum().item(),
                           (loss(x64, bg64 + eps * vg, bu64) - loss(x64, bg64 - eps * vg, bu64)) / (2 * eps)),
                          ("dup_bias", (out["dup_bias"].double().cpu() * vu).sum().item(),
                           (loss(x64, bg64, bu64 + eps * vu) - loss(x64, bg64, bu64 - eps * vu)) / (2 * eps))):
        # g and u were stored in bfloat16: each of the sum's terms is off by up to about 2^-8, and terms cancel
        size = {"dx": out["dx"].double().cpu().norm() * vx.norm() / np.sqrt(vx.numel()),
                "dgate_bias": out["dgate_bias"].double().cpu().norm(), "dup_bias": out["dup_bias"].double().cpu().norm()}[name].item()
        say(f"  {name}: {got:.6g} against {dn:.6g}, size {size:.3g}")
        assert abs(got - dn) <= 6 * 2.0 ** -8 * size


# ---- norms -----------------------------------------------------------------------

def norm_case(gen, M, D, dt, rt, pre, post, bias, groups):
    c, g = {"pre": pre, "post": post, "scale": 0.75, "eps": 1e-5}, {}
    y, y64 = rand(gen, M, D, dtype=dt)
    r, r64 = rand(gen, M, D, dtype=rt, scale=2.0)
    for name, kind in (("pre", pre), ("post", post)):
        g[name + "_weight"], c[name + "_w"] = rand(gen, D, dtype=dt, scale=0.2, mean=1.0) if kind != "none" else (None, None)
        g[name + "_bias"], c[name + "_b"] = rand(gen, D, dtype=dt) if bias and kind != "none" else (None, None)
    rows = None
    c["gate"], g["gate"] = None, None
    if groups:
        rows = -(-M // groups)
        groups = -(-M // rows)
        g["gate"], gate64 = rand(gen, groups, D, dtype=dt)
        c["gate"] = gate64[torch.arange(M) // rows]
    return y, y64, r, r64, c, dict(g, gate_rows=rows, pre_norm=NORMS[pre], post_norm=NORMS[post], scale=0.75)


NORM_SHAPES = [(1, 1), (1, 64), (1, 2048), (2, 7), (3, 513), (5, 2048), (17, 1000), (64, 4096), (33, 4100), (7, 8192),
               (4, 16384), (3, 32768), (2, 20001), (300, 40), (1000, 256)]


@pytest.mark.parametrize("M,D", NORM_SHAPES)
@pytest.mark.parametrize("dt,rt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")])
def test_block_norm(M, D, dt, rt):
    gen = torch.Generator().manual_seed(M * 5 + D)
    dt, rt = DT[dt], DT[rt]
    for pre, post, bias, groups in (("rms", "none", False, 0), ("rms", "rms", False, 1), ("layer", "layer", True, 3),
                                    ("none", "rms", True, M)):
        say(f"norm M={M} D={D} {dt} {rt} {pre} {post} gate {groups}")
        y, y64, r, r64, c, g = norm_case(gen, M, D, dt, rt, pre, post, bias, groups)
        r1, n, stats = Q.block_norm(r, y, save_stats=True, **g)
        w1, wn, ws = R.block_norm(r64, y64, c)
        near(r1, w1, max(U[rt], F32 if rt == torch.float32 else 0), "r'")
        # binary32 arithmetic ahead of the rounding; a row of one value cancels to its bias
        near(stats, ws, F32, "stats")
        if pre == "none":
            assert n is None
        elif D > 1:
            near(n, wn, U[dt] + F32, "n")
        else:
            assert (n.double().cpu() - wn).abs().max() <= U[dt] * wn.abs().max() + F32 * max(1.0, ws[:, 3].max().item())


@pytest.mark.parametrize("M,D", [(1, 64), (9, 333), (40, 2048)])
def test_block_norm_first_norm_and_in_place(M, D):
    gen = torch.Generator().manual_seed(M)
    r, r64 = rand(gen, M, D)
    w, w64 = rand(gen, D, scale=0.1, mean=1.0)
    r1, n, stats = Q.block_norm(r, pre_weight=w, save_stats=True)
    assert r1 is r
    c = dict(pre="rms", post="none", pre_w=w64, pre_b=None, post_w=None, post_b=None, gate=None, scale=1.0, eps=1e-5)
    near(n, R.block_norm(r64, None, c)[1], U[torch.bfloat16] + F32, "n")
    dn, dn64 = rand(gen, M, D)
    out = Q.block_norm_backward(r, None, stats, dn, pre_weight=w)
    assert set(out) == {"dr", "pre_dw"}
    x = r64.clone().requires_grad_()
    (R.norm(x, "rms", w64, None, 1e-5)[0] * dn64).sum().backward()
    near(out["dr"], x.grad, U[torch.bfloat16] + F32, "dr")
    y, _ = rand(gen, M, D)
    want = Q.block_norm(r, y, pre_weight=w)
    got = Q.block_norm(r, y, pre_weight=w, r_out=r)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0].data_ptr() == r.data_ptr()


@pytest.mark.parametrize("M,D", NORM_SHAPES)
@pytest.mark.parametrize("dt,rt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_block_norm_backward(M, D, dt, rt):
    """Against the derivative that autograd takes of the binary64 forward form."""
    gen = torch.Generator().manual_seed(M * 3 + D)
    dt, rt = DT[dt], DT[rt]
    for pre, post, bias, groups in (("rms", "none", False, 0), ("rms", "rms", False, 1), ("layer", "layer", True, 3),
                                    ("none", "rms", True, M), ("layer", "rms", True, max(1, M // 2))):
        if D == 1 and "layer" in (pre, post):
            continue                       # a norm of one centred value is constant: its gradient is rounding noise
        say(f"norm backward M={M} D={D} {dt} {rt} {pre} {post} gate {groups}")
        y, y64, r, r64, c, g = norm_case(gen, M, D, dt, rt, pre, post, bias, groups)
        stats = Q.block_norm(r, y, save_stats=True, **g)[2] if pre != "none" or post != "none" else None
        # r plays r': the statistics of the pre norm are those of r itself
        own = R.block_norm(r64, None, dict(c, post="none"))[2] if pre != "none" else None
        if own is not None:
            stats[:, 2:] = own[:, 2:].float().cuda()
        dn, dn64 = rand(gen, M, D, dtype=dt, scale=0.1) if pre != "none" else (None, None)
        dr, dr64 = rand(gen, M, D, dtype=rt, scale=0.1)
        out = Q.block_norm_backward(r, y, stats, dn, dr, **g)
        # G by the pre norm alone, then the rest from G
        v = {k: c[k].clone().requires_grad_() for k in ("pre_w", "pre_b", "post_w", "post_b") if c[k] is not None}
        rr = r64.clone().requires_grad_()
        G = dr64
        if pre != "none":
            (R.norm(rr, pre, v.get("pre_w"), v.get("pre_b"), 1e-5)[0] * dn64).sum().backward()
            G = dr64 + rr.grad
        yy = y64.clone().requires_grad_()
        p = R.norm(yy, post, v.get("post_w"), v.get("post_b"), 1e-5)[0]
        gate = None if c["gate"] is None else c["gate"].clone().requires_grad_()
        (0.75 * (p if gate is None else gate * p) * G).sum().backward()
        near(out["dr"], G, U[rt] + F32, "dr")
        # dy = (t - hat (t . hat) / D - ..) rstd with binary32 statistics: 2^-22 of the terms, which cancel at D = 1
        rstd = R.norm(y64, post, None, None, 1e-5)[2]
        t = 0.75 * G * (1 if gate is None else c["gate"]) * (1 if c["post_w"] is None else c["post_w"]) * rstd
        near(out["dy"], yy.grad, U[dt] + 5 * F32 + 2.0 ** -22 * (t.norm() / yy.grad.norm()).item(), "dy")
        if gate is not None:
            rows = g["gate_rows"]
            want = torch.stack([t.sum(0) for t in gate.grad.split(rows)])
            near(out["dgate"], want, U[dt] + F32, "dgate")
        for name, key in (("pre_dw", "pre_w"), ("pre_db", "pre_b"), ("post_dw", "post_w"), ("post_db", "post_b")):
            if key in v:
                near(out[name], v[key].grad, F32, name)
        again = Q.block_norm_backward(r, y, stats, dn, dr, **g)
        assert all(torch.equal(out[k], again[k]) for k in out), "not deterministic"


def test_block_norm_bad_rows_stay_alone():
    gen = torch.Generator().manual_seed(1)
    M, D = 6, 300
    y, _ = rand(gen, M, D)
    r, _ = rand(gen, M, D)
    clean = Q.block_norm(r, y, post_norm=Q.Q4_NORM_RMS)
    y[2, 5], r[4, 7] = float("nan"), float("inf")
    r1, n, _ = Q.block_norm(r, y, post_norm=Q.Q4_NORM_RMS)
    for m in (0, 1, 3, 5):
        assert torch.equal(r1[m], clean[0][m]) and torch.equal(n[m], clean[1][m])
    assert torch.isnan(n[2]).all() and not torch.isfinite(r1[4, 7])


# ---- the operators together: streams, graphs, long offsets --------------------------------

def chain(w, t, stream=None):
    r1, n, stats = Q.block_norm(t["r"], t["y"], pre_weight=t["pw"], save_stats=True, stream=stream)
    h, g, u = Q.q4_gated(w[0], w[1], n, save_pre=True, stream=stream)
    z = Q.q4_linear(w[2], h, residual=r1, stream=stream)
    d = Q.q4_linear_backward(w[2], t["dz"], stream=stream)["dx"]
    b = Q.q4_gated_backward(w[0], w[1], d, g, u, bias_grad=True, stream=stream)
    e = Q.block_norm_backward(r1, t["y"], stats, b["dx"], t["dz"], pre_weight=t["pw"], stream=stream)
    return [r1, n, h, z, d] + [b[k] for k in sorted(b)] + [e[k] for k in sorted(e)]


def chain_inputs(M, D, N):
    gen = torch.Generator().manual_seed(M + D)
    w = [weight("q4_0", N, D, 1)[0], weight("q4_0", N, D, 2)[0], weight("affine4", D, N, 3)[0]]
    t = {k: rand(gen, M, D)[0] for k in ("r", "y", "dz")}
    t["pw"] = rand(gen, D, scale=0.1, mean=1.0)[0]
    return w, t


@pytest.mark.parametrize("M", [1, 24, 150])
def test_chain_on_another_stream(M):
    w, t = chain_inputs(M, 256, 512)
    want = chain(w, t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = chain(w, t)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = chain(w, t, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("M", [1, 24, 150])
def test_chain_in_a_graph(M):
    w, t = chain_inputs(M, 256, 512)
    chain(w, t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(w, t)
    for i in range(3):
        t["r"].normal_(generator=torch.Generator("cuda").manual_seed(i))
        t["dz"].normal_(generator=torch.Generator("cuda").manual_seed(50 + i))
        for o in out:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = chain(w, t)
        assert all(torch.equal(a, b) for a, b in zip(out, want)), f"replay {i}"


def test_offsets_past_32_bits():
    """Outputs of more than 2^31 values: the last rows equal the same rows of a small call."""
    w, _ = weight("q4_0", 8192, 64, 1)
    M = (1 << 31) // 8192 + 300
    x = torch.randn(M, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    y = Q.q4_linear(w, x)
    tail = Q.q4_linear(w, x[-256:].contiguous())
    assert torch.equal(y[-256:], tail)
    out = Q.q4_linear_backward(w, y, act=Q.Q4_ACT_SILU, pre=y)
    small = Q.q4_linear_backward(w, y[-256:].contiguous(), act=Q.Q4_ACT_SILU, pre=y[-256:].contiguous())
    assert torch.equal(out["dz"][-256:], small["dz"])
    near(out["dx"][-256:], small["dx"].double().cpu(), 2.0 ** -8, "dx")     # another split of the sum
    del out, y
    M, D = (1 << 31) // 32768 + 40, 32768
    r = torch.randn(M, D, device="cuda", dtype=torch.bfloat16, generator=torch.Generator("cuda").manual_seed(2))
    r1, n, stats = Q.block_norm(r, r, post_norm=Q.Q4_NORM_RMS, save_stats=True)
    a = r[-16:].contiguous()
    b1, bn, bs = Q.block_norm(a, a, post_norm=Q.Q4_NORM_RMS, save_stats=True)
    assert torch.equal(r1[-16:], b1) and torch.equal(n[-16:], bn) and torch.equal(stats[-16:], bs)
    out = Q.block_norm_backward(r1, r, stats, n, r1, post_norm=Q.Q4_NORM_RMS)
    small = Q.block_norm_backward(b1, a, bs, bn, b1, post_norm=Q.Q4_NORM_RMS)
    assert torch.equal(out["dr"][-16:], small["dr"]) and torch.equal(out["dy"][-16:], small["dy"])
