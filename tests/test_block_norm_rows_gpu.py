"""block_norm and its gradients where a workgroup takes several rows: one norm (before
the block, after it, or the stream's alone) and two, one and several waves a row,
gates whose rows do not divide the workgroup's.  Against the binary64 forms of
block_reference (run on the GPU), all rows and all sums; a repeated call gives the
same bits.

Tolerances as in test_block_gpu: an output's rounding (2^-8, 2^-11, 2^-24) and
2e-5 for binary32 sums and statistics; dy's terms cancel at few values only.
"""
import pytest
import torch

import block_reference as R
import gemv_q4_affine_amd as Q
import test_block_gpu as G

pytestmark = pytest.mark.gpu

# rows well above what the forward grid holds at once (256 CUs: 16 to 2 workgroups
# each at these widths), and 3 to 10 rows a workgroup backward
SHAPES = [(2500, 4096), (4100, 1537), (9000, 1000), (5000, 2048), (1300, 8192), (9000, 520),
          (700, 16392), (520, 32768)]
# pre, post, bias, with y, rows of a gate (None: no gate; 0: all)
FORMS = [("rms", "none", False, True, None), ("layer", "none", True, True, 7), ("none", "rms", False, True, 0),
         ("none", "layer", True, True, 3), ("rms", "none", False, False, None), ("layer", "none", True, False, None),
         ("rms", "rms", False, True, 11), ("layer", "layer", True, True, None)]
TYPES = [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")]


def case(M, D, types, form):
    pre, post, bias, with_y, rows = form
    dt, rt = (G.DT[t] for t in types)
    gen = torch.Generator().manual_seed(M + 7 * D)
    groups = 0 if rows is None else 1 if rows == 0 else -(-M // rows)
    y, y64, r, r64, c, g = G.norm_case(gen, M, D, dt, rt, pre, post, bias, groups)
    if not with_y:
        y = y64 = None
        g = dict(g, dtype=dt)
    wide = [None if t is None else t.cuda() for t in (y64, r64)]
    return gen, dt, rt, y, wide[0], r, wide[1], {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}, g


def small(gen, M, D, dtype):
    return (torch.randn(M, D, generator=gen, device="cpu") * 0.1).to(dtype).cuda()


def near(got, want, limit, what):
    """G.near, the error taken on the GPU."""
    if got.dtype == torch.float16 and want.norm() > 0:
        limit += 2.0 ** -25 * want.numel() ** 0.5 / want.norm().item()
    e = ((got.double() - want).norm() / want.norm()).item()
    G.say(f"  {what}: {e:.3g} (limit {limit:.3g})")
    assert got.shape == want.shape and e <= limit, f"{what}: {e} > {limit}"


@pytest.mark.parametrize("M,D", SHAPES)
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(str(v) for v in f))
@pytest.mark.parametrize("types", TYPES, ids="/".join)
def test_forward(M, D, types, form):
    gen, dt, rt, y, y64, r, r64, c, g = case(M, D, types, form)
    G.say(f"norm rows M={M} D={D} {types} {form}")
    r1, n, stats = Q.block_norm(r, y, save_stats=True, **g)
    with torch.device("cuda"):
        w1, wn, ws = R.block_norm(r64, y64, c)
    near(r1, w1, G.U[rt] + G.F32, "r'")
    near(stats, ws, G.F32, "stats")
    # each row for itself: one row's statistics out of 9000 would not show in the norm of all
    assert ((stats.double() - ws).abs().amax(1) <= G.F32 * ws.abs().amax(1)).all()
    if n is not None:
        near(n, wn, G.U[dt] + G.F32, "n")
    for _ in range(3):
        again = Q.block_norm(r, y, save_stats=True, **g)
        assert torch.equal(again[0], r1) and torch.equal(again[2], stats) and (n is None or torch.equal(again[1], n))


@pytest.mark.parametrize("M,D", SHAPES)
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(str(v) for v in f))
@pytest.mark.parametrize("types", TYPES, ids="/".join)
def test_backward(M, D, types, form):
    with torch.device("cuda"):
        backward(M, D, types, form)


def backward(M, D, types, form):
    with torch.device("cpu"):
        gen, dt, rt, y, y64, r, r64, c, g = case(M, D, types, form)
    pre, post, scale = form[0], form[1], g["scale"]
    G.say(f"norm rows backward M={M} D={D} {types} {form}")
    # r plays r': the statistics of the pre norm are those of r itself
    ws = [R.norm(r64, pre, None, None, 1e-5)[1:], R.norm(y64, post, None, None, 1e-5)[1:] if y is not None else None]
    stats64 = torch.cat([*(ws[1] or (r64[:, :1] * 0, r64[:, :1] * 0 + 1)), *ws[0]], 1)
    stats = stats64.float()
    dn = small(gen, M, D, dt) if pre != "none" else None
    dr = small(gen, M, D, rt)
    dr64 = dr.double()
    out = Q.block_norm_backward(r, y, stats, dn, dr, **g)
    v = {k: c[k].clone().requires_grad_() for k in ("pre_w", "pre_b", "post_w", "post_b") if c[k] is not None}
    want = {}
    total = dr64
    if pre != "none":
        rr = r64.clone().requires_grad_()
        (R.norm(rr, pre, v.get("pre_w"), v.get("pre_b"), 1e-5)[0] * dn.double()).sum().backward()
        total = dr64 + rr.grad
    want["dr"] = (total, G.U[rt] + G.F32)
    if y is not None:
        yy = y64.clone().requires_grad_()
        p = R.norm(yy, post, v.get("post_w"), v.get("post_b"), 1e-5)[0]
        gate = None if c["gate"] is None else c["gate"].clone().requires_grad_()
        (scale * (p if gate is None else gate * p) * total).sum().backward()
        want["dy"] = (yy.grad, G.U[dt] + 5 * G.F32)
        if gate is not None:
            want["dgate"] = (torch.stack([t.sum(0) for t in gate.grad.split(g["gate_rows"])]), G.U[dt] + G.F32)
    for name, key in (("pre_dw", "pre_w"), ("pre_db", "pre_b"), ("post_dw", "post_w"), ("post_db", "post_b")):
        if key in v:
            want[name] = (v[key].grad, G.F32)
    assert set(out) == set(want)
    for name, (value, limit) in want.items():
        near(out[name], value, limit, name)
    for _ in range(3):
        again = Q.block_norm_backward(r, y, stats, dn, dr, **g)
        assert all(torch.equal(out[k], again[k]) for k in out), "not deterministic"
