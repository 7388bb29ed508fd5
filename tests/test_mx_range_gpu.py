"""The operators on microscaled numbers at the ends of their ranges: values beside
borders between codes below binary32's normal numbers, scales from the first to
the last.  Tolerances: test_mx_gpu's, where nothing else is said."""
import math

import numpy as np
import pytest
import torch

import block_reference as R
import gemv_q4_affine_amd as Q
import mx_reference as X
from test_mx_gpu import NORMS, TYPES, say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _done():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    yield
    torch.cuda.synchronize()


# ---- norm ------------------------------------------------------------------------

def beside_borders(kind, byte, columns, rng):
    """Values v, within half a step of binary32 beside a border between two codes under the scale byte (but not on
    it), whose blocks of 32 have that scale."""
    t = X.table(kind)
    t = np.unique(np.abs(t[np.isfinite(t)]))
    step = 2.0 ** (byte - 127)
    border = (t[1:] + t[:-1]) / 2 * step
    v = rng.choice(border, columns)
    ulp = np.maximum(np.spacing(v.astype(np.float32)).astype(np.float64), 2.0 ** -149)
    v = (v + rng.uniform(0.05, 0.45, columns) * rng.choice([-1, 1], columns) * ulp) * rng.choice([-1, 1], columns)
    v[::32] = 2.0 ** X.TOP[kind] * 1.25 * step              # keeps the scale
    return v


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("pre", ["rms", "layer"])
@pytest.mark.parametrize("byte", [0, 1, 2, 3, 4, 5, 6, 7, 8, 20])
def test_norm_codes_beside_borders(kind, pre, byte):
    """Weights that bring n beside borders: rounded to binary32 first, about half of them would lie on one, and a tie
    goes to the even code, not to the nearer one.  Below 2^-126 binary32 steps evenly, by 2^-149."""
    rng = np.random.default_rng(byte)
    D, eps = 4096, float(np.float32(1e-5))
    v = beside_borders(kind, byte, D, rng)
    r = np.where(np.arange(D) % 2, -1.0, 1.0)               # mean 0, mean square 1
    rstd = 1 / math.sqrt(1 + eps)
    # the nearest binary32 weight, one step either side: n = r rstd w, where w's own steps allow
    w = (np.abs(v) / rstd).astype(np.float32)
    w = np.stack([w, np.nextafter(w, np.float32(0)), np.nextafter(w, np.float32(1))]).astype(np.float64)
    off = np.abs(w * rstd - np.abs(v))
    w = w[off.argmin(0), np.arange(D)] * np.sign(v) * r
    W, T = torch.from_numpy(w.astype(np.float32)), torch.from_numpy(r.astype(np.float32))[None]
    c = dict(pre=pre, post="none", pre_w=W.double(), pre_b=None, post_w=None, post_b=None, gate=None, scale=1.0, eps=eps)
    n = R.block_norm(T.double(), None, c)[1].numpy()
    c64, s64 = X.quantize(n, kind)
    assert (s64 == byte).all()
    twice = X.quantize(n.astype(np.float32).astype(np.float64), kind)[0]
    say(f"{kind} {pre} {byte}: {(twice != c64).sum()} codes would differ after two roundings")
    if byte < 7 and kind == "fp8":
        assert (twice != c64).sum() > 100                   # the case is one where it counts
    _, (codes, scales), _ = Q.block_norm_mx(T.cuda(), pre_norm=NORMS[pre], pre_weight=W.cuda(), eps=eps, n_type=TYPES[kind])
    assert np.array_equal(scales.cpu().numpy(), s64), "scales"
    assert np.array_equal(X.unpacked(codes.cpu().numpy(), kind), c64), "codes"


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_norm_past_binary32(kind):
    """An n past binary32's largest number is taken as that number; below its smallest, n's codes are zeros."""
    D, top = 96, float(np.finfo(np.float32).max)
    r = torch.zeros(1, D)
    r[0, ::32], r[0, 1::32] = 1.0, 0.5
    w = torch.full((D,), top)
    w[32:64] = 2.0 ** -149
    w[64:] = top / 16
    c = dict(pre="rms", post="none", pre_w=w.double(), pre_b=None, post_w=None, post_b=None, gate=None, scale=1.0, eps=float(np.float32(1e-5)))
    n = R.block_norm(r.double(), None, c)[1].numpy()
    assert np.abs(n).max() > 2 * top and np.abs(n[0, 64:]).max() < top
    c64, s64 = X.quantize(n.clip(-top, top), kind)
    _, (codes, scales), _ = Q.block_norm_mx(r.cuda(), pre_weight=w.cuda(), n_type=TYPES[kind])
    assert np.array_equal(scales.cpu().numpy(), s64) and np.array_equal(X.unpacked(codes.cpu().numpy(), kind), c64)


# ---- scales ------------------------------------------------------------------------

def weights(scales, seed):
    """Planes of any codes under the given scale bytes [N, K / 32], and their binary64 values, on the GPU."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    N, K = scales.shape[0], scales.shape[1] * 32
    q = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    code = torch.stack((q & 15, q >> 4), 2).view(N, K).long()
    table = torch.from_numpy(X.table("fp4")).cuda()
    s = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
    return (q, scales.to(torch.uint8)), table[code] * s


def by_element(got, x, W, what, extra=0.0):
    """Every output within its own rounding and K + 8 binary32 roundings of the sum of its terms' magnitudes, where those
    lie inside binary32's normal numbers (and the output inside its type)."""
    want, terms = x @ W.T, x.abs() @ W.abs().T
    top = min(float(torch.finfo(got.dtype).max), 2.0 ** 126)
    inside = (terms < top * 0.99) & (terms > 2.0 ** -100)
    slack = want.abs() * (torch.finfo(got.dtype).eps / 2) + terms * ((x.shape[1] + 8) * 2.0 ** -24 + extra)
    if got.dtype == torch.float16:
        slack += 2.0 ** -25
    e = ((got.double() - want).abs() / slack)[inside]
    say(f"  {what}: {inside.double().mean().item():.2f} of the outputs, {e.max().item() if e.numel() else 0:.3g} of the slack")
    assert torch.isfinite(got[inside]).all() and (e <= 1).all(), what
    return inside


#: 255 rows of W, each under a scale of its own, times `more`; the routes by rows, on 16-bit x.
ROUTES = [(1, 1, 160), (4, 1, 2080), (5, 1, 160), (20, 1, 544), (40, 1, 8192), (64, 1, 160), (65, 1, 160), (100, 1, 544), (300, 1, 544),
          (700, 32, 544)]


@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("M,more,K", ROUTES)
def test_every_scale_of_the_weights(x, M, more, K):
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[x]
    w, W = weights(torch.arange(255, device="cuda").repeat(more)[:, None].expand(255 * more, K // 32).contiguous(), M)
    gen = torch.Generator(device="cuda").manual_seed(M)
    seen = torch.zeros(255 * more, dtype=torch.bool, device="cuda")
    for e in (-100, -50, 0, 50, 100) if x == "bf16" else (-13, -6, 0, 6, 12):
        v = (torch.randn(M, K, generator=gen, device="cuda").clamp(-4, 4) * 2.0 ** e).to(dt)
        seen |= by_element(Q.mx_linear(w, v), v.double(), W, f"{x} {M} 2^{e}").any(0)
    assert seen[:255].all() if x == "bf16" else seen[85:135].all()


@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("M,more,K", ROUTES)
def test_blocks_of_very_different_scales(x, M, more, K):
    """Blocks of W that x's own range balances, so that all of them count: 2^+-100 in bfloat16, 2^+-15 in binary16."""
    dt, far = {"bf16": (torch.bfloat16, 100), "f16": (torch.float16, 14)}[x]
    gen = torch.Generator(device="cuda").manual_seed(M)
    N, nb = 255 * more, K // 32
    e = torch.tensor([0, far, -far, 3], device="cuda")[torch.arange(nb, device="cuda") % 4]
    w, W = weights(120 + e + torch.randint(0, 3, (N, nb), generator=gen, device="cuda"), M)
    v = (torch.randn(M, K, generator=gen, device="cuda") * torch.exp2(-e.double()).repeat_interleave(32)).to(dt)
    by_element(Q.mx_linear(w, v), v.double(), W, f"{x} {M}")


@pytest.mark.parametrize("M", [1, 3, 12, 40, 64])
def test_largest_scales_and_infinities(M):
    """Scales of 2^126 and 2^127 beside ordinary ones: an infinity or a NaN in x gives what its terms give, and no other
    row or column sees it."""
    K, N = 352, 100
    gen = torch.Generator(device="cuda").manual_seed(M)
    s = torch.randint(118, 124, (N, K // 32), generator=gen, device="cuda")
    s[7::8, 3], s[5::8, 10] = 254, 253
    w, W = weights(s, M)
    v = torch.randn(M, K, generator=gen, device="cuda")
    v[:, 96:128] *= 2.0 ** -110                              # the large blocks' values
    v[:, 320:] *= 2.0 ** -110
    v = v.bfloat16()
    by_element(Q.mx_linear(w, v), v.double(), W, "large")
    clean = Q.mx_linear(w, v)
    for k in (5, 100, 340):
        bad, row = v.clone(), M // 2
        bad[row, k] = math.inf
        got = Q.mx_linear(w, bad)
        others = [m for m in range(M) if m != row]
        assert torch.equal(got[others], clean[others])
        col = W[:, k]
        assert torch.equal(torch.isnan(got[row]), col == 0)
        assert (got[row][col > 0] == math.inf).all() and (got[row][col < 0] == -math.inf).all()
        bad[row, k] = math.nan
        got = Q.mx_linear(w, bad)
        assert torch.isnan(got[row]).all() and torch.equal(got[others], clean[others])


# ---- gradients ---------------------------------------------------------------------

@pytest.mark.parametrize("M,N,blocks", [(1, 33, 255), (5, 64, 255), (70, 2048, 255), (300, 511, 255), (700, 100, 510)])
def test_gradients_under_every_scale(M, N, blocks):
    """Columns of W under scales of their own: dx = dz W, dz in binary16 (2^-12 of each term)."""
    w, W = weights((torch.arange(blocks, device="cuda") % 255)[None].expand(N, blocks).contiguous(), M)
    gen = torch.Generator(device="cuda").manual_seed(N)
    seen = torch.zeros(blocks * 32, dtype=torch.bool, device="cuda")
    for e in (-100, -50, 0, 50, 100):
        dy = (torch.randn(M, N, generator=gen, device="cuda") * 2.0 ** e).bfloat16()
        got = Q.mx_linear_backward(w, dy, bias_grad=True)
        seen |= by_element(got["dx"], dy.double(), W.T, f"{M} 2^{e}", 2.0 ** -12).any(0)
    assert seen.all()


@pytest.mark.parametrize("M,N,blocks", [(1, 33, 5), (9, 100, 16), (70, 2048, 17), (300, 511, 40), (65, 9000, 129), (40, 40000, 15)])
def test_gradients_of_rows_of_different_scales(M, N, blocks):
    """Rows of W over 2^36 of scales in every block of columns, all of whose terms count: dy balances them."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    e = torch.tensor([0, 18, -18, 3, -7], device="cuda")[torch.arange(N, device="cuda") % 5]
    u, U = weights((110 - e // 2)[:, None] + torch.randint(0, 3, (N, blocks), generator=gen, device="cuda"), M + 1)
    w, W = weights((120 + e)[:, None] - torch.randint(0, 3, (N, blocks), generator=gen, device="cuda"), M)
    bad = (w[0], w[1].clone())
    bad[1][N // 2, blocks // 2] = 255
    dy = (torch.randn(M, N, generator=gen, device="cuda") * torch.exp2(-e.double() / 3)).bfloat16()
    got = Q.mx_linear_backward(w, dy)["dx"]
    by_element(got, dy.double(), W.T, f"{M} {N}", 2.0 ** -12)
    spoilt = Q.mx_linear_backward(bad, dy)["dx"].view(M, blocks, 32)
    fine = torch.arange(blocks, device="cuda") != blocks // 2
    assert torch.isnan(spoilt[:, ~fine]).all() and torch.equal(spoilt[:, fine], got.view(M, blocks, 32)[:, fine])
    # both matrices of a gated product, of which either may have the larger scales
    gp, up = (torch.randn(M, N, generator=gen, device="cuda").bfloat16() for _ in range(2))
    for a, A, b, B in ((w, W, u, U), (u, U, w, W)):
        g = Q.mx_gated_backward(a, b, dy, gp, up, act=Q.Q4_ACT_RELU)
        dg, du = (dy.double() * up.double() * (gp > 0)), dy.double() * gp.double().clamp(min=0)
        by_element(g["dx"], torch.cat((dg, du), 1), torch.cat((A, B), 0).T, "gated", 2.0 ** -12)
