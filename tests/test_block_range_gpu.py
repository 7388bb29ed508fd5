"""The products over the whole range of their operands' types, on both sides of the
few-row kernels (64 rows): against binary64, row by row.  Tolerances as in
test_block_gpu (`bar`), and bfloat16's absolute spacing below 2^-126 (2^-133).
"""
import pytest
import torch

import block_reference as R
import gemv_q4_affine_amd as Q
import test_block_gpu as G

pytestmark = pytest.mark.gpu

ROWS = [1, 3, 4, 5, 16, 17, 33, 64, 65, 200]


def rows_near(got, want, dtype, what):
    got, want = got.double().cpu(), want.double().cpu()
    for m in range(got.shape[0]):
        e, n = (got[m] - want[m]).norm().item(), want[m].norm().item()
        assert e <= G.bar(dtype) * n + 2.0 ** -132 * want.shape[1] ** 0.5, (what, m, e / n)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("fmt", R.FMTS)
@pytest.mark.parametrize("K", [64, 512, 4096])
def test_largest_and_smallest_x(fmt, M, K):
    """bfloat16 x up to the type's largest value, in either sign or all of one, and
    down to its normal range's end; outputs are in range.  Where x is all of one sign,
    W's codes are what they are: sums of whole blocks at the top of the range."""
    gen = torch.Generator().manual_seed(M * 7 + K)
    N = 48
    (w, W), (u, U) = G.weight(fmt, N, K, M, scale=1e-3), G.weight(fmt, N, K, M + 1, scale=1e-3)
    top = torch.finfo(torch.bfloat16).max
    x = torch.rand(M, K, generator=gen) * torch.tensor([-1.0, 1.0])[torch.randint(0, 2, (M, K), generator=gen)]
    kind = torch.arange(M) % 5
    x[kind == 1] = x[kind == 1].abs()
    x[kind == 2] = 1.0
    size = torch.tensor([top, top, top, 2.0 ** -110, 2.0 ** -120])[(kind + M) % 5]
    # a row whose exact sums leave the type takes 1/4, 1/16 .. of the size
    for m in range(M):
        while ((x[m].double() * size[m].double()) @ torch.stack([W, U]).transpose(1, 2)).abs().max() > 0.9 * top:
            size[m] /= 4
    x = (x.double() * size[:, None].double()).bfloat16()
    assert torch.isfinite(x).all()
    y, pre = Q.q4_linear(w, x.cuda(), save_pre=True)
    rows_near(y, x.double() @ W.T, torch.bfloat16, "y")
    assert torch.equal(pre, y)
    _, g, up = Q.q4_gated(w, u, x.cuda(), act=Q.Q4_ACT_RELU, save_pre=True)
    rows_near(g, x.double() @ W.T, torch.bfloat16, "gate")
    rows_near(up, x.double() @ U.T, torch.bfloat16, "up")


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("fmt", R.FMTS)
def test_largest_codes(fmt, M):
    """Every code the largest (and the smallest) and every x the largest: the block
    sums are as large as they get."""
    N, K = 32, 256
    top = torch.finfo(torch.bfloat16).max
    for code in (0, 255):
        q = torch.full((N, K // (1 if fmt == "affine8" else 2)), code, dtype=torch.uint8, device="cuda")
        most = 255 if fmt == "affine8" else 15
        if fmt == "q4_0":
            d = torch.full((N, K // 32), 2.0 ** -13).half()
            w, value = (q.view(N, K // 32, 16), d.view(torch.int16).cuda()), 2.0 ** -13 * (code % 16 - 8)
        else:
            s, b = torch.full((N, K // 64), 2.0 ** -18).bfloat16(), torch.full((N, K // 64), -(2.0 ** -12)).bfloat16()
            w, value = (q, s.view(torch.int16).cuda(), b.view(torch.int16).cuda()), 2.0 ** -18 * min(code, most) - 2.0 ** -12
        x = torch.full((M, K), top).bfloat16()
        rows_near(Q.q4_linear(w, x.cuda()), torch.full((M, N), top * value * K, dtype=torch.float64), torch.bfloat16, code)


def same_kind(got, want, dtype, what):
    """Infinities and NaN where binary64 has them; the rest near, row by row."""
    got, want = got.double().cpu(), want.double().cpu()
    assert torch.equal(got.isnan(), want.isnan()), (what, (got.isnan() != want.isnan()).nonzero()[:5])
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf]), what
    ok = torch.isfinite(want)
    assert torch.isfinite(got[ok]).all(), what
    rows_near(torch.where(ok, got, 0), torch.where(ok, want, 0), dtype, what)


def times(x, W):
    """x . W^T by its definition: a zero weight and an infinity make a NaN, a zero x and a
    finite weight do not."""
    return torch.stack([(row * W).sum(1) for row in x])


def spoil(x, largest):
    """One infinity of either sign, beside large values; two of the same and of opposite
    signs; a NaN; in rows of their own."""
    for m in range(x.shape[0]):
        k = (37 * m + 11) % x.shape[1]
        j = (k + 20) % x.shape[1]
        kind = m % 7
        if kind in (0, 2):
            x[m, k] = float("inf" if kind == 0 else "-inf")
            x[m, (k + 1) % x.shape[1]] = -largest
        elif kind in (1, 3):
            x[m, k] = float("inf")
            x[m, j] = float("inf" if kind == 1 else "-inf")
        elif kind == 4:
            x[m, k] = float("nan")
    return x


@pytest.mark.parametrize("M", [1, 2, 3, 4, 16, 20, 33, 64, 65, 200])
@pytest.mark.parametrize("fmt", R.FMTS)
@pytest.mark.parametrize("K", [192, 8192])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_infinities_in_x(fmt, M, K, dt):
    """A row with an infinity is what its infinite terms make it, and no other row is."""
    gen = torch.Generator().manual_seed(M + K)
    N, dt = 40, G.DT[dt]
    (w, W), (u, U) = G.weight(fmt, N, K, M), G.weight(fmt, N, K, M + 1)
    x = spoil(torch.randn(M, K, generator=gen), 3e38 if dt == torch.bfloat16 else 6e4).to(dt)
    g64, u64 = times(x.double(), W), times(x.double(), U)
    y, pre = Q.q4_linear(w, x.cuda(), act=Q.Q4_ACT_GELU, save_pre=True)
    same_kind(pre, g64, dt, "pre")
    same_kind(Q.q4_linear(w, x.cuda()), g64, dt, "y")
    _, g, up = Q.q4_gated(w, u, x.cuda(), save_pre=True)
    same_kind(g, g64, dt, "gate")
    same_kind(up, u64, dt, "up")


@pytest.mark.parametrize("M", [1, 9, 64, 200])
@pytest.mark.parametrize("fmt", R.FMTS)
def test_infinities_in_gradients(fmt, M):
    gen = torch.Generator().manual_seed(M)
    N, K = 40, 128
    (w, W), (u, U) = G.weight(fmt, N, K, M), G.weight(fmt, N, K, M + 1)
    dy = spoil(torch.randn(M, N, generator=gen), 3e38).bfloat16()
    pre = torch.randn(M, N, generator=gen).bfloat16()
    same_kind(Q.q4_linear_backward(w, dy.cuda())["dx"], times(dy.double(), W.T), torch.bfloat16, "dx")
    dz = R.linear_grad(W, dy.double(), pre.double(), "relu")[1]
    dz = dz.bfloat16().double()                        # exact: dy or zero (an infinity times zero: NaN)
    out = Q.q4_linear_backward(w, dy.cuda(), act=Q.Q4_ACT_RELU, pre=pre.cuda())
    same_kind(out["dz"], dz, torch.bfloat16, "dz")
    same_kind(out["dx"], times(dz, W.T), torch.bfloat16, "dx, relu")
    # dh is finite, dh u is not: the row's largest value is met in u only
    up = spoil(torch.randn(M, N, generator=gen) * 1e30, 1e38).bfloat16()
    dh = torch.ones(M, N).bfloat16()
    gate = (torch.rand(M, N, generator=gen) + 0.5).bfloat16()
    out = Q.q4_gated_backward(w, u, dh.cuda(), gate.cuda(), up.cuda(), act=Q.Q4_ACT_RELU)
    dup = gate.double()
    same_kind(out["dgate"], up.double(), torch.bfloat16, "dgate")
    same_kind(out["dx"], times(up.double(), W.T) + times(dup, U.T), torch.bfloat16, "dx, gated")


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_slopes_of_every_size(act):
    """dz = dy act'(pre) for pre of either sign over bfloat16's range: where the slope has
    reached 0 or 1, and where pre^3 leaves binary32's range."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    pre = torch.cat([bits, bits + 0x8000 - (1 << 16)]).to(torch.int16).view(torch.bfloat16).view(-1, 64)
    M = pre.shape[0]
    w, _ = G.weight("q4_0", 64, 64, 1)
    dz = Q.q4_linear_backward(w, torch.ones(M, 64).bfloat16().cuda(), act=G.ACTS[act], pre=pre.cuda())["dz"].double().cpu()
    z = pre.double().clamp(-1e3, 1e3)                     # the slopes there are 0 and 1 to 1e-400
    want = R.act(z, act)[1]
    # half a unit of the rounding, 1.5e-7 of GELU's distribution function times two, binary32's own
    assert ((dz - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all(), (pre.flatten()[((dz - want).abs() - 2.0 ** -8 * want.abs()).argmax()])
    one = torch.ones(M, 64).bfloat16().cuda()
    gated = Q.q4_gated_backward(w, w, one, pre.cuda(), one, act=G.ACTS[act])
    assert torch.equal(gated["dgate"].double().cpu(), dz)
    value = R.act(z, act)[0]
    value = torch.where(pre.double() > 1e3, pre.double(), value)
    got = gated["dup"].double().cpu()
    assert ((got - value).abs() <= 2.0 ** -8 * value.abs() + 1e-6).all()
