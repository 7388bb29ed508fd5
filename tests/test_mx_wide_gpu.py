"""The products on microscaled numbers at the sizes that take every tile and
split, with offsets past 32 bits, at once on two streams, and on planes that
they refuse.  Tolerances: test_mx_gpu's."""
import math

import pytest
import torch

import gemv_q4_affine_amd as Q
from test_mx_gpu import ACTS, DT, F32, U, bar, near, say

pytestmark = pytest.mark.gpu


def planes(R, K, bits, seed):
    """Random planes on the GPU: any 4-bit code, 8-bit ones within a few powers of two, scales around 1."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if bits == 4:
        q = torch.randint(0, 256, (R, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    else:
        q = torch.randint(32, 120, (R, K), generator=gen, device="cuda", dtype=torch.uint8)
        q |= torch.randint(0, 2, (R, K), generator=gen, device="cuda", dtype=torch.uint8) << 7
    return q, torch.randint(119, 125, (R, K // 32), generator=gen, device="cuda", dtype=torch.uint8)


def values(p):
    """Binary64 values by the dequantiser, which test_mx_gpu holds to every code and scale."""
    return Q.mx_dequantize(p, dtype=torch.float32).double()


def act64(z, kind):
    if kind == "silu":
        return z * torch.sigmoid(z)
    return z * 0.5 * torch.erfc(-z / math.sqrt(2)) if kind == "gelu" else z


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,N,K", [(4096, 4096, 2080), (2050, 12289, 544), (1030, 4100, 1024), (33000, 100, 2048), (130, 640, 16384),
                                   (70, 264, 9984), (500, 3000, 128), (256, 8192, 256), (2048, 3104, 64)])
def test_every_tile(bits, M, N, K):
    kind, tol = ("fp8" if bits == 8 else "fp4"), 2.0
    w, x = planes(N, K, 4, M), planes(M, K, bits, N)
    W, X = values(w), values(x)
    for dt, act, extra in (("bf16", "none", False), ("f16", "silu", True), ("bf16", "gelu", True)):
        say(f"linear {kind} M={M} N={N} K={K} {dt} {act}")
        gen = torch.Generator(device="cuda").manual_seed(5)
        b = torch.randn(N, generator=gen, device="cuda").to(DT[dt]) if extra else None
        r = torch.randn(M, N, generator=gen, device="cuda").to(DT[dt]) if extra else None
        got = Q.mx_linear(w, x, bias=b, act=ACTS[act], residual=r, save_pre=extra, dtype=DT[dt])
        z = X @ W.T
        z = z if b is None else z + b.double()
        y = act64(z, act)
        y = y if r is None else y + r.double()
        # an activation's slope is at most 1.13, and its value's error that of z, which may be the larger
        grow = max(1.0, 1.13 * (z.norm() / y.norm()).item())
        near(got[0] if extra else got, y.cpu(), grow * bar(DT[dt], kind), "y")
        if extra:
            near(got[1], z.cpu(), bar(DT[dt], kind), "pre")
    u = planes(N, K, 4, M + 1)
    h, g, up = Q.mx_gated(w, u, x, save_pre=True)
    g64, u64 = X @ W.T, X @ values(u).T
    h64 = act64(g64, "silu") * u64
    grow = max(1.0, 1.13 * ((g64.abs() * u64.abs()).norm() / h64.norm()).item())
    near(h, h64.cpu(), U[torch.bfloat16] + tol * grow * (bar(torch.bfloat16, kind) - U[torch.bfloat16]), "h")
    near(g, g64.cpu(), bar(torch.bfloat16, kind), "g")
    near(up, u64.cpu(), bar(torch.bfloat16, kind), "u")
    assert torch.equal(Q.mx_gated(w, u, x), h), "with and without the projections"


def columns(w, x, y, rows, cols):
    """Outputs at some rows and columns against binary64."""
    W, X = values((w[0][cols], w[1][cols])), (x[rows].double() if isinstance(x, torch.Tensor) else values((x[0][rows], x[1][rows])))
    near(y[rows][:, cols], (X @ W.T).cpu(), bar(y.dtype, "fp8") + F32, "sample")


@pytest.mark.parametrize("M,x", [(1, "fp8"), (3, "fp8"), (20, "fp8"), (80, "fp8"), (1, "bf16"), (3, "bf16"), (20, "bf16")])
def test_weights_past_32_bits(M, x):
    N, K = 70000, 131072                                    # 4.6 GB of codes
    w = planes(N, K, 4, 3)
    xs = planes(M, K, 8, 4) if x == "fp8" else torch.randn(M, K, device="cuda").bfloat16()
    y = Q.mx_linear(w, xs)
    columns(w, xs, y, torch.arange(M, device="cuda")[::7], torch.tensor([0, 1, 35000, 65535, 65537, N - 1], device="cuda"))


@pytest.mark.parametrize("bits", [8, 4])
def test_rows_and_outputs_past_32_bits(bits):
    M, N, K = 40000, 96, 131072 * 8 // bits                 # 5.2 GB of codes of x
    w, x = planes(N, K, 4, 3), planes(M, K, bits, 4)
    y = Q.mx_linear(w, x)
    columns(w, x, y, torch.tensor([0, 255, 32767, 32769, M - 1], device="cuda"), torch.arange(N, device="cuda")[::5])
    del x, y
    M, N, K = 70000, 40008, 96                              # 5.6 GB of outputs
    w, x = planes(N, K, 4, 5), planes(M, K, bits, 6)
    y = Q.mx_linear(w, x)
    columns(w, x, y, torch.tensor([0, 53681, 53690, M - 1], device="cuda"), torch.tensor([0, 7, 20000, N - 1], device="cuda"))


def test_planes_past_32_bits():
    v = torch.randn(70000, 32768, device="cuda", dtype=torch.bfloat16)
    q, s = Q.mx_quantize(v, Q.Q4_MXFP8)
    back = Q.mx_dequantize((q, s), dtype=torch.bfloat16)
    for rows in (slice(0, 3), slice(65533, 65540), slice(69998, 70000)):
        alone = Q.mx_quantize(v[rows].contiguous(), Q.Q4_MXFP8)
        assert torch.equal(q[rows], alone[0]) and torch.equal(s[rows], alone[1])
        assert torch.equal(back[rows], Q.mx_dequantize(alone, dtype=torch.bfloat16))


@pytest.mark.parametrize("M", [1, 16, 50, 300])
def test_two_streams_at_once(M):
    N, K = 2048, 4096
    w, u = planes(N, K, 4, 1), planes(N, K, 4, 2)
    xs = [planes(M, K, 8, s) for s in (3, 4)]
    want = [(Q.mx_linear(w, x), Q.mx_gated(w, u, x)) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(8):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append((Q.mx_linear(w, xs[k]), Q.mx_gated(w, u, xs[k])))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for k in (0, 1) for g in got[k] for a, b in zip(g, want[k]))


def test_refused_tensors():
    w, x = planes(64, 96, 4, 1), planes(5, 96, 8, 2)
    with pytest.raises(ValueError):
        Q.mx_linear((w[0].t().contiguous().t(), w[1]), x)                    # not contiguous
    with pytest.raises(ValueError):
        Q.mx_linear(w, (x[0].cpu(), x[1]))
    with pytest.raises(ValueError):
        Q.mx_linear((w[0].cpu(), w[1]), x)
    with pytest.raises(ValueError):
        Q.mx_linear(w, x, residual=torch.zeros(5, 64, device="cuda", dtype=torch.float16))
    with pytest.raises(Q.Q4Error):
        Q.mx_linear((w[0][1:], w[1][1:]), x)                                   # scales from byte 3 on: not aligned
    with pytest.raises(Q.Q4Error):
        Q.mx_linear(w, planes(100, 96, 8, 2), workspace=None)                  # needs one
    with pytest.raises(TypeError):
        Q.mx_linear(w, torch.zeros(5, 96, device="cuda", dtype=torch.float64))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,N,K", [(33, 12290, 4128), (50, 9000, 2048), (64, 5000, 4096), (64, 4096, 4096), (40, 70000, 64), (32, 12290, 4128)])
def test_gated_by_columns_or_tiles(M, N, K, bits):
    """33 to 64 rows: where the row tiles make one round of the GPU they are streamed, else multiplied as tiles."""
    kind = "fp8" if bits == 8 else "fp4"
    w, u, x = planes(N, K, 4, M), planes(N, K, 4, M + 1), planes(M, K, bits, N)
    h, g, up = Q.mx_gated(w, u, x, save_pre=True)
    g64, u64 = values(x) @ values(w).T, values(x) @ values(u).T
    h64 = act64(g64, "silu") * u64
    grow = max(1.0, 1.13 * ((g64.abs() * u64.abs()).norm() / h64.norm()).item())
    near(h, h64.cpu(), U[torch.bfloat16] + 2.0 * grow * (bar(torch.bfloat16, kind) - U[torch.bfloat16]), "h")
    near(g, g64.cpu(), bar(torch.bfloat16, kind), "g")
    near(up, u64.cpu(), bar(torch.bfloat16, kind), "u")
    for m in (0, M - 1):                                     # rows do not depend on their neighbours
        assert torch.allclose(Q.mx_linear(w, (x[0][m:m + 1].clone(), x[1][m:m + 1].clone())).float(), g[m].float(), rtol=2.0 ** -6, atol=1e-4 * g64.abs().max().item())


@pytest.mark.parametrize("scale", [104, 140])
def test_smallest_and_largest_scales_of_the_images(scale):
    """2^-23 to 2^13: every 4-bit code is exact in binary16, forward and transposed."""
    M, N, K = 70, 96, 256
    w = planes(N, K, 4, 7)
    w[1].fill_(scale)
    gen = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    near(Q.mx_linear(w, x), (x.double() @ values(w).T).cpu(), bar(torch.bfloat16), "y")
    dy = torch.randn(M, N, generator=gen, device="cuda").bfloat16()
    near(Q.mx_linear_backward(w, dy)["dx"], (dy.double() @ values(w)).cpu(), bar(torch.bfloat16), "dx")


@pytest.mark.parametrize("M,N,K", [(65, 200, 4128), (128, 3000, 1056), (129, 9000, 2048), (300, 9001, 320), (700, 8200, 544), (1000, 30, 96)])
def test_bf16_by_columns_or_images(M, N, K):
    """More than 64 rows of bfloat16: 64 at a time where that is few turns, else images; the residual in place."""
    w, u = planes(N, K, 4, M), planes(N, K, 4, M + 1)
    gen = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    r = torch.randn(M, N, generator=gen, device="cuda").bfloat16()
    b = torch.randn(N, generator=gen, device="cuda").bfloat16()
    z = x.double() @ values(w).T + b.double()
    y, r64 = r.clone(), r.double()
    got = Q.mx_linear(w, x, bias=b, residual=y, y=y, save_pre=True)
    near(y, (z + r64).cpu(), bar(torch.bfloat16), "y")
    near(got[1], z.cpu(), bar(torch.bfloat16), "pre")
    h, g, up = Q.mx_gated(w, u, x, save_pre=True)
    g64, u64 = x.double() @ values(w).T, x.double() @ values(u).T
    h64 = act64(g64, "silu") * u64
    grow = max(1.0, 1.13 * ((g64.abs() * u64.abs()).norm() / h64.norm()).item())
    near(h, h64.cpu(), U[torch.bfloat16] + 2.0 * grow * (bar(torch.bfloat16) - U[torch.bfloat16]), "h")
    near(g, g64.cpu(), bar(torch.bfloat16), "g")
    near(up, u64.cpu(), bar(torch.bfloat16), "u")


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,N,K", [(65, 4096, 4128), (128, 4000, 4096), (200, 500, 8192), (1000, 20, 4096), (129, 5000, 4096)])
def test_long_sums_of_a_few_more_rows(bits, M, N, K):
    kind = "fp8" if bits == 8 else "fp4"
    w, x = planes(N, K, 4, M), planes(M, K, bits, N)
    r = torch.randn(M, N, device="cuda").bfloat16()
    y = r.clone()
    z = values(x) @ values(w).T
    got = Q.mx_linear(w, x, residual=y, y=y, save_pre=True)
    near(got[0], (z + r.double()).cpu(), bar(torch.bfloat16, kind), "y")
    near(got[1], z.cpu(), bar(torch.bfloat16, kind), "pre")
