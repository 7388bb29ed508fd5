"""The feed-forward operators in binary64 on the CPU, from their definitions:
what the GPU tests compare with.  Shares no code with the library."""
import math

import numpy as np
import torch

FMTS = ("q4_0", "affine4", "affine8")


def planes(fmt, N, K, seed, scale=0.02):
    """Random planes (numpy, bit patterns) of an [N, K] matrix and its binary64 values."""
    rng = np.random.default_rng(seed)
    if fmt == "q4_0":
        codes = rng.integers(0, 16, (N, K // 32, 32), dtype=np.uint8)
        d = (rng.standard_normal((N, K // 32)) * scale / 4).astype(np.float16)
        W = (codes.astype(np.float64) - 8) * d.astype(np.float64)[..., None]
        return (codes[..., :16] | (codes[..., 16:] << 4), d.view(np.int16)), torch.from_numpy(W.reshape(N, K))
    top = 15 if fmt == "affine4" else 255
    codes = rng.integers(0, top + 1, (N, K), dtype=np.uint8)
    s = torch.from_numpy(rng.uniform(0.5, 1.5, (N, K // 64)) * scale * 4 / top).bfloat16()
    b = torch.from_numpy(rng.uniform(-2.5, -1.5, (N, K // 64)) * scale).bfloat16()
    W = torch.from_numpy(codes.astype(np.float64)).view(N, K // 64, 64) * s.double()[..., None] + b.double()[..., None]
    q = codes if fmt == "affine8" else codes[:, 0::2] | (codes[:, 1::2] << 4)
    return (np.ascontiguousarray(q), s.view(torch.int16).numpy(), b.view(torch.int16).numpy()), W.view(N, K)


def act(z, kind):
    """Value and slope of an activation."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return torch.clamp(z, min=0), (z > 0).double()
    if kind == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if kind == "gelu":
        F = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * F, F + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    v = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    t = torch.tanh(v)
    return z * (1 + t) / 2, (1 + t) / 2 + z * (1 - t * t) / 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)


def linear(x, W, bias, kind, residual):
    z = x @ W.T if bias is None else x @ W.T + bias
    y = act(z, kind)[0]
    return (y if residual is None else y + residual), z


def linear_grad(W, dy, pre, kind):
    dz = dy if kind == "none" else dy * act(pre, kind)[1]
    return dz @ W, dz, dz.sum(0)


def gated(x, Wg, Wu, bg, bu, kind):
    g, u = linear(x, Wg, bg, "none", None)[0], linear(x, Wu, bu, "none", None)[0]
    return act(g, kind)[0] * u, g, u


def gated_grad(Wg, Wu, dh, g, u, kind):
    value, slope = act(g, kind)
    dg, du = dh * u * slope, dh * value
    return dg @ Wg + du @ Wu, dg, du, dg.sum(0), du.sum(0)


def norm(v, kind, w, b, eps):
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros(v.shape[0], 1, dtype=v.dtype)
    rstd = 1 / torch.sqrt(((v - mean) ** 2).mean(1, keepdim=True) + eps)
    if kind == "none":
        return v, mean * 0, rstd * 0 + 1
    out = (v - mean) * rstd
    out = out if w is None else out * w
    return (out if b is None else out + b), mean, rstd


def block_norm(r, y, c):
    """c: pre, post, pre_w, pre_b, post_w, post_b, gate (one row per row of r, or None), scale, eps."""
    M = r.shape[0]
    m0, i0 = torch.zeros(M, 1, dtype=r.dtype), torch.ones(M, 1, dtype=r.dtype)
    if y is not None:
        p, m0, i0 = norm(y, c["post"], c["post_w"], c["post_b"], c["eps"])
        r = r + c["scale"] * (p if c["gate"] is None else c["gate"] * p)
    n, m1, i1 = norm(r, c["pre"], c["pre_w"], c["pre_b"], c["eps"])
    return r, n, torch.cat([m0, i0, m1, i1], 1)


def rel(got, want):
    got, want = got.double().cpu(), want.double().cpu()
    d = (got - want).norm().item()
    n = want.norm().item()
    return d / n if n else (0.0 if d == 0 else math.inf)
