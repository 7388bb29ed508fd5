"""Microscaled (MX) numbers in binary64 on the CPU, from their definition: what
the tests compare with.  Shares no code with the library; the activations,
norms and gradients are block_reference's."""
import numpy as np
import torch

#: Magnitudes by code.
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)])
E4M3[127] = np.nan
TOP = {"fp4": 2, "fp8": 8}
BITS = {"fp4": 4, "fp8": 8}


def table(kind):
    """Values of all codes of a type."""
    t = E2M1 if kind == "fp4" else E4M3
    return np.concatenate([t, -t])


def quantize(v, kind):
    """(codes one per value, scale bytes) of v [R, K] (binary64 numpy)."""
    R, K = v.shape
    b = v.reshape(R, K // 32, 32)
    finite = np.isfinite(b).all(2)
    amax = np.where(finite, np.abs(np.where(np.isfinite(b), b, 0)).max(2), 0)
    _, e = np.frexp(amax)                                  # amax = f 2^e, 1/2 <= f < 1
    e = np.where(amax > 0, np.maximum(e - 1 - TOP[kind], -127), -127)
    t = np.abs(np.where(finite[..., None], b, 0)) / 2.0 ** e[..., None].astype(float)
    mags = E2M1 if kind == "fp4" else E4M3[:127]
    up = np.searchsorted(mags, t).clip(0, len(mags) - 1)   # the first magnitude at or above
    down = (up - 1).clip(0)
    high, low = mags[up] - t, t - mags[down]
    c = np.where(high < low, up, np.where(low < high, down, np.where(up % 2 == 0, up, down)))
    c = np.where(t >= mags[-1], len(mags) - 1, c)
    sign = np.signbit(b) & finite[..., None]
    c = c + sign * (8 if kind == "fp4" else 128)
    return c.reshape(R, K).astype(np.uint8), np.where(finite, e + 127, 255).astype(np.uint8)


def values(codes, scales, kind):
    s = 2.0 ** (scales.astype(float) - 127)
    s[scales == 255] = np.nan
    return table(kind)[codes] * np.repeat(s, 32, 1)


def planes(codes, kind):
    """The code plane as the library lays it out."""
    return codes if kind == "fp8" else codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpacked(plane, kind):
    if kind == "fp8":
        return plane
    out = np.empty((plane.shape[0], plane.shape[1] * 2), np.uint8)
    out[:, 0::2], out[:, 1::2] = plane & 15, plane >> 4
    return out


def tensor(R, K, kind, seed, scale=1.0, spread=3):
    """Random planes (torch, on the CPU) of [R, K] numbers around `scale`, and their binary64 values."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16 if kind == "fp4" else 256, (R, K)).astype(np.uint8)
    if kind == "fp8":
        codes = np.where(codes & 127 == 127, codes - 1, codes).astype(np.uint8)      # NaNs
        codes = np.where((codes & 127) < 64, codes + 32, codes).astype(np.uint8)     # within a few powers of two
    at = int(np.floor(np.log2(scale))) - (0 if kind == "fp4" else 6)
    scales = (127 + at + rng.integers(-spread, spread + 1, (R, K // 32))).astype(np.uint8)
    return (torch.from_numpy(planes(codes, kind)), torch.from_numpy(scales)), torch.from_numpy(values(codes, scales, kind))
