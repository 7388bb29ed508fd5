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
