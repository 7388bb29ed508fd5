"""q4_linear and q4_gated at up to 64 rows and many columns, where a workgroup takes one,
two or three tiles of 16 columns and the last one ends inside them: against
binary64 (tolerances as in test_block_gpu), the last columns by themselves too.
"""
import pytest
import torch

import block_reference as R
import gemv_q4_affine_amd as Q
import test_block_gpu as G

pytestmark = pytest.mark.gpu


def near(got, want, limit, what):
    G.near(got, want, limit, what)
    # 49 columns: the last tile of 16 and a workgroup's before it.  The fewer the values, the less even a rounding error's size
    G.near(got[:, -49:], want[:, -49:], 1.5 * limit, what + ", last columns")


# 256 CUs: one tile a workgroup up to N = 4096, two to 8192, three to 12288 (8 bits: at 5 to 16 rows), then two
@pytest.mark.parametrize("N", [4111, 8176, 8193, 8241, 10007, 12288, 12289, 16401])
@pytest.mark.parametrize("M", [1, 3, 4, 5, 8, 16, 17, 32, 40, 64])
@pytest.mark.parametrize("fmt", R.FMTS)
def test_wide(fmt, M, N):
    gen = torch.Generator().manual_seed(M + N)
    K = 64 * (1 + (M + N) % 13)                         # inside one step of 256 (128) and over several
    (w, W), (u, U) = G.weight(fmt, N, K, M), G.weight(fmt, N, K, M + 1)
    for dt in (torch.bfloat16, torch.float16):
        G.say(f"wide {fmt} M={M} N={N} K={K} {dt}")
        x, x64 = G.rand(gen, M, K, dtype=dt)
        b, b64 = G.rand(gen, N, dtype=dt)
        r, r64 = G.rand(gen, M, N, dtype=dt)
        y, pre = Q.q4_linear(w, x, bias=b, act=Q.Q4_ACT_SILU, residual=r, save_pre=True)
        y64, z64 = R.linear(x64, W, b64, "silu", r64)
        near(y, y64, G.bar(dt), "y")
        near(pre, z64, G.bar(dt), "pre")
        if N in (8193, 12289):
            near(Q.q4_gated(w, u, x, up_bias=b), R.gated(x64, W, U, None, b64, "silu")[0], G.bar(dt, 4), "h")
        assert torch.equal(Q.q4_linear(w, x, bias=b, act=Q.Q4_ACT_SILU, residual=r), y), "not deterministic"
