"""The feed-forward operators at the edges of their arguments, on the GPU."""
import pytest
import torch

import gemv_q4_affine_amd as Q

pytestmark = pytest.mark.gpu


def used_memory(*shape, dtype):
    """Leaves memory of this size, full of NaN, for the next allocation of it."""
    t = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    del t


@pytest.mark.parametrize("stream", [False, True])
def test_norm_gradients_of_no_rows(stream):
    """Sums over no rows are zeros: the gate's gradient among them."""
    D, groups, dt = 96, 5, torch.bfloat16
    none = torch.zeros(0, D, dtype=dt, device="cuda")
    w, gate = torch.ones(D, dtype=dt, device="cuda"), torch.ones(groups, D, dtype=dt, device="cuda")
    s = torch.cuda.Stream() if stream else None
    with torch.cuda.stream(s):
        used_memory(groups, D, dtype=dt)
        used_memory(D, dtype=torch.float32)
    out = Q.block_norm_backward(none, none, torch.zeros(0, 4, device="cuda"), none, none, pre_weight=w, pre_bias=w,
                                post_norm=Q.Q4_NORM_LAYER, post_weight=w, post_bias=w, gate=gate, stream=s)
    torch.cuda.synchronize()
    assert out["dr"].shape == out["dy"].shape == (0, D) and out["dgate"].shape == (groups, D)
    for name in ("dgate", "pre_dw", "pre_db", "post_dw", "post_db"):
        assert (out[name] == 0).all(), name


def test_a_dz_that_would_be_dy_is_refused():
    """Without an activation dz is dy: the C ABI refuses a dz output, and so does the
    binding, which must not leave the caller's tensor unwritten."""
    w = Q.q4_quantize(torch.randn(64, 64, device="cuda"))
    dy = torch.ones(3, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(Q.Q4Error):
        Q.q4_linear_backward(w, dy, dz=torch.empty_like(dy))
    assert set(Q.q4_linear_backward(w, dy)) == {"dx"}
    dz = torch.zeros_like(dy)
    out = Q.q4_linear_backward(w, dy, act=Q.Q4_ACT_RELU, pre=dy, dz=dz)
    assert out["dz"] is dz and torch.equal(dz, dy)


def test_more_rows_than_one_launch_of_the_packers():
    """2^25 rows and more: the row packers' 1024 threads for each eight rows pass 2^32."""
    M, N, K = (1 << 25) + 4 * 1024 + 40, 8, 64
    gen = torch.Generator("cuda").manual_seed(1)
    w = Q.q4_quantize(torch.randn(N, K, device="cuda", generator=gen))
    x = torch.randn(M, K, device="cuda", generator=gen, dtype=torch.bfloat16)
    y = Q.q4_linear(w, x)
    ends = [slice(0, 128), slice((1 << 24) - 64, (1 << 24) + 64), slice(M - 128, M)]
    for part in ends:
        assert torch.equal(y[part], Q.q4_linear(w, x[part].contiguous())), part
    del x
    pre = torch.randn(M, N, device="cuda", generator=gen, dtype=torch.bfloat16)
    out = Q.q4_linear_backward(w, y, act=Q.Q4_ACT_SILU, pre=pre, bias_grad=True)
    for part in ends:
        small = Q.q4_linear_backward(w, y[part].contiguous(), act=Q.Q4_ACT_SILU, pre=pre[part].contiguous())
        assert torch.equal(out["dx"][part], small["dx"]) and torch.equal(out["dz"][part], small["dz"]), part
    # dz as it was summed, before its rounding; binary32 sums of 2^25 terms in groups of eight, then in order
    s = torch.sigmoid(pre.double())
    want = (y.double() * s * (1 + pre.double() * (1 - s))).sum(0)
    size = (y.double() * s * (1 + pre.double() * (1 - s))).square().sum(0).sqrt()
    assert ((out["dbias"].double() - want).abs() <= 1e-3 * size + 1e-6 * want.abs()).all()
