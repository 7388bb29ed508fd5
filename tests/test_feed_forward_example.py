"""examples/feed_forward.py on the GPU: the three operators together, forward and
backward, against the same layer in binary64 on dequantised weights."""
import importlib.util
import os

import pytest
import torch

import gemv_q4_affine_amd as Q

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(layer, r, y, w):
    Wg, Wu, Wd = (Q.q4_dequantize(*p, out_dtype=torch.float32).double().cpu() for p in (layer.gate, layer.up, layer.down))
    r1 = r + y
    n = r1 / torch.sqrt((r1 * r1).mean(1, keepdim=True) + layer.eps) * w
    g = n @ Wg.T
    return r1 + (g * torch.sigmoid(g) * (n @ Wu.T)) @ Wd.T


@pytest.mark.parametrize("M", [1, 9, 40, 200])
def test_layer_and_its_gradients(M):
    """n and h are rounded to bfloat16 on the way (2^-8 each) and the output once
    more; the gradients also pass dh and dn through bfloat16."""
    layer, _ = example().random_layer(256, 704, seed=M)
    gen = torch.Generator().manual_seed(M)
    r, y, d = (torch.randn(M, 256, generator=gen).bfloat16() for _ in range(3))
    with torch.no_grad():
        out = layer(r.cuda(), y.cuda())
    rc, yc = r.cuda().requires_grad_(), y.cuda().requires_grad_()
    layer.weight.requires_grad_()
    trained = layer(rc, yc)
    assert torch.equal(trained.detach(), out)
    trained.backward(d.cuda())
    r64, y64 = r.double().requires_grad_(), y.double().requires_grad_()
    w64 = layer.weight.detach().double().cpu().requires_grad_()
    want = reference(layer, r64, y64, w64)
    want.backward(d.double())
    u = 2.0 ** -8
    for got, exact, limit in ((out, want.detach(), 3 * u), (rc.grad, r64.grad, 4 * u), (yc.grad, y64.grad, 4 * u),
                              (layer.weight.grad, w64.grad, 4 * u)):
        e = ((got.double().cpu() - exact).norm() / exact.norm()).item()
        assert e <= limit, (e, limit)
    layer.weight.requires_grad_(False)


def test_example_runs(capsys):
    example().main()
    out = capsys.readouterr().out
    assert "one token" in out and "training step" in out
