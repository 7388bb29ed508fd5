"""The feed-forward half of a transformer layer on quantised weights.

    r' = r + y                    y: the attention block's output, r: the residual stream
    n  = rms_norm(r') * weight
    h  = silu(n Wgate^T) * (n Wup^T)
    out = r' + h Wdown^T

``FeedForward`` runs it with the library's block_norm, q4_gated and q4_linear:
three launches for a token.  With gradients wanted it is a torch autograd
function, for training adapters or norms around the frozen weights.

    python examples/feed_forward.py          # a token, a prompt and a training step, timed
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemv_q4_affine_amd as Q  # noqa: E402


class _Train(torch.autograd.Function):
    @staticmethod
    def forward(ctx, r, y, weight, layer):
        r1, n, stats = Q.block_norm(r, y, pre_weight=weight, eps=layer.eps, save_stats=True)
        h, gate_pre, up_pre = Q.q4_gated(layer.gate, layer.up, n, save_pre=True)
        ctx.layer = layer
        ctx.save_for_backward(r1, y, weight, stats, gate_pre, up_pre)
        return Q.q4_linear(layer.down, h, residual=r1)

    @staticmethod
    def backward(ctx, d):
        r1, y, weight, stats, gate_pre, up_pre = ctx.saved_tensors
        layer, d = ctx.layer, d.contiguous()
        dh = Q.q4_linear_backward(layer.down, d)["dx"]
        dn = Q.q4_gated_backward(layer.gate, layer.up, dh, gate_pre, up_pre)["dx"]
        g = Q.block_norm_backward(r1, y, stats, dn, d, pre_weight=weight)
        return g["dr"], g["dy"], g["pre_dw"].to(weight.dtype), None


class FeedForward:
    """gate, up [N, D] and down [D, N]: planes of one of the library's formats
    (what its quantisers return); weight: the norm's, bfloat16 [D]."""

    def __init__(self, gate, up, down, weight, eps=1e-5):
        self.gate, self.up, self.down, self.weight, self.eps = gate, up, down, weight, eps

    def __call__(self, r, y):
        """r, y bfloat16 [M, D] -> the stream after the block, [M, D]."""
        if torch.is_grad_enabled() and any(t.requires_grad for t in (r, y, self.weight)):
            return _Train.apply(r, y, self.weight, self)
        r1, n, _ = Q.block_norm(r, y, pre_weight=self.weight, eps=self.eps)
        return Q.q4_linear(self.down, Q.q4_gated(self.gate, self.up, n), residual=r1)


def random_layer(D, N, seed=0, scale=0.02):
    """A layer with random Q4_0 weights, and the weights before quantisation."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dense = [torch.randn(*shape, generator=gen, device="cuda") * scale for shape in ((N, D), (N, D), (D, N))]
    weight = (torch.randn(D, generator=gen, device="cuda") * 0.1 + 1).bfloat16()
    return FeedForward(*(Q.q4_quantize(w) for w in dense), weight), dense


def main():
    D, N = 2048, 8192
    layer, _ = random_layer(D, N)
    for M, what in ((1, "decode, one token"), (512, "prompt, 512 tokens")):
        r, y = (torch.randn(M, D, device="cuda").bfloat16() for _ in range(2))
        for _ in range(20):
            out = layer(r, y)
        torch.cuda.synchronize()
        start = time.perf_counter()
        for _ in range(100):
            out = layer(r, y)
        torch.cuda.synchronize()
        print(f"{what}: {(time.perf_counter() - start) * 1e4:.1f} us, |out| {out.float().norm().item():.1f}", flush=True)
    r, y = (torch.randn(512, D, device="cuda").bfloat16().requires_grad_() for _ in range(2))
    layer.weight.requires_grad_()
    out = layer(r, y)
    loss = out.float().square().mean()
    loss.backward()
    print(f"training step, 512 tokens: loss {loss.item():.4f}, |dr| {r.grad.float().norm().item():.4g}, "
          f"|dweight| {layer.weight.grad.float().norm().item():.4g}", flush=True)


if __name__ == "__main__":
    main()
