"""A mixture-of-experts feed-forward layer for many tokens, forward and backward, with dense_gemm_11_gb300.

Forward: the router's choice sorted by expert and the tokens' rows copied into
that order, one product for the gates and the other inputs of all experts, the
gated activation (which keeps its inputs in 8 bits), the product down, and the
rows back to their tokens.  Backward: the same path the other way.  What is kept
between the two: the sorted rows and the experts' results in 16 bits, the inputs
of the activation in 8.

    python examples/moe_training.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_11_gb300 as g  # noqa: E402

BF16 = torch.bfloat16


def empty(*shape, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="cuda")


class MoELayer:
    """y = sum_j w_j down[e_j] (silu(gate[e_j] x) * (up[e_j] x)), w the softmax of the top_k largest logits x router.

    The experts' weights are BF16, the router (width x experts) FP32; gradients are FP32 and summed over calls of backward().
    """

    def __init__(self, experts, top_k, width, inner, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return (torch.randn(shape, generator=gen, device="cuda") * shape[-1] ** -0.5).to(BF16)

        self.top_k, self.inner = top_k, inner
        self.router = torch.randn(width, experts, generator=gen, device="cuda") * width ** -0.5
        self.gate_up = normal(experts, 2 * inner, width)  # gates in the first rows of each, the others below
        self.down = normal(experts, width, inner)
        self.grads = {n: torch.zeros(getattr(self, n).shape, device="cuda") for n in ("router", "gate_up", "down")}

    def forward(self, x):
        T, H = x.shape
        E, k, I, n = self.router.shape[1], self.top_k, self.inner, x.shape[0] * self.top_k
        logits = empty(T, E, dtype=torch.float32)
        g.gemm_f32(x.float(), self.router, logits)
        top, chosen = logits.topk(k, dim=1)
        self.x, self.chosen, self.w = x, chosen, torch.softmax(top, dim=1)
        self.offsets, self.rows = empty(E + 1, dtype=torch.int32), empty(T, k, dtype=torch.int32)
        self.xs, gu, h, self.ys, y = empty(n, H), empty(n, 2 * I), empty(n, I), empty(n, H), empty(T, H)
        self.kept = [*g.fp8_empty(n, I), *g.fp8_empty(n, I)]
        g.moe_dispatch(chosen.int(), x, self.xs, self.offsets, self.rows)
        g.gemm_grouped(self.xs, self.gate_up, gu, self.offsets)
        g.fp8_gated_act(gu[:, :I], gu[:, I:], h, *self.kept)
        g.gemm_grouped(h, self.down, self.ys, self.offsets)
        g.moe_combine(self.ys, self.rows, y, self.w)
        return y

    def backward(self, dy):
        """Gradient of x; those of the weights are added to grads."""
        n, H = self.xs.shape
        I = self.inner
        dys, dw = empty(n, H), torch.empty_like(self.w)
        g.moe_combine_grad(dy, self.ys, self.rows, self.w, dys, dw)
        dh, dgu, h, dxs, dx = empty(n, I), empty(n, 2 * I), empty(n, I), empty(n, H), empty(*dy.shape)
        g.gemm_grouped(dys, self.down, dh, self.offsets, b_trans=False)
        g.fp8_gated_act_grad(dh, *self.kept, dgu[:, :I], dgu[:, I:], h)
        g.gemm_grouped_wgrad(dys, h, self.grads["down"], self.offsets, beta=1.0)
        g.gemm_grouped_wgrad(dgu, self.xs, self.grads["gate_up"], self.offsets, beta=1.0)
        g.gemm_grouped(dgu, self.gate_up, dxs, self.offsets, b_trans=False)
        g.moe_combine(dxs, self.rows, dx)
        # the softmax of the chosen logits, and the router's product
        dlogits = torch.zeros(dy.shape[0], self.router.shape[1], device="cuda")
        dlogits.scatter_(1, self.chosen, self.w * (dw - (dw * self.w).sum(1, keepdim=True)))
        g.gemm_f32(self.x.float().t().contiguous(), dlogits, self.grads["router"], beta=1.0)
        dx_router = empty(*dy.shape, dtype=torch.float32)
        g.gemm_f32(dlogits, self.router.t().contiguous(), dx_router)
        return (dx.float() + dx_router).to(BF16)

    def step(self, lr):
        for name, grad in self.grads.items():
            w = getattr(self, name)
            w.copy_(w.float() - lr * grad)
            grad.zero_()


def train(tokens=1000, experts=16, top_k=3, width=512, inner=384, steps=20, lr=20.0, seed=1):
    """Losses of a fit to another random layer."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, width, generator=gen, device="cuda").to(BF16)
    target = MoELayer(experts, top_k, width, inner, seed=5).forward(x).float()
    layer, losses = MoELayer(experts, top_k, width, inner), []
    for _ in range(steps):
        diff = layer.forward(x).float() - target
        losses.append(float((diff ** 2).mean()))
        layer.backward((diff * (2 / diff.numel())).to(BF16))
        layer.step(lr)
    return losses


def main():
    losses = train()
    print("mixture of experts: loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], len(losses)))
    assert g.check() == g.GEMM_OK


if __name__ == "__main__":
    main()
