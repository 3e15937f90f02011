"""8-bit block-scaled layers, trained and served with dense_gemm_11_gb300.

train():  a linear layer fitted to random targets.  Every step quantizes the
          weights, the activations and the output gradient, and takes the three
          products of the layer from their 8-bit forms: y = x W^T + b (bias in
          the epilogue), dx = dy W and dW = dy^T x (summed into FP32 gradients).
serve():  a mixture-of-experts feed-forward layer whose expert matrices are
          quantized once; decode steps of a few tokens replay a CUDA graph of
          norm-free residual layers, one kernel a layer.

    python examples/fp8_layers.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_11_gb300 as g  # noqa: E402


class Linear8:
    """y = x W^T + b with FP32 master weights and 8-bit products."""

    def __init__(self, n_in, n_out, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.W = torch.randn(n_out, n_in, generator=gen, device="cuda") * n_in ** -0.5
        self.b = torch.zeros(n_out, device="cuda")
        self.dW, self.db = torch.zeros_like(self.W), torch.zeros_like(self.b)
        self.Wq = g.fp8_empty(n_out, n_in, "blocks")
        g.fp8_quantize(self.W, *self.Wq, "blocks")

    def forward(self, x):
        T, n_in = x.shape
        self.x = x
        xq = g.fp8_empty(T, n_in, "rows")
        g.fp8_quantize(x, *xq, "rows")
        y = torch.empty(T, self.W.shape[0], dtype=torch.bfloat16, device="cuda")
        g.gemm_fp8(*xq, *self.Wq, y, bias=self.b)
        return y

    def backward(self, dy):
        """Gradient of x; those of W and b are added to dW and db."""
        T, n_out = dy.shape
        rows, cols = g.fp8_empty(T, n_out, "rows", torch.float8_e5m2), g.fp8_empty(T, n_out, "cols", torch.float8_e5m2)
        xc = g.fp8_empty(*self.x.shape, "cols")
        g.fp8_quantize(dy, *rows, "rows")
        g.fp8_quantize(dy, *cols, "cols")
        g.fp8_quantize(self.x, *xc, "cols")
        dx = torch.empty_like(self.x)
        g.gemm_fp8(*rows, *self.Wq, dx, b_trans=False)
        g.gemm_fp8(*cols, *xc, self.dW, beta=1.0, b_scales="rows")
        self.db += dy.float().sum(0)
        return dx

    def step(self, lr):
        self.W -= lr * self.dW
        self.b -= lr * self.db
        self.dW.zero_()
        self.db.zero_()
        g.fp8_quantize(self.W, *self.Wq, "blocks")


def train(tokens=1000, n_in=1024, n_out=768, steps=30, lr=0.5, seed=1):
    """Losses of a fit to a random linear map."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, n_in, generator=gen, device="cuda").bfloat16()
    target = x.float() @ (torch.randn(n_in, n_out, generator=gen, device="cuda") * n_in ** -0.5)
    layer, losses = Linear8(n_in, n_out), []
    for _ in range(steps):
        diff = layer.forward(x).float() - target
        losses.append(float((diff ** 2).mean()))
        layer.backward((diff / tokens).bfloat16())
        layer.step(lr)
    return losses


class MoE8:
    """A mixture-of-experts feed-forward layer with 8-bit expert matrices."""

    def __init__(self, experts, top_k, width, inner, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.top_k = top_k
        self.router = (torch.randn(experts, width, generator=gen, device="cuda") * width ** -0.5).bfloat16()
        self.mats, self.scales = [], []
        for rows, cols in ((inner, width), (inner, width), (width, inner)):
            Q = torch.empty(experts, rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
            S = torch.empty(experts, -(-rows // 128), -(-cols // 128), device="cuda")
            for e in range(experts):
                w = torch.randn(rows, cols, generator=gen, device="cuda") * cols ** -0.5
                g.fp8_quantize(w, Q[e], S[e], "blocks")
            self.mats.append(Q)
            self.scales.append(S)

    def __call__(self, x, y):
        g.moe_few_tokens(x, self.router, *self.mats, y, self.top_k, scales=self.scales)


def serve(tokens=4, experts=16, top_k=2, width=1024, inner=512, layers=3, steps=5):
    """Hidden states after `steps` replays of the captured layers, and the same without a graph."""
    stack = [MoE8(experts, top_k, width, inner, seed=i) for i in range(layers)]
    x, y = torch.empty(tokens, width, dtype=torch.bfloat16, device="cuda"), torch.empty(tokens, width, dtype=torch.bfloat16, device="cuda")

    def decode():
        for layer in stack:
            layer(x, y)
            x.add_(y, alpha=0.5)

    gen = torch.Generator(device="cuda").manual_seed(7)
    start = torch.randn(tokens, width, generator=gen, device="cuda").bfloat16()
    x.copy_(start)
    for _ in range(steps):
        decode()
    plain = x.clone()
    graph = torch.cuda.CUDAGraph()
    x.copy_(start)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        decode()
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    return x.clone(), plain


def main():
    losses = train()
    print("8-bit linear layer: loss %.4f -> %.5f in %d steps" % (losses[0], losses[-1], len(losses)))
    captured, plain = serve()
    print("8-bit mixture of experts: %d tokens decoded, graph and plain calls %s" % (len(captured), "agree" if torch.equal(captured, plain) else "differ"))
    assert g.check() == g.GEMM_OK


if __name__ == "__main__":
    main()
