"""The operators of a mixture-of-experts layer for many tokens in a run, as the example uses them."""
import importlib.util
import os

import pytest
import torch

import dense_gemm_11_gb300 as g
from conftest import ROOT, gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_training", os.path.join(ROOT, "examples", "moe_training.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def exact(layer, x, weights):
    """The layer in FP64, the experts as the layer chose them."""
    router, gate_up, down = weights
    w = torch.softmax((x @ router).gather(1, layer.chosen), dim=1)
    y = torch.zeros_like(x)
    for e in range(router.shape[1]):
        t, j = (layer.chosen == e).nonzero(as_tuple=True)
        gu = x[t] @ gate_up[e].t()
        h = torch.nn.functional.silu(gu[:, :layer.inner]) * gu[:, layer.inner:]
        y = y.index_add(0, t, (h @ down[e].t()) * w[t, j][:, None])
    return y


def relative(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("tokens,experts,top_k,width,inner", [(300, 8, 2, 256, 136), (1, 5, 3, 64, 48), (777, 40, 4, 128, 200)])
def test_layer_and_gradients(example, tokens, experts, top_k, width, inner):
    layer = example.MoELayer(experts, top_k, width, inner, seed=tokens)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, dy = torch.randn(tokens, width, generator=gen, device="cuda").to(BF16), torch.randn(tokens, width, generator=gen, device="cuda").to(BF16)
    y = layer.forward(x)
    dx = layer.backward(dy)
    assert g.check() == g.GEMM_OK
    leaves = [t.double().requires_grad_() for t in (x, layer.router, layer.gate_up, layer.down)]
    want = exact(layer, leaves[0], leaves[1:])
    want.backward(dy.double())
    # y: four roundings to BF16 on the way (2^-8 each at most), the activation's slope below 1.1
    assert relative(y, want.detach()) <= 4 * 1.1 * 2.0 ** -8
    # gradients: besides these the copies in e4m3, 2^-4 at most in each of g and u
    bound = 2 * 2.0 ** -4 + 8 * 2.0 ** -8
    for got, leaf in zip((dx, layer.grads["router"], layer.grads["gate_up"], layer.grads["down"]), leaves):
        assert relative(got, leaf.grad) <= bound
    # against differences: the layer along a direction of x, in FP64
    d = torch.randn(tokens, width, generator=gen, device="cuda").double()
    step = 1e-6
    up, low = (exact(layer, x.double() + s * step * d, [t.detach() for t in leaves[1:]]) for s in (1, -1))
    slope = float((((up - low) / (2 * step)) * dy.double()).sum())
    assert abs(float((dx.double() * d).sum()) - slope) <= bound * float(leaves[0].grad.norm() * d.norm())


def test_gradients_add_up(example):
    layer = example.MoELayer(4, 2, 64, 32)
    x = torch.randn(50, 64, device="cuda").to(BF16)
    layer.forward(x)
    layer.backward(x)
    once = {n: t.clone() for n, t in layer.grads.items()}
    layer.backward(x)
    for n, t in layer.grads.items():
        # twice the sum, one more addition's rounding
        assert torch.allclose(t, 2 * once[n], rtol=2.0 ** -22, atol=0)


def test_example_runs(example):
    losses = example.train(tokens=200, experts=6, top_k=2, width=128, inner=64, steps=3)
    assert len(losses) == 3 and all(torch.isfinite(torch.tensor(losses)))
    assert g.check() == g.GEMM_OK


class Job:
    """All calls of a layer's forward and backward pass on fixed tensors, with products that share scratch."""

    def __init__(self, seed, T=40, E=6, k=2, H=4096, I=256):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(BF16)  # noqa: E731
        n = T * k
        self.ids = torch.randint(0, E, (T, k), generator=gen, device="cuda").int()
        self.x, self.w13, self.wd, self.dy = r(T, H), r(E, 2 * I, H) / 64, r(E, H, I) / 16, r(T, H)
        self.weights = torch.rand(T, k, generator=gen, device="cuda")
        self.offsets, self.rows = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda")
        z = lambda *s, t=BF16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
        self.xs, self.gu, self.h, self.ys, self.y = z(n, H), z(n, 2 * I), z(n, I), z(n, H), z(T, H)
        self.kept = [*g.fp8_empty(n, I), *g.fp8_empty(n, I)]
        self.dys, self.dw, self.dh, self.dgu, self.hh, self.dxs, self.dx = z(n, H), z(T, k, t=torch.float32), z(n, I), z(n, 2 * I), z(n, I), z(n, H), z(T, H)
        self.gd, self.g13 = z(E, H, I, t=torch.float32), z(E, 2 * I, H, t=torch.float32)
        self.I = I

    def run(self, stream=None):
        I, s = self.I, {"stream": stream}
        g.moe_dispatch(self.ids, self.x, self.xs, self.offsets, self.rows, **s)
        g.gemm_grouped(self.xs, self.w13, self.gu, self.offsets, **s)
        g.fp8_gated_act(self.gu[:, :I], self.gu[:, I:], self.h, *self.kept, **s)
        g.gemm_grouped(self.h, self.wd, self.ys, self.offsets, **s)
        g.moe_combine(self.ys, self.rows, self.y, self.weights, **s)
        g.moe_combine_grad(self.dy, self.ys, self.rows, self.weights, self.dys, self.dw, **s)
        g.gemm_grouped(self.dys, self.wd, self.dh, self.offsets, b_trans=False, **s)
        g.fp8_gated_act_grad(self.dh, *self.kept, self.dgu[:, :I], self.dgu[:, I:], self.hh, **s)
        g.gemm_grouped_wgrad(self.dys, self.hh, self.gd, self.offsets, **s)
        g.gemm_grouped_wgrad(self.dgu, self.xs, self.g13, self.offsets, **s)
        g.gemm_grouped(self.dgu, self.w13, self.dxs, self.offsets, b_trans=False, **s)
        g.moe_combine(self.dxs, self.rows, self.dx, **s)

    def results(self):
        return [t.clone() for t in (self.offsets, self.rows, self.xs, self.gu, self.h, self.y, self.dys, self.dw, self.dgu, self.gd, self.g13, self.dx)]

    def clear(self):
        for t in (self.offsets, self.rows, self.xs, self.gu, self.h, self.ys, self.y, self.dys, self.dw, self.dh, self.dgu, self.hh, self.dxs, self.dx, self.gd, self.g13):
            t.zero_()


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_repeats_and_streams():
    """The same bits every time, on streams of their own at the same time, and through stream=."""
    jobs, want = [Job(i) for i in range(3)], []
    for j in jobs:
        j.run()
        torch.cuda.synchronize()
        want.append(j.results())
        j.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for i in range(6):
        for j, s in zip(jobs, streams):
            if i % 2:
                j.run(stream=s)
            else:
                with torch.cuda.stream(s):
                    j.run()
    torch.cuda.synchronize()
    assert g.check() == g.GEMM_OK
    for j, w in zip(jobs, want):
        assert same(j.results(), w)


def test_graphs_of_one_stream_overlap():
    """Two graphs captured on one stream, replayed at the same time, new inputs between replays."""
    jobs = [Job(10), Job(11)]
    jobs[0].run()
    assert any("splitk" in plan for plan in plans(jobs[0]))  # products that need scratch are among them
    capture, graphs = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    for j in jobs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=capture):
            j.run()
        graphs.append(graph)
    for seed in (20, 30):
        fresh = [Job(seed), Job(seed + 1)]
        want = []
        for f in fresh:
            f.run()
            torch.cuda.synchronize()
            want.append(f.results())
        for j, f in zip(jobs, fresh):
            j.clear()
            for name in ("ids", "x", "w13", "wd", "dy", "weights"):
                getattr(j, name).copy_(getattr(f, name))
        torch.cuda.synchronize()
        side = [torch.cuda.Stream() for _ in jobs]
        for _ in range(3):
            for s, graph in zip(side, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        assert g.check() == g.GEMM_OK
        for j, w in zip(jobs, want):
            assert same(j.results(), w)


def plans(job):
    """The plans of the job's products."""
    seen = []
    for a, b, c, bt in ((job.xs, job.w13, job.gu, True), (job.h, job.wd, job.ys, True), (job.dgu, job.w13, job.dxs, False)):
        g.gemm_grouped(a, b, c, job.offsets, b_trans=bt)
        seen.append(g.last_plan())
    torch.cuda.synchronize()
    return seen
