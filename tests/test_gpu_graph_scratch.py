"""Library scratch under stream capture: each graph has its own, for as long as it lives.

PyTorch captures every graph on one stream, so scratch that went by the stream
would be shared by all of them.
"""
import gc

import numpy as np
import pytest
import torch

import dense_gemm_11_gb300 as g
from conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]
BF16 = torch.bfloat16


def rand(*shape, seed, dtype=torch.float32):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32)).cuda().to(dtype)


def fp8_product(seed, M=1024, N=1024, K=8192):
    A, B = g.fp8_empty(M, K, "rows"), g.fp8_empty(N, K, "blocks")
    g.fp8_quantize(rand(M, K, seed=seed, dtype=BF16), *A, "rows")
    g.fp8_quantize(rand(N, K, seed=seed + 1, dtype=BF16), *B, "blocks")
    C = torch.empty(M, N, device="cuda")
    return (lambda: g.gemm_fp8(*A, *B, C)), C, "fp8_pair_256x256_splitk"


def moe_layer(seed, T=16, E=16, H=1024, I=1024):
    X, router = rand(T, H, seed=seed, dtype=BF16), rand(E, H, seed=seed + 1, dtype=BF16) / 32
    mats = [rand(E, *s, seed=seed + 2 + i, dtype=BF16) / 32 for i, s in enumerate(((I, H), (I, H), (H, I)))]
    Y = torch.empty(T, H, device="cuda")
    return (lambda: g.moe_few_tokens(X, router, *mats, Y, 4)), Y, "moe_few_tokens"


def fp32_split(seed, n=256, K=4096):
    A, B, C = rand(n, K, seed=seed), rand(K, n, seed=seed + 1), torch.empty(n, n, device="cuda")
    return (lambda: g.gemm_f32(A, B, C)), C, "splitk"


def three_tf32(seed, n=512):
    A, B, C = rand(n, n, seed=seed), rand(n, n, seed=seed + 1), torch.empty(n, n, device="cuda")
    return (lambda: g.gemm_f32_3xtf32(A, B, C)), C, "tf32x3_pair"


def fp32_repacked(seed, n=1500):
    A, B = rand(n, n + 1, seed=seed)[:, :n], rand(n, n + 1, seed=seed + 1)[:, :n]
    C = torch.empty(n, n, device="cuda")
    return (lambda: g.gemm_f32(A, B, C)), C, ""


JOBS = [fp8_product, moe_layer, fp32_split, three_tf32, fp32_repacked]


def eager(job):
    call, out, plan = job
    torch.cuda.synchronize()
    out.fill_(float("nan"))
    call()
    assert plan in g.last_plan()
    torch.cuda.synchronize()
    assert g.check() == g.GEMM_OK and torch.isfinite(out).all()
    return out.clone()


def captured(*calls, repeat=1):
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for _ in range(repeat):
            for call in calls:
                call()
    return graph


def free_memory():
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()  # as a capture does
    return torch.cuda.mem_get_info()[0]


@pytest.mark.parametrize("make", JOBS)
def test_graphs_replayed_at_once(make):
    """Two graphs of the same shapes on two streams, with calls on a third."""
    jobs = [make(seed) for seed in (10, 20, 30)]
    want = [eager(job) for job in jobs]
    graphs = [captured(job[0], repeat=10) for job in jobs[:2]]
    streams = [torch.cuda.Stream() for _ in jobs]
    for _, out, _ in jobs:
        out.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        with torch.cuda.stream(streams[2]):
            for _ in range(5):
                jobs[2][0]()
    torch.cuda.synchronize()
    assert g.check() == g.GEMM_OK
    for (_, out, _), w in zip(jobs, want):
        assert torch.equal(out, w)


@pytest.mark.parametrize("make,size", [(fp8_product, 16 << 20), (three_tf32, 4 << 20)])
def test_each_graph_allocates_its_own_and_gives_it_back(make, size):
    """16 tiles of 256 x 256 FP32 sums at least (16 MB and more), or four FP32 copies of 512 x 512."""
    job = make(40)
    eager(job)
    captured(job[0]).replay()  # what a first graph costs beside the scratch
    eager(job)
    before, graphs = free_memory(), []
    for i in range(1, 4):
        graphs.append(captured(job[0]))
        assert before - free_memory() >= i * size, i
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    del graphs, graph
    gc.collect()
    eager(job)  # a call frees it
    assert before - free_memory() < size


def test_many_graphs_one_after_the_other():
    """Captured, replayed and dropped with no call outside a capture: the memory of the last ones comes back."""
    job = fp8_product(60)
    want = eager(job)
    low = []
    for _ in range(12):
        graph = captured(job[0])
        job[1].fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(job[1], want)
        del graph
        low.append(free_memory())
    assert low[3] - low[-1] < (16 << 20)


@pytest.mark.parametrize("make,small,large", [(moe_layer, {"T": 2}, {"T": 120}), (fp32_split, {"n": 128}, {"n": 512}), (three_tf32, {"n": 256}, {"n": 1024}),
                                              (fp8_product, {"M": 512, "N": 512, "K": 16384}, {"M": 1024, "N": 1024, "K": 8192})])
def test_scratch_that_grows(make, small, large):
    """Within a capture, and in calls outside it, between replays of a graph that was captured with less."""
    a, b = make(50, **small), make(70, **large)
    plans = [job[2] for job in (a, b)]
    a, b = ((job[0], job[1], "") for job in (a, b))
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        want_a = eager(a)
        first = torch.cuda.CUDAGraph()
        with torch.cuda.graph(first, stream=stream):
            a[0]()
        want_b = eager(b)  # the stream's own scratch grows
        assert plans[1] in g.last_plan()
        both = torch.cuda.CUDAGraph()
        with torch.cuda.graph(both, stream=stream):
            a[0]()
            b[0]()  # the capture's grows
            a[0]()
        for _ in range(3):
            a[1].fill_(0)
            first.replay()
            torch.cuda.synchronize()
            assert torch.equal(a[1], want_a)
            a[1].fill_(0), b[1].fill_(0)
            both.replay()
            torch.cuda.synchronize()
            assert torch.equal(a[1], want_a) and torch.equal(b[1], want_b)
        assert torch.equal(eager(b), want_b)
    assert g.check() == g.GEMM_OK


def test_branches_of_one_capture():
    """Two streams that take part in one capture work at the same time."""
    jobs = [fp32_split(80), fp32_split(90)]
    want = [eager(job) for job in jobs]
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(10):
            jobs[0][0]()
        with torch.cuda.stream(side):
            for _ in range(10):
                jobs[1][0]()
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for _, out, _ in jobs:
            out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        for (_, out, _), w in zip(jobs, want):
            assert torch.equal(out, w)
