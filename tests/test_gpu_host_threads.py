"""Calls of two host threads on one stream: each has the stream's scratch for itself, however many launches it makes (GB300)."""
import threading

import pytest
import torch

import dense_gemm_11_gb300 as g
from conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]
BF16, F32 = torch.bfloat16, torch.float32
REPEATS = 40


def rand(*shape, seed, dtype=BF16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def offsets_of(*sizes):
    return torch.tensor([0, *sizes], device="cuda").cumsum(0).int()


# Each: the call into an output, the output's shape and type, part of the plan, its launches
def rows(seed, sizes=(1, 1), N=1024, K=8192):
    A, B, off = rand(sum(sizes), K, seed=seed), rand(len(sizes), N, K, seed=seed + 1), offsets_of(*sizes)
    return (lambda C, s: g.gemm_grouped(A, B, C, off, stream=s)), (sum(sizes), N), BF16, "grouped_pair_splitk", 2


def more_rows(seed):
    return rows(seed, (100, 150, 60, 90))


def weights(seed, M=100, N=130):
    off = offsets_of(20000, 0, 9001)
    A, B = rand(29001, M + 4, seed=seed)[:, :M], rand(29001, N + 6, seed=seed + 1)[:, :N]
    return (lambda C, s: g.gemm_grouped_wgrad(A, B, C, off, stream=s)), (3, M, N), F32, "grouped_wgrad_pair_splitk", 2


def fp8_product(seed, M=1024, N=1024, K=8192):
    A, B = g.fp8_empty(M, K, "rows"), g.fp8_empty(N, K, "blocks")
    g.fp8_quantize(rand(M, K, seed=seed), *A, "rows")
    g.fp8_quantize(rand(N, K, seed=seed + 1), *B, "blocks")
    return (lambda C, s: g.gemm_fp8(*A, *B, C, stream=s)), (M, N), F32, "fp8_pair_256x256_splitk", 2


def fp32_repacked(seed, n=1500):
    A, B = rand(n, n + 1, seed=seed, dtype=F32)[:, :n], rand(n, n + 1, seed=seed + 1, dtype=F32)[:, :n]
    return (lambda C, s: g.gemm_f32(A, B, C, stream=s)), (n, n), F32, "repack", None


def three_tf32(seed, n=512):
    A, B = rand(n, n, seed=seed, dtype=F32), rand(n, n, seed=seed + 1, dtype=F32)
    return (lambda C, s: g.gemm_f32_3xtf32(A, B, C, stream=s)), (n, n), F32, "tf32x3", None


def few_tokens(seed, T=16, E=16, H=1024, I=1024):
    X, router = rand(T, H, seed=seed), rand(E, H, seed=seed + 1) / 32
    mats = [rand(E, *s, seed=seed + 2 + i) / 32 for i, s in enumerate(((I, H), (I, H), (H, I)))]
    return (lambda C, s: g.moe_few_tokens(X, router, *mats, C, 4, stream=s)), (T, H), F32, "moe_few_tokens", 1


# The second of a pair asks for more scratch than the first.
@pytest.mark.parametrize("first,second", [(rows, rows), (rows, more_rows), (weights, more_rows), (rows, fp8_product), (fp8_product, fp8_product),
                                          (fp32_repacked, fp32_repacked), (three_tf32, three_tf32), (few_tokens, more_rows)])
def test_two_threads_on_one_stream(first, second):
    jobs = [first(10), second(20)]
    want, outs = [], []
    for call, shape, t, plan, launches in jobs:
        want.append(torch.full(shape, float("nan"), device="cuda", dtype=t))
        call(want[-1], None)
        assert plan in g.last_plan() and launches in (None, g.last_launch_count())
        outs.append(torch.full((REPEATS, *shape), float("nan"), device="cuda", dtype=t))
    torch.cuda.synchronize()
    assert all(torch.isfinite(w).all() for w in want)
    stream, ready, errors = torch.cuda.Stream(), threading.Barrier(2), []  # without scratch yet: it grows meanwhile

    def work(call, out):
        try:
            ready.wait(30)
            for o in out:
                call(o, stream)
        except Exception as e:  # noqa: BLE001 (reported by the test)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(job[0], out)) for job, out in zip(jobs, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and g.check() == g.GEMM_OK
    for w, out in zip(want, outs):
        assert all(torch.equal(o, w) for o in out)
