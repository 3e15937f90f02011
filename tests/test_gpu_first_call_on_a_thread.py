"""A host thread's first CUDA call may be one of the library's: it has no current context yet (GB300)."""
import threading

import pytest
import torch

import dense_gemm_11_gb300 as g
from conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]
BF16 = torch.bfloat16


def rand(*shape, dtype=BF16):
    return torch.randn(shape, device="cuda").to(dtype)


def calls():
    A, B, W = rand(256, 512), rand(512, 384), rand(4, 384, 512)
    off = torch.tensor([0, 100, 100, 250, 256], device="cuda").int()
    F, G = rand(256, 512, dtype=torch.float32), rand(512, 384, dtype=torch.float32)
    Aq, Bq = g.fp8_empty(256, 512, "rows"), g.fp8_empty(384, 512, "blocks")
    g.fp8_quantize(A, *Aq, "rows")
    g.fp8_quantize(B.t().contiguous(), *Bq, "blocks")
    router, mats = rand(8, 512) / 16, [rand(8, *s) / 16 for s in ((256, 512), (256, 512), (512, 256))]
    few = A[:4].contiguous()
    ids = torch.randint(0, 4, (256, 1), device="cuda").int()
    offsets, rows = torch.empty(5, device="cuda").int(), torch.empty(256, 1, device="cuda").int()
    new = lambda *s, t=torch.float32: (lambda: torch.zeros(s, dtype=t, device="cuda"))  # noqa: E731
    return {
        "f32": (lambda C: g.gemm_f32(F, G, C), new(256, 384)),
        "3xtf32": (lambda C: g.gemm_f32_3xtf32(F, G, C), new(256, 384)),
        "16 bits": (lambda C: g.gemm_tc(A, B, C), new(256, 384)),
        "batch": (lambda C: g.gemm_tc_batched(A.reshape(4, 64, 512), W, C, b_trans=True), new(4, 64, 384)),
        "8 bits": (lambda C: g.gemm_fp8(*Aq, *Bq, C), new(256, 384)),
        "few tokens": (lambda C: g.moe_few_tokens(few, router, *mats, C, 2), new(4, 512)),
        "rows by expert": (lambda C: g.moe_dispatch(ids, A, C, offsets, rows), new(256, 512, t=BF16)),
        "experts' rows": (lambda C: g.gemm_grouped(A, W, C, off), new(256, 384)),
        "experts' weights": (lambda C: g.gemm_grouped_wgrad(A, A, C, off), new(4, 512, 512)),
    }


@pytest.mark.parametrize("name", ["f32", "3xtf32", "16 bits", "batch", "8 bits", "few tokens", "rows by expert", "experts' rows", "experts' weights"])
def test_first_call_of_a_thread(name):
    torch.manual_seed(2)
    call, new = calls()[name]
    want, got, errors = new(), new(), []
    call(want)  # what a process does once is done
    torch.cuda.synchronize()

    def work():
        try:
            call(got)
        except Exception as e:  # noqa: BLE001 (reported by the test)
            errors.append(e)

    thread = threading.Thread(target=work)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert g.check() == g.GEMM_OK and torch.equal(got, want) and bool((got != 0).any())
