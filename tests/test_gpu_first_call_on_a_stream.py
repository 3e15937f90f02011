"""The first call on a stream clears its counters in that stream's order.

The default stream is kept busy while the first calls on a fresh non-blocking
stream run: what they clear must not wait behind it, since the kernels do not.
Memory that the counters may come from is filled with ones first.
"""
import numpy as np
import pytest
import torch

import dense_gemm_11_gb300 as g
from conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def test_counters_are_clear_before_the_first_kernel():
    gen = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(4, 512, generator=gen, device="cuda").bfloat16()
    router = torch.randn(8, 512, generator=gen, device="cuda").bfloat16()
    mats = [torch.randn(8, 512, 512, generator=gen, device="cuda").bfloat16() / 23 for _ in range(3)]
    A, B = torch.randn(256, 4096, generator=gen, device="cuda"), torch.randn(4096, 256, generator=gen, device="cuda")
    Y, C = torch.empty(4, 512, device="cuda"), torch.empty(256, 256, device="cuda")
    g.moe_few_tokens(X, router, *mats, Y, 2)
    g.gemm_f32(A, B, C)
    want = Y.clone(), C.clone()
    for i in range(3):
        stream = torch.cuda.Stream(priority=-1)  # no other test has used it, so the call allocates
        Y.fill_(float("nan")), C.fill_(float("nan"))
        dirty = [torch.full((1 << 18,), -1, dtype=torch.int32, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        del dirty
        torch.cuda.empty_cache()
        torch.cuda._sleep(40_000_000)  # about 20 ms of the default stream
        g.gemm_f32(A, B, C, stream=stream)
        stream.synchronize()
        assert not torch.cuda.current_stream().query(), "the default stream was to be busy still"
        g.moe_few_tokens(X, router, *mats, Y, 2, stream=stream)  # a cooperative launch waits for the device
        torch.cuda.synchronize()
        assert g.check() == g.GEMM_OK
        assert np.array_equal(Y.cpu().numpy(), want[0].cpu().numpy()) and np.array_equal(C.cpu().numpy(), want[1].cpu().numpy())
