"""The mixture of experts' long sums round to nearest: an FP32 Y against the definition in 64 bits, by norm.

What FP32 sums leave of normal data, of the norm.  The matrix instruction adds a
box of 64 or 128 k in 4 to 16 steps that truncate, half of 2^-23 of the sum on
average, most of it in the last steps: at most 16 * 2^-24 = 1e-6, typically 3e-7,
of independent sign from box to box.  At most 128 boxes then add up to nearest,
sqrt(128) 2^-25 = 3e-7.  The two factors of h err by 4e-7 each, 6e-7 together,
the activation by 2^-22, and the down projection's sums again by 4e-7: 8e-7, and
2e-6 is checked.  Chains of all k in the matrix instruction truncate up to 768
times one after the other and leave 7e-6.
"""
import pytest
import torch

import dense_gemm_11_gb300 as g
import fp8_ref as ref
from conftest import gpu_available
from test_gpu_moe import layer

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.mark.parametrize("xt,fp8", [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True), (torch.float16, True)])
@pytest.mark.parametrize("T", [1, 20])
def test_error_by_norm(xt, fp8, T):
    X, router, mats, scales = layer(T, 2, 4096, 8192, xt, fp8, seed=T)
    Y = torch.empty(T, 4096, device="cuda")
    g.moe_few_tokens(X, router, *mats, Y, 2, scales=scales)
    assert g.check() == g.GEMM_OK
    y, _, _, _ = ref.moe(X, router, *mats, 2, scales)
    off = float((Y.double().cpu() - y).norm() / y.norm())
    assert off <= 2e-6, off
