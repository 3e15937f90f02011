"""The mixture-of-experts layer at its limits, with FP32 routers for many tokens and with uneven routing.

Bounds and the exactness of the logits as in test_gpu_moe.py (for H = 32768 the
partial sums of a logit stay below 2^24 steps as well: they are random walks of
32768 steps of about 1400, 3e5).
"""
import pytest
import torch

import dense_gemm_11_gb300 as g
from conftest import gpu_available
from test_gpu_moe import check_layer, layer

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,k,H", [(31, 40, 3, 272), (32, 40, 3, 272), (33, 5, 2, 1040), (100, 61, 6, 512), (128, 130, 8, 256)])
def test_fp32_router(xt, T, E, k, H):
    """Weights that no 16-bit type holds: steps of 2^-13 from -1 to 1, on tokens of one significant bit, so that logits stay exact."""
    X, router, mats, _ = layer(T, E, H, 64, xt)
    gen = torch.Generator(device="cuda").manual_seed(T)
    X = torch.randint(-1, 2, X.shape, generator=gen, device="cuda").to(xt)
    router = torch.randint(-8191, 8192, router.shape, generator=gen, device="cuda").float() / 8192 / 16
    assert not torch.equal(router.to(xt).float(), router)
    check_layer(X, router, mats, None, k)
    check_layer(X, router, mats, None, k, torch.float32, renorm=False)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,E,k,H,I", [(64, 512, 16, 64, 32), (128, 512, 8, 48, 64), (31, 512, 16, 32, 32), (1, 512, 16, 256, 128), (64, 16, 16, 128, 144),
                                       (3, 2, 1, 32768, 32), (40, 2, 2, 32768, 64), (128, 3, 1, 32768, 16), (2, 2, 1, 32, 32768)])
def test_limits(fp8, T, E, k, H, I):
    check_layer(*layer(T, E, H, I, torch.bfloat16, fp8, seed=T + E), k)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [20, 128])
def test_uneven_routing(fp8, T):
    """Half the tokens choose the same two of 40 experts, most experts get none."""
    X, router, mats, scales = layer(T, 40, 256, 272, torch.bfloat16, fp8)
    X[:, 0], X[: T // 2, 0] = 0, 3.875
    router[:, 0] = 0
    router[7, 0], router[31, 0] = 8, 4
    check_layer(X, router, mats, scales, 2)
