"""Sizes whose indices would not fit 32 bits are refused on the host (no GPU)."""
import os

import pytest

import dense_gemm_11_gb300 as g
from test_fp8_abi import MOE, PROD, QUANT

TOP = 2 ** 31 - 1
LIMIT = 2 ** 31 - 512


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(g.LIB_PATH):
        g.build()
    return g.lib()


@pytest.mark.parametrize("size", [TOP, TOP - 100, LIMIT + 1])
@pytest.mark.parametrize("which", ["rows", "cols"])
@pytest.mark.parametrize("layout", [g.GEMM_FP8_ROWS, g.GEMM_FP8_COLS, g.GEMM_FP8_BLOCKS])
def test_quantize(L, which, size, layout):
    change = {which: size, "ldx": TOP, "ldq": TOP, "lds": TOP, "layout": layout}
    assert L.gemm_fp8_quantize_block128(*{**QUANT, **change}.values()) == g.GEMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("size", [TOP, TOP - 100, LIMIT + 1])
@pytest.mark.parametrize("which", ["M", "N", "K"])
def test_product(L, which, size):
    ld = 2 ** 31
    change = {which: size, "lda": ld, "ldb": ld, "ldc": ld, "ldsa": ld, "ldsb": ld}
    assert L.gemm_fp8_block128(*{**PROD, **change}.values()) == g.GEMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("change", [dict(T=64, top_k=16, E=16, H=16, I=2 ** 21), dict(T=128, top_k=1, E=8, H=16, I=2 ** 24),
                                    dict(E=256, I=2 ** 23, H=16)])
def test_moe(L, change):
    assert L.gemm_moe_few_tokens(*{**MOE, **change}.values()) == g.GEMM_ERR_UNSUPPORTED
