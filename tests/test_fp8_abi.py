"""Host-side argument checks of the 8-bit entry points (no GPU: every case is refused, or empty, before any CUDA call)."""
import os

import pytest

import dense_gemm_11_gb300 as g

FAKE = 0x10000
E4, E5 = g.GEMM_DTYPE_E4M3, g.GEMM_DTYPE_E5M2
QUANT = dict(rows=4, cols=256, X=FAKE, x_type=g.GEMM_DTYPE_BF16, ldx=256, Q=FAKE, q_type=E4, ldq=256, S=FAKE, lds=4,
             layout=g.GEMM_FP8_ROWS, stream=None)
PROD = dict(M=8, N=256, K=256, alpha=1.0, A=FAKE, a_type=E4, lda=256, SA=FAKE, ldsa=8, B=FAKE, b_type=E4, ldb=256, SB=FAKE,
            ldsb=2, b_trans=1, b_layout=g.GEMM_FP8_BLOCKS, beta=0.0, C=FAKE, c_type=g.GEMM_DTYPE_BF16, ldc=256, bias=None,
            act=0, stream=None)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(g.LIB_PATH):
        g.build()
    return g.lib()


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(cols=-1), dict(x_type=E4), dict(x_type=-1), dict(q_type=g.GEMM_DTYPE_F16), dict(q_type=5),
    dict(layout=-1), dict(layout=3), dict(ldx=255), dict(ldq=255), dict(lds=3), dict(X=None), dict(Q=None), dict(S=None),
    dict(layout=g.GEMM_FP8_COLS, ldq=3, lds=256), dict(layout=g.GEMM_FP8_COLS, lds=255), dict(layout=g.GEMM_FP8_BLOCKS, lds=1),
])
def test_quantize_rejects(L, change):
    assert L.gemm_fp8_quantize_block128(*{**QUANT, **change}.values()) == g.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(act=4), dict(act=-1), dict(a_type=g.GEMM_DTYPE_BF16), dict(b_type=0), dict(c_type=E4),
    dict(b_trans=2), dict(b_layout=g.GEMM_FP8_COLS), dict(b_layout=g.GEMM_FP8_ROWS, b_trans=0), dict(lda=255), dict(ldb=255),
    dict(ldc=255), dict(ldsa=7), dict(ldsb=1), dict(b_layout=g.GEMM_FP8_ROWS, ldsb=255), dict(A=None), dict(SA=None),
    dict(B=None), dict(SB=None), dict(C=None),
])
def test_product_rejects(L, change):
    assert L.gemm_fp8_block128(*{**PROD, **change}.values()) == g.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(A=FAKE + 8), dict(B=FAKE + 8), dict(SA=FAKE + 4), dict(lda=257), dict(ldb=264), dict(ldsa=9),
    dict(b_layout=g.GEMM_FP8_ROWS, ldsb=257), dict(b_layout=g.GEMM_FP8_ROWS, ldsb=256, SB=FAKE + 4),
])
def test_product_does_not_support(L, change):
    assert L.gemm_fp8_block128(*{**PROD, **change}.values()) == g.GEMM_ERR_UNSUPPORTED


def test_empty(L):
    none = dict(X=None, Q=None, S=None)
    for change in (dict(rows=0), dict(cols=0)):
        assert L.gemm_fp8_quantize_block128(*{**QUANT, **none, **change}.values()) == g.GEMM_OK
    none = dict(A=None, B=None, SA=None, SB=None, C=None)
    for change in (dict(M=0), dict(N=0)):
        assert L.gemm_fp8_block128(*{**PROD, **none, **change}.values()) == g.GEMM_OK
        assert g.last_launch_count() == 0


def test_fp8_empty_strides():
    import torch
    for layout in ("rows", "cols", "blocks"):
        Q, S = g.fp8_empty(130, 257, layout, device="cpu")
        assert (Q.shape, S.shape) == tuple(map(torch.Size, g._fp8_shapes(130, 257, layout)))
        assert Q.stride(0) % 16 == 0 and S.stride(0) % 4 == 0 and Q.dtype == torch.float8_e4m3fn


MOE = dict(T=4, E=8, top_k=2, H=256, I=128, X=FAKE, x_type=g.GEMM_DTYPE_BF16, ldx=256, router=FAKE, router_type=g.GEMM_DTYPE_BF16,
           gate=FAKE, up=FAKE, down=FAKE, w_type=E4, s_gate=FAKE, s_up=FAKE, s_down=FAKE, act=g.GEMM_ACT_SILU, renormalize=1,
           Y=FAKE, y_type=g.GEMM_DTYPE_BF16, ldy=256, ids=None, weights=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(E=-1), dict(E=0), dict(H=-1), dict(I=-1), dict(I=0), dict(top_k=0), dict(top_k=9), dict(x_type=0), dict(x_type=E4),
    dict(router_type=g.GEMM_DTYPE_F16), dict(w_type=g.GEMM_DTYPE_F16), dict(w_type=E5), dict(y_type=E4), dict(act=5), dict(act=-1),
    dict(renormalize=2), dict(ldx=255), dict(ldy=255), dict(X=None), dict(router=None), dict(gate=None), dict(down=None),
    dict(Y=None), dict(s_gate=None), dict(s_up=None), dict(s_down=None),
])
def test_moe_rejects(L, change):
    assert L.gemm_moe_few_tokens(*{**MOE, **change}.values()) == g.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(T=129), dict(E=513), dict(E=32, top_k=17), dict(T=128, top_k=16, E=64), dict(H=264, ldx=264, ldy=264), dict(I=120), dict(H=32784, ldx=32784, ldy=32784),
    dict(X=FAKE + 2), dict(router=FAKE + 2), dict(gate=FAKE + 1), dict(up=FAKE + 1), dict(down=FAKE + 8), dict(ldx=257),
])
def test_moe_does_not_support(L, change):
    assert L.gemm_moe_few_tokens(*{**MOE, **change}.values()) == g.GEMM_ERR_UNSUPPORTED


def test_moe_empty(L):
    for change in (dict(T=0), dict(H=0)):
        assert L.gemm_moe_few_tokens(*{**MOE, **dict(X=None, Y=None), **change}.values()) == g.GEMM_OK
        assert g.last_launch_count() == 0
