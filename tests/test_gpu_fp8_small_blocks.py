"""The quantizer on blocks of zeros and of very small values.

Every step of q = round8(x (F / a)) is a correctly rounded FP32 operation, so q
and s are compared bit for bit, with the floor under a block's maximum that keeps
s and F / a normal numbers: F 2^-126 rounded up to a power of two.  What a value
reads back as is off by half a step of its rounding at most, the quotients' own
roundings (2^-24 each) on top.
"""
import numpy as np
import pytest
import torch

import dense_gemm_11_gb300 as g
import fp8_ref as ref
from conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
FLOOR = {E4: np.float32(2.0 ** -117), E5: np.float32(2.0 ** -110)}


def quantized(x, layout, dtype, monkeypatch):
    monkeypatch.setattr(ref, "TINY", FLOOR[dtype])
    Q, S = g.fp8_empty(*x.shape, layout, dtype)
    g.fp8_quantize(x, Q, S, layout)
    assert g.check() == g.GEMM_OK
    q, s = ref.quantize(x.float().cpu().numpy(), dtype, layout)
    assert np.array_equal(S.double().cpu().numpy(), s, equal_nan=True)
    assert np.array_equal(Q.float().double().cpu().numpy(), q, equal_nan=True)
    return Q, S


@pytest.mark.parametrize("dtype", [E4, E5])
@pytest.mark.parametrize("layout", ["rows", "cols", "blocks"])
@pytest.mark.parametrize("xt", [torch.float32, torch.float16, torch.bfloat16])
def test_zeros(dtype, layout, xt, monkeypatch):
    x = torch.zeros(300, 200, dtype=xt, device="cuda")
    x[150:, 140:] = 2.0
    Q, S = quantized(x, layout, dtype, monkeypatch)
    back = ref.dequantize(Q, S, "blocks" if layout == "blocks" else "rows")
    assert torch.equal((back.t() if layout == "cols" else back).float(), x.float())
    assert (S > 0).all() and torch.isfinite(S).all()


@pytest.mark.parametrize("dtype", [E4, E5])
@pytest.mark.parametrize("layout", ["rows", "cols", "blocks"])
def test_small_values(dtype, layout, monkeypatch):
    """Block maxima from 2^-149 to 2^-100, over both floors."""
    bits, low = ref.GRID[dtype]
    for power in list(range(-149, -100, 3)) + [-117, -118, -112, -111, -110, -109]:
        x = torch.from_numpy(np.ldexp(np.random.default_rng(-power).uniform(-1, 1, (130, 140)), power).astype(np.float32)).cuda()
        Q, S = quantized(x, layout, dtype, monkeypatch)
        back, q, s = ref.dequantize(Q, S, "blocks" if layout == "blocks" else "rows"), Q.double().abs(), S.double().max()
        back = back.t() if layout == "cols" else back
        half_step = 2.0 ** -(bits + 1) * torch.maximum(x.double().abs() * (1 + 2.0 ** -bits), 2.0 ** low * s)
        assert ((back - x.double()).abs() <= half_step + 2.0 ** -22 * x.double().abs()).all(), power
        assert torch.isfinite(q).all()


@pytest.mark.parametrize("dtype", [E4, E5])
@pytest.mark.parametrize("layout", ["rows", "cols", "blocks"])
def test_special_values(dtype, layout, monkeypatch):
    """Zeros, NaN, an infinity and a very large value, each in a block of its own or beside ordinary ones."""
    x = torch.from_numpy(np.random.default_rng(5).standard_normal((256, 256))).float().cuda()
    x[:128, :128] = 0.0
    x[3, 200], x[200, 3] = float("nan"), float("-inf")
    x[130, 130:256] *= 2.0 ** -130
    x[255, 255] = 3.0e38
    quantized(x, layout, dtype, monkeypatch)


def test_gradient_with_rows_of_zeros():
    """Masked tokens in an e5m2 gradient leave the others' products alone."""
    dy = torch.from_numpy(np.random.default_rng(1).standard_normal((40, 256))).float().cuda()
    dy[7] = 0
    dy[20:30] = 0
    W = torch.from_numpy(np.random.default_rng(2).standard_normal((256, 300))).float().cuda()
    A, W8 = g.fp8_empty(40, 256, "rows", E5), g.fp8_empty(256, 300, "blocks")
    g.fp8_quantize(dy, *A, "rows")
    g.fp8_quantize(W, *W8, "blocks")
    dx = torch.empty(40, 300, device="cuda")
    g.gemm_fp8(*A, *W8, dx, b_trans=False)
    assert torch.isfinite(dx).all() and not dx[7].any() and not dx[20:30].any() and dx[8].any()
