"""The gated activation with 8-bit copies of its inputs, and its backward pass from them (GB300)."""
import pytest
import torch

import dense_gemm_11_gb300 as g
from experts_ref import act, close, kept, rounded

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


def mat(rows, cols, dtype, pad, shift=0, scale=1.0, fill=None):
    full = torch.full(((rows + 1) * (cols + pad) + shift,), 0.0 if fill is None else fill, device="cuda").to(dtype)
    m = full[shift:].as_strided((rows, cols), (cols + pad, 1))
    if fill is None:
        m.copy_(torch.randn(rows, cols, device="cuda") * scale)
    return m


def pair(rows, cols, q, pad):
    Q = torch.zeros(rows, cols + pad, device="cuda").to(q)[:, :cols]
    S = torch.zeros(-(-cols // 128), rows + pad, device="cuda")[:, :rows]
    return Q, S


# rows, columns, type, padding, first element
SHAPES = [(1, 1, F32, 0, 0), (1, 128, BF16, 0, 0), (5, 129, F16, 0, 0), (16, 256, BF16, 8, 0), (33, 1000, BF16, 0, 0), (17, 264, F32, 3, 1), (300, 127, F16, 1, 0), (64, 2056, BF16, 0, 3)]


@pytest.mark.parametrize("code", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("rows,cols,t,pad,shift", SHAPES)
def test_forward_and_backward(rows, cols, t, pad, shift, gated, code):
    torch.manual_seed(rows + cols + code)
    q = E5 if (rows + code) % 2 else E4
    G, U = mat(rows, cols, t, pad, shift, scale=3.0), mat(rows, cols, t, pad, shift) if gated else None
    H = mat(rows, cols, t, pad, shift, fill=-7.0)
    (GQ, GS), (UQ, US) = pair(rows, cols, q, pad), pair(rows, cols, q, pad) if gated else (None, None)
    g.fp8_gated_act(G, U, H, GQ, GS, UQ, US, act=code)
    assert g.check() == g.GEMM_OK
    a, _, e, _ = act(G.double(), code)
    u = U.double() if gated else torch.ones_like(a)
    close(H, a * u, rounded((e + 2.0 ** -24 * (a.abs() + e)) * u.abs(), a * u, t), "h")
    for X, Q, S in ((G, GQ, GS), (U, UQ, US)):
        if X is None:
            continue
        wq, ws = pair(rows, cols, q, pad)
        g.fp8_quantize(X, wq, ws, "rows")
        assert torch.equal(Q.contiguous().view(torch.uint8), wq.contiguous().view(torch.uint8)) and torch.equal(S, ws)
    if pad:
        assert (H.as_strided((rows, pad), (cols + pad, 1), storage_offset=H.storage_offset() + cols) == -7.0).all()

    dH = mat(rows, cols, t, pad, shift)
    dG, dU, back = (mat(rows, cols, t, pad, shift, fill=-7.0) for _ in range(3))
    g.fp8_gated_act_grad(dH, GQ, GS, UQ, US, dG, dU if gated else None, back, act=code)
    assert g.check() == g.GEMM_OK
    # g' is one FP32 product; its rounding moves act and its slope by 2^-24 |g'| times their slopes (2 at most, and 2)
    gk, uk = kept(GQ, GS), kept(UQ, US) if gated else torch.ones_like(a)
    a, s, ea, es = act(gk, code)
    ea, es = ea + 2.0 ** -23 * gk.abs(), es + (2.0 ** -23 * gk.abs() if code not in (0, 2) else 0)
    dh = dH.double()
    want = dh * uk * s
    close(dG, want, rounded(dh.abs() * uk.abs() * (es + 4 * 2.0 ** -24 * (s.abs() + es)), want, t), "dg")
    if gated:
        close(dU, dh * a, rounded(dh.abs() * (ea + 2.0 ** -24 * (a.abs() + ea)), dh * a, t), "du")
    close(back, a * uk, rounded(uk.abs() * (ea + 3 * 2.0 ** -24 * (a.abs() + ea)), a * uk, t), "h from the copies")
    alone = mat(rows, cols, t, pad, shift, fill=-7.0)
    g.fp8_gated_act_grad(dH, GQ, GS, UQ, US, alone, dU if gated else None, act=code)
    assert torch.equal(alone, dG)


@pytest.mark.parametrize("code", [1, 3, 4])
def test_backward_against_differences(code):
    """The slope at the copies, against differences of the FP64 activation."""
    G, U = torch.linspace(-6, 6, 256, device="cuda").reshape(2, 128), torch.ones(2, 128, device="cuda")
    (GQ, GS), (UQ, US) = pair(2, 128, E4, 0), pair(2, 128, E4, 0)
    H, dG, dU = (torch.empty(2, 128, device="cuda") for _ in range(3))
    g.fp8_gated_act(G, U, H, GQ, GS, UQ, US, act=code)
    g.fp8_gated_act_grad(torch.ones(2, 128, device="cuda"), GQ, GS, UQ, US, dG, dU, act=code)
    x, step = kept(GQ, GS), 1e-4
    slope = (act(x + step, code)[0] - act(x - step, code)[0]) / (2 * step)
    # the differences' own error is step^2 / 6 times the third derivative (2 at most); u' is within 2^-23 of 1
    assert ((dG.double() - slope * kept(UQ, US)).abs() <= 1e-5).all()


def test_special_values():
    G = torch.zeros(3, 256, device="cuda")
    G[0, 5], G[1, 7], G[2, 130] = float("nan"), float("inf"), -1e30
    U = torch.ones(3, 256, device="cuda")
    for code in (1, 2, 3, 4):
        (GQ, GS), (UQ, US) = pair(3, 256, E4, 0), pair(3, 256, E4, 0)
        H = torch.empty(3, 256, device="cuda")
        g.fp8_gated_act(G, U, H, GQ, GS, UQ, US, act=code)
        assert g.check() == g.GEMM_OK
        assert H[0, 5].isnan() and H[1, 7] == float("inf") and H[2, 130] == 0 and (H[0, 6:] == 0).all() and (H[2, :128] == 0).all()
        assert (kept(GQ, GS)[0, 6:] == 0).all() and kept(GQ, GS)[0, 5].isnan()
        dG, dU, back = (torch.empty(3, 256, device="cuda") for _ in range(3))
        g.fp8_gated_act_grad(U, GQ, GS, UQ, US, dG, dU, back, act=code)
        assert dG[2, 130] == 0 and dU[2, 130] == 0 and back[2, 130] == 0 and torch.isfinite(dG[2]).all()


def test_what_the_copies_lose():
    """The gradients from the 8-bit copies are near those from the values: e4m3 is within 1/16 of a value."""
    torch.manual_seed(3)
    G, U, dH = torch.randn(64, 512, device="cuda"), torch.randn(64, 512, device="cuda"), torch.randn(64, 512, device="cuda")
    (GQ, GS), (UQ, US) = pair(64, 512, E4, 0), pair(64, 512, E4, 0)
    H, dG, dU = (torch.empty(64, 512, device="cuda") for _ in range(3))
    g.fp8_gated_act(G, U, H, GQ, GS, UQ, US)
    g.fp8_gated_act_grad(dH, GQ, GS, UQ, US, dG, dU)
    a, s, _, _ = act(G.double(), 4)
    for got, want in ((dG, dH.double() * U.double() * s), (dU, dH.double() * a)):
        assert float((got.double() - want).norm() / want.norm()) <= 1 / 16 + 1 / 16


# 2432 blocks of 16 rows x 128 columns and more: a CTA takes four column blocks of its rows, two at a time (FP32 forwards: two in all), and
# the last CTA of a row one, two or three; ragged last rows and columns.
MANY = [(2500, 2100, BF16, 0, 0), (4001, 1290, F16, 0, 0), (2500, 2100, F32, 0, 0), (3100, 1800, BF16, 3, 1), (40000, 129, F16, 0, 0)]


@pytest.mark.parametrize("code", [1, 2, 4])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("rows,cols,t,pad,shift", MANY)
def test_many_blocks(rows, cols, t, pad, shift, gated, code):
    assert -(-rows // 16) * -(-cols // 128) >= 16 * torch.cuda.get_device_properties(0).multi_processor_count
    test_forward_and_backward(rows, cols, t, pad, shift, gated, code)


# largest value, half a step relative to a value, half of the smallest step
FORMATS = {E4: (448.0, 2.0 ** -4, 2.0 ** -10), E5: (57344.0, 2.0 ** -3, 2.0 ** -17)}


@pytest.mark.parametrize("q", [E4, E5])
@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_what_the_copies_lose_beside_a_large_value(t, q):
    """A copy is off by half a step of its type at most: relative to the value, or, below the type's normal numbers, to its block's scale.

    Beside a value of 2^12 those below 2^-14.8 of it (e4m3) are that small, and those below half of a step are zeros.
    """
    torch.manual_seed(4)
    G, U = torch.randn(20, 700, device="cuda").to(t), (torch.randn(20, 700, device="cuda") * 0.1).to(t)
    G[:, ::128], U[::2, 5] = 2.0 ** 12, -(2.0 ** 12)
    G[:, 1::7] *= 2.0 ** -10
    (GQ, GS), (UQ, US) = pair(20, 700, q, 0), pair(20, 700, q, 0)
    H = torch.empty_like(G)
    g.fp8_gated_act(G, U, H, GQ, GS, UQ, US)
    assert g.check() == g.GEMM_OK
    top, relative, smallest = FORMATS[q]
    for X, Q, S in ((G, GQ, GS), (U, UQ, US)):
        x = X.double()
        padded = torch.nn.functional.pad(x.abs(), (0, 768 - 700)).reshape(20, 6, 128)
        scale = (padded.amax(2) / top).repeat_interleave(128, 1)[:, :700]
        # the scale, its reciprocal and the product with it are FP32: 2^-24 each, which may move a value over the middle of a step
        bound = torch.maximum(relative * x.abs(), smallest * scale) * (1 + 2.0 ** -3 * 2.0 ** -18) + 4 * 2.0 ** -24 * x.abs()
        close(kept(Q, S), x, bound)
        small = x.abs() < 0.99 * smallest * scale
        assert (kept(Q, S)[small] == 0).all()
    if q == E4:
        assert bool((kept(GQ, GS) == 0).any()) and bool(((kept(GQ, GS) - G.double()).abs() > 0.0625 * G.double().abs()).any())  # more than 2^-4 of a value


@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_an_infinity_takes_its_block(t):
    """h has it where it belongs; the copies' scale is infinite, and the gradients are NaN in the 128 columns of that block of the row."""
    torch.manual_seed(5)
    G, U, dH = (torch.randn(5, 400, device="cuda").to(t) for _ in range(3))
    G[2, 200] = float("inf")
    clean = torch.ones(5, 400, dtype=torch.bool, device="cuda")
    clean[2, 128:256] = False
    (GQ, GS), (UQ, US) = pair(5, 400, E4, 0), pair(5, 400, E4, 0)
    H, dG, dU, back = (torch.empty_like(G) for _ in range(4))
    g.fp8_gated_act(G, U, H, GQ, GS, UQ, US)
    g.fp8_gated_act_grad(dH, GQ, GS, UQ, US, dG, dU, back)
    assert g.check() == g.GEMM_OK
    assert H[2, 200].abs() == float("inf") and int(torch.isfinite(H.float()).sum()) == 5 * 400 - 1
    assert GS[1, 2] == float("inf") and int(torch.isfinite(GS).sum()) == GS.numel() - 1
    for out in (dG, dU, back):
        assert torch.isfinite(out[clean].float()).all() and out[~clean].isnan().all()
