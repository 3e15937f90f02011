"""The mixture-of-experts layer for a few tokens against its definition in 64 bits.

Inputs are made so that every partial sum of a logit is exact in FP32 (tokens
in steps of 1/32, router weights in steps of 2^-13), so the chosen experts are
compared exactly, ties included.

Bound of y.  h is held in 11 bits or more: rounding errs by at most 2^-12 of
|h| where an FP16 number holds it (2^-17 and 2^-22 with two numbers), plus
2^-20 of the slot's largest |h|; together under 2^-11 of S = sum_j w_j |Wdown|
|h_j| for the data here.  h itself errs by the FP32 sums of its two factors,
1e-5 of sum |W||x| each, which for normal data of width H <= 4096 is at most
1e-5 * 0.8 sqrt(H) / 0.8 of its size where that is typical (64e-5 relative,
averaged over the sum by the signs); activations in __expf and rcp.approx add
2^-20.  With FP32 sums of the down projection at 1e-5 S: 2^-11 S + 7e-4 S,
rounded up to 1.5e-3 S, plus one rounding of the output.
"""
import numpy as np
import pytest
import torch

import dense_gemm_11_gb300 as g
import fp8_ref as ref
from conftest import gpu_available
from helpers import assert_within

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]
E4 = torch.float8_e4m3fn
OUT = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
TOL = 1.5e-3


def layer(T, E, H, I, xt=torch.bfloat16, fp8=False, gated=True, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    X = (rn(T, H).clamp(-3.9, 3.9) * 32).round().div(32).to(xt)
    router = (rn(E, H) / H ** 0.5 * 8192).round().clamp(-256, 256).div(8192).to(xt)
    mats, scales = [], []
    for rows, cols in ((I, H), (I, H), (H, I)):
        w = rn(E, rows, cols) / cols ** 0.5
        if fp8:
            Q = torch.empty(E, rows, cols, dtype=E4, device="cuda")
            S = torch.empty(E, -(-rows // 128), -(-cols // 128), device="cuda")
            for e in range(E):
                g.fp8_quantize(w[e], Q[e], S[e], "blocks")
            mats.append(Q)
            scales.append(S)
        else:
            mats.append(w.to(xt))
    if not gated:
        mats[1] = None
    return X, router, mats, (tuple(scales) if fp8 else None)


def check_layer(X, router, mats, scales, k, yt=None, act=g.GEMM_ACT_SILU, renorm=True, stream=None):
    T, H = X.shape
    yt = X.dtype if yt is None else yt
    Y = torch.full((T, H), float("nan"), dtype=yt, device="cuda")
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    g.moe_few_tokens(X, router, *mats, Y, k, scales=scales, act=act, renormalize=renorm, ids=ids, weights=w)
    assert g.check() == g.GEMM_OK and g.last_launch_count() == 1
    y, want_ids, want_w, S = ref.moe(X, router, *mats, k, scales, act, renorm)
    assert torch.equal(ids.cpu().long(), want_ids)
    assert (w.double().cpu() - want_w).abs().max() <= 2e-6
    assert_within(Y.double().cpu().numpy(), y.numpy(), S.numpy(), TOL, out=OUT[yt])
    return Y


@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 1, 1, 16, 16), (1, 8, 2, 512, 1024), (1, 64, 8, 1040, 528), (2, 5, 5, 128, 128), (3, 7, 1, 144, 2064), (5, 13, 3, 1008, 784),
    (8, 4, 2, 256, 640), (9, 2, 1, 512, 512), (16, 32, 4, 640, 272), (33, 3, 2, 384, 400), (64, 64, 6, 256, 128), (128, 8, 8, 128, 256),
    (128, 1, 1, 272, 144), (100, 300, 10, 64, 48),
])
def test_layer(xt, fp8, T, E, k, H, I):
    check_layer(*layer(T, E, H, I, xt, fp8, seed=T + E), k)


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("act", [g.GEMM_ACT_NONE, g.GEMM_ACT_GELU, g.GEMM_ACT_RELU, g.GEMM_ACT_GELU_TANH, g.GEMM_ACT_SILU])
def test_activations_and_output_types(gated, act):
    for fp8, yt in ((False, torch.float32), (True, torch.float16)):
        check_layer(*layer(11, 6, 272, 400, fp8=fp8, gated=gated), 2, yt, act, renorm=not gated)


def test_fp32_router_and_strided_rows():
    X, router, mats, _ = layer(6, 9, 256, 128)
    check_layer(X, router.float(), mats, None, 3)
    room = torch.zeros(6, 320, dtype=X.dtype, device="cuda")
    room[:, 8:264] = X
    check_layer(room[:, 8:264], router, mats, None, 3)
    big = torch.zeros(6, 300, device="cuda")
    g.moe_few_tokens(X, router, *mats, big[:, 7:263], 3)
    y, _, _, S = ref.moe(X, router, *mats, 3)
    assert_within(big[:, 7:263].double().cpu().numpy(), y.numpy(), S.numpy(), TOL)
    assert not big[:, :7].any() and not big[:, 263:].any()


def test_every_token_to_one_expert_and_ties():
    X, router, mats, _ = layer(40, 6, 128, 128)
    router[:] = 0  # all logits equal: the lowest indices
    check_layer(X, router, mats, None, 2)
    router[4] = X[:, :].abs().amax() / 64
    check_layer(X.abs(), router, mats, None, 1)


def test_extreme_logits():
    X, router, mats, _ = layer(4, 8, 64, 64)
    X[1] = 0
    X[2] *= 64
    check_layer(X, router * 64, mats, None, 3)
    check_layer(X, router * 64, mats, None, 3, renorm=False)


@pytest.mark.parametrize("power", [15, -12])
@pytest.mark.parametrize("xt,fp8", [(torch.float16, False), (torch.float16, True), (torch.bfloat16, True), (torch.bfloat16, False)])
@pytest.mark.parametrize("T", [2, 40])
def test_hidden_values_outside_fp16(xt, fp8, power, T):
    """|h| above FP16's largest number, or so small that FP16 would lose bits."""
    X, router, mats, scales = layer(T, 6, 256, 208, xt, fp8)
    if fp8:
        scales[1].mul_(2.0 ** power)
    else:
        mats[1].mul_(2.0 ** power)
    Y = torch.empty(T, 256, device="cuda")
    g.moe_few_tokens(X, router, *mats, Y, 2, scales=scales)
    y, _, _, S = ref.moe(X, router, *mats, 2, scales)
    # (the absolute floor of the comparison, 1e-6, is scaled away)
    assert_within((Y.double() * 2.0 ** -power).cpu().numpy(), y.numpy() * 2.0 ** -power, S.numpy() * 2.0 ** -power, TOL)


def test_infinite_weight_reaches_its_tokens_only():
    X, router, mats, _ = layer(12, 6, 128, 128, torch.float16)
    ids = torch.empty(12, 2, dtype=torch.int32, device="cuda")
    Y = torch.empty_like(X)
    g.moe_few_tokens(X, router, *mats, Y, 2, ids=ids)
    clean, hit = Y.clone(), (ids == int(ids[0, 0])).any(dim=1)
    mats[1][int(ids[0, 0])] = float("inf")
    g.moe_few_tokens(X, router, *mats, Y, 2)
    assert torch.equal(Y[~hit], clean[~hit]) and not torch.isfinite(Y[hit].float()).all(dim=1).any()


def test_nan_token_stays_alone():
    X, router, mats, scales = layer(5, 6, 128, 128, fp8=True)
    clean = check_layer(X, router, mats, scales, 2)
    X[3, 5] = float("nan")
    Y = torch.empty_like(X)
    ids = torch.empty(5, 2, dtype=torch.int32, device="cuda")
    g.moe_few_tokens(X, router, *mats, Y, 2, scales=scales, ids=ids)
    assert torch.isnan(Y[3]).all() and ((ids >= 0) & (ids < 6)).all() and ids[3, 0] != ids[3, 1]
    for t in (0, 1, 2, 4):
        assert torch.equal(Y[t], clean[t])


def test_repeats_and_streams():
    jobs = [(layer(T, 16, 512, 256, fp8=f, seed=T), T) for T, f in ((1, False), (24, True))]
    want = [check_layer(*job, 4) for job, _ in jobs]
    outs = [[torch.empty(T, 512, dtype=torch.bfloat16, device="cuda") for _ in range(10)] for _, T in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(10):
        for (job, _), o, st in zip(jobs, outs, streams):
            g.moe_few_tokens(*job[:2], *job[2], o[i], 4, scales=job[3], stream=st)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(x, w) for x in o)


def test_captured():
    X, router, mats, _ = layer(3, 8, 256, 256)
    Y = torch.empty_like(X)
    g.moe_few_tokens(X, router, *mats, Y, 2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.moe_few_tokens(X, router, *mats, Y, 2)
    for seed in (3, 4):
        X.copy_(layer(3, 8, 256, 256, seed=seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        y, _, _, S = ref.moe(X, router, *mats, 2)
        assert_within(Y.double().cpu().numpy(), y.numpy(), S.numpy(), TOL, out="bf16")


def test_refusals():
    X, router, mats, scales = layer(4, 6, 128, 128, fp8=True)
    Y = torch.empty_like(X)
    with pytest.raises(ValueError):
        g.moe_few_tokens(X, router, *mats, Y, 2)
    with pytest.raises(ValueError):
        g.moe_few_tokens(X, router, *mats, Y[:3], 2, scales=scales)
    with pytest.raises(ValueError):
        g.moe_few_tokens(X, router, mats[0], mats[1], mats[2][:5], Y, 2, scales=scales)
    with pytest.raises(TypeError):
        g.moe_few_tokens(X.float(), router, *mats, Y, 2, scales=scales)
    with pytest.raises(TypeError):
        g.moe_few_tokens(X, router, *[m.view(torch.uint8) for m in mats], Y, 2, scales=scales)
    with pytest.raises(TypeError):
        g.moe_few_tokens(X, router, *mats, Y, 2, scales=scales, ids=torch.empty(4, 2, device="cuda"))
    for k, status in ((0, g.GEMM_ERR_INVALID_ARG), (7, g.GEMM_ERR_INVALID_ARG)):
        with pytest.raises(g.GemmError) as e:
            g.moe_few_tokens(X, router, *mats, Y, k, scales=scales)
        assert e.value.status == status
    g.moe_few_tokens(X[:0], router, *mats, Y[:0], 2, scales=scales)
    assert g.last_launch_count() == 0
