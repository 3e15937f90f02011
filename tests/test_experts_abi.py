"""Refusals of the mixture-of-experts operators for many tokens (no GPU: every case ends on the host)."""
import os
import struct

import pytest
import torch

import dense_gemm_11_gb300 as g
from conftest import gpu_available

FAKE = 0x10000
F32, F16, BF16, E4 = g.GEMM_DTYPE_F32, g.GEMM_DTYPE_F16, g.GEMM_DTYPE_BF16, g.GEMM_DTYPE_E4M3
BIG = 2 ** 31 - 1

DISPATCH = dict(T=4, E=8, top_k=2, H=64, ids=FAKE, X=FAKE, x_type=BF16, ldx=64, Xs=FAKE, ldxs=64, offsets=FAKE, rows=FAKE, stream=None)
COMBINE = dict(T=4, top_k=2, H=64, R=8, Ys=FAKE, type=BF16, ldys=64, rows=FAKE, weights=FAKE, Y=FAKE, ldy=64, stream=None)
GRAD = dict(T=4, top_k=2, H=64, R=8, dY=FAKE, type=BF16, lddy=64, Ys=FAKE, ldys=64, rows=FAKE, weights=FAKE, dYs=FAKE, lddys=64, dweights=FAKE, stream=None)
ROWS = dict(E=4, R=8, N=64, K=64, alpha=1.0, A=FAKE, lda=64, B=FAKE, ldb=64, stride_b=4096, ab_type=BF16, b_trans=1, beta=0.0, C=FAKE, c_type=F32, ldc=64,
            offsets=FAKE, stream=None)
WEIGHTS = dict(E=4, R=8, M=64, N=64, alpha=1.0, A=FAKE, lda=64, B=FAKE, ldb=64, ab_type=BF16, beta=0.0, C=FAKE, c_type=F32, ldc=64, stride_c=4096, offsets=FAKE,
               stream=None)
ACT = dict(rows=4, cols=256, G=FAKE, ldg=256, U=FAKE, ldu=256, type=BF16, H=FAKE, ldh=256, GQ=FAKE, ldgq=256, GS=FAKE, ldgs=4, UQ=FAKE, lduq=256, US=FAKE, ldus=4,
           q_type=E4, act=4, stream=None)
ACT_GRAD = dict(rows=4, cols=256, dH=FAKE, lddh=256, type=BF16, GQ=FAKE, ldgq=256, GS=FAKE, ldgs=4, UQ=FAKE, lduq=256, US=FAKE, ldus=4, q_type=E4, dG=FAKE, lddg=256,
                dU=FAKE, lddu=256, H=FAKE, ldh=256, act=4, stream=None)
CALLS = {"gemm_moe_dispatch": DISPATCH, "gemm_moe_combine": COMBINE, "gemm_moe_combine_grad": GRAD, "gemm_grouped_f32acc": ROWS,
         "gemm_grouped_wgrad_f32acc": WEIGHTS, "gemm_fp8_gated_act": ACT, "gemm_fp8_gated_act_grad": ACT_GRAD}


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(g.LIB_PATH):
        g.build()
    return g.lib()


def call(L, name, **change):
    return getattr(L, name)(*{**CALLS[name], **change}.values())


INVALID = [
    ("gemm_moe_dispatch", [dict(T=-1), dict(E=-1), dict(H=-1), dict(top_k=0), dict(x_type=E4), dict(x_type=-1), dict(ldx=63), dict(ldxs=63), dict(ids=None),
                           dict(X=None), dict(Xs=None), dict(offsets=None), dict(rows=None)]),
    ("gemm_moe_combine", [dict(T=-1), dict(H=-1), dict(R=-1), dict(top_k=0), dict(type=E4), dict(ldys=63), dict(ldy=63), dict(Ys=None), dict(rows=None), dict(Y=None)]),
    ("gemm_moe_combine_grad", [dict(T=-1), dict(H=-1), dict(R=-1), dict(top_k=0), dict(type=3), dict(lddy=63), dict(ldys=63), dict(lddys=63), dict(dY=None),
                               dict(Ys=None), dict(rows=None), dict(weights=None), dict(dYs=None), dict(dweights=None)]),
    ("gemm_grouped_f32acc", [dict(E=-1), dict(R=-1), dict(N=-1), dict(K=-1), dict(ab_type=F32), dict(ab_type=E4), dict(c_type=E4), dict(b_trans=2), dict(lda=63),
                             dict(ldb=63), dict(ldc=63), dict(stride_b=4095), dict(stride_b=0), dict(A=None), dict(B=None), dict(C=None), dict(offsets=None)]),
    ("gemm_grouped_wgrad_f32acc", [dict(E=-1), dict(R=-1), dict(M=-1), dict(N=-1), dict(ab_type=F32), dict(c_type=E4), dict(lda=63), dict(ldb=63), dict(ldc=63),
                                   dict(stride_c=4095), dict(stride_c=0), dict(A=None), dict(B=None), dict(C=None), dict(offsets=None)]),
    ("gemm_fp8_gated_act", [dict(rows=-1), dict(cols=-1), dict(type=E4), dict(q_type=BF16), dict(act=5), dict(act=-1), dict(ldg=255), dict(ldu=255), dict(ldh=255),
                            dict(ldgq=255), dict(lduq=255), dict(ldgs=3), dict(ldus=3), dict(G=None), dict(H=None), dict(GQ=None), dict(GS=None), dict(UQ=None),
                            dict(US=None), dict(U=None)]),
    ("gemm_fp8_gated_act_grad", [dict(rows=-1), dict(cols=-1), dict(type=E4), dict(q_type=BF16), dict(act=5), dict(act=-1), dict(lddh=255), dict(lddg=255),
                                 dict(lddu=255), dict(ldh=255), dict(ldgq=255), dict(lduq=255), dict(ldgs=3), dict(ldus=3), dict(dH=None), dict(GQ=None),
                                 dict(GS=None), dict(dG=None), dict(dU=None), dict(US=None), dict(UQ=None)]),
]


@pytest.mark.parametrize("name,change", [(n, c) for n, cs in INVALID for c in cs])
def test_invalid(L, name, change):
    assert call(L, name, **change) == g.GEMM_ERR_INVALID_ARG


UNSUPPORTED = [
    ("gemm_moe_dispatch", [dict(E=4097), dict(top_k=129), dict(T=BIG), dict(T=2 ** 28, top_k=8), dict(H=2 ** 30, ldx=2 ** 30, ldxs=2 ** 30)]),
    ("gemm_moe_combine", [dict(top_k=129), dict(T=BIG), dict(T=2 ** 28, top_k=8), dict(R=BIG), dict(H=BIG, ldys=BIG, ldy=BIG)]),
    ("gemm_moe_combine_grad", [dict(top_k=129), dict(T=BIG), dict(T=2 ** 28, top_k=8), dict(R=BIG), dict(H=BIG, lddy=BIG, ldys=BIG, lddys=BIG)]),
    ("gemm_grouped_f32acc", [dict(A=FAKE + 8), dict(B=FAKE + 2), dict(lda=68), dict(ldb=68, stride_b=8000), dict(stride_b=4100), dict(R=BIG), dict(E=BIG),
                             dict(N=BIG, ldc=BIG, stride_b=2 ** 50), dict(K=BIG, lda=2 ** 31, ldb=2 ** 31, stride_b=2 ** 50), dict(lda=2 ** 38),
                             dict(E=2 ** 20, R=2 ** 20, N=2 ** 12, ldc=2 ** 12, stride_b=2 ** 18)]),
    ("gemm_grouped_wgrad_f32acc", [dict(A=FAKE + 8), dict(B=FAKE + 2), dict(lda=68), dict(ldb=68), dict(R=BIG), dict(E=BIG), dict(M=BIG, lda=2 ** 31, stride_c=2 ** 50),
                                   dict(lda=2 ** 38), dict(ldb=2 ** 38)]),
    ("gemm_fp8_gated_act", [dict(rows=BIG, ldgs=BIG, ldus=BIG), dict(rows=2 ** 30, cols=2 ** 13, ldgs=2 ** 30, ldus=2 ** 30,
                                                                    **{k: 2 ** 13 for k in ("ldg", "ldu", "ldh", "ldgq", "lduq")})]),
    ("gemm_fp8_gated_act_grad", [dict(rows=BIG, ldgs=BIG, ldus=BIG)]),
]


@pytest.mark.parametrize("name,change", [(n, c) for n, cs in UNSUPPORTED for c in cs])
def test_unsupported(L, name, change):
    assert call(L, name, **change) == g.GEMM_ERR_UNSUPPORTED


# The kernels' 32-bit indices run over the last slot, of 2^31 - 32,768 at most, by less than 2^15, and over the last column, of
# 2^31 - 4096 at most, by 4096.
BEYOND = [
    ("gemm_moe_dispatch", [dict(T=2 ** 31 - 32767, top_k=1), dict(T=2 ** 31 - 512, top_k=1, X=None, Xs=None), dict(T=2 ** 24 - 255, top_k=128, X=None, Xs=None)]),
    ("gemm_moe_combine", [dict(H=h, ldys=2 ** 31, ldy=2 ** 31) for h in (2 ** 31 - 4095, 2 ** 31 - 2048, 2 ** 31 - 512)]),
    ("gemm_moe_combine_grad", [dict(H=h, lddy=2 ** 31, ldys=2 ** 31, lddys=2 ** 31) for h in (2 ** 31 - 4095, 2 ** 31 - 2048, 2 ** 31 - 512)]),
]


@pytest.mark.parametrize("name,change", [(n, c) for n, cs in BEYOND for c in cs])
def test_indices_that_would_pass_32_bits(L, name, change):
    assert call(L, name, **change) == g.GEMM_ERR_UNSUPPORTED


WORD_CALLS = list(CALLS)  # in the order of gemm_word_call


def words(name, **change):
    args = {**CALLS[name], **change}
    fmt = "".join("d" if n in ("alpha", "beta") else "q" for n in args)
    return struct.pack("=" + fmt, *(0 if v is None else v for v in args.values())), len(args)


@pytest.mark.parametrize("name,change", [(n, c) for n, cs in INVALID + UNSUPPORTED for c in cs])
def test_the_same_as_words(L, name, change):
    packed, n = words(name, **change)
    assert L.gemm_call_words(WORD_CALLS.index(name), packed, n) == call(L, name, **change) != g.GEMM_OK


def test_words_that_do_not_fit(L):
    for i, name in enumerate(WORD_CALLS):
        packed, n = words(name)
        for bad in (n - 1, n + 1, 0, -1):
            assert L.gemm_call_words(i, packed, bad) == g.GEMM_ERR_INVALID_ARG
        assert L.gemm_call_words(i, None, n) == g.GEMM_ERR_INVALID_ARG
        for first in (2 ** 31, -2 ** 31 - 1, 2 ** 40):  # an int that is none: not cut to one that would pass
            assert L.gemm_call_words(i, struct.pack("=q", first) + packed[8:], n) == g.GEMM_ERR_INVALID_ARG
    for i in (-1, len(WORD_CALLS)):
        assert L.gemm_call_words(i, words("gemm_moe_dispatch")[0], 13) == g.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("name,change", [
    ("gemm_moe_combine", dict(T=0, Ys=None, rows=None, Y=None)), ("gemm_moe_combine", dict(H=0, Ys=None, rows=None, Y=None)), ("gemm_moe_combine_grad", dict(T=0, rows=None, dY=None)),
    ("gemm_grouped_f32acc", dict(E=0, A=None, B=None, C=None, offsets=None)), ("gemm_grouped_f32acc", dict(R=0, A=None, C=None)), ("gemm_grouped_f32acc", dict(N=0, B=None, C=None)),
    ("gemm_grouped_wgrad_f32acc", dict(E=0, C=None, offsets=None)), ("gemm_grouped_wgrad_f32acc", dict(M=0, A=None, C=None)), ("gemm_grouped_wgrad_f32acc", dict(N=0, B=None, C=None)),
    ("gemm_fp8_gated_act", dict(rows=0, G=None, H=None)), ("gemm_fp8_gated_act", dict(cols=0, G=None, GQ=None)), ("gemm_fp8_gated_act_grad", dict(rows=0, dH=None)),
])
def test_empty(L, name, change):
    assert call(L, name, **change) == g.GEMM_OK
    assert g.last_launch_count() == 0


# ---------------------------------------------------------------- the binding
host_only = pytest.mark.skipif(gpu_available(), reason="host pointers stand in for device ones")
B16, I32, F = torch.bfloat16, torch.int32, torch.float32
E4T = torch.float8_e4m3fn


class OnCuda(torch.Tensor):
    """A CPU tensor that says it is a CUDA tensor: only its properties are looked at here."""
    is_cuda = True

    def get_device(self):
        return 0


def on(*shape, dtype=B16):
    return torch.zeros(shape).to(dtype).as_subclass(OnCuda)


def arguments():
    return {
        "moe_dispatch": dict(ids=on(4, 2, dtype=I32), X=on(4, 16), Xs=on(8, 16), offsets=on(7, dtype=I32), rows=on(4, 2, dtype=I32)),
        "moe_combine": dict(Ys=on(8, 16), rows=on(4, 2, dtype=I32), Y=on(4, 16), weights=on(4, 2, dtype=F)),
        "moe_combine_grad": dict(dY=on(4, 16), Ys=on(8, 16), rows=on(4, 2, dtype=I32), weights=on(4, 2, dtype=F), dYs=on(8, 16), dweights=on(4, 2, dtype=F)),
        "gemm_grouped": dict(A=on(8, 16), B=on(6, 24, 16), C=on(8, 24), offsets=on(7, dtype=I32)),
        "gemm_grouped_wgrad": dict(A=on(8, 16), B=on(8, 24), C=on(6, 16, 24, dtype=F), offsets=on(7, dtype=I32)),
        "fp8_gated_act": dict(G=on(4, 256), U=on(4, 256), H=on(4, 256), GQ=on(4, 256, dtype=E4T), GS=on(2, 4, dtype=F), UQ=on(4, 256, dtype=E4T), US=on(2, 4, dtype=F)),
        "fp8_gated_act_grad": dict(dH=on(4, 256), GQ=on(4, 256, dtype=E4T), GS=on(2, 4, dtype=F), UQ=on(4, 256, dtype=E4T), US=on(2, 4, dtype=F), dG=on(4, 256), dU=on(4, 256),
                                   H=on(4, 256)),
    }


NAMES = [(f, n) for f, a in arguments().items() for n in a]


@host_only
@pytest.mark.parametrize("function,name", NAMES)
@pytest.mark.parametrize("value", [3, "text", [1.0]])
def test_not_a_tensor(function, name, value):
    with pytest.raises(TypeError):
        getattr(g, function)(**{**arguments()[function], name: value})


@host_only
@pytest.mark.parametrize("function,name", NAMES)
@pytest.mark.parametrize("how", ["type", "shape", "device", "expanded"])
def test_wrong_tensor(function, name, how):
    args = arguments()[function]
    t = args[name]
    if how == "type":
        args[name] = on(*t.shape, dtype=torch.float64)
    elif how == "shape":
        args[name] = on(*t.shape[:-1], t.shape[-1] + (2 if name != "offsets" else 1), dtype=t.dtype)
        if function == "moe_dispatch" and name == "offsets":
            pytest.skip("any number of experts")
    elif how == "device":
        args[name] = torch.zeros(t.shape).to(t.dtype)
    else:
        args[name] = torch.zeros(1).to(t.dtype).expand(t.shape).as_subclass(OnCuda)
    with pytest.raises(TypeError if how in ("type", "device") else ValueError):
        getattr(g, function)(**args)


@host_only
@pytest.mark.parametrize("function,change", [
    ("moe_dispatch", dict(Xs=on(7, 16))), ("moe_dispatch", dict(Xs=on(8, 16, dtype=F))), ("moe_dispatch", dict(X=None)), ("moe_dispatch", dict(Xs=None)),
    ("moe_dispatch", dict(ids=on(4, 0, dtype=I32), rows=on(4, 0, dtype=I32))), ("moe_dispatch", dict(offsets=on(0, dtype=I32))), ("moe_dispatch", dict(offsets=on(3, 2, dtype=I32))),
    ("moe_combine", dict(Y=on(4, 16, dtype=F))), ("moe_combine_grad", dict(dYs=on(9, 16))), ("moe_combine_grad", dict(dYs=on(8, 16, dtype=torch.float16))),
    ("gemm_grouped", dict(B=on(6, 24, 16, dtype=torch.float16))), ("gemm_grouped", dict(b_trans=False)), ("gemm_grouped", dict(offsets=on(6, dtype=I32))),
    ("gemm_grouped", dict(B=on(24, 16))), ("gemm_grouped", dict(B=on(1, 24, 16).expand(6, 24, 16).as_subclass(OnCuda))),
    ("gemm_grouped", dict(B=on(6, 16, 24).transpose(1, 2).as_subclass(OnCuda))),
    ("gemm_grouped_wgrad", dict(B=on(9, 24))), ("gemm_grouped_wgrad", dict(C=on(1, 16, 24, dtype=F).expand(6, 16, 24).as_subclass(OnCuda))),
    ("fp8_gated_act", dict(U=None)), ("fp8_gated_act", dict(UQ=None)), ("fp8_gated_act", dict(UQ=on(4, 256, dtype=torch.float8_e5m2))), ("fp8_gated_act", dict(H=on(4, 256, dtype=F))),
    ("fp8_gated_act_grad", dict(UQ=None)), ("fp8_gated_act_grad", dict(dU=None)), ("fp8_gated_act_grad", dict(GS=on(4, 2, dtype=F))),
])
def test_what_does_not_fit(function, change):
    with pytest.raises((TypeError, ValueError)):
        getattr(g, function)(**{**arguments()[function], **change})


@host_only
@pytest.mark.parametrize("function", list(arguments()))
def test_other_device(function, monkeypatch):
    g._load_codes()
    monkeypatch.setattr(g, "_device_now", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        getattr(g, function)(**arguments()[function])
