"""How many bits of h the mixture-of-experts layer keeps between its two halves.

With no gate, no activation, one expert a token and a down projection that is
the identity, Y is h itself.  Tokens and weights are integers whose products sum
to less than 2^24, so h is exact in FP32 in whatever order it is summed, and what
Y differs by is what holding h as 16-bit numbers dropped.

Bounds, of a token's largest |h|.  BF16 weights: three numbers of 8 bits hold
all 24, and adding them up again in FP32 rounds to 2^-23 at most: 2^-22.  FP16
and e4m3 weights: two numbers of 11 bits leave 2^-23, and 2^-21 where the second
is subnormal; with the sum 2^-20.  One number fewer leaves 2^-17 or 2^-12,
beyond either bound, which the last test shows on the 64-bit values.
"""
import numpy as np
import pytest
import torch

import dense_gemm_11_gb300 as g
from conftest import gpu_available

E4 = torch.float8_e4m3fn
N = 256
# tokens, weights: the largest integers, and the bound
KINDS = {"bf16": (torch.bfloat16, torch.bfloat16, 255, 255, 2.0 ** -22), "f16": (torch.float16, torch.float16, 255, 255, 2.0 ** -20),
         "e4m3_f16": (torch.float16, E4, 2047, 15, 2.0 ** -20), "e4m3_bf16": (torch.bfloat16, E4, 255, 15, 2.0 ** -20)}


def integers(kind, T, signs=True, small=1):
    """(X, gate, h) of float64 integers: two experts, the first for even tokens."""
    _, _, x_max, w_max, _ = KINDS[kind]
    rng = np.random.default_rng(T)
    x = rng.integers(-x_max if signs else 0, x_max + 1, (T, N)).astype(np.float64)
    w = rng.integers(0, w_max // small + 1, (2, N, N)).astype(np.float64)
    x[:, 0], x[1::2, 1], x[0::2, 1] = 1, 16, 0  # what the router looks at
    w[:, :, :2] = 0
    h = np.einsum("eij,tj->eti", w, x)
    return x, w, np.where((np.arange(T) % 2 == 0)[:, None], h[0], h[1])


@pytest.mark.gpu
@pytest.mark.skipif(not gpu_available(), reason="needs a GPU")
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 9, 40])
@pytest.mark.parametrize("small", [1, 15])
def test_hidden_values_keep_their_bits(kind, T, small):
    """small: h inside FP16's range for some tokens, as well as outside."""
    xt, wt, _, _, bound = KINDS[kind]
    x, w, h = integers(kind, T, small=small)
    assert np.abs(np.einsum("eij,tj->eti", w, np.abs(x))).max() < 2 ** 24
    dev = lambda a, t: torch.from_numpy(a).float().cuda().to(t)  # noqa: E731
    router = torch.zeros(2, N, dtype=xt, device="cuda")
    router[0, 0], router[1, 1] = 8.0, 1.0
    gate, down = dev(w, wt), dev(np.broadcast_to(np.eye(N), (2, N, N)).copy(), wt)
    scales = None if wt != E4 else (torch.ones(2, 2, 2, device="cuda"), None, torch.ones(2, 2, 2, device="cuda"))
    Y = torch.empty(T, N, device="cuda")
    ids = torch.empty(T, 1, dtype=torch.int32, device="cuda")
    g.moe_few_tokens(dev(x, xt), router, gate, None, down, Y, 1, scales=scales, act=g.GEMM_ACT_NONE, ids=ids)
    assert g.check() == g.GEMM_OK
    assert np.array_equal(ids.cpu().numpy()[:, 0], np.arange(T) % 2)
    off = np.abs(Y.double().cpu().numpy() - h).max(axis=1) / np.abs(h).max(axis=1)
    assert off.max() <= bound, off.max()


def held(h, numbers, dtype):
    """h as the sum of so many 16-bit numbers."""
    rest, total = torch.from_numpy(h), torch.zeros(h.shape, dtype=torch.float64)
    for _ in range(numbers):
        part = rest.to(torch.float32).to(dtype).double()
        total, rest = total + part, rest - part
    return total.numpy()


@pytest.mark.parametrize("kind", KINDS)
def test_bounds_tell_a_lost_number(kind):
    _, _, h = integers(kind, 9)
    h = h / 2.0 ** np.ceil(np.log2(np.abs(h).max() / 2 ** 15))  # where FP16 holds it
    dtype, all_of_it = (torch.bfloat16, 3) if kind == "bf16" else (torch.float16, 2)
    off = lambda n: (np.abs(held(h, n, dtype) - h).max(axis=1) / np.abs(h).max(axis=1)).max()  # noqa: E731
    assert off(all_of_it) <= KINDS[kind][-1] / 2 and off(all_of_it - 1) > 2 * KINDS[kind][-1]
