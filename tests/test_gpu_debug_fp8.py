"""The 8-bit operators and the mixture of experts in the GEMM11_DEBUG build.

Child processes load the debug library: a subset of these operators' tests
passes with its synchronous pipelines and index checks, and with the extent of
the result made smaller than the result (GEMM11_DEBUG_SHRINK_C) the checks fire,
the stores past it are skipped and the rest is right.  The memory is as large as
without the shrink, so no access leaves it either way.
"""
import pytest

from conftest import gpu_available
from test_gpu_debug_build import _child

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def test_operators_with_the_debug_library():
    rc, out = _child(["-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu", "tests/test_gpu_fp8.py", "tests/test_gpu_fp8_small_blocks.py",
                      "tests/test_gpu_fp8_many_tiles.py", "tests/test_gpu_moe.py", "tests/test_moe_hidden_bits.py",
                      "-k", "test_quantize or test_zeros or test_product or cut_along_k and not graph or test_layer or hidden_values or uneven or strided"], {})
    assert rc == 0, out[-3000:]
    assert " passed" in out


SHRINK_SCRIPT = r"""
import torch
import dense_gemm_11_gb300 as g
assert g.debug_build()

def fires(call, out, want):
    out.fill_(-1)
    try:
        call()
        raise SystemExit("the check did not fire")
    except g.GemmError as e:
        assert e.status == g.GEMM_ERR_DEBUG_CHECK, g.status_string(e.status)
    got, want = out.reshape(-1).float().cpu(), want.reshape(-1).float().cpu()
    assert (got[-8:] == -1).all(), got[-8:]          # past the extent: not stored
    assert torch.equal(got[:-8], want[:-8])          # the rest, of small integers: exact
    assert g.check() == g.GEMM_OK                    # reported once, by the call

gen = torch.Generator(device="cuda").manual_seed(1)
ints = lambda *s: torch.randint(-4, 5, s, generator=gen, device="cuda").float()
E4 = torch.float8_e4m3fn
for M, N, K in ((40, 65, 256), (300, 203, 256), (4, 128, 2048)):   # whole tiles, CTA pairs into odd rows, split over a cluster
    a, b, C = ints(M, K), ints(N, K), torch.empty(M, N, device="cuda")
    ones = lambda *s: torch.ones(s[0], (s[1] + 3) // 4 * 4, device="cuda")[:, :s[1]]
    fires(lambda: g.gemm_fp8(a.to(E4), ones(K // 128, M), b.to(E4), ones(-(-N // 128), K // 128), C), C, a @ b.t())
for layout in ("rows", "blocks", "cols"):
    x = ints(128, 128)
    x[:, 0], x[0, :] = 448, 448  # every scale is one
    Q, S = torch.empty(128, 128, dtype=E4, device="cuda"), torch.empty((1, 1) if layout == "blocks" else (1, 128), device="cuda")
    fires(lambda: g.fp8_quantize(x, Q, S, layout), Q, x.t() if layout == "cols" else x)
X, router = ints(5, 64).bfloat16(), torch.zeros(3, 64, device="cuda").bfloat16()
gate, down, Y = ints(3, 48, 64).bfloat16(), ints(3, 64, 48).bfloat16(), torch.empty(5, 64, device="cuda")
fires(lambda: g.moe_few_tokens(X, router, gate, None, down, Y, 1, act=g.GEMM_ACT_NONE), Y, X.float() @ gate[0].float().t() @ down[0].float().t())
print("shrink ok")
"""


def test_checks_fire_and_skip_the_store():
    rc, out = _child(["-c", SHRINK_SCRIPT], {"GEMM11_DEBUG_SHRINK_C": "8"})
    assert rc == 0 and "shrink ok" in out, out[-3000:]
