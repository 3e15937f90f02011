"""The mixture-of-experts operators for many tokens in the GEMM11_DEBUG build.

Child processes load the debug library: these operators' tests pass with its
synchronous pipelines and index checks, and with the extent of the result made
smaller than the result (GEMM11_DEBUG_SHRINK_C) the checks fire, the stores past
it are skipped and the rest is right.  The memory is as large as without the
shrink, so no access leaves it either way.
"""
import pytest

from conftest import gpu_available
from test_gpu_debug_build import _child

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def test_operators_with_the_debug_library():
    rc, out = _child(["-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu", "tests/test_gpu_moe_rows.py", "tests/test_gpu_grouped.py",
                      "tests/test_gpu_gated_act.py", "tests/test_gpu_moe_layer.py", "-k", "not graphs and not test_example"], {})
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
T, k, H = 6, 2, 8
ids = torch.arange(T * k, device="cuda").reshape(T, k).int()
rows, offsets = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T * k + 1, dtype=torch.int32, device="cuda")
x, xs = ints(T, H), torch.empty(T * k, H, device="cuda")
fires(lambda: g.moe_dispatch(ids, x, xs, offsets, rows), xs, x.repeat_interleave(k, 0))
rows = torch.arange(T * k, device="cuda").int().reshape(T, k)
ys, y = ints(T * k, 16), torch.empty(T, 16, device="cuda")
fires(lambda: g.moe_combine(ys, rows, y), y, ys.reshape(T, k, 16).sum(1))
dys, dy, w = torch.empty(T * k, 16, device="cuda"), ints(T, 16), ints(T, k)
fires(lambda: g.moe_combine_grad(dy, ys, rows, w, dys, torch.empty(T, k, device="cuda")), dys, dy.repeat_interleave(k, 0) * w.reshape(-1, 1))
off = torch.tensor([0, 30, 40], device="cuda").int()
for K in (64, 8192):  # whole, and shared contractions
    a, b, c = ints(40, K).bfloat16(), ints(2, 24, K).bfloat16(), torch.empty(40, 24, device="cuda")
    want = torch.cat([a[:30].float() @ b[0].float().t(), a[30:].float() @ b[1].float().t()])
    fires(lambda: g.gemm_grouped(a, b, c, off), c, want)
for R in (40, 40000):
    off = torch.tensor([0, R // 2 - 3, R], device="cuda").int()
    a, b, c = ints(R, 16).bfloat16(), ints(R, 24).bfloat16(), torch.empty(2, 16, 24, device="cuda")
    s = [slice(0, R // 2 - 3), slice(R // 2 - 3, R)]
    fires(lambda: g.gemm_grouped_wgrad(a, b, c, off), c, torch.stack([a[i].float().t() @ b[i].float() for i in s]))
G, h = ints(3, 64), torch.empty(3, 64, device="cuda")
Q, S = g.fp8_empty(3, 64)
fires(lambda: g.fp8_gated_act(G, None, h, Q, S, act=g.GEMM_ACT_RELU), h, G.relu())
fires(lambda: g.fp8_gated_act_grad(G, Q, S, None, None, h, None, act=g.GEMM_ACT_NONE), h, G)
print("shrink ok")
"""


def test_checks_fire_and_skip_the_store():
    rc, out = _child(["-c", SHRINK_SCRIPT], {"GEMM11_DEBUG_SHRINK_C": "8"})
    assert rc == 0 and "shrink ok" in out, out[-3000:]
