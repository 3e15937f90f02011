"""Matrices whose rows share memory are refused (no GPU: the refusal comes before any call).

A column of n rows expanded from one element has row stride 0, which is not a
leading dimension: read with 1 it would run n - 1 elements past its memory.
"""
import pytest
import torch

import dense_gemm_11_gb300 as g
from conftest import gpu_available

pytestmark = pytest.mark.skipif(gpu_available(), reason="host pointers stand in for device ones")
E4 = torch.float8_e4m3fn


class OnCuda(torch.Tensor):
    """A CPU tensor that says it is a CUDA tensor: only its properties are looked at here."""
    is_cuda = True


def mat(rows, cols, dtype=torch.float32, expanded=False):
    t = torch.zeros(1, cols, dtype=torch.float32).to(dtype).expand(rows, cols) if expanded else torch.zeros(rows, cols).to(dtype)
    return t.as_subclass(OnCuda)


@pytest.mark.parametrize("cols", [1, 16])
@pytest.mark.parametrize("bad", ["X", "Q", "S"])
def test_quantize(bad, cols):
    args = {"X": mat(300, cols), "Q": mat(300, cols, E4), "S": mat(1, 300)}
    layout = "rows"
    if bad == "S":
        args, layout = {"X": mat(300, cols), "Q": mat(cols, 300, E4), "S": mat(3, cols)}, "cols"
    args[bad] = mat(*args[bad].shape, args[bad].dtype, expanded=True)
    with pytest.raises(ValueError, match=f"{bad} needs a row stride"):
        g.fp8_quantize(*args.values(), layout)


@pytest.mark.parametrize("bad", ["A", "SA", "B", "SB", "C"])
def test_product(bad):
    M, N, K = (1, 1, 300) if bad in ("SA", "SB") else (40, 1, 1) if bad in ("A", "C") else (1, 40, 1)
    args = {"A": mat(M, K, E4), "SA": mat(-(-K // 128), M), "B": mat(N, K, E4), "SB": mat(-(-K // 128), N), "C": mat(M, N)}
    args[bad] = mat(*args[bad].shape, args[bad].dtype, expanded=True)
    with pytest.raises(ValueError, match=f"^{bad} needs a row stride"):
        g.gemm_fp8(*args.values(), b_scales="rows")


@pytest.mark.parametrize("bad", [0, 1, 2])
def test_dense(bad):
    args = [mat(40, 40), mat(40, 40), mat(40, 40)]
    args[bad] = mat(40, 1, expanded=True)
    with pytest.raises(ValueError, match="needs a row stride"):
        g.gemm_f32(*args)


def test_what_is_fine():
    """One row, no rows, no columns, and a view of a wider matrix."""
    for t in (mat(1, 8, expanded=True), mat(0, 8), mat(5, 0), mat(5, 16)[:, :3], mat(1, 1, expanded=True)):
        _, ld, rows, cols, _ = g._typed_mat(t, "X", g._FLOATS)
        assert (rows, cols) == tuple(t.shape) and ld >= max(1, cols)
        assert g._mat(t, "X", torch.float32)[1] >= max(1, cols)
