"""Arguments of moe_few_tokens that are no tensors, or of the wrong kind, are refused by name (no GPU)."""
import pytest
import torch

import dense_gemm_11_gb300 as g
from conftest import gpu_available
from test_row_strides import OnCuda

pytestmark = pytest.mark.skipif(gpu_available(), reason="host pointers stand in for device ones")
E4 = torch.float8_e4m3fn


def on(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape).to(dtype).as_subclass(OnCuda)


def arguments(fp8):
    wt = E4 if fp8 else torch.bfloat16
    args = dict(X=on(4, 32), router=on(6, 32), gate=on(6, 16, 32, dtype=wt), up=on(6, 16, 32, dtype=wt), down=on(6, 32, 16, dtype=wt), Y=on(4, 32), top_k=2)
    return args, [on(6, 1, 1, dtype=torch.float32) for _ in range(3)] if fp8 else None


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", ["X", "router", "gate", "up", "down", "Y"])
@pytest.mark.parametrize("value", [None, 3, [1.0]])
def test_not_a_tensor(fp8, name, value):
    if name == "up" and value is None:
        pytest.skip("a layer without a gate")
    args, scales = arguments(fp8)
    with pytest.raises(TypeError):
        g.moe_few_tokens(**{**args, name: value}, scales=scales)


@pytest.mark.parametrize("i", [0, 1, 2])
@pytest.mark.parametrize("value", [None, 1.0, "half"])
def test_scales(i, value):
    args, scales = arguments(True)
    scales[i] = scales[i].half() if value == "half" else value
    with pytest.raises(TypeError, match=rf"scales\[{i}\]"):
        g.moe_few_tokens(**args, scales=scales)


@pytest.mark.parametrize("name", ["ids", "weights"])
def test_outputs(name):
    args, _ = arguments(False)
    for value in ([[0, 1]] * 4, on(4, 2), on(2, 4, dtype=torch.int32 if name == "ids" else torch.float32)):
        with pytest.raises(TypeError, match=name):
            g.moe_few_tokens(**args, **{name: value})
