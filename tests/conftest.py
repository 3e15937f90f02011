import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")


def gpu_available():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


# Tests whose expected value is known to be wrong, with the reason.  They run as
# they were written and have to fail.
WRONG_EXPECTATIONS = {
    "tests/test_gpu_fp8.py::test_quantize_special_values":
        "its reference divides 57344 by 2^-117, which overflows FP32, so that it expects NaN for a block of zeros in "
        "e5m2; test_gpu_fp8_small_blocks.py has the same inputs with the floor that keeps zeros",
}


def pytest_collection_modifyitems(items):
    for item in items:
        reason = WRONG_EXPECTATIONS.get(item.nodeid.split("[")[0])
        if reason:
            item.add_marker(pytest.mark.xfail(strict=True, reason=reason))
