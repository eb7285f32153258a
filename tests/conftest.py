import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (runs through the HIP C-ABI library)")


# What these cases end with, residual gradient == grad_y on every row, is not the gradient: y is 0 behind the last row
# whatever the residual holds, so it is 0 there.  test_gpu_experts_edges.py runs the same inputs against that (and
# checks y, dx, dw and db of them as these do).
def _wrong_residual_gradient(item):
    if item.path.name != "test_gpu_experts.py" or item.originalname not in ("test_product",
                                                                            "test_product_unaligned_storage"):
        return False
    return item.callspec.params["residual"] and item.callspec.params["dropped"] > 0


def pytest_collection_modifyitems(items):
    for item in items:
        if _wrong_residual_gradient(item):
            item.add_marker(pytest.mark.xfail(strict=True, raises=AssertionError,
                                              reason="asserts grad_y as the residual's gradient of rows that are 0"))
