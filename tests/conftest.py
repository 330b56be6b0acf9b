import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (runs through the HIP library)")
    config.addinivalue_line("markers", "slow: large CPU work")


# Tests kept as they were written whose expected value is not the contract's: they have to fail.
OUTDATED = {
    "test_gpu_mx.py::test_rmsnorm_tiny_and_huge_rows":
        "expects zeros for a finite row of 1e25, where include/lora.h's formula gives h / rms; "
        "test_gpu_mx_range.py::test_rmsnorm_rows_of_every_size holds the formula's values",
}


def pytest_collection_modifyitems(items):
    for item in items:
        reason = OUTDATED.get("::".join((item.path.name, item.name)))
        if reason:
            item.add_marker(pytest.mark.xfail(reason=reason, strict=True, raises=AssertionError))
