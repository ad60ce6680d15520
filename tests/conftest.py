import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: long-running CPU test")


#: Tests that assert what the framework no longer does, with the reason.  They stay as they were written, and run where there
#: is no GPU: on one, the call that they expect to be refused would start kernels on addresses that are no memory.
OVERTAKEN = {
    "test_dense_abi.py::test_forward":
        "refuses MXFP8 products of 64 columns: the format's blocks are 32 columns, and moe_gated writes such rows; "
        "test_dense_edges_abi.py makes the test's other assertions",
}


def pytest_collection_modifyitems(items):
    for item in items:
        for name, reason in OVERTAKEN.items():
            if item.nodeid.split("[")[0].endswith(name):
                item.add_marker(pytest.mark.xfail(reason=reason, run=not os.path.exists("/dev/kfd")))
