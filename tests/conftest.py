import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: long CPU test")


def gpu_available() -> bool:
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


@pytest.fixture(scope="session")
def require_gpu():
    if not gpu_available():
        pytest.skip("no GPU visible")


# Tests whose expected value is not what include/qgemv.h defines.  They run as
# they stand and are expected to fail; the test named beside each has the value
# that the oracle gives.
CONTRADICTED = {
    "test_gpu_kv.py::test_length_past_the_table_counts_as_the_tables":
        "expects a length of 10^9 over a table of 64 slots to give the rows of a length of 64; row t is the token at "
        "len - (start[b+1] - t), so both rows stand past the table and see 64 tokens, not 63 and 64 "
        "(test_gpu_kv_edges.py::test_lengths_far_past_the_table)",
}


def pytest_collection_modifyitems(items):
    for item in items:
        reason = CONTRADICTED.get(item.nodeid.rsplit("/", 1)[-1])
        if reason:
            item.add_marker(pytest.mark.xfail(reason=reason, raises=AssertionError, strict=True))
