import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: full-size workloads (minutes of host work)")


@pytest.fixture(scope="session")
def oracle_mod():
    import oracle
    return oracle


# Tests that hold a value the contract does not have; they stay as they were and are run, and are meant to fail.
SUPERSEDED = {
    "test_gpu_kv_cache.py::test_evict_with_missing_pages":
        "expects kept places for tokens on missing pages, whose new places are then never written but count as tokens; "
        "test_gpu_kv_contract.py::test_evicted_tokens_are_there has the same lengths, budget and missing pages",
}


def pytest_collection_modifyitems(items):
    for item in items:
        for name, reason in SUPERSEDED.items():
            if item.nodeid.endswith(name):
                item.add_marker(pytest.mark.xfail(reason=reason, raises=AssertionError, strict=True))
