import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


# Tests that expect a wrong value: they stay as they were written and have to fail, at an assertion.
WRONG = {
    "test_gpu_serving4.py::test_a_run_of_prompts_tokens_reads_and_evictions":
        "counts positions from the lengths that an eviction has shrunk, while the kept keys stay turned by their former "
        "positions; test_gpu_serving_positions.py has the same run with the positions counted",
}


def pytest_collection_modifyitems(items):
    for item in items:
        for name, why in WRONG.items():
            if name in item.nodeid:
                item.add_marker(pytest.mark.xfail(reason=why, raises=AssertionError, strict=True))


@pytest.fixture(scope="session", autouse=True)
def _oracle_built():
    import oracle
    if not os.path.exists(os.path.join(ROOT, "oracle", "liboracle.so")):
        oracle.build()
    yield


def golden(name):
    """Parse a tests/golden/*.txt fixture: '#' comments, 'key value...' lines."""
    out = {}
    with open(os.path.join(ROOT, "tests", "golden", name)) as f:
        for line in f:
            line = line.strip()
            if not line or line.startswith("#"):
                continue
            k, *vals = line.split()
            out[k] = vals
    return out
