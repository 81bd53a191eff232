import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")


# Tests whose expected values contradict include/lora_decode.h.  They still run,
# and have to fail.
_WRONG_VALUES = {
    "test_decode_pages_gpu.py::test_random_steps":
        "its model leaves a sequence that is cut inside a shared page on that page; the header shares full pages only. "
        "test_decode_shared_pages_gpu.py::test_random_steps is the same run with the sequence's own page",
}


def pytest_collection_modifyitems(items):
    for item in items:
        reason = _WRONG_VALUES.get(item.nodeid.rsplit("/", 1)[-1])
        if reason:
            item.add_marker(pytest.mark.xfail(reason=reason, strict=True))


@pytest.fixture(scope="session")
def oracle_mod():
    import oracle
    oracle.lib()
    return oracle
