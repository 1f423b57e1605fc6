import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")
    config.addinivalue_line("markers", "slow: long-running (full-size workloads)")


# Modules whose kernels wait on barriers: every test of theirs looks whether a wait gave up, which only the count tells
_WAITING = ("attention", "mx4_cache", "unseen_rows", "answers", "rotary")


@pytest.fixture(autouse=True)
def waits_have_ended(request):
    yield
    name = request.module.__name__
    if request.node.get_closest_marker("gpu") is not None and any(part in name for part in _WAITING):
        import extended_precision_gemm_gb300 as ddg

        assert ddg.wait_timeouts() == 0
