"""Test configuration: the ``gpu`` marker and the repository root on sys.path."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a B200 (sm_100a) and the built CUDA library")


@pytest.fixture(autouse=True, scope="module")
def ordinary_waits_end(request):
    """No bounded wait may run out in the ordinary key-weight tests: a missed one can leave
    the result right and the status clear, a second late."""
    if not request.module.__name__.endswith(("test_gpu_key_weights", "test_gpu_key_weight_parts")):
        yield
        return
    import speculative_decoding_tree_va_b200 as va
    before = va.device_timeouts()
    yield
    assert va.device_timeouts() == before
