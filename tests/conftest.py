import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200, sm_100a)")
    config.addinivalue_line("markers", "slow: long-running CPU test")


@pytest.fixture(scope="session")
def cuda_device():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def bounds_flag_stays_clear(request):
    """On the bounds-checked build a GPU test also fails if one of its calls
    that left the status word to the binding computed an index outside a
    buffer (calls with a status word of their own assert on that)."""
    yield
    if request.node.get_closest_marker("gpu") is None:
        return
    from tree_speculative_decoding_ancestor_b200 import binding
    for word in binding._status.values():
        assert not int(word.item()) & binding.DEV_BOUNDS
