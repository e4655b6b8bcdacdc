import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")


@pytest.fixture(autouse=True)
def _free_blocks_of_zeros(request):
    """test_serve_native_binding compares whole outputs of two calls, among them rows that belong to no sequence:
    those are not written and hold what their memory held. It begins with small free blocks of zeros, in
    whatever order the tests run."""
    if request.module.__name__.rpartition(".")[2] == "test_serve_native_binding" and request.node.get_closest_marker("gpu"):
        import torch
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        # Requests of up to 1 MB come from one pool, whose free blocks these become.
        held = [torch.zeros(1 << 18, dtype=torch.int32, device="cuda") for _ in range(16)]
        torch.cuda.synchronize()
        del held
    yield
