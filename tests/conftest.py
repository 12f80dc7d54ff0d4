import glob
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
    config.addinivalue_line("markers", "slow: long CPU test")


# Tests that hand made-up addresses to the library: never beside a GPU, also
# where torch, which the file itself asks for one, cannot be imported.
MADE_UP_ADDRESSES = "test_token_ops_cpu.py"


def gpu_nodes():
    return glob.glob("/dev/nvidia[0-9]*")


def pytest_collection_modifyitems(items):
    if gpu_nodes():
        for item in items:
            if item.path.name == MADE_UP_ADDRESSES:
                item.add_marker(pytest.mark.skip(reason="made-up addresses stay away from a GPU"))


@pytest.fixture(scope="session")
def cuda_device():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")
