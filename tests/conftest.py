import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


# Modules whose calls pass every check with descriptors of host memory and then
# fail to launch for want of a GPU; where there is one they would run on that memory.
HOST_MEMORY = ("test_abi_operators_cpu", "test_cache_overlap_cpu")


def pytest_runtest_setup(item):
    if item.module.__name__ in HOST_MEMORY:
        import torch

        if torch.cuda.is_available():
            pytest.skip("descriptors of host memory: the launches would run")
