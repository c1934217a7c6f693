import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (runs through the C-ABI library)")
    config.addinivalue_line("markers", "slow: long-running CPU test")


# Host checks hand the library made-up pointers and expect a refusal before any launch.
# This one also makes a call that the library rightly accepts (append does not look at the
# order pools): without a GPU the launch fails, with one it would fault.
REACHES_THE_GPU = {"test_pools_without_pages"}


def pytest_collection_modifyitems(items):
    here = [x for x in items if x.name in REACHES_THE_GPU]
    if here:
        import torch
        if torch.cuda.is_available():
            for x in here:
                x.add_marker(pytest.mark.skip(reason="made-up pointers: only without a GPU"))


@pytest.fixture(scope="session")
def oracle_mod():
    import oracle
    oracle.build()
    return oracle
