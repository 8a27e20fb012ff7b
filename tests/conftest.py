import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GB300 (sm_103) device; runs the CUDA path")


# Host tests whose call passes every check, with fake addresses, before they ask whether
# there is a GPU: beside one it would be a real launch, so they are skipped before it.
CALLS_BEFORE_ASKING = {"test_valid_arguments_reach_the_device_check", "test_strided_accepts_views_and_nope192_shapes"}


def pytest_runtest_setup(item):
    if item.name in CALLS_BEFORE_ASKING:
        import torch
        if torch.cuda.is_available():
            pytest.skip("a GPU is present; covered by the GPU tests")


@pytest.fixture(scope="session")
def built_library():
    """Build libmlaqp.so if it is missing or stale, then load it."""
    from mla_decode_query_gb300 import build, load_library
    build.build_library()
    return load_library()


@pytest.fixture(scope="session")
def cuda_device(built_library):
    """The GPU tests must run on the CUDA path: fail (never skip) without it."""
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU test selected but CUDA is not available")
    torch.cuda.init()
    return torch.device("cuda:0")
