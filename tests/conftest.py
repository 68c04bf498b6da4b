import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

ADDRESS_TESTS = {"test_packed_host.py", "test_rope_in_place_host.py"}


def pytest_configure(config):
    config.addinivalue_line(
        "markers", "gpu: runs CUDA kernels; needs a GB300 (sm_103a) GPU")


def pytest_collection_modifyitems(config, items):
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        has_gpu = False
    if has_gpu:
        # calls that pass every check with addresses that are not memory: with
        # a GPU they would be launched
        skip = pytest.mark.skip(reason="addresses that no kernel may follow: without a GPU only")
        for item in items:
            if item.path.name in ADDRESS_TESTS:
                item.add_marker(skip)
        return
    skip = pytest.mark.skip(reason="no CUDA device in this process")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)
