import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


# Tests that hold a value which was found wrong.  They stay as they were written and run; that they fail is expected.
WRONG_VALUES = {
    "test_gpu_layer_ops.py::test_page_plan_by_hand[too-many-tokens]":
        "expects lengths and pages of all 30 new tokens beside positions of the 17 that are kept: attention places a "
        "request's rows by its length, so those of the request that is cut would be off by the 3 tokens that are not "
        "there (test_gpu_plan_cut.py has the case, and a prompt in two such steps)",
}


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a) and the built library")
    config.addinivalue_line("markers", "slow: long-running CPU test")


def pytest_collection_modifyitems(config, items):
    for it in items:
        reason = WRONG_VALUES.get(it.nodeid.split("/")[-1])
        if reason:
            it.add_marker(pytest.mark.xfail(reason=reason, strict=True))
    # GPU tests need a device; skip them cleanly where there is none so that
    # `-m "not gpu"` and plain runs on a CPU host stay green.
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        has_gpu = False
    if has_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for it in items:
        if "gpu" in it.keywords:
            it.add_marker(skip)
