"""Shared test setup: the `gpu` marker and import paths."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")


# Cases that hold a value which is wrong; they still run.
WRONG = {
    "test_gpu_kv_cache.py::test_evict[256-16-1-33-33-0]":
        "expects rows 16-31 of a sequence, whose page does not exist, to be kept and their places to stay as they were: "
        "there they hold NaN scales, so all queries over the evicted pages would be NaN (tests/test_gpu_kv_holes.py)",
}


def pytest_collection_modifyitems(items):
    for item in items:
        for name, why in WRONG.items():
            if item.nodeid.endswith(name):
                item.add_marker(pytest.mark.xfail(raises=AssertionError, strict=True, reason=why))
