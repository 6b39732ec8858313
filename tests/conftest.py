import glob
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

# Modules whose tests call the library with addresses that are none: it refuses the calls or, where no GPU is, fails to launch.  On a machine with a GPU a
# call that is accepted after all, by a check that was relaxed or an expectation that is wrong, would launch a kernel on them.
FAKE_ADDRESSES = {"test_boundary.py", "test_step_host.py", "test_step_edges_host.py", "test_packed_host.py", "test_packed_scratch_host.py",
                  "test_zz_no_alloc.py"}


def keep_off_gpus(items, gpu):
    for item in items:
        if gpu and item.path.name in FAKE_ADDRESSES and not item.get_closest_marker("gpu"):
            item.add_marker(pytest.mark.skip(reason="fake addresses must never reach a GPU"))


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built libqgemv")


def pytest_collection_modifyitems(items):
    keep_off_gpus(items, bool(glob.glob("/dev/nvidia[0-9]*")) or os.path.exists("/dev/nvidiactl"))
