import os
import sys

REPO = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if REPO not in sys.path:
    sys.path.insert(0, REPO)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a); runs through the C-ABI library")
    config.addinivalue_line("markers", "slow: large-workload parity case")


def pytest_collection_modifyitems(items):
    # the tests of offsets past 32 bits hold tens of GB on the device
    for item in items:
        if "offsets_past_32_bits" in item.name:
            item.add_marker("slow")
