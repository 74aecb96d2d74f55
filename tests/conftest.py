import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200, sm_100a)")


def read_golden(name):
    """Non-comment lines of a fixture under tests/golden/."""
    path = os.path.join(ROOT, "tests", "golden", name)
    with open(path, encoding="utf-8") as f:
        return [ln.strip() for ln in f if ln.strip() and not ln.startswith("#")]


def golden_table(name):
    out = {}
    for ln in read_golden(name):
        key, rest = ln.split("=", 1)
        out[key.strip()] = float(rest.split(";", 1)[0])
    return out


# These modules pass made-up addresses to entry points and expect the call to end at
# the check for a device.  Where there is one, the kernels would run on them.
MADE_UP_ADDRESSES = ("test_abi", "test_adapter_host", "test_adapter_limits", "test_adapter_overlap")


def skip_made_up_addresses(items, have_device):
    for item in items if have_device else ():
        if item.module.__name__ in MADE_UP_ADDRESSES:
            item.add_marker(pytest.mark.skip(reason="made-up addresses: only on a machine without a GPU"))


def pytest_collection_modifyitems(config, items):
    if any(item.module.__name__ in MADE_UP_ADDRESSES for item in items if hasattr(item, "module")):
        import torch
        skip_made_up_addresses(items, torch.cuda.is_available())
