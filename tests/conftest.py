import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")
    config.addinivalue_line("markers", "slow: takes more than a few seconds")


# Tests that hold a wrong value, and why it is wrong.  They run, and are expected to fail.
WRONG = {
    "test_draft_capi_cpu.py::test_oracle_trees_closed_forms":
        "of a tree's own slots it has a chain see all before it under any window; a chain sees what attention has it see, which is "
        "no slot at or before its own less the window (test_oracle_chain_under_a_window_sees_what_attention_sees); its other lines "
        "are test_oracle_ways_masks_and_branches",
}


def pytest_collection_modifyitems(items):
    for item in items:
        reason = WRONG.get(item.nodeid.split("/")[-1])   # wherever the run is rooted
        if reason:
            item.add_marker(pytest.mark.xfail(reason=reason, raises=AssertionError, strict=True))
