"""The page calls without a GPU: how they are launched."""
import os

import sliding_window_gqa_prep_gb300 as swa

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(swa.__file__))), "sliding_window_gqa_prep_gb300", "csrc")


def test_no_call_asks_for_every_SM_at_once():
    """A cooperative launch waits until all its blocks fit beside what other streams run, and is refused where a process
    has fewer SMs than the device: counts in place need none."""
    with open(os.path.join(CSRC, "swa_pages.cu")) as h:
        s = h.read()
    assert "Cooperative" not in s and "this_grid" not in s
