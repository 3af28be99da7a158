"""The page calls without a GPU: how they are launched, and sizes that the call has to refuse, not the binding."""
import os

import pytest
import torch

import sliding_window_gqa_prep_gb300 as swa
from sliding_window_gqa_prep_gb300 import paged4

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(swa.__file__))), "sliding_window_gqa_prep_gb300", "csrc")


def test_no_call_asks_for_every_SM_at_once():
    """A cooperative launch waits until all its blocks fit beside what other streams run, and is refused where a process
    has fewer SMs than the device: counts in place need none."""
    with open(os.path.join(CSRC, "swa_pages.cu")) as h:
        s = h.read()
    assert "Cooperative" not in s and "this_grid" not in s

def test_pools_without_pages():
    """Empty pools came out as a division by zero: the call itself refuses them."""
    assert paged4._pools([torch.zeros(0, 2, 16, 64)], 0, -1)[:2] == (0, 1)
    with pytest.raises(ValueError):
        paged4._pools([torch.zeros(4, 2, 16, 64)], 0, -1)
