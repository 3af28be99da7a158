"""The checks that the binding of the paged calls makes before it packs a struct, on CPU tensors
(whose device number is -1) in the place of CUDA ones."""
import pytest
import torch

import sliding_window_gqa_prep_gb300 as swa
from sliding_window_gqa_prep_gb300 import paged

CPU = -1


def parts():
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 3, dtype=torch.int32)
    return pool, pool.clone(), table, torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)


def test_cache_fields():
    k, v, table, start, lens = parts()
    fields, cap = paged._cache(k, v, table, start, lens, CPU)
    assert fields[:6] == (1, 2, 64, 16, 4, 3) and cap == 48
    assert fields[7:] == (k.data_ptr(), v.data_ptr(), table.data_ptr(), start.data_ptr(), lens.data_ptr())
    # one pool in both places, as swa.h allows for the calls that only read
    assert paged._cache(k, k, table, start, lens, CPU)[0][7:9] == (k.data_ptr(), k.data_ptr())


def test_no_values_are_not_taken_for_the_keys():
    """cache_v=None once stood for cache_k: the attention's result came from the keys."""
    k, v, table, start, lens = parts()
    with pytest.raises(ValueError):
        paged._cache(k, None, table, start, lens, CPU)


@pytest.mark.parametrize("which", range(5))
def test_what_is_no_tensor_is_refused(which):
    a = list(parts())
    if which == 3:
        a[which] = 5                      # row_start: None has a meaning (paged_evict)
    else:
        a[which] = None
    with pytest.raises(ValueError):
        paged._cache(*a, CPU)


def test_evict_workspace_of_sizes_past_the_limit():
    """B * nk <= 2^24, as the call has it: beyond, the bytes passed 64 bits and came out as few."""
    assert swa.paged_evict_workspace_size(65535, 256, 16, 1 << 26, 1 << 30) == 65535 * 256 * (1 << 30) * 24
    for b, nk in ((65535, 257), (65535, 65535), (0, 1)):
        with pytest.raises(swa.SwaError):
            swa.paged_evict_workspace_size(b, nk, 16, 1 << 26, 1 << 30)
