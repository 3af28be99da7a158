"""The page calls with their counts in place, beside other work on the GPU."""
import numpy as np
import pytest
import torch

import sliding_window_gqa_prep_gb300 as swa

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test collected on a machine without a GPU")
    yield


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def batch(B, width, num_pages, seed):
    """Ragged tables of pages of 16 slots, some shared, and pools of two page sizes."""
    rng = np.random.default_rng(seed)
    order, lens, table, refs = rng.permutation(num_pages).tolist(), [], [], [0] * num_pages
    for b in range(B):
        n = int(rng.integers(1, (width - 1) * 16))
        row = [table[-1][0]] if b % 3 else []
        row += [order.pop() for _ in range(-(-n // 16) - len(row))]
        lens.append(n)
        table.append(row + [-1] * (width - len(row)))
        for p in row:
            refs[p] += 1
    pools = [torch.randint(0, 1 << 30, (num_pages, k), dtype=torch.int32, device="cuda") for k in (64, 5000)]
    return pools, i32(table), i32(lens), i32(refs), i32(rng.integers(-1, B, 2 * B)), i32(rng.integers(0, 30, 2 * B))


def test_counts_in_place_beside_other_streams():
    """Two streams whose calls overlap, and a third that keeps the SMs busy: every call gives what it gives alone with counts
    apart."""
    torch.cuda.synchronize()
    states, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        pools, table, lens, refs, parent, room = batch(40, 12, 3000, 70 + i)
        alone = swa.paged_fork(pools, table, lens, refs, parent, 16, room=room)
        packed = swa.paged_compact([], table, refs)
        states.append((pools, table, lens, refs, parent, room, alone, packed, [x.clone() for x in pools]))
    busy, a = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    got = [[], []]
    for it in range(30):
        with torch.cuda.stream(busy):
            a @ a
        for i, s in enumerate(streams):
            pools, table, lens, refs, parent, room, *_ = states[i]
            with torch.cuda.stream(s):
                mine = refs.clone()
                f = swa.paged_fork(pools, table, lens, mine, parent, 16, room=room, refs_out=mine)
                again, where = refs.clone(), table.clone()
                c = swa.paged_compact([torch.empty_like(pools[0])], where, again, table_out=where, refs_out=again)
                got[i].append((f, c))
    torch.cuda.synchronize()
    for (pools, *_, alone, packed, after), calls in zip(states, got):
        assert all(torch.equal(x, y) for x, y in zip(pools, after))
        for f, c in calls:
            assert all(torch.equal(x, y) for x, y in zip(f, alone))
            assert all(torch.equal(x, y) for x, y in zip(c, packed))
