"""A key that is NaN (a 4-bit block that held an infinity or NaN, or a NaN in a 16-bit pool) makes the rows that
see it NaN, and no others: in every kernel, wherever the keys are cut."""
import pytest
import torch

import sliding_window_gqa_prep_gb300 as swa
from paged4_f64 import Cache, U8

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test collected on a machine without a GPU")
    yield


# one CTA an item; items that are cut; the tensor-core kernel with one share of the keys and with several
CASES = [dict(t=[1], lens=[300], nh=4, nk=2, wide=0), dict(t=[2, 1], lens=[700, 300], nh=8, nk=2, wide=40), dict(t=[1], lens=[9000], nh=4, nk=1, wide=0),
         dict(t=[70], lens=[400], nh=4, nk=1, wide=0), dict(t=[40], lens=[3624], nh=8, nk=1, wide=0), dict(t=[130, 1], lens=[4000, 4000], nh=4, nk=2, wide=0)]


def batches(kw, hd, seed=3):
    """(name, q, K pool and the NaN that a key's first features become, call) of both caches."""
    nh, nk = kw["nh"], kw["nk"]
    bt = Cache(kw["t"], kw["lens"], nk, hd, 64, seed=seed, wide=kw["wide"])
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(bt.T, nh, hd, generator=g, device="cuda").to(torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = lambda: (torch.empty(bt.T, nh, hd, device="cuda"), torch.empty(bt.T, nh, device="cuda"))   # noqa: E731

    def in4():
        out, lse = new()
        swa.paged4_attend(q, *bt.args, hd ** -0.5, max_rows=max(kw["t"]), out=out, lse=lse, err=err)
        return out, lse
    yield bt, bt.pools[1].view(U8), 127, in4
    k16, v16 = (torch.randn(bt.pools[0].shape[0], nk, 64, hd, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))

    def in16():
        out, lse = new()
        swa.paged_attend(q, k16, v16, *bt.args[4:], hd ** -0.5, max_rows=max(kw["t"]), out=out, lse=lse, err=err)
        return out, lse
    yield bt, k16, float("nan"), in16


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("kw", CASES)
def test_nan_keys_reach_the_rows_that_see_them(kw, hd):
    for bt, pool, nan, call in batches(kw, hd):
        n, t = bt.n[0], bt.t[0]
        fine = call()
        assert fine[0].isfinite().all() and fine[1].isfinite().all()
        # every key of a stretch: the rows' last keys, one alone, and from the start of each tile on, so that some share of
        # the keys has nothing else
        for lo, hi in [(n - t, n - t + 1), (n - t + t // 2, n), (5, n // 3), (0, 1)] + [(x, n) for x in range(64, n, 64)]:
            keep = pool.clone()
            j = torch.arange(lo, hi, device="cuda")
            pool[bt.table[0].long()[j // bt.page], :, j % bt.page, 0] = nan
            out, lse = call()
            pool.copy_(keep)
            sees = torch.tensor([n - t + i >= lo for i in range(t)], device="cuda")
            assert out[:t][sees].isnan().all() and lse[:t][sees].isnan().all(), (lo, hi, out[:t][sees].isnan().float().mean())
            # vectors that share a warp's running maxima may be scaled elsewhere: two roundings of weights to bf16
            assert ((out - fine[0])[:t][~sees].abs() <= 2.0 ** -7 * 6.0).all() and ((lse - fine[1])[:t][~sees].abs() <= 2.0 ** -7).all(), (lo, hi)
            assert torch.equal(out[t:], fine[0][t:]) and torch.equal(lse[t:], fine[1][t:])
