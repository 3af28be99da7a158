"""The 4-bit paged cache at the sizes where its calls choose other code than for small batches: shares that
count items' starts, more sequences than threads, more heads than a block takes. Against float64
(paged4_f64.py); tolerances are those of test_gpu_paged4.py."""
import numpy as np
import pytest
import torch

import sliding_window_gqa_prep_gb300 as swa
from paged4_f64 import Cache

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test collected on a machine without a GPU")
    yield


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def zero():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def tiny(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def attend_and_check(bt, nh, dtype, window=0, sinks=0, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(bt.T, nh, bt.hd, generator=g, device="cuda").to(dtype)
    scale = bt.hd ** -0.5 * 0.5 * 2.0 ** -bt.exps[0]
    out = torch.full((bt.T, nh, bt.hd), 5.0, device="cuda")
    lse, err = torch.full((bt.T, nh), 77.0, device="cuda"), zero()
    swa.paged4_attend(q, *bt.args, scale, max_rows=max(bt.t), window=window, sinks=sinks, out=out, lse=lse, err=err, **bt.exp)
    assert int(err.item()) == 0
    ro, rl, av, sa = bt.attend(q, scale, window, sinks)
    live = bt.live
    n = torch.zeros(live, 1, 1, dtype=torch.float64, device="cuda")
    for b, x in enumerate(bt.n):
        n[bt.start[b]:bt.start[b + 1]] = max(x, 1)
    d = bt.hd * 2.0 ** -24 * sa[:live, :, None]
    vmax = 6.0 * 2.0 ** bt.exps[1]
    tol = ((2.0 ** -11 + 2 * (d + 2.0 ** -19) + n * 2.0 ** -24) * av[:live] + n * 2.0 ** -36 * vmax + 2.0 ** -24 * ro[:live].abs()
           + tiny(FP))
    off = (out[:live].double() - ro[:live]).abs()
    assert (off <= tol).all(), ((off / tol).max().item(), (~(off <= tol)).nonzero()[:4].tolist())
    none = rl[:live].isneginf()
    assert torch.equal(lse[:live].isneginf(), none)
    tl = d[..., 0] + 2.0 ** -19 + n[..., 0] * 2.0 ** -24 + 2.0 ** -22 * rl[:live].abs()
    assert ((lse[:live].double() - rl[:live]).abs() <= tl)[~none].all()
    assert (out[live:] == 5.0).all() and (lse[live:] == 77.0).all()


# (hd, query heads a KV head, rows): one to four tiles of 8 vectors, and four CTAs an SM at most
@pytest.mark.parametrize("hd,hpg,rows", [(64, 1, 1), (64, 4, 3), (64, 16, 2), (128, 4, 1), (128, 3, 4), (128, 8, 4), (256, 1, 1), (256, 4, 4)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_attend_where_shares_count_starts(hd, hpg, rows, dtype):
    """Eight tiles a CTA and more: shares count what an item's start costs, and are cut inside starts too."""
    nk, kt = 4, 64 if hd == 256 else 128
    rng = np.random.default_rng(hd + hpg)
    t, lens, tiles = [], [], 0
    while tiles * nk < 4 * 8 * sms() + 100:                  # kWeighed tiles for each CTA of at most four an SM
        r = int(rng.integers(0, rows + 1)) if rng.random() < 0.7 else rows
        n = int(rng.integers(1, 40)) if rng.random() < 0.2 else int(rng.integers(1, 6000))
        n = max(n, r)
        t.append(r)
        lens.append(n)
        tiles += -(-n // kt) if r else 0
    t[0] = rows
    lens[0] = max(lens[0], rows)
    bt = Cache(t, lens, nk, hd, 64, seed=21, pad=2, exps=(1, -2))
    attend_and_check(bt, nk * hpg, dtype)


@pytest.mark.parametrize("hd,hpg,rows,window", [(128, 2, 1, 0), (256, 4, 4, 3000), (64, 8, 4, 2500)])
def test_attend_of_one_and_two_long_sequences(hd, hpg, rows, window):
    """Items of hundreds of shares, and a window and sinks over them."""
    kt = 64 if hd == 256 else 128
    n = (4 * 8 * sms() // 2 + 77) * kt
    bt = Cache([rows, 1], [n, n // 5], 2, hd, 256, seed=22, exps=(0, 0))
    attend_and_check(bt, 2 * hpg, BF)
    if window:
        attend_and_check(bt, 2 * hpg, HF, window=window, sinks=5)


@pytest.mark.parametrize("hd,wide,most", [(64, 80, 300), (128, 80, 1280), (256, 80, 1280)])
def test_attend_of_more_sequences_than_threads(hd, wide, most):
    """400 sequences in the form that cuts items: several sequences a thread of the scan, some without rows."""
    rng = np.random.default_rng(hd)
    t = [int(x) for x in rng.choice([0, 1, 1, 2], 400)]
    t[-1] = 1
    lens = [max(a, int(x)) for a, x in zip(t, rng.integers(0, most, 400))]
    attend_and_check(Cache(t, lens, 2, hd, 16, seed=23, wide=wide, pad=1), 6, BF)


# ------------------------------------------------------------------ read
@pytest.mark.parametrize("nk,page,t", [(300, 16, 40), (513, 32, 3), (256, 16, 700)])
@pytest.mark.parametrize("dtype", [FP, BF])
def test_read_of_many_heads(nk, page, t, dtype):
    """More KV heads than a block takes."""
    bt = Cache([t, 2], [t + 5, 2], nk, 64, page, seed=32, pad=1, exps=(1, -1))
    out = [torch.full((bt.T, nk, 64), 5.0, dtype=dtype, device="cuda") for _ in range(2)]
    err = zero()
    swa.paged4_read(*bt.args, k_out=out[0], v_out=out[1], err=err, **bt.exp)
    assert int(err.item()) == 0
    for b in range(2):
        for got, ref in zip(out, bt.keys(b)):
            assert torch.equal(got[bt.start[b]:bt.start[b + 1]].double(), ref[bt.n[b] - bt.t[b]:])
    assert (out[0][bt.live:] == 5.0).all() and (out[1][bt.live:] == 5.0).all()
