"""What the softmax weights of paged_attend lose in the cache's type, against float64.

The scores are made exact, so that nothing else hides it: q is 1 in one feature and 0 elsewhere,
so <q, k> is one feature of k. With the score s (in log2 units at most 2^-23 |s| off: two f32
roundings), the subtraction of the maximum (2^-24 of at most max|s|) and the 2^x (2^-21), a weight
is off by e = 2^-22 max|s| + 2^-20 relative before it is rounded, in numerator and sum. Sums of n
terms in f32 add n 2^-24. With r for what the type takes from a weight:
  |out - ref| <= (r + 2 e + n 2^-24) mean|v| + 2^-24 |ref|        (f32 output)
"""
import numpy as np
import pytest
import torch

import sliding_window_gqa_prep_gb300 as swa

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test collected on a machine without a GPU")
    yield


def scored(scores, rows, hpg, hd, dtype, v, page=64, max_pages=None):
    """One KV head whose key j has the score scores[j] (of the cache's type) against every query
    vector: (out in f32, the scores and values as the cache holds them)."""
    n = len(scores)
    need = -(-n // page)
    g = torch.Generator().manual_seed(7)
    order = torch.randperm(need, generator=g)
    k = torch.full((need, 1, page, hd), float("nan"))
    vv = torch.full((need, 1, page, hd), float("nan"))
    for i in range(need):
        m = min(page, n - i * page)
        k[order[i], 0, :m] = 0.0
        k[order[i], 0, :m, 3] = scores[i * page:i * page + m]
        vv[order[i], 0, :m] = v[i * page:i * page + m]
    k, vv = k.to(dtype).cuda(), vv.to(dtype).cuda()
    table = torch.zeros(1, max_pages or need, dtype=torch.int32)
    table[0, :need] = order.to(torch.int32)
    q = torch.zeros(rows, hpg, hd, dtype=dtype)
    q[..., 3] = 1.0
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    err = i32([0])
    out = swa.paged_attend(q.cuda(), k, vv, table.cuda(), i32([0, rows]), i32([n]), 1.0, max_rows=rows,
                           out=torch.empty(rows, hpg, hd, device="cuda"), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out.double().cpu().numpy(), scores.to(dtype).double().numpy(), v.to(dtype).double().numpy()


def reference(s, v, lim):
    p = np.exp(s[:lim] - s[:lim].max())
    return p @ v[:lim] / p.sum(), p @ np.abs(v[:lim]) / p.sum()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hd", [64, 128, 256])
# whole items, split and joined ones; one vector and a full block of 16; several rows
@pytest.mark.parametrize("n,rows,hpg", [(40, 1, 1), (64, 1, 16), (300, 4, 4), (1500, 1, 8)])
def test_weights_of_few_vectors_are_not_rounded_once(n, rows, hpg, hd, dtype):
    g = torch.Generator().manual_seed(n + hd)
    scores, v = torch.randn(n, generator=g), torch.randn(n, hd, generator=g)
    out, s, v = scored(scores, rows, hpg, hd, dtype, v)
    u = torch.finfo(dtype).eps / 2
    e = 2.0 ** -22 * np.abs(s).max() + 2.0 ** -20
    for i in range(rows):
        ref, absv = reference(s, v, n - rows + i + 1)
        # the rounding and its rest: u^2; in f16 the rest has no bits below 2^-25 of a weight of 2^15
        r = u * u
        floor = n * 2.0 ** -40 * np.abs(v).max() if dtype == HF else 0.0
        tol = (r + 2 * e + n * 2.0 ** -24) * absv + 2.0 ** -24 * np.abs(ref) + floor
        for h in range(hpg):
            assert (np.abs(out[i, h] - ref) <= tol).all(), np.abs(out[i, h] - ref).max()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("n,rows,hpg", [(300, 20, 1), (700, 8, 4), (900, 50, 2)])   # 20, 32 and 100 vectors
def test_weights_of_many_vectors_are_rounded_once(n, rows, hpg, hd, dtype):
    g = torch.Generator().manual_seed(n + hd)
    scores, v = torch.randn(n, generator=g), torch.randn(n, hd, generator=g)
    out, s, v = scored(scores, rows, hpg, hd, dtype, v)
    e = 2.0 ** -22 * np.abs(s).max() + 2.0 ** -20
    for i in range(rows):
        ref, absv = reference(s, v, n - rows + i + 1)
        # f16 has no bits below 2^-25, of a largest weight of 2^11 or 2^15
        floor = n * 2.0 ** -36 * np.abs(v).max() if dtype == HF else 0.0
        tol = (torch.finfo(dtype).eps / 2 + 2 * e + n * 2.0 ** -24) * absv + 2.0 ** -24 * np.abs(ref) + floor
        for h in range(hpg):
            assert (np.abs(out[i, h] - ref) <= tol).all(), np.abs(out[i, h] - ref).max()


# log2 e * 1419 / 512 = 3.9984 and * 1420 / 512 = 4.0012: the tensor-core kernel's f16 form raises
# its running maximum for a tile whose maximum is 2^4 times the last one or more
@pytest.mark.parametrize("peaks", [
    {3: 0.0}, {5000: 0.0}, {3: -1419 / 512, 5000: 0.0}, {3: -1420 / 512, 5000: 0.0},
    {3: -8.0, 700: -1420 / 512, 5000: 0.0}, {3: 0.0, 5000: -1420 / 512},
])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("rows,wide", [(1, None), (40, None), (150, None), (150, 2048)])
def test_f16_small_weights_count(rows, wide, hd, peaks):
    """8192 keys, nearly all at 3e-7 of the largest weight: a quarter of a percent together, which
    must not vanish from the product where it counts in the sum."""
    n = 8192
    scores, v = torch.full((n,), -15.0), torch.ones(n, hd)
    for j, x in peaks.items():
        scores[j], v[j] = x, -1.0
    out, s, v = scored(scores, rows, 1, hd, HF, v, max_pages=wide)
    e = 2.0 ** -22 * np.abs(s).max() + 2.0 ** -20
    for i in (0, rows // 2, rows - 1):
        ref, absv = reference(s, v, n - rows + i + 1)
        tol = (2.0 ** -11 + 2 * e + n * 2.0 ** -24) * absv + 2.0 ** -24 * np.abs(ref) + n * 2.0 ** -36
        assert (np.abs(out[i, 0] - ref) <= tol).all(), np.abs(out[i, 0] - ref).max()
        # the peaks alone would give -1
        assert (ref > -1 + 4e-3).all()
