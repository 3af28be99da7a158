"""What the softmax weights of paged4_attend lose in f16, against float64.

The scores are exact, so that nothing else hides it: q is 1 in one feature and 0 elsewhere, so <q, k> is
one feature of k, which the cache holds exactly and q's power of two does not change. As in
test_gpu_paged_weights.py a weight is off by e = 2^-22 max|s| + 2^-20 relative before it is rounded, in
numerator and sum; sums of n terms in f32 add n 2^-24. With r for what f16 takes from a weight, and bits below
2^-25 of one whose largest is 2^11 or more (2^-36 of the row's):
  |out - ref| <= (r + 2 e + n 2^-24) mean|v| + n 2^-36 max|v| + 2^-24 |ref|        (f32 output)
r is 2^-11 for a weight that is rounded once, 2^-22 for one whose rest is kept.
"""
import numpy as np
import pytest
import torch

import sliding_window_gqa_prep_gb300 as swa
from paged4_f64 import E4, U8, decode

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test collected on a machine without a GPU")
    yield


def scored(n, rows, hpg, hd, dtype, seed, page=64, wide=0):
    """One KV head of n keys that are 0 but in feature 3, and a q that reads it: (out in f32, the keys'
    scores, the values)."""
    g = torch.Generator().manual_seed(seed)
    need = max(-(-n // page), wide)
    order = torch.randperm(need, generator=g)
    k, v = (torch.zeros(need, 1, page, hd // 2, dtype=U8) for _ in range(2))
    ks, vs = (torch.full((need, 1, page, hd // 16), 127, dtype=U8) for _ in range(2))
    j = torch.arange(n)
    at = order[j // page], 0, j % page
    k[at[0], at[1], at[2], 1] = (torch.randint(0, 16, (n,), generator=g) << 4).to(U8)      # feature 3: an upper half
    ks[at] = torch.randint(40, 57, (n, hd // 16), generator=g, dtype=torch.int32).to(U8)   # 1/4 .. 1: scores within 6
    v[at] = torch.randint(0, 256, (n, hd // 2), generator=g, dtype=torch.int32).to(U8)
    vs[at] = torch.randint(40, 57, (n, hd // 16), generator=g, dtype=torch.int32).to(U8)
    s, vv = decode(k[at], ks[at], 0)[:, 3].numpy(), decode(v[at], vs[at], 0).numpy()
    q = torch.zeros(rows, hpg, hd, dtype=dtype)
    q[..., 3] = 1.0
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    err = i32([0])
    out = swa.paged4_attend(q.cuda(), k.cuda(), ks.cuda().view(E4), v.cuda(), vs.cuda().view(E4), i32([order.tolist()]),
                            i32([0, rows]), i32([n]), 1.0, max_rows=rows, out=torch.empty(rows, hpg, hd, device="cuda"), err=err)
    assert int(err.item()) == 0
    return out.double().cpu().numpy(), s, vv


def check(out, s, v, r):
    n, rows = len(s), out.shape[0]
    e = 2.0 ** -22 * np.abs(s).max() + 2.0 ** -20
    for i in range(rows):
        lim = n - rows + i + 1
        p = np.exp(s[:lim] - s[:lim].max())
        ref, absv = p @ v[:lim] / p.sum(), p @ np.abs(v[:lim]) / p.sum()
        tol = (r + 2 * e + n * 2.0 ** -24) * absv + n * 2.0 ** -36 * np.abs(v).max() + 2.0 ** -24 * np.abs(ref)
        assert (np.abs(out[i] - ref) <= tol).all(), (np.abs(out[i] - ref) / tol).max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hd", [64, 128, 256])
# whole items, split and joined ones; one vector, a full tile of 8 and two; several rows
@pytest.mark.parametrize("n,rows,hpg,wide", [(40, 1, 1, 0), (64, 1, 8, 0), (64, 1, 16, 0), (48, 4, 4, 0), (40, 1, 8, 64), (100, 2, 6, 64), (1500, 1, 8, 0),
                                              (50, 2, 2, 0), (60, 1, 4, 64), (45, 4, 1, 64)])
def test_weights_of_few_vectors_are_not_rounded_once(n, rows, hpg, wide, hd, dtype):
    check(*scored(n, rows, hpg, hd, dtype, n + hd, wide=wide), 2.0 ** -22)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("n,rows,hpg", [(60, 20, 1), (64, 8, 4), (300, 20, 1), (900, 50, 2)])     # 20, 32 and 100 vectors
def test_weights_of_many_vectors_are_rounded_once(n, rows, hpg, hd, dtype):
    check(*scored(n, rows, hpg, hd, dtype, n + hd), 2.0 ** -11)
