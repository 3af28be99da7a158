"""The 4-bit paged cache and the calls that share pages against the float64 oracle
(oracle/paged4_oracle.py).

Tolerances (u: half a step of the type, eps / 2):
  codes, scales, tables, counts, copies: exact. (What append stores is defined by the exact
           rotated key; the oracle's own angles are off by some 2^-53 pos, so that inputs at a border of
           the encoding, which are those that do not turn, are the only ones where that could matter.)
  read     exact in f32 and bf16; one rounding in f16
  q of append  8 * 2^-24 + 2^-21 of |u| + |v| and one rounding, as swa_rotary's
  attend   a weight enters the value product in f16: 2^-11 relative, and at most 2^-36 of the
           row's scale where it is small; keys and values are exact; a score is a sum of hd
           products in f32: off by at most hd * 2^-24 * sum |q_i k_i| scale =: d; q itself loses at
           most 2^-39 of its largest value in each feature (part of d's hd * 2^-24 for the sizes
           here); scaling, subtraction and 2^x 2^-19; in numerator and sum:
           |out - ref| <= (2^-11 + 2 (d + 2^-19) + n 2^-24) mean|v| + n 2^-36 max|v| + u |ref|.
  lse      d + 2^-19 + n 2^-24 + 2^-22 |lse|
"""
import numpy as np
import pytest
import torch

from oracle import paged4_oracle as p4, paged_oracle as po
from sliding_window_gqa_prep_gb300 import _abi
import sliding_window_gqa_prep_gb300 as swa

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
U8, E4 = torch.uint8, torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test collected on a machine without a GPU")
    yield


def f64(x):
    return x.detach().double().cpu().numpy()


def bits(x):
    return x.detach().view(U8).cpu().numpy()


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def zero():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


class Batch4:
    """A ragged chunk over a 4-bit paged cache: random codes, scales around 1; slots that no
    sequence holds have scale NaN."""

    def __init__(self, t, lens, nh, nk, hd, page, dtype=BF, seed=0, pad=0, spare=2, sharp=1.0, exps=(0, 0), window=0, sinks=0):
        g = torch.Generator().manual_seed(seed)
        self.t, self.n, self.nh, self.nk, self.hd, self.page, self.dtype = t, lens, nh, nk, hd, page, dtype
        self.exp = {"exp_k": exps[0], "exp_v": exps[1]}
        self.mask = {"window": window, "sinks": sinks}
        B = len(t)
        need = [max(1, -(-x // page)) for x in lens]
        self.max_pages = max(need)
        pool = sum(need) + spare
        order = torch.randperm(pool, generator=g)
        self.table = torch.full((B, self.max_pages), -7, dtype=torch.int32)
        codes = lambda: torch.randint(0, 256, (pool, nk, page, hd // 2), generator=g, dtype=torch.int32).to(U8)
        self.k, self.v = codes().cuda(), codes().cuda()
        ks, vs = (torch.full((pool, nk, page, hd // 16), 127, dtype=U8) for _ in range(2))
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]].to(torch.int32)
            at += need[b]
            first = lens[b] - t[b]                       # the first row's slot
            for j in range(lens[b]):
                if window and sinks <= j <= first - window:
                    continue                             # no row sees it
                p = int(self.table[b, j // page])
                for s in (ks, vs):                       # 2^-3 .. 1, all mantissas
                    s[p, :, j % page] = torch.randint(32, 57, (nk, hd // 16), generator=g, dtype=torch.int32).to(U8)
        self.ks, self.vs = ks.cuda().view(E4), vs.cuda().view(E4)
        self.start = [0]
        for x in t:
            self.start.append(self.start[-1] + x)
        self.T = self.start[-1] + pad
        self.q = (torch.randn(self.T, nh, hd, generator=g) * sharp).to(dtype).cuda()
        self.scale = hd ** -0.5 * 0.5 * 2.0 ** -exps[0]
        self.cap = self.max_pages * page
        self.pools = (self.k, self.ks, self.v, self.vs)
        self.args = (*self.pools, self.table.cuda(), dev(self.start), dev(lens))

    def values(self):
        with np.errstate(invalid="ignore"):
            k = p4.decode(bits(self.k), bits(self.ks), self.exp["exp_k"])
            v = p4.decode(bits(self.v), bits(self.vs), self.exp["exp_v"])
        return k, v

    def oracle(self):
        k, v = self.values()
        return p4.attend(f64(self.q), k, v, self.table.numpy(), self.start, self.n, self.scale, **self.mask)

    def attend(self, **kw):
        kw.setdefault("max_rows", max(max(self.t), 1))
        err = zero()
        lse = torch.full((self.T, self.nh), 77.0, device="cuda")
        out = kw.pop("out", None)
        if out is None:
            out = torch.full((self.T, self.nh, self.hd), 5.0, dtype=self.dtype, device="cuda")
        args = kw.pop("args", self.args)
        swa.paged4_attend(kw.pop("q", self.q), *args, self.scale, out=out, lse=lse, err=err, **self.exp, **self.mask, **kw)
        torch.cuda.synchronize()
        return out, lse, int(err.item())

    def check(self, out, lse, ref=None):
        ro, rl, av, sa = ref if ref is not None else self.oracle()
        live = self.start[-1]
        n = max(max(self.n), 1)
        d = self.hd * 2.0 ** -24 * sa[:live, :, None]
        o, ro, av = f64(out)[:live], ro[:live], av[:live]
        vmax = float(np.nan_to_num(np.abs(self.values()[1])).max())
        tol = ((2.0 ** -11 + 2 * (d + 2.0 ** -19) + n * 2.0 ** -24) * av + n * 2.0 ** -36 * vmax + unit(out.dtype) * np.abs(ro)
               + tiny(out.dtype))
        bad = ~(np.abs(o - ro) <= tol)
        assert not bad.any(), (int(bad.sum()), np.abs(o - ro).max(), np.argwhere(bad)[:4])
        g, rl = f64(lse)[:live], rl[:live]
        empty = np.isneginf(rl)
        assert (np.isneginf(g) == empty).all()
        tl = d[..., 0] + 2.0 ** -19 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(empty, 0, rl))
        assert (np.abs(np.where(empty, 0, g) - np.where(empty, 0, rl)) <= tl).all()
        # rows of no sequence are left as they were
        assert (out[live:] == 5.0).all() and (lse[live:] == 77.0).all()


# ------------------------------------------------------------------ append and read
APPEND = [
    dict(t=[1], lens=[1], nh=2, nk=1, hd=64, page=16, rot=64),
    dict(t=[1, 1, 1], lens=[17, 16, 300], nh=8, nk=2, hd=128, page=16, rot=128),
    dict(t=[5, 0, 33, 1], lens=[5, 9, 100, 64], nh=6, nk=3, hd=64, page=32, rot=32, pad=3),
    dict(t=[30, 7], lens=[131, 500], nh=4, nk=4, hd=256, page=128, rot=20),
    dict(t=[3, 2], lens=[40, 2], nh=4, nk=1, hd=128, page=64, rot=0),
    dict(t=[6], lens=[70], nh=3, nk=3, hd=256, page=256, rot=254),
    dict(t=[9], lens=[70], nh=2, nk=2, hd=128, page=16, rot=70),
]


def projection(bt, src, seed, pad=8):
    """q, k, v as rows inside a wider packed projection."""
    g = torch.Generator().manual_seed(seed)
    nh, nk, hd, T = bt.nh, bt.nk, bt.hd, bt.T
    proj = torch.randn(T, (nh + 2 * nk) * hd + pad, generator=g)
    proj *= torch.exp2(torch.randint(-12, 5, (T, 1), generator=g).float())      # rows of all sizes
    proj[torch.rand(proj.shape, generator=g) < 0.05] = 0
    proj = proj.to(src).cuda()
    return (proj[:, :nh * hd].unflatten(1, (nh, hd)), proj[:, nh * hd:(nh + nk) * hd].unflatten(1, (nk, hd)),
            proj[:, (nh + nk) * hd:(nh + 2 * nk) * hd].unflatten(1, (nk, hd)))


def stored(bt, before, k, v):
    """The pools after rows k, v (f64 values) entered, by the oracle."""
    want = [bits(x).copy() for x in before]
    for b in range(len(bt.t)):
        for i in range(bt.t[b]):
            r, slot = bt.start[b] + i, bt.n[b] - bt.t[b] + i
            p = int(bt.table[b, slot // bt.page])
            for at, x, e in ((0, k, "exp_k"), (2, v, "exp_v")):
                c, s = p4.encode(x[r], bt.exp[e])
                want[at][p, :, slot % bt.page], want[at + 1][p, :, slot % bt.page] = c, s
    return want


@pytest.mark.parametrize("src,dtype", [(BF, BF), (HF, HF), (FP, BF), (FP, HF), (BF, HF)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("kw", APPEND)
def test_append(kw, inter, src, dtype):
    kw = dict(kw)
    rot = kw.pop("rot")
    bt = Batch4(seed=5, exps=(1, -4), **kw)
    q, k, v = projection(bt, src, 6)
    g = torch.Generator().manual_seed(7)
    pos = torch.randint(0, 100000, (bt.T,), generator=g, dtype=torch.int32)
    pos[0] = 0
    turns, freqs = (swa.rotary_turns(rot), swa.rotary_freqs(rot).numpy()) if rot else (None, [])
    before = [x.clone() for x in bt.pools]
    q_out = torch.full((bt.T, bt.nh, bt.hd), 5.0, dtype=dtype, device="cuda")
    err = zero()
    swa.paged4_append(k, v, pos.cuda(), *bt.args, q=q, q_out=q_out, turns=turns, interleaved=inter, mag=1.25 if rot == 70 else 1.0,
                      err=err, **bt.exp)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    mag = 1.25 if rot == 70 else 1.0
    turn = lambda x: po.rotary(f64(x), pos.numpy(), freqs, inter, False, mag)
    want = stored(bt, before, turn(k), f64(v))
    for name, got, ref in zip(("k", "k scale", "v", "v scale"), bt.pools, want):
        assert (bits(got) == ref).all(), (name, np.argwhere(bits(got) != ref)[:4])
    live, rq, a = bt.start[-1], turn(q), np.abs(f64(q))
    other, h = a.copy(), rot // 2
    if inter:
        other[..., 0:rot:2], other[..., 1:rot:2] = a[..., 1:rot:2], a[..., 0:rot:2]
    else:
        other[..., :h], other[..., h:rot] = a[..., h:rot], a[..., :h]
    tol = (8 * 2.0 ** -24 + 2.0 ** -21) * mag * (a + other) + unit(dtype) * np.abs(rq) + tiny(dtype)
    assert (np.abs(f64(q_out) - rq)[:live] <= tol[:live]).all() and (q_out[live:] == 5.0).all()


def test_append_at_the_borders():
    """Values on the borders between two codes and blocks on those between two scales, of every type
    that holds them; and one step of the type to either side."""
    for src, exp in ((FP, 0), (BF, -3), (HF, 2), (FP, 20), (FP, -32)):
        eps = torch.finfo(src).eps
        blocks = []
        for s in range(1, 127):
            u = p4.E4M3[s] * 2.0 ** exp
            for f in (1.0, 1.0 + eps, 1.0 - eps / 2):
                blocks.append([x * u * f for x in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)] + [6 * u] + [-x * u * f for x in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.0)])
                mid = 3 * (p4.E4M3[s] + p4.E4M3[s - 1]) * 2.0 ** exp        # 6 times the middle of two scales
                blocks.append([mid * f] + [mid / 7] * 15)
        blocks += [[0.0] * 16, [1e-30] * 16, [3000.0 * 2.0 ** min(exp, 3)] * 16, [6 * 2.0 ** (exp - 10)] * 16, [6.1 * 2.0 ** (exp - 10)] * 16]
        while len(blocks) % 4:
            blocks.append([0.0] * 16)
        x = torch.tensor(blocks, dtype=torch.float64).to(src).view(-1, 1, 64)
        n = x.shape[0]
        bt = Batch4(t=[n], lens=[n], nh=1, nk=1, hd=64, page=16, seed=8, exps=(exp, exp))
        before = [y.clone() for y in bt.pools]
        swa.paged4_append(x.cuda(), x.cuda(), None, *bt.args, **bt.exp)
        want = stored(bt, before, f64(x), f64(x))
        for got, ref in zip(bt.pools, want):
            assert (bits(got) == ref).all(), (src, exp, np.argwhere(bits(got) != ref)[:4])


def test_append_rotated_next_to_borders():
    """Keys whose rotation lands next to a border: found by turning border values back in f64, so
    that f32 angles would settle many of them wrongly."""
    rot, hd, T = 64, 64, 128
    g = torch.Generator().manual_seed(9)
    pos = torch.randint(1, 500, (T,), generator=g, dtype=torch.int32)
    freqs = swa.rotary_freqs(rot).numpy()
    want = np.random.default_rng(3).choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], (T, 1, hd)) * 0.8125
    want[..., ::16] = 6 * 0.8125
    back = po.rotary(want, pos.numpy(), freqs, False, True)
    k = torch.tensor(back).float()
    bt = Batch4(t=[T], lens=[T], nh=1, nk=1, hd=hd, page=64, seed=9)
    before = [x.clone() for x in bt.pools]
    swa.paged4_append(k.cuda(), k.cuda(), pos.cuda(), *bt.args, turns=swa.rotary_turns(rot))
    ref = stored(bt, before, po.rotary(f64(k), pos.numpy(), freqs), f64(k))
    for got, r in zip(bt.pools, ref):
        assert (bits(got) == r).all(), np.argwhere(bits(got) != r)[:4]


def test_append_of_infinities_and_nan():
    x = torch.randn(3, 2, 64, generator=torch.Generator().manual_seed(1))
    x[0, 0, 3], x[1, 1, 20], x[2, 0, 63] = float("inf"), float("nan"), float("-inf")
    bt = Batch4(t=[3], lens=[3], nh=2, nk=2, hd=64, page=16)
    before = [y.clone() for y in bt.pools]
    swa.paged4_append(x.cuda(), x.cuda(), None, *bt.args)
    for got, ref in zip(bt.pools, stored(bt, before, f64(x), f64(x))):
        assert (bits(got) == ref).all()
    k, v = swa.paged4_read(*bt.args, T=3)
    want = x.isfinite().unflatten(-1, (4, 16)).all(-1, keepdim=True).expand(3, 2, 4, 16).flatten(-2)
    assert torch.equal(k.isfinite().cpu(), want) and torch.equal(v.isnan().cpu(), ~want)


def test_append_reports_and_skips():
    """A chunk longer than its length, a bad page and rows out of range: reported, nothing
    else written; read gives zeros there and leaves rows of no sequence."""
    bt = Batch4(t=[4, 2, 3], lens=[40, 20, 17], nh=2, nk=1, hd=64, page=16, seed=7)
    x = torch.randn(9, 1, 64, generator=torch.Generator().manual_seed(8)).to(BF).cuda()
    err = zero()
    before = [y.clone() for y in bt.pools]
    table = bt.args[4].clone()
    table[1, 1] = 1 << 30                                    # slots 18, 19 of sequence 1
    where = (table, dev([0, 4, 6, 50]), dev([2, 20, 17]))    # the last sequence reaches past T
    swa.paged4_append(x, x, None, *bt.pools, *where, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == _abi.SWA_DERR_META | _abi.SWA_DERR_PAGE | _abi.SWA_DERR_SEGMENT
    p = int(table[0, 0])
    want = [bits(y).copy() for y in before]
    for i in (2, 3):                                         # rows 2, 3 of sequence 0 have slots 0, 1
        for at in (0, 2):
            c, s = p4.encode(f64(x[i]), 0)
            want[at][p, :, i - 2], want[at + 1][p, :, i - 2] = c, s
    for got, ref in zip(bt.pools, want):
        assert (bits(got) == ref).all()
    err, k = zero(), torch.full((9, 1, 64), 3.0, dtype=BF, device="cuda")
    swa.paged4_read(*bt.pools, *where, k_out=k, err=err)
    assert int(err.item()) == _abi.SWA_DERR_META | _abi.SWA_DERR_PAGE | _abi.SWA_DERR_SEGMENT
    assert not k[[0, 1, 4, 5]].any() and (k[6:] == 3.0).all() and k[2:4].abs().sum() > 0


@pytest.mark.parametrize("dtype", [FP, BF, HF])
@pytest.mark.parametrize("kw", [
    dict(t=[1], lens=[1], nh=1, nk=1, hd=64, page=16), dict(t=[5, 0, 33, 1], lens=[5, 9, 100, 64], nh=3, nk=3, hd=128, page=32, pad=3),
    dict(t=[200, 131], lens=[300, 131], nh=2, nk=2, hd=256, page=64), dict(t=[2000, 900], lens=[2000, 901], nh=1, nk=1, hd=64, page=128),
    dict(t=[3, 30000], lens=[70, 30000], nh=2, nk=1, hd=64, page=256)])
def test_read(kw, dtype):
    bt = Batch4(seed=12, exps=(3, -5), **kw)
    out = [torch.full((bt.T, bt.nk, bt.hd), 5.0, dtype=dtype, device="cuda") for _ in range(2)]
    err = zero()
    swa.paged4_read(*bt.args, k_out=out[0], v_out=out[1], err=err, **bt.exp)
    assert int(err.item()) == 0
    live = bt.start[-1]
    for x, got in zip(bt.values(), out):
        ref = np.concatenate([np.zeros((0, bt.nk, bt.hd))] + [
            np.stack([po.gather(x, bt.table.numpy(), b, g, bt.n[b])[bt.n[b] - bt.t[b]:] for g in range(bt.nk)], 1)
            for b in range(len(bt.t))])
        # scales are normal e4m3 here: f16 holds the values of exponents -5 and 3 too
        assert (f64(got)[:live] == ref).all() and (got[live:] == 5.0).all()
    one = torch.full_like(out[0], 5.0)
    assert swa.paged4_read(*bt.args, v_out=one, **bt.exp)[0] is None and torch.equal(one, out[1])


# ------------------------------------------------------------------ attend
ATTEND = [
    # one token: lengths of one, inside a page, page ends, many tiles
    dict(t=[1], lens=[1], nh=1, nk=1, hd=64, page=16),
    dict(t=[1], lens=[133], nh=8, nk=2, hd=64, page=16),
    dict(t=[1, 1, 1, 1], lens=[64, 65, 63, 1], nh=4, nk=4, hd=128, page=64),
    dict(t=[1, 1, 1], lens=[1000, 16, 4097], nh=16, nk=2, hd=128, page=32),
    dict(t=[1, 1], lens=[2050, 700], nh=8, nk=2, hd=256, page=128),
    dict(t=[1], lens=[300], nh=32, nk=1, hd=128, page=256),
    dict(t=[1, 1, 1], lens=[500, 129, 128], nh=9, nk=1, hd=64, page=16),
    # few rows, empty sequences, rows behind the last one, a length of zero with rows
    dict(t=[3, 0, 8], lens=[3, 50, 200], nh=12, nk=4, hd=64, page=16, pad=5),
    dict(t=[8, 8], lens=[8, 519], nh=32, nk=8, hd=128, page=64),
    dict(t=[2, 1], lens=[0, 5], nh=2, nk=1, hd=64, page=16),
    dict(t=[5], lens=[2], nh=4, nk=2, hd=128, page=16),              # its first three rows see nothing
    dict(t=[0, 0], lens=[5, 0], nh=2, nk=1, hd=64, page=16, pad=2),
    dict(t=[7, 1], lens=[100, 33], nh=5, nk=1, hd=256, page=16),
    # a window, with and without first slots that stay
    dict(t=[1, 1], lens=[700, 90], nh=8, nk=2, hd=128, page=16, window=100, sinks=4),
    dict(t=[1], lens=[2000], nh=4, nk=1, hd=64, page=64, window=1, sinks=0),
    dict(t=[1, 1], lens=[3000, 2], nh=4, nk=1, hd=256, page=32, window=1, sinks=1),
    dict(t=[4, 1, 0], lens=[1111, 64, 9], nh=6, nk=2, hd=128, page=256, window=257, sinks=130),
    dict(t=[6], lens=[900], nh=4, nk=2, hd=256, page=16, window=3, sinks=17),
    dict(t=[5], lens=[5], nh=4, nk=2, hd=64, page=16, window=2, sinks=1),
    dict(t=[3], lens=[400], nh=4, nk=4, hd=128, page=16, window=1000, sinks=4),
    dict(t=[2], lens=[400], nh=4, nk=4, hd=128, page=16, window=50, sinks=1000),
    # chunks: row blocks, causal diagonals across tiles, odd head groups
    dict(t=[130], lens=[130], nh=4, nk=1, hd=64, page=16),
    dict(t=[257, 64], lens=[300, 900], nh=8, nk=2, hd=128, page=64),
    dict(t=[100, 1, 33], lens=[612, 800, 33], nh=6, nk=2, hd=128, page=32, pad=1),
    dict(t=[40, 0, 90], lens=[1000, 10, 90], nh=5, nk=1, hd=64, page=128),
    dict(t=[70, 129], lens=[290, 129], nh=4, nk=2, hd=256, page=16),
    dict(t=[300], lens=[200], nh=2, nk=1, hd=128, page=16),          # 100 rows see nothing
    dict(t=[35], lens=[1111], nh=32, nk=1, hd=128, page=256),
    dict(t=[513, 3], lens=[2000, 3], nh=1, nk=1, hd=128, page=16),
    dict(t=[10, 10], lens=[10, 700], nh=8, nk=2, hd=128, page=32),
    dict(t=[9, 9, 9], lens=[9, 64, 1000], nh=4, nk=2, hd=256, page=64),
    # chunks under a window
    dict(t=[300], lens=[900], nh=2, nk=1, hd=128, page=16, window=70, sinks=4),
    dict(t=[200, 90, 1], lens=[200, 2000, 700], nh=4, nk=2, hd=64, page=64, window=128, sinks=0),
    dict(t=[150], lens=[1500], nh=4, nk=2, hd=256, page=128, window=33, sinks=300),
    dict(t=[260, 130], lens=[2600, 130], nh=3, nk=1, hd=128, page=32, window=1, sinks=2),
    dict(t=[400], lens=[300], nh=2, nk=1, hd=64, page=16, window=40, sinks=3),       # 100 rows see nothing
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kw", ATTEND)
def test_attend(kw, dtype):
    bt = Batch4(dtype=dtype, seed=11, exps=(2, -3), **kw)
    ref = bt.oracle()
    out, lse, err = bt.attend()
    assert err == 0
    bt.check(out, lse, ref)
    again, lse2, _ = bt.attend()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    wide = torch.full((bt.T, bt.nh, bt.hd), 5.0, device="cuda")
    bt.check(*bt.attend(out=wide)[:2], ref)


@pytest.mark.parametrize("kw", [dict(t=[1, 2], lens=[700, 90], nh=8, nk=2, hd=128, page=16),
                                dict(t=[150], lens=[400], nh=2, nk=1, hd=64, page=32, window=64, sinks=2),
                                dict(t=[40], lens=[400], nh=4, nk=1, hd=256, page=64)])
def test_attend_of_large_and_small_queries(kw):
    """q's range is wider than f16's: rows are scaled by powers of two, so that rows of any size give
    what the formula gives, down to rows whose scores vanish."""
    bt = Batch4(dtype=BF, seed=13, **kw)
    for mul in (2.0 ** 100, 2.0 ** -60, 2.0 ** -126):
        q = (bt.q.float() * mul).to(BF)
        small = Batch4(dtype=BF, seed=13, **kw)
        small.q, small.scale = q, bt.scale / mul if mul > 2.0 ** -100 else bt.scale
        small.check(*small.attend()[:2])
    z = Batch4(dtype=BF, seed=13, **kw)
    z.q = torch.zeros_like(z.q)
    z.check(*z.attend()[:2])
    z.scale = 0.0
    z.q = bt.q
    z.check(*z.attend()[:2])


@pytest.mark.parametrize("kw", [dict(t=[2, 1], lens=[300, 90], nh=4, nk=2, hd=128, page=16),
                                dict(t=[90, 140], lens=[300, 140], nh=2, nk=1, hd=128, page=64)])
def test_attend_reports(kw):
    """Bad pages read as zeros, lengths and rows out of range are reported; the other sequences'
    results stay."""
    bt = Batch4(seed=14, **kw)
    ref = bt.attend()
    table = bt.args[4].clone()
    table[0, 0] = 1 << 29
    out, lse, err = bt.attend(args=(*bt.pools, table, *bt.args[5:]))
    assert err == _abi.SWA_DERR_PAGE and torch.equal(out[bt.start[1]:], ref[0][bt.start[1]:])
    k, v = bt.values()
    ro = p4.attend(f64(bt.q), k, v, table.cpu().numpy(), bt.start, bt.n, bt.scale)
    bt.check(out, lse, ro)
    lens = bt.args[6].clone()
    lens[0] = -3
    out, lse, err = bt.attend(args=(*bt.args[:6], lens))
    assert err == _abi.SWA_DERR_META and torch.equal(out[bt.start[1]:], ref[0][bt.start[1]:])
    assert not out[:bt.start[1]].any() and torch.isneginf(lse[:bt.start[1]]).all()
    out, lse, err = bt.attend(args=(*bt.args[:5], dev([0, bt.start[1], 1 << 20]), bt.args[6]))
    assert err == _abi.SWA_DERR_SEGMENT and torch.equal(out[:bt.start[1]], ref[0][:bt.start[1]])
    assert (out[bt.start[1]:] == 5.0).all()


@pytest.mark.parametrize("kw", [dict(t=[1, 3], lens=[300, 90], nh=4, nk=2, hd=128, page=16),
                                dict(t=[90, 140], lens=[300, 140], nh=2, nk=1, hd=64, page=64)])
def test_attend_strided_q_and_row_bounds(kw):
    bt = Batch4(seed=15, **kw)
    ref = bt.attend()
    wide = torch.full((bt.T, bt.nh + 3, bt.hd), float("nan"), dtype=BF, device="cuda")
    wide[:, 1:1 + bt.nh] = bt.q
    got = bt.attend(q=wide[:, 1:1 + bt.nh])
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    # a looser bound of the rows may choose another kernel
    bt.check(*bt.attend(max_rows=max(bt.t) + 200)[:2])


# ------------------------------------------------------------------ pages
def pools_for(num_pages, page, seed=0):
    """A 16-bit pool, codes and scales: three of different page sizes."""
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(num_pages, 2, page, 64, generator=g).to(BF).cuda(),
            torch.randint(0, 256, (num_pages, 2, page, 32), generator=g, dtype=torch.int32).to(U8).cuda(),
            torch.randint(0, 127, (num_pages, 2, page, 4), generator=g, dtype=torch.int32).to(U8).cuda().view(E4)]


def sequences(lens, page, num_pages, width, seed, share=0, extra=0):
    """A consistent table: `share` leading pages in common, `extra` pages behind the last key."""
    order = np.random.default_rng(seed).permutation(num_pages).tolist()
    common = [order.pop() for _ in range(share)]
    table, refs = [], [0] * num_pages
    for n in lens:
        need = -(-n // page)
        row = common[:need] + [order.pop() for _ in range(max(0, need - share) + extra)]
        table.append(row + [-1] * (width - len(row)))
        for p in row:
            refs[p] += 1
    return table, refs


FORK = [
    dict(lens=[40, 33], parent=[0, 1], room=[1, 1]),                         # one step: nothing to copy
    dict(lens=[40, 33], parent=[0, 0, 0, 1], room=[1, 1, 1, 1]),             # branches
    dict(lens=[48, 32, 0], parent=[1, 1, 0, -1, 2, 0], room=[1, 0, 17, 40, 3, 100]),   # full pages, an empty parent
    dict(lens=[40, 33, 7], parent=[-1, -1, -1], room=[0, 0, 5]),             # all end, one begins
    dict(lens=[70, 70, 70, 70], parent=[3, 3, 0, 1], room=None, share=4),    # beams over a common prefix
    dict(lens=[20, 20], parent=[0, 1, 1], room=[1, 1, 1], share=2),          # both hold the page that is written next
    dict(lens=[20, 35], parent=[0, 1], room=[1, 1], share=3),                # .. and one of them is past it
    dict(lens=[20, 20], parent=[0, 0], room=[1, 1], held=True),              # .. and a holder outside the table
    dict(lens=[5] * 40, parent=[i % 40 for i in range(0, 700, 7)], room=[2] * 100, num_pages=400),
    dict(lens=[40, 33], parent=[0, 0, 0, 1], room=[1, 1, 1, 1], num_pages=9000),     # the passes on a cluster
    dict(lens=[100, 90], parent=[0, 1], room=[1, 1], extra=2),               # pages behind the last key are let go
    dict(lens=[40, 33], parent=[0, 0, 0, 1], room=[500, 1, 1, 1], num_pages=12, lacking=True),
    dict(lens=[33] * 5, parent=[0, 0, 0, 0, 1, 2, 3, 4], room=[0] * 8, num_pages=16, lacking=True),
]


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("kw", FORK)
def test_fork(kw, page):
    kw = dict(kw)
    lens, parent, room = kw["lens"], kw["parent"], kw["room"]
    if page == 64:
        lens = [n * 4 - (n % 3 if n % 16 else 0) for n in lens]
    num_pages, width = kw.get("num_pages", 60), 12
    table, refs = sequences(lens, page, num_pages, width, 3, kw.get("share", 0), kw.get("extra", 0))
    if kw.get("held"):
        refs[table[0][lens[0] // page]] += 1
    want = p4.fork(table, lens, refs, parent, room, page, num_pages)
    pools = pools_for(num_pages, page)
    before = [x.clone() for x in pools]
    err = zero()
    args = (dev(table), dev(lens), dev(refs), dev(parent))
    got = swa.paged_fork(pools, *args, page, room=None if room is None else dev(room), err=err)
    torch.cuda.synchronize()
    assert got[0].tolist() == want[0] and got[1].tolist() == want[1] and got[2].tolist() == want[2] and got[3].item() == want[3]
    full = bool(kw.get("lacking"))
    past = room is not None and any(n + x > width * page for n, x in zip(want[1], room))     # the table's width
    assert int(err.item()) == (_abi.SWA_DERR_FULL if full else 0) | (_abi.SWA_DERR_META if past else 0)
    assert full == (want[3] < 0)
    for x, y in zip(pools, before):
        y = y.view(U8)
        for src, dst in want[4]:
            y[dst] = y[src]
        assert torch.equal(x.view(U8), y)
    # every page is held as often as it is counted
    if not full:
        held = np.bincount([p for row in want[0] for p in row if p >= 0], minlength=num_pages)
        outside = np.array(refs) - np.bincount([p for row in table for p in row if p >= 0], minlength=num_pages)
        assert (held + outside == np.array(want[2])).all()
    # again, and with the counts in place
    again = swa.paged_fork(pools, *args, page, room=None if room is None else dev(room))
    assert all(torch.equal(x, y) for x, y in zip(got, again))
    mine = args[2].clone()
    swa.paged_fork(pools, args[0], args[1], mine, args[3], page, room=None if room is None else dev(room), refs_out=mine)
    assert torch.equal(mine, got[2]) and all(torch.equal(x.view(U8), y.view(U8)) for x, y in zip(pools, before))


def test_fork_reports():
    """Parents, lengths and pages out of range."""
    table, refs = sequences([40, 33], 16, 60, 4, 3)
    table[1][1] = 99
    pools, err = pools_for(60, 16), zero()
    got = swa.paged_fork(pools, dev(table), dev([40, 33]), dev(refs), dev([0, 1]), 16, err=err)
    want = p4.fork(table, [40, 33], refs, [0, 1], None, 16, 60)
    assert int(err.item()) == _abi.SWA_DERR_PAGE and got[0].tolist() == want[0] and got[2].tolist() == want[2]
    for lens, parent in (([40, 1000], [0, 1]), ([-5, 33], [0, 1]), ([40, 33], [2, 0]), ([40, 33], [-9, 1])):
        table, refs = sequences([40, 64], 16, 60, 4, 3)
        err = zero()
        got = swa.paged_fork(pools, dev(table), dev(lens), dev(refs), dev(parent), 16, err=err)
        want = p4.fork(table, lens, refs, parent, None, 16, 60)
        assert int(err.item()) == _abi.SWA_DERR_META, (lens, parent)
        assert [x.tolist() for x in got[:3]] == list(want[:3])
    table, refs = sequences([40, 33], 16, 60, 4, 3)
    refs[table[0][0]] = 0                                     # fewer holders than the table has
    err = zero()
    got = swa.paged_fork(pools, dev(table), dev([40, 33]), dev(refs), dev([-1, 1]), 16, err=err)
    assert int(err.item()) == _abi.SWA_DERR_META and got[2][table[0][0]].item() == -1


@pytest.mark.parametrize("B,R,width,num_pages", [(300, 900, 40, 30000), (1, 5000, 3, 20000), (5000, 1, 9, 70001)])
def test_fork_of_large_batches(B, R, width, num_pages):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, (width - 1) * 16, B).tolist()
    table, refs = sequences(lens, 16, num_pages, width, 3)
    parent, room = rng.integers(-1, B, R).tolist(), rng.integers(0, 20, R).tolist()
    pools = [torch.arange(num_pages, dtype=torch.int32, device="cuda").view(-1, 1).expand(num_pages, 4).contiguous()]
    want = p4.fork(table, lens, refs, parent, room, 16, num_pages)
    got = swa.paged_fork(pools, dev(table), dev(lens), dev(refs), dev(parent), 16, room=dev(room))
    assert [x.tolist() for x in got[:3]] == list(want[:3]) and got[3].item() == want[3]
    moved = np.arange(num_pages)
    for src, dst in want[4]:
        moved[dst] = src
    assert (pools[0][:, 0].cpu().numpy() == moved).all()


@pytest.mark.parametrize("lens,num_pages", [([40, 33], 60), ([16], 1), ([0], 7), ([100] * 9, 64), ([700, 1, 333], 70001), ([2000] * 40, 5001)])
def test_compact(lens, num_pages):
    width = max(-(-max(lens) // 16), 1) + 1
    table, refs = sequences(lens, 16, num_pages, width, 5)
    if num_pages > 100:
        refs[num_pages - 2] += 3                              # a holder outside the table
    want = p4.compact(table, refs, num_pages)
    pools = pools_for(num_pages, 16) if num_pages < 100 else [torch.arange(num_pages * 4, dtype=torch.int32, device="cuda").view(-1, 4)]
    before, err = [x.clone() for x in pools], zero()
    t, r = dev(table), dev(refs)
    got = swa.paged_compact(pools, t, r, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert [x.tolist() for x in got[:3]] == list(want[:3]) and got[3].item() == want[3]
    for x, y in zip(pools, before):
        y = y.view(U8)
        if want[4]:
            src, dst = dev([c[0] for c in want[4]], torch.int64), dev([c[1] for c in want[4]], torch.int64)
            y[dst] = y[src]
        assert torch.equal(x.view(U8), y)
    again = swa.paged_compact(pools, t, r)
    assert all(torch.equal(x, y) for x, y in zip(got, again))
    assert all(torch.equal(x.view(U8), y.view(U8)) for x, y in zip(pools, before))
    swa.paged_compact(pools, t, r, table_out=t, refs_out=r)
    assert torch.equal(t, got[0]) and torch.equal(r, got[1])


def test_compact_reports():
    table, refs = sequences([40, 33], 16, 20, 4, 6)
    refs[table[0][0]] = 0                                     # the table names a free page
    refs[table[0][1]] = -2
    err = zero()
    got = swa.paged_compact(pools_for(20, 16), dev(table), dev(refs), err=err)
    want = p4.compact(table, refs, 20)
    assert int(err.item()) == _abi.SWA_DERR_META | _abi.SWA_DERR_PAGE
    assert [x.tolist() for x in got[:3]] == list(want[:3]) and got[0][0, 0].item() == -1
