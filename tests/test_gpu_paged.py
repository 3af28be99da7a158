"""Rotary and paged-cache kernels against the float64 oracle (oracle/paged_oracle.py).

Tolerances (u: half a step of the type, eps / 2):
  rotary   the angle is good to 2^-33 turns plus its rounding to f32 (2^-24 of at most pi)
           and sincospif's own error (2 ulp); two products and a sum in f32: 8 * 2^-24 of
           |u| + |v|, times mag; then one rounding.
  attend   each weight is rounded to the type once (u, relative) and the result once. A
           score is a sum of hd products in f32: off by at most hd * 2^-24 * sum |q_i k_i|
           scale =: d; with the scaling, the subtraction and the 2^x (2^-21) a weight is off
           by d + 2^-19 relative, in numerator and sum:
           |out - ref| <= (u + 2 (d + 2^-19) + n 2^-24) * mean|v| + u |ref|.
  lse      d + 2^-19 + n 2^-24 (the sum) + 2^-22 |lse|
  weigh    the same weights without rounding, against the given lse (its product with log2 e
           adds 2^-23 |lse|): relative d + 2^-19 + 2^-22 |lse| + 2^-24 per term added.
  evict, slots, lengths: exact.
A rounding to f16 is off by up to 2^-25 absolute where the value is below 2^-14: the grid's
step is 2^-24 there (`tiny`). The weights are rounded times 2^15, so that they lose at most
2^-40 of the largest each: n 2^-40 max|v| in the result.
"""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as po
from sliding_window_gqa_prep_gb300 import _abi
import sliding_window_gqa_prep_gb300 as swa

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test collected on a machine without a GPU")
    yield


def f64(x):
    return x.detach().double().cpu().numpy()


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half a step of the type's grid below its smallest normal number."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


class Batch:
    """A ragged chunk over a paged cache whose unused slots and pages hold NaN."""

    def __init__(self, t, lens, nh, nk, hd, page, dtype=BF, seed=0, pad=0, spare=2, scale=None, sharp=1.0):
        g = torch.Generator().manual_seed(seed)
        self.t, self.n, self.nh, self.nk, self.hd, self.page, self.dtype = t, lens, nh, nk, hd, page, dtype
        B = len(t)
        need = [max(1, -(-x // page)) for x in lens]
        self.max_pages = max(need)
        pool = sum(need) + spare
        order = torch.randperm(pool, generator=g)
        self.table = torch.full((B, self.max_pages), -7, dtype=torch.int32)
        k = torch.full((pool, nk, page, hd), float("nan"))
        v = torch.full((pool, nk, page, hd), float("nan"))
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]].to(torch.int32)
            at += need[b]
            for i in range(need[b]):
                p, n = int(self.table[b, i]), min(page, lens[b] - i * page)
                if n > 0:
                    k[p, :, :n] = torch.randn(nk, n, hd, generator=g) * sharp
                    v[p, :, :n] = torch.randn(nk, n, hd, generator=g)
        self.k, self.v = k.to(dtype).cuda(), v.to(dtype).cuda()
        self.start = [0]
        for x in t:
            self.start.append(self.start[-1] + x)
        self.T = self.start[-1] + pad
        self.q = torch.randn(self.T, nh, hd, generator=g).to(dtype).cuda()
        self.scale = hd ** -0.5 if scale is None else scale
        self.cap = self.max_pages * page
        self.args = (self.k, self.v, self.table.cuda(), dev(self.start), dev(lens))

    def oracle(self):
        k, v = f64(self.k), f64(self.v)
        return po.attend(f64(self.q), k, v, self.table.numpy(), self.start, self.n, self.scale)

    def attend(self, **kw):
        kw.setdefault("max_rows", max(max(self.t), 1))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        lse = torch.full((self.T, self.nh), 77.0, device="cuda")
        out = kw.pop("out", None)
        if out is None:
            out = torch.full((self.T, self.nh, self.hd), 5.0, dtype=self.dtype, device="cuda")
        swa.paged_attend(kw.pop("q", self.q), *self.args, self.scale, out=out, lse=lse, err=err, **kw)
        torch.cuda.synchronize()
        return out, lse, int(err.item())

    def check(self, out, lse, ref=None):
        ro, rl, av, sa = ref if ref is not None else self.oracle()
        live = self.start[-1]
        u = unit(self.dtype)
        n = max(max(self.n), 1)
        d = self.hd * 2.0 ** -24 * sa[:live, :, None]
        o, ro, av = f64(out)[:live], ro[:live], av[:live]
        uo = unit(out.dtype)
        tol = (u + 2 * (d + 2.0 ** -19) + n * 2.0 ** -24) * av + uo * np.abs(ro) + tiny(out.dtype)
        if self.dtype == HF:
            tol = tol + n * 2.0 ** -40 * float(self.v.nan_to_num(0).abs().max())
        bad = ~(np.abs(o - ro) <= tol)
        assert not bad.any(), (int(bad.sum()), np.abs(o - ro).max(), np.argwhere(bad)[:4])
        g, rl = f64(lse)[:live], rl[:live]
        empty = np.isneginf(rl)
        assert (np.isneginf(g) == empty).all()
        tl = d[..., 0] + 2.0 ** -19 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(empty, 0, rl))
        assert (np.abs(np.where(empty, 0, g) - np.where(empty, 0, rl)) <= tl).all()
        # rows of no sequence are left as they were
        assert (out[live:] == 5.0).all() and (lse[live:] == 77.0).all()


# ------------------------------------------------------------------ rotary
ROTARY = [
    dict(T=1, H=1, hd=8, rot=8), dict(T=7, H=3, hd=64, rot=64), dict(T=5, H=40, hd=128, rot=64),
    dict(T=3, H=2, hd=64, rot=20), dict(T=2, H=5, hd=256, rot=2), dict(T=301, H=9, hd=128, rot=128),
    dict(T=4000, H=6, hd=64, rot=48), dict(T=2, H=2, hd=1024, rot=1000), dict(T=2, H=2500, hd=8, rot=6),
    dict(T=700, H=5, hd=32, rot=28), dict(T=33, H=3, hd=256, rot=136),
]


@pytest.mark.parametrize("dtype", [FP, BF, HF])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("kw", ROTARY)
def test_rotary(kw, inter, dtype):
    T, H, hd, rot = kw["T"], kw["H"], kw["hd"], kw["rot"]
    g = torch.Generator().manual_seed(T + rot)
    x = torch.randn(T, H, hd, generator=g).to(dtype)
    pos = torch.randint(-5, 1 << 20, (T,), generator=g, dtype=torch.int32)
    pos[0] = 2147483647 if T > 1 else 3
    f = swa.rotary_freqs(rot).numpy()
    turns = swa.rotary_turns(rot)
    for inverse, mag in ((False, 1.0), (True, 1.25)):
        y = swa.rotary(x.cuda(), pos.cuda(), turns, interleaved=inter, inverse=inverse, mag=mag)
        ref = po.rotary(f64(x), pos.numpy(), f, inter, inverse, mag)
        a = np.abs(f64(x))
        other = a.copy()
        h = rot // 2
        if inter:
            other[..., 0:rot:2], other[..., 1:rot:2] = a[..., 1:rot:2], a[..., 0:rot:2]
        else:
            other[..., :h], other[..., h:rot] = a[..., h:rot], a[..., :h]
        # positions up to 2^31: the oracle's own f64 angle is good to 2^31 * 2^-53 * 2
        tol = (8 * 2.0 ** -24 + 2.0 ** -21) * mag * (a + other) + unit(dtype) * np.abs(ref) + tiny(dtype)
        tol[..., rot:] = 0
        assert (np.abs(f64(y) - ref) <= tol).all()


def test_rotary_gradient():
    """inverse is the transpose: <R x, g> = <x, R' g>, and central differences."""
    g = torch.Generator().manual_seed(3)
    x, gy = torch.randn(6, 2, 32, generator=g).cuda(), torch.randn(6, 2, 32, generator=g).cuda()
    pos, turns = dev([0, 1, 5, 1000, 77777, -4]), swa.rotary_turns(24)
    for inter in (False, True):
        gx = swa.rotary(gy, pos, turns, interleaved=inter, inverse=True, mag=0.7)
        y = swa.rotary(x, pos, turns, interleaved=inter, mag=0.7)
        a, b = float((y.double() * gy.double()).sum()), float((x.double() * gx.double()).sum())
        # 2 * 384 products of values good to 16 * 2^-24
        assert abs(a - b) <= 16 * 2.0 ** -24 * float((y.abs().double() * gy.abs().double()).sum()
                                                     + (x.abs().double() * gx.abs().double()).sum())
        for at in ((0, 0, 0), (3, 1, 7), (4, 0, 20), (5, 1, 31)):
            e = torch.zeros_like(x)
            e[at] = 0.5
            yp = swa.rotary(x + e, pos, turns, interleaved=inter, mag=0.7)
            ym = swa.rotary(x - e, pos, turns, interleaved=inter, mag=0.7)
            diff = float(((yp.double() - ym.double()) * gy.double()).sum())
            # linear: the difference over a step of 1 is the derivative, up to f32 rounding of y
            # (|y| < 4 in two features, |gy| < 4)
            assert abs(diff - float(gx[at])) <= 64 * 16 * 2.0 ** -24


def test_rotary_strided_and_in_place():
    """q and k heads inside packed rows, heads before rows, and in place."""
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn(9, 8, 64, generator=g).to(BF).cuda()
    pos, turns = dev(range(100, 109)), swa.rotary_turns(64)
    want = swa.rotary(qkv[:, :6].contiguous(), pos, turns)
    got = qkv.clone()
    swa.rotary(got[:, :6], pos, turns, out=got[:, :6])
    assert torch.equal(got[:, :6], want) and torch.equal(got[:, 6:], qkv[:, 6:])
    heads_first = qkv[:, :6].transpose(0, 1).contiguous()
    out = torch.empty_like(heads_first)
    swa.rotary(heads_first.transpose(0, 1), pos, turns, out=out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), want)
    with pytest.raises(swa.SwaError):
        swa.rotary(got[:, :4], pos, turns, out=got[:, 2:6])          # overlapping, not the same
    with pytest.raises(ValueError):
        swa.rotary(got, pos[:3], turns)
    with pytest.raises(ValueError):
        swa.rotary(got, pos.cpu(), turns)
    with pytest.raises(ValueError):
        swa.rotary(got, pos, turns, out=got[:, :4])                 # another shape
    with pytest.raises(ValueError):
        swa.rotary(got, pos, turns, out=got.float())                # another type
    assert swa.rotary(got[:0], pos[:0], turns).shape == (0, 8, 64)
    assert torch.equal(swa.rotary(x=qkv[:, :6], pos=pos, turns=turns), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = swa.rotary(qkv[:, :6], pos, turns, stream=side)
    side.synchronize()
    assert torch.equal(y, want)


# ------------------------------------------------------------------ append
APPEND = [
    dict(t=[1], lens=[1], nh=2, nk=1, hd=64, page=16, rot=64),
    dict(t=[1, 1, 1], lens=[17, 16, 300], nh=8, nk=2, hd=128, page=16, rot=128),
    dict(t=[5, 0, 33, 1], lens=[5, 9, 100, 64], nh=6, nk=3, hd=64, page=32, rot=32, pad=3),
    dict(t=[130, 7], lens=[131, 500], nh=4, nk=4, hd=256, page=128, rot=20),
    dict(t=[3, 2], lens=[40, 2], nh=4, nk=1, hd=128, page=64, rot=0),
]


@pytest.mark.parametrize("dtype,src", [(BF, BF), (HF, HF), (BF, FP), (HF, FP)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("kw", APPEND)
def test_append(kw, inter, dtype, src):
    kw = dict(kw)
    rot = kw.pop("rot")
    bt = Batch(dtype=dtype, seed=5, **kw)
    g = torch.Generator().manual_seed(6)
    nh, nk, hd, T = bt.nh, bt.nk, bt.hd, bt.T
    # rows inside a wider packed projection
    proj = torch.randn(T, (nh + 2 * nk) * hd + 8, generator=g).to(src).cuda()
    q = proj[:, :nh * hd].unflatten(1, (nh, hd))
    k = proj[:, nh * hd:(nh + nk) * hd].unflatten(1, (nk, hd))
    v = proj[:, (nh + nk) * hd:(nh + 2 * nk) * hd].unflatten(1, (nk, hd))
    pos = torch.randint(0, 100000, (T,), generator=g, dtype=torch.int32).cuda()
    turns = swa.rotary_turns(rot) if rot else None
    before_k, before_v = bt.k.clone(), bt.v.clone()
    slot_pos = torch.full((len(bt.t), nk, bt.cap), -9, dtype=torch.int32, device="cuda")
    weight = torch.full((len(bt.t), nk, bt.cap), 3.0, device="cuda")
    q_out = torch.full((T, nh, hd), 5.0, dtype=dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    swa.paged_append(k, v, pos, *bt.args, q=q, q_out=q_out, turns=turns, interleaved=inter, slot_pos=slot_pos,
                     weight=weight, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    # the rotation itself is the rotary kernel's, tested above: the same bits here
    def turned(x):
        x = x.float().contiguous()
        return (swa.rotary(x, pos, turns, interleaved=inter) if rot else x).to(dtype)
    wq, wk, wv = turned(q), turned(k), v.to(dtype)
    live = bt.start[-1]
    assert torch.equal(q_out[:live], wq[:live]) and (q_out[live:] == 5.0).all()
    want_k, want_v = before_k, before_v
    for b in range(len(bt.t)):
        for i in range(bt.t[b]):
            r, slot = bt.start[b] + i, bt.n[b] - bt.t[b] + i
            p = int(bt.table[b, slot // bt.page])
            want_k[p, :, slot % bt.page], want_v[p, :, slot % bt.page] = wk[r], wv[r]
            assert (slot_pos[b, :, slot] == pos[r]).all() and (weight[b, :, slot] == 0).all()
    same = lambda a, b: bool(((a == b) | (a.isnan() & b.isnan())).all())
    assert same(bt.k, want_k) and same(bt.v, want_v)
    assert int((slot_pos != -9).sum()) <= live * nk and int((weight == 0).sum()) == live * nk


def test_append_reports_and_skips():
    """A chunk longer than its length, a bad page and rows out of range: reported, nothing
    else written."""
    bt = Batch(t=[4, 2, 3], lens=[40, 20, 17], nh=2, nk=1, hd=64, page=16, seed=7)
    g = torch.Generator().manual_seed(8)
    x = torch.randn(9, 1, 64, generator=g).to(BF).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k0 = bt.k.clone()
    table = bt.args[2].clone()
    table[1, 1] = 1 << 30                                    # slots 18, 19 of sequence 1
    starts = dev([0, 4, 6, 50])                              # the last sequence reaches past T
    swa.paged_append(x, x, None, bt.k, bt.v, table, starts, dev([2, 20, 17]), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == _abi.SWA_DERR_META | _abi.SWA_DERR_PAGE | _abi.SWA_DERR_SEGMENT
    p = int(table[0, 0])
    assert torch.equal(bt.k[p, 0, :2], x[2:4, 0])            # rows 2, 3 of sequence 0 have slots 0, 1
    bt.k[p, 0, :2] = k0[p, 0, :2]
    assert bool(((bt.k == k0) | (bt.k.isnan() & k0.isnan())).all())


# ------------------------------------------------------------------ attend
ATTEND = [
    # one token: lengths of one, inside a page, page ends, many tiles
    dict(t=[1], lens=[1], nh=1, nk=1, hd=64, page=16),
    dict(t=[1], lens=[133], nh=8, nk=2, hd=64, page=16),
    dict(t=[1, 1, 1, 1], lens=[64, 65, 63, 1], nh=4, nk=4, hd=128, page=64),
    dict(t=[1, 1, 1], lens=[1000, 16, 4097], nh=16, nk=2, hd=128, page=32),
    dict(t=[1, 1], lens=[2050, 700], nh=8, nk=2, hd=256, page=128),
    dict(t=[1], lens=[300], nh=32, nk=1, hd=128, page=256),
    # few rows, empty sequences, rows behind the last one, a length of zero with rows
    dict(t=[3, 0, 8], lens=[3, 50, 200], nh=12, nk=4, hd=64, page=16, pad=5),
    dict(t=[8, 8], lens=[8, 519], nh=32, nk=8, hd=128, page=64),
    dict(t=[2, 1], lens=[0, 5], nh=2, nk=1, hd=64, page=16),
    dict(t=[5], lens=[2], nh=4, nk=2, hd=128, page=16),              # its first three rows see nothing
    dict(t=[0, 0], lens=[5, 0], nh=2, nk=1, hd=64, page=16, pad=2),
    dict(t=[7, 1], lens=[100, 33], nh=5, nk=1, hd=256, page=16),
    # chunks: row blocks, causal diagonals across tiles, odd head groups
    dict(t=[130], lens=[130], nh=4, nk=1, hd=64, page=16),
    dict(t=[257, 64], lens=[300, 900], nh=8, nk=2, hd=128, page=64),
    dict(t=[100, 1, 33], lens=[612, 800, 33], nh=6, nk=2, hd=128, page=32, pad=1),
    dict(t=[40, 0, 90], lens=[1000, 10, 90], nh=5, nk=1, hd=64, page=128),
    dict(t=[70, 129], lens=[290, 129], nh=4, nk=2, hd=256, page=16),
    dict(t=[300], lens=[200], nh=2, nk=1, hd=128, page=16),          # 100 rows see nothing
    dict(t=[35], lens=[1111], nh=32, nk=1, hd=128, page=256),
    dict(t=[513, 3], lens=[2000, 3], nh=1, nk=1, hd=128, page=16),
    # equal rows of 33 to 64 vectors, and of 17 and more at hd 256: tensor cores
    dict(t=[10, 10], lens=[10, 700], nh=8, nk=2, hd=128, page=32),
    dict(t=[16], lens=[300], nh=4, nk=1, hd=64, page=16),
    dict(t=[9, 9, 9], lens=[9, 64, 1000], nh=4, nk=2, hd=256, page=64),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kw", ATTEND)
def test_attend(kw, dtype):
    bt = Batch(dtype=dtype, seed=11, **kw)
    out, lse, err = bt.attend()
    assert err == 0
    bt.check(out, lse)


@pytest.mark.parametrize("kw", [ATTEND[3], ATTEND[13], ATTEND[16]])
def test_attend_scales_and_types(kw):
    """f32 output, a sharp softmax, scale 0 and padded q rows."""
    bt = Batch(dtype=BF, seed=12, sharp=6.0, **kw)
    out = torch.full((bt.T, bt.nh, bt.hd), 5.0, device="cuda")
    bt.check(*bt.attend(out=out)[:2])
    wide = torch.zeros(bt.T, bt.nh * bt.hd + 24, dtype=BF, device="cuda")
    wide[:, :bt.nh * bt.hd] = bt.q.view(bt.T, -1)
    o2, l2, _ = bt.attend(q=wide[:, :bt.nh * bt.hd].unflatten(1, (bt.nh, bt.hd)))
    o1, l1, _ = bt.attend()
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    bt.scale = 0.0
    bt.check(*bt.attend()[:2])


def test_attend_f16_small_weights():
    """Many keys far below the largest: their weights must not vanish from the product."""
    bt = Batch(t=[1], lens=[8192], nh=1, nk=1, hd=64, page=64, dtype=HF, seed=13, scale=1.0)
    bt.q.zero_()
    bt.q[0, 0, 0] = 1.0
    bt.k.nan_to_num_(0)
    bt.k[..., 0] = -15.0                                     # weight 3e-7 against the one of 1
    p = int(bt.table[0, 0])
    bt.k[p, 0, 3, 0] = 0.0
    bt.v.nan_to_num_(0)
    bt.v.fill_(1.0)
    bt.v[p, 0, 3] = -1.0
    out, lse, _ = bt.attend()
    bt.check(out, lse)


def test_attend_reports():
    """Bad pages are zero keys, a length past the table is clamped, a chunk over max_rows is
    skipped; the other sequences are not touched by it."""
    bt = Batch(t=[1, 2, 9, 1], lens=[90, 70, 64, 30], nh=4, nk=2, hd=64, page=16, seed=14, pad=1)
    table = bt.table.clone()
    table[1, 2] = bt.k.shape[0]
    bt.args = (bt.k, bt.v, table.cuda(), dev(bt.start), dev([90, 70, 64, 1 << 20]))
    # the clamped sequence then reads pages its table does not name: give it real ones
    table[3, :] = torch.tensor([int(table[0, 0])] * bt.max_pages)
    bt.args = (bt.k, bt.v, table.cuda(), dev(bt.start), dev([90, 70, 64, 1 << 20]))
    out, lse, err = bt.attend(max_rows=2)
    assert err == _abi.SWA_DERR_META | _abi.SWA_DERR_PAGE | _abi.SWA_DERR_SEGMENT
    bt.table, bt.n = table, [90, 70, 64, bt.cap]
    ref = bt.oracle()
    keep = [r for r in range(bt.start[-1]) if not 3 <= r < 12]
    skipped = out[3:12], lse[3:12]
    assert (skipped[0] == 5.0).all() and (skipped[1] == 77.0).all()
    bt.start, t = [0, 4], bt.T
    pick = lambda x: x[keep]
    o, l = torch.cat((out[keep], out[-1:])), torch.cat((lse[keep], lse[-1:]))
    bt.check(o, l, tuple(pick(x) for x in ref))


def _many(seed, B, lo, hi, rows):
    """Many short sequences: several items and units a CTA, odd and even ones, some without
    rows or keys."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(lo, hi + 1, (B,), generator=g).tolist()
    t = [rows[int(x)] for x in torch.randint(0, len(rows), (B,), generator=g)]
    for b in range(0, B, 37):
        lens[b] = 0
    return t, lens


MANY = [
    dict(seed=1, B=400, lo=0, hi=300, rows=[0, 1, 1, 1, 2], nh=4, nk=2, hd=64, page=16),
    dict(seed=2, B=700, lo=1, hi=90, rows=[0, 1], nh=2, nk=1, hd=128, page=32),
    dict(seed=3, B=230, lo=100, hi=600, rows=[1, 3], nh=8, nk=2, hd=128, page=64),
    dict(seed=4, B=120, lo=1, hi=700, rows=[1, 2], nh=4, nk=2, hd=256, page=128),
    # short sequences and chunks in one call
    dict(seed=5, B=150, lo=60, hi=300, rows=[0, 1, 1, 7, 40], nh=8, nk=2, hd=64, page=16),
    dict(seed=6, B=60, lo=100, hi=500, rows=[1, 90, 33], nh=4, nk=1, hd=128, page=256),
    dict(seed=7, B=40, lo=130, hi=500, rows=[1, 129], nh=2, nk=1, hd=256, page=16),
]


@pytest.mark.parametrize("kw", MANY)
def test_attend_many_sequences(kw):
    kw = dict(kw)
    t, lens = _many(*(kw.pop(x) for x in ("seed", "B", "lo", "hi", "rows")))
    bt = Batch(t=t, lens=lens, dtype=BF, seed=16, pad=3, **kw)
    out, lse, err = bt.attend()
    assert err == 0
    bt.check(out, lse)
    # a loose bound of the rows takes the other path and gives the same values
    out, lse, err = bt.attend(max_rows=2147483647)
    assert err == 0
    bt.check(out, lse)


def test_attend_same_bits_and_streams():
    """The same call gives the same bits; on another stream; two at once with their own
    workspaces; captured and replayed with a poisoned workspace."""
    bt = Batch(t=[1, 40, 3], lens=[3000, 700, 900], nh=8, nk=2, hd=128, page=64, seed=15)
    o1, l1, _ = bt.attend()
    need = swa.paged_attend_workspace_size(3, bt.T, 8, 2, 128, 64, bt.max_pages, 40)
    ws = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(o1) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, w, o in zip(streams, ws, outs):
            swa.paged_attend(bt.q, *bt.args, bt.scale, max_rows=40, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[:44], o1[:44])
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(o1)
    with torch.cuda.graph(g):
        swa.paged_attend(bt.q, *bt.args, bt.scale, max_rows=40, out=out)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:44], o1[:44])


def test_attend_far_offsets():
    """A pool whose elements pass 2^31: the last pages are read."""
    pool, nk, page, hd = 2100, 8, 256, 512 // 4
    pages = (1 << 31) // (nk * page * hd) + 8
    ck = torch.empty(pages, nk, page, hd, dtype=BF, device="cuda")
    cv = torch.empty_like(ck)
    g = torch.Generator(device="cuda").manual_seed(1)
    ck[-3:] = torch.randn(3, nk, page, hd, generator=g, device="cuda").to(BF)
    cv[-3:] = torch.randn(3, nk, page, hd, generator=g, device="cuda").to(BF)
    small_k, small_v = ck[-3:].clone(), cv[-3:].clone()
    for t, nh in ((1, 8), (70, 16)):
        q = torch.randn(t, nh, hd, generator=g, device="cuda").to(BF)
        lens, start = dev([700]), dev([0, t])
        a = swa.paged_attend(q, ck, cv, dev([[pages - 1, pages - 3, pages - 2]]), start, lens, 0.1, max_rows=t)
        b = swa.paged_attend(q, small_k, small_v, dev([[2, 0, 1]]), start, lens, 0.1, max_rows=t)
        assert torch.equal(a, b) and not a.isnan().any()


def test_attend_refusals_of_the_binding():
    bt = Batch(t=[1, 2], lens=[90, 70], nh=4, nk=2, hd=64, page=16, seed=17)
    k, v, tab, start, lens = bt.args
    call = lambda q=bt.q, k=k, v=v, tab=tab, start=start, lens=lens, **kw: swa.paged_attend(
        q, k, v, tab, start, lens, 0.1, **{"max_rows": 2, **kw})
    for kw in (dict(q=bt.q.float()), dict(q=bt.q[:, :, :32]), dict(v=v.to(HF)), dict(tab=tab.long()), dict(start=start[:2]),
               dict(lens=lens.cpu()), dict(k=k.transpose(1, 2)), dict(start=None), dict(out=torch.empty(3, 4, 64, device="cuda").half()),
               dict(lse=torch.empty(3, 2, device="cuda")), dict(q=bt.q.transpose(0, 1))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(max_rows=0), dict(q=torch.zeros(3, 5, 64, dtype=BF, device="cuda")),
               dict(workspace=torch.empty(512, dtype=torch.uint8, device="cuda")[8:])):
        with pytest.raises(swa.SwaError):
            call(**kw)
    out = call()
    assert out.shape == (3, 4, 64) and out.dtype == BF
    assert call(out=torch.zeros(3, 4, 64, device="cuda")).dtype == FP
    assert swa.paged_attend(bt.q[:0], k, v, tab, dev([0, 0, 0]), lens, 0.1, max_rows=1).shape == (0, 4, 64)


# ------------------------------------------------------------------ weigh
WEIGH = [
    dict(t=[1], lens=[1], nh=1, nk=1, hd=64, page=16),
    dict(t=[1, 1, 0], lens=[100, 65, 30], nh=8, nk=2, hd=128, page=16),
    dict(t=[9, 33], lens=[9, 500], nh=6, nk=2, hd=64, page=32, pad=2),
    dict(t=[64, 3], lens=[700, 2], nh=32, nk=1, hd=128, page=64),
    dict(t=[130], lens=[260], nh=4, nk=2, hd=256, page=128),
    dict(t=[300, 20], lens=[250, 400], nh=3, nk=1, hd=128, page=16),
    dict(t=[1100], lens=[1500], nh=2, nk=1, hd=64, page=256),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kw", WEIGH)
def test_weigh(kw, dtype):
    bt = Batch(dtype=dtype, seed=21, **kw)
    _, rl, _, sa = bt.oracle()
    lse = torch.tensor(rl, dtype=torch.float32).cuda()
    lse[bt.start[-1]:] = float("nan")
    B = len(bt.t)
    g = torch.Generator().manual_seed(22)
    w = torch.rand(B, bt.nk, bt.cap, generator=g)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((B, bt.nk, bt.cap), 5.0, device="cuda")
    args = (bt.q, lse, bt.k, *bt.args[2:], bt.scale)
    kwm = dict(max_rows=max(max(bt.t), 1), err=err)
    swa.paged_weigh(*args, weight=w.cuda(), out=out, **kwm)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    f32_lse = f64(lse)
    f32_lse[np.isneginf(f32_lse)] = 0
    ref = po.weigh(f64(bt.q), f32_lse, f64(bt.k), bt.table.numpy(), bt.start, bt.n, bt.scale, f64(w))
    live = bt.start[-1]
    d = bt.hd * 2.0 ** -24 * (sa[:live].max() if live else 0.0)
    lmax = np.abs(np.where(np.isneginf(rl), 0, rl)).max() if live else 0.0
    terms = max(bt.t) * bt.nh // bt.nk + 1
    tol = (d + 2.0 ** -19 + 2.0 ** -22 * lmax + terms * 2.0 ** -24) * np.abs(ref) + 1e-30
    got = f64(out)
    for b in range(B):
        assert (np.abs(got[b, :, :bt.n[b]] - ref[b, :, :bt.n[b]]) <= tol[b, :, :bt.n[b]]).all()
        assert (got[b, :, bt.n[b]:] == 5.0).all()
    # in place, and without weights
    x = w.cuda()
    swa.paged_weigh(*args, weight=x, out=x, **kwm)
    z = swa.paged_weigh(*args, **kwm)
    for b in range(B):
        n = bt.n[b]
        assert torch.equal(x[b, :, :n], out[b, :, :n]) and torch.equal(x[b, :, n:].cpu(), w[b, :, n:])
        assert torch.equal(w[b, :, :n].cuda() + z[b, :, :n], out[b, :, :n])


@pytest.mark.parametrize("kw", MANY + [
    # query tiles kept (two of them), and streamed (more)
    dict(seed=8, B=150, lo=300, hi=1500, rows=[40, 64], nh=8, nk=2, hd=128, page=64),
    dict(seed=9, B=70, lo=500, hi=1500, rows=[100, 20], nh=8, nk=2, hd=64, page=32),
    dict(seed=10, B=80, lo=200, hi=900, rows=[100, 3], nh=8, nk=2, hd=256, page=64),
    # one, two and more of them in one share
    dict(seed=11, B=170, lo=200, hi=900, rows=[20, 50, 0, 60, 100], nh=8, nk=2, hd=128, page=64),
    dict(seed=12, B=170, lo=100, hi=700, rows=[12, 30, 31, 70], nh=4, nk=1, hd=256, page=32),
    # groups of heads that do not divide a query tile
    dict(seed=13, B=60, lo=300, hi=900, rows=[100, 17], nh=10, nk=2, hd=256, page=64),
    dict(seed=14, B=40, lo=100, hi=800, rows=[60, 9, 21], nh=24, nk=2, hd=64, page=16),
    dict(seed=15, B=30, lo=100, hi=800, rows=[30, 7], nh=31, nk=1, hd=128, page=64),
])
def test_weigh_many_units(kw):
    """Several units a CTA, of one half and of two, and back to back calls."""
    kw = dict(kw)
    t, lens = _many(*(kw.pop(x) for x in ("seed", "B", "lo", "hi", "rows")))
    bt = Batch(t=t, lens=lens, dtype=HF, seed=23, pad=1, **kw)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.zeros(bt.T, bt.nh, device="cuda")
    # lse as the attention gives it (tested above); the exact weights against it
    swa.paged_attend(bt.q, *bt.args, bt.scale, max_rows=max(t), lse=lse, err=err)
    runs = [swa.paged_weigh(bt.q, lse, bt.k, *bt.args[2:], bt.scale, max_rows=max(t), err=err) for _ in range(20)]
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for r in runs[1:]:
        assert torch.equal(r, runs[0])
    k, q, l = bt.k.double(), bt.q.double(), lse.double()
    hpg, got = bt.nh // bt.nk, runs[0].double()
    for b in range(len(t)):
        n, r0, r1 = lens[b], bt.start[b], bt.start[b + 1]
        idx = torch.arange(n)
        rows = k[bt.table[b][idx // bt.page].long().cuda(), :, (idx % bt.page).cuda()]       # [n][nk][hd]
        x = torch.einsum("rghd,ngd->rghn", q[r0:r1].view(r1 - r0, bt.nk, hpg, bt.hd), rows) * bt.scale
        sabs = torch.einsum("rghd,ngd->rghn", q[r0:r1].abs().view(r1 - r0, bt.nk, hpg, bt.hd), rows.abs()) * bt.scale
        i = torch.arange(r1 - r0, device="cuda")
        seen = torch.arange(n, device="cuda")[None, :] < (n - (r1 - r0) + i + 1)[:, None]
        w = torch.exp(x - l[r0:r1].view(r1 - r0, bt.nk, hpg, 1))
        w = torch.where(seen[:, None, None, :], w, torch.zeros_like(w)).sum((0, 2))          # [nk][n]
        d = bt.hd * 2.0 ** -24 * (float(sabs.max()) if sabs.numel() else 0.0)
        lm = float(l[r0:r1].nan_to_num(neginf=0).abs().max()) if r1 > r0 else 0.0
        tol = (d + 2.0 ** -19 + 2.0 ** -22 * lm + ((r1 - r0) * hpg + 1) * 2.0 ** -24) * w + 1e-30
        assert ((got[b, :, :n] - w).abs() <= tol).all(), b
        assert (got[b, :, n:] == 0).all()


# ------------------------------------------------------------------ evict
EVICT = [
    dict(lens=[1], nk=1, hd=64, page=16, keep=1),
    dict(lens=[20, 0, 7], nk=2, hd=64, page=16, keep=7),
    dict(lens=[300, 64, 128], nk=3, hd=128, page=64, keep=100),
    dict(lens=[2112, 2050], nk=2, hd=128, page=32, keep=2048),
    dict(lens=[5000], nk=1, hd=256, page=128, keep=17),
    dict(lens=[1500, 1024, 1025], nk=1, hd=64, page=256, keep=1024),
    dict(lens=[40], nk=2, hd=64, page=16, keep=1000),
]


@pytest.mark.parametrize("kind", ["spread", "ties", "special"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kw", EVICT)
def test_evict(kw, dtype, kind):
    kw = dict(kw)
    keep = kw.pop("keep")
    lens = kw["lens"]
    B = len(lens)
    bt = Batch(t=[0] * B, nh=kw["nk"], dtype=dtype, seed=31, **kw)
    g = torch.Generator().manual_seed(32)
    shape = (B, bt.nk, bt.cap)
    w = torch.exp(2 * torch.randn(shape, generator=g))
    if kind == "ties":
        w = torch.randint(0, 3, shape, generator=g).float()
    elif kind == "special":
        some = torch.rand(shape, generator=g)
        w = torch.where(some < 0.1, torch.full_like(w, float("nan")), w)
        w = torch.where((some > 0.1) & (some < 0.2), torch.full_like(w, -0.0), w)
        w = torch.where((some > 0.2) & (some < 0.3), torch.full_like(w, float("inf")), w)
        w = torch.where((some > 0.3) & (some < 0.5), -w, w)
    pos = torch.rand(B, bt.nk, 2 * bt.cap, generator=g).argsort(-1)[..., :bt.cap].to(torch.int32).contiguous()
    sinks = 0 if kind == "ties" else 4
    recent = None if kind == "ties" else torch.randint(bt.cap, 2 * bt.cap, (B,), generator=g, dtype=torch.int32)
    k0, v0 = bt.k.clone(), bt.v.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    wo = torch.full(shape, 5.0, device="cuda")
    pout = torch.full(shape, -3, dtype=torch.int32, device="cuda")

    def call():
        n, _, _ = swa.paged_evict(bt.k, bt.v, bt.args[2], dev(lens), w.cuda(), pos.cuda(), keep, sinks=sinks,
                                  recent_from=None if recent is None else recent.cuda(), weight_out=wo,
                                  slot_pos_out=pout, err=err)
        torch.cuda.synchronize()
        return n
    got_n = call()
    assert int(err.item()) == 0
    want_k, want_v = k0.clone(), v0.clone()
    want_w, want_p = np.full(shape, 5.0), np.full(shape, -3)
    for b in range(B):
        for h in range(bt.nk):
            wl, pl = w[b, h].numpy().copy(), pos[b, h].numpy().copy()
            new, moves = po.evict(wl, pl, lens[b], keep, sinks, None if recent is None else int(recent[b]))
            for to, of in moves:
                wl[to], pl[to] = wl[of], pl[of]
                a, z = int(bt.table[b, to // bt.page]), int(bt.table[b, of // bt.page])
                want_k[a, h, to % bt.page], want_v[a, h, to % bt.page] = k0[z, h, of % bt.page], v0[z, h, of % bt.page]
            want_w[b, h, :new], want_p[b, h, :new] = wl[:new], pl[:new]
    assert got_n.tolist() == [min(x, keep) for x in lens]
    same = lambda a, b: bool(((a == b) | (a.isnan() & b.isnan())).all())
    for _ in range(2):
        assert same(bt.k, want_k) and same(bt.v, want_v)
        np.testing.assert_array_equal(wo.cpu().numpy(), want_w.astype(np.float32))
        np.testing.assert_array_equal(pout.cpu().numpy(), want_p)
        call()                                               # the same inputs again: the same result


@pytest.mark.parametrize("kind", ["spread", "ties", "special"])
@pytest.mark.parametrize("kw", [
    # the most slots that eight CTAs hold in registers; in shared memory; and more than that
    dict(lens=[32768, 9000], nk=2, hd=64, page=256, keep=2000),
    dict(lens=[40000, 100, 33000], nk=1, hd=128, page=64, keep=2500),
    dict(lens=[350000], nk=1, hd=64, page=256, keep=3001),
])
def test_evict_long(kw, kind):
    test_evict(kw, BF, kind)


def test_evict_reports():
    bt = Batch(t=[0, 0], lens=[64, 30], nh=1, nk=1, hd=64, page=16, seed=33)
    table = bt.args[2].clone()
    table[0, 0] = 999
    w = torch.arange(64, dtype=torch.float32, device="cuda").repeat(2, 1, 1)
    pos = torch.arange(64, dtype=torch.int32, device="cuda").repeat(2, 1, 1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k0 = bt.k.clone()
    n, wo, _ = swa.paged_evict(bt.k, bt.v, table, dev([64, -4]), w, pos, 32, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == _abi.SWA_DERR_PAGE | _abi.SWA_DERR_META
    assert n.tolist() == [32, 0] and wo[0, 0, :32].tolist() == list(range(32, 64))
    # slots 0 .. 15 lie on the bad page: only 16 .. 31 moved in
    p, z = int(table[0, 1]), int(table[0, 3])
    assert torch.equal(bt.k[p, 0], k0[z, 0])


# ------------------------------------------------------------------ a run of them
def test_step_captured_and_on_a_stream():
    """Append, attend, weigh and evict of one decode step, eager, on another stream, and
    captured into a graph whose workspaces are its own: the same bits."""
    B, nh, nk, hd, page, lens = 6, 8, 2, 128, 32, [700, 33, 64, 1, 1000, 257]
    g = torch.Generator().manual_seed(51)
    turns = swa.rotary_turns(hd)
    x = torch.randn(B, (nh + 2 * nk), hd, generator=g).to(BF).cuda()
    q, k, v = x[:, :nh], x[:, nh:nh + nk], x[:, nh + nk:]
    pos = dev([n - 1 for n in lens])

    def fresh():
        bt = Batch(t=[1] * B, lens=lens, nh=nh, nk=nk, hd=hd, page=page, seed=52)
        gg = torch.Generator().manual_seed(53)
        w = torch.rand(B, nk, bt.cap, generator=gg).cuda()
        p = torch.arange(bt.cap, dtype=torch.int32).repeat(B, nk, 1).cuda()
        return bt, w, p, [torch.zeros(B, nh, hd, dtype=BF, device="cuda"), torch.zeros(B, nh, device="cuda"),
                          torch.zeros(B, nk, bt.cap, device="cuda"), torch.zeros(B, nk, bt.cap, device="cuda"),
                          torch.zeros(B, nk, bt.cap, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")]

    def step(bt, w, p, o, stream=None):
        qr = swa.paged_append(k, v, pos, *bt.args, q=q, turns=turns, slot_pos=p, weight=w, stream=stream)
        swa.paged_attend(qr, *bt.args, hd ** -0.5, max_rows=1, out=o[0], lse=o[1], stream=stream)
        swa.paged_weigh(qr, o[1], bt.k, *bt.args[2:], hd ** -0.5, max_rows=1, weight=w, out=o[2], stream=stream)
        swa.paged_evict(bt.k, bt.v, bt.args[2], bt.args[4], o[2], p, 100, weight_out=o[3], slot_pos_out=o[4], lens_out=o[5],
                        stream=stream)
        return [y.clone() for y in o] + [bt.k.nan_to_num(9), bt.v.nan_to_num(9)]
    a = fresh()
    want = step(*a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = fresh()
    torch.cuda.synchronize()
    step(*b, stream=s)
    torch.cuda.synchronize()
    for y, z in zip([*b[3], b[0].k.nan_to_num(9), b[0].v.nan_to_num(9)], want):
        assert torch.equal(y, z)
    c = fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*c)
    k0, v0, w0, p0 = c[0].k.clone(), c[0].v.clone(), c[1].clone(), c[2].clone()
    for _ in range(2):
        for y, z in ((c[0].k, k0), (c[0].v, v0), (c[1], w0), (c[2], p0)):
            y.copy_(z)
        graph.replay()
        torch.cuda.synchronize()
        for y, z in zip([*c[3], c[0].k.nan_to_num(9), c[0].v.nan_to_num(9)], want):
            assert torch.equal(y, z)


@pytest.mark.parametrize("kw", [dict(t=[1, 1, 1], lens=[1500, 1400, 700]), dict(t=[90, 33, 1], lens=[1500, 1400, 700])])
def test_graphs_at_once_over_shared_pages(kw):
    """Sequences that read the same pages (a prefix they share), and two captured graphs over
    them replayed on two streams together: the bits of the calls alone."""
    bt = Batch(nh=8, nk=2, hd=128, page=64, seed=54, **kw)
    table = bt.table.clone()
    table[1, :10] = table[0, :10]
    table[2, :10] = table[0, :10]
    bt.table, bt.args = table, (bt.k, bt.v, table.cuda(), *bt.args[3:])
    out, lse, err = bt.attend()
    assert err == 0
    bt.check(out, lse)
    rows = max(bt.t)
    want = out, lse, swa.paged_weigh(bt.q, lse, bt.k, *bt.args[2:], bt.scale, max_rows=rows)
    graphs, got = [], []
    for _ in range(2):
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        w = torch.zeros_like(want[2])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            swa.paged_attend(bt.q, *bt.args, bt.scale, max_rows=rows, out=o, lse=l)
            swa.paged_weigh(bt.q, l, bt.k, *bt.args[2:], bt.scale, max_rows=rows, out=w)
        graphs.append(g)
        got.append((o, l, w))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, l, w in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1]) and torch.equal(w, want[2])


def test_layer_steps_with_a_budget():
    """A prompt chunk, then decode steps: append, attend, weigh, and an eviction whenever
    the cache passes its budget, against the same steps in float64 on the values the cache
    holds."""
    B, nh, nk, hd, page, rot = 2, 4, 2, 64, 16, 32
    budget, slack = 48, 4
    cap_pages = 5
    g = torch.Generator().manual_seed(41)
    ck = torch.full((B * cap_pages, nk, page, hd), float("nan"), dtype=BF, device="cuda")
    cv = ck.clone()
    table = torch.randperm(B * cap_pages, generator=g).view(B, cap_pages).to(torch.int32)
    cap = cap_pages * page
    weight = torch.zeros(B, nk, cap, device="cuda")
    slot_pos = torch.full((B, nk, cap), -1, dtype=torch.int32, device="cuda")
    turns, freqs = swa.rotary_turns(rot), swa.rotary_freqs(rot).numpy()
    lens, seen = [0, 0], [0, 0]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    evictions = 0
    for step in range(12):
        t = [60, 37] if step == 0 else [1, 1]
        T = sum(t)
        start = [0, t[0], T]
        lens = [n + x for n, x in zip(lens, t)]
        pos = torch.tensor(sum([list(range(seen[b], seen[b] + t[b])) for b in range(B)], []), dtype=torch.int32)
        seen = [n + x for n, x in zip(seen, t)]
        x = torch.randn(T, (nh + 2 * nk) * hd, generator=g)
        q = x[:, :nh * hd].view(T, nh, hd).cuda()
        k = x[:, nh * hd:(nh + nk) * hd].unflatten(1, (nk, hd)).cuda()
        v = x[:, (nh + nk) * hd:].unflatten(1, (nk, hd)).cuda()
        shared = (table.cuda(), dev(start), dev(lens))
        qr = swa.paged_append(k, v, pos.cuda(), ck, cv, *shared, q=q, turns=turns, slot_pos=slot_pos, weight=weight,
                              err=err)
        lse = torch.empty(T, nh, device="cuda")
        out = swa.paged_attend(qr, ck, cv, *shared, hd ** -0.5, max_rows=max(t), lse=lse, err=err)
        swa.paged_weigh(qr, lse, ck, *shared, hd ** -0.5, max_rows=max(t), weight=weight, out=weight, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        wq = po.rotary(f64(q), pos.numpy(), freqs)
        # f32 rotation (2^-21 of |u| + |v| <= 2 max|x|), then one rounding
        assert (np.abs(f64(qr) - wq) <= 2.0 ** -20 * np.abs(f64(q)).max() + unit(BF) * np.abs(wq)).all()
        ro, rl, av, sa = po.attend(f64(qr), f64(ck), f64(cv), table.numpy(), start, lens, hd ** -0.5)
        d = hd * 2.0 ** -24 * sa[..., None]
        tol = (unit(BF) + 2 * (d + 2.0 ** -19) + max(lens) * 2.0 ** -24) * av + unit(BF) * np.abs(ro)
        assert (np.abs(f64(out) - ro) <= tol).all()
        # every row and head has given its weight of one, less what was evicted
        if evictions == 0:
            total = f64(weight).sum(-1)
            np.testing.assert_allclose(total, np.array([[n * nh // nk] * nk for n in seen]), rtol=1e-4)
        if max(lens) > budget + slack:
            recent = dev([n - 8 for n in seen])
            n2, weight, slot_pos = swa.paged_evict(ck, cv, shared[0], shared[2], weight, slot_pos, budget,
                                                   recent_from=recent, sinks=2, err=err)
            lens = n2.tolist()
            evictions += 1
            for b in range(B):
                if seen[b] > budget:
                    for h in range(nk):
                        held = set(slot_pos[b, h, :lens[b]].tolist())
                        assert len(held) == lens[b]
                        assert {0, 1} <= held and set(range(seen[b] - 8, seen[b])) <= held
    assert evictions >= 2
