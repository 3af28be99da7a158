"""Uses of the paged calls that their documentation allows, next to the plain ones of
test_gpu_paged.py: captured steps whose caches grow under them, calls from several host threads,
rows in front of the first sequence, tables far wider than the lengths, groups of heads that send
single tokens to the tensor cores. Tolerances are those derived there."""
import threading

import numpy as np
import pytest
import torch

from oracle import paged_oracle as po
import sliding_window_gqa_prep_gb300 as swa
from test_gpu_paged import BF, HF, Batch, dev, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test collected on a machine without a GPU")
    yield


@pytest.mark.parametrize("hd,nh,nk", [(64, 4, 2), (128, 32, 8), (256, 8, 2)])
def test_a_captured_step_over_growing_caches(hd, nh, nk):
    """One graph of append, attend and weigh, replayed while lengths grow inside a table made for the
    longest: what the calls give one at a time, from a length of one on, across tiles and pages."""
    B, page, max_pages = 3, 32, 40
    g = torch.Generator().manual_seed(61)
    pool = lambda: torch.full((B * max_pages, nk, page, hd), float("nan"), dtype=BF, device="cuda")
    table = torch.randperm(B * max_pages, generator=g).view(B, max_pages).to(torch.int32).cuda()
    start, turns = dev(range(B + 1)), swa.rotary_turns(hd)
    x = torch.zeros(B, nh + 2 * nk, hd, dtype=BF, device="cuda")
    lens, pos = dev([0] * B), dev([0] * B)
    cap = max_pages * page

    def state():
        return dict(k=pool(), v=pool(), out=torch.zeros(B, nh, hd, dtype=BF, device="cuda"),
                    lse=torch.zeros(B, nh, device="cuda"), w=torch.zeros(B, nk, cap, device="cuda"),
                    err=torch.zeros(1, dtype=torch.int32, device="cuda"))

    def step(s):
        cache = (s["k"], s["v"], table, start, lens)
        q = swa.paged_append(x[:, nh:nh + nk], x[:, nh + nk:], pos, *cache, q=x[:, :nh], turns=turns, weight=s["w"], err=s["err"])
        swa.paged_attend(q, *cache, hd ** -0.5, max_rows=1, out=s["out"], lse=s["lse"], err=s["err"])
        swa.paged_weigh(q, s["lse"], s["k"], table, start, lens, hd ** -0.5, max_rows=1, weight=s["w"], out=s["w"], err=s["err"])
    a, b = state(), state()
    warm = state()
    lens.fill_(1)
    step(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for s in (b,):                                           # the capture ran nothing
        assert not s["out"].any()
    held = [0, 600, 1100]
    # the longer ones hold something already
    fill_k, fill_v = (torch.randn(B * max_pages, nk, page, hd, generator=g).to(BF) for _ in range(2))
    for s in (a, b):
        for i, n in enumerate(held):
            for j in range(-(-n // page)):
                p, m = int(table[i, j]), min(page, n - j * page)
                s["k"][p, :, :m], s["v"][p, :, :m] = fill_k[p, :, :m].cuda(), fill_v[p, :, :m].cuda()
    for it in range(70):
        x.copy_(torch.randn(B, nh + 2 * nk, hd, generator=g).to(BF))
        held = [n + 1 for n in held]
        lens.copy_(torch.tensor(held, dtype=torch.int32))
        pos.copy_(lens - 1)
        torch.cuda.synchronize()
        step(a)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("out", "lse", "w"):
            assert torch.equal(a[name], b[name]), (it, name)
    assert int(a["err"].item()) == 0 and int(b["err"].item()) == 0
    for name in ("k", "v"):
        assert torch.equal(a[name].nan_to_num(7), b[name].nan_to_num(7))
    # every step's row gave each KV head a weight of one a query head: to the keys it saw
    total = f64(a["w"]).sum(-1)
    np.testing.assert_allclose(total, 70 * nh // nk, rtol=1e-4)


def test_calls_from_several_threads():
    """Host threads with a stream each, their first calls at the same time: the bits of the calls
    alone."""
    kinds = [dict(t=[1, 1], lens=[900, 1300], nh=8, nk=2, hd=64, page=16), dict(t=[90, 3], lens=[900, 300], nh=8, nk=2, hd=64, page=32),
             dict(t=[1, 1], lens=[700, 90], nh=8, nk=2, hd=256, page=64), dict(t=[70], lens=[700], nh=4, nk=2, hd=128, page=64)]
    batches = [Batch(dtype=dt, seed=62 + i, **kw) for i, kw in enumerate(kinds) for dt in (BF, HF)]
    torch.cuda.synchronize()
    got, faults = [None] * len(batches), []
    gate = threading.Barrier(len(batches))

    def work(i):
        try:
            bt, s = batches[i], torch.cuda.Stream()
            gate.wait(60)
            rows = max(bt.t)
            for _ in range(20):
                lse = torch.empty(bt.T, bt.nh, device="cuda")
                s.wait_stream(torch.cuda.current_stream())
                o = swa.paged_attend(bt.q, *bt.args, bt.scale, max_rows=rows, lse=lse, stream=s)
                w = swa.paged_weigh(bt.q, lse, bt.k, *bt.args[2:], bt.scale, max_rows=rows, stream=s)
                s.synchronize()
                if got[i] is None:
                    got[i] = (o, lse, w)
                assert all(torch.equal(a, b) for a, b in zip(got[i], (o, lse, w)))
        except BaseException as e:                           # noqa: BLE001 (told to the test's thread)
            faults.append((i, repr(e)))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(batches))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not faults, faults
    for bt, (o, lse, w) in zip(batches, got):
        o1, l1, err = bt.attend()
        assert err == 0 and torch.equal(o, o1) and torch.equal(lse, l1)


USES = [
    # single tokens of wide groups: the tensor-core kernel with a row a sequence
    dict(t=[1, 1, 1], lens=[1, 700, 65], nh=32, nk=1, hd=256, page=16),
    dict(t=[1] * 70, lens=[(37 * i) % 300 + 1 for i in range(70)], nh=34, nk=2, hd=256, page=32),
    # many KV heads of one query head
    dict(t=[1, 2], lens=[130, 70], nh=96, nk=96, hd=64, page=16),
    dict(t=[40], lens=[100], nh=20, nk=20, hd=128, page=64),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kw", USES)
def test_attend_uses(kw, dtype):
    bt = Batch(dtype=dtype, seed=63, **kw)
    out, lse, err = bt.attend()
    assert err == 0
    bt.check(out, lse)


@pytest.mark.parametrize("wide", [1, 9, 700])
@pytest.mark.parametrize("kw", [
    dict(t=[1, 1], lens=[133, 20], nh=8, nk=2, hd=64, page=16), dict(t=[5, 2], lens=[700, 90], nh=8, nk=2, hd=128, page=32),
    dict(t=[256], lens=[512], nh=8, nk=2, hd=128, page=64), dict(t=[130, 1, 40], lens=[300, 900, 77], nh=8, nk=2, hd=64, page=16),
    dict(t=[50, 1], lens=[300, 500], nh=4, nk=1, hd=256, page=128),
])
def test_wide_tables(kw, wide):
    """A table for many more keys than the sequences hold: entries behind them are not read."""
    bt = Batch(dtype=BF, seed=64, **kw)
    lens = torch.tensor(bt.n)
    table = torch.full((len(bt.t), bt.max_pages * wide), -1, dtype=torch.int32)
    table[:, :bt.max_pages] = bt.table
    for b, n in enumerate(lens.tolist()):
        table[b, -(-n // bt.page):] = -1                     # would be reported
    bt.args = (bt.k, bt.v, table.cuda(), *bt.args[3:])
    out, lse, err = bt.attend()
    assert err == 0
    bt.check(out, lse)
    w = swa.paged_weigh(bt.q, lse, bt.k, *bt.args[2:], bt.scale, max_rows=max(bt.t))
    got = f64(w)
    ref = po.weigh(f64(bt.q), f64(lse), f64(bt.k), bt.table.numpy(), bt.start, bt.n, bt.scale,
                   np.zeros((len(bt.t), bt.nk, bt.cap)))
    # weights of at most a few units each; scores good to hd 2^-24 sum|q k|, see test_weigh
    np.testing.assert_allclose(got[..., :bt.cap], ref, rtol=2.0 ** -12, atol=2.0 ** -20)
    assert not got[..., bt.cap:].any()


@pytest.mark.parametrize("rows", [1, 9, 70])
def test_rows_in_front_of_the_first_sequence(rows):
    """row_start may begin behind row 0: rows in front belong to no sequence, like those behind."""
    bt = Batch(t=[rows, 2], lens=[200, 60], nh=4, nk=2, hd=64, page=16, seed=65, pad=2)
    ref = bt.oracle()
    out, lse, err = bt.attend()
    bt.check(out, lse, ref)
    front = 3
    q = torch.cat((torch.randn(front, 4, 64).to(BF).cuda(), bt.q))
    start = dev([x + front for x in bt.start])
    o = torch.full((bt.T + front, 4, 64), 5.0, dtype=BF, device="cuda")
    l = torch.full((bt.T + front, 4), 77.0, device="cuda")
    args = (*bt.args[:3], start, bt.args[4])
    swa.paged_attend(q, *args, bt.scale, max_rows=rows + 1, out=o, lse=l)
    assert torch.equal(o[front:], out) and torch.equal(l[front:], lse)
    assert (o[:front] == 5.0).all() and (l[:front] == 77.0).all()
    k = torch.randn(bt.T + front, 2, 64, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    a, b = [(bt.k.clone(), bt.v.clone()) for _ in range(2)]
    qa, qb = (torch.full((n, 4, 64), 5.0, dtype=BF, device="cuda") for n in (bt.T + front, bt.T))
    swa.paged_append(k, k, None, *a, bt.args[2], start, bt.args[4], q=q, q_out=qa)
    swa.paged_append(k[front:], k[front:], None, *b, *bt.args[2:], q=bt.q, q_out=qb)
    for x, y in zip(a, b):
        assert torch.equal(x.nan_to_num(9), y.nan_to_num(9))
    assert torch.equal(qa[front:], qb) and (qa[:front] == 5.0).all()


def test_weigh_the_last_rows_alone_and_scale_zero():
    """q may hold the last rows of a chunk alone; with scale 0 every key seen gets the same."""
    bt = Batch(t=[60, 20], lens=[300, 150], nh=8, nk=2, hd=128, page=64, seed=66)
    out, lse, _ = bt.attend()
    last = [16, 7]
    pick = torch.cat([torch.arange(bt.start[b + 1] - n, bt.start[b + 1]) for b, n in enumerate(last)]).cuda()
    w = swa.paged_weigh(bt.q[pick].contiguous(), lse[pick].contiguous(), bt.k, bt.args[2], dev([0, 16, 23]), bt.args[4],
                        bt.scale, max_rows=16)
    ref = po.weigh(f64(bt.q[pick]), f64(lse[pick]), f64(bt.k), bt.table.numpy(), [0, 16, 23], bt.n, bt.scale,
                   np.zeros((2, 2, bt.cap)))
    np.testing.assert_allclose(f64(w), ref, rtol=2.0 ** -12, atol=2.0 ** -20)
    bt.scale = 0.0
    out, lse, _ = bt.attend()
    bt.check(out, lse)
    w = f64(swa.paged_weigh(bt.q, lse, bt.k, *bt.args[2:], 0.0, max_rows=60))
    for b in range(2):
        n, t = bt.n[b], bt.t[b]
        seen = np.array([sum(4.0 / (n - t + i + 1) for i in range(t) if j < n - t + i + 1) for j in range(bt.cap)])
        # each weight is 2^(log2 of its share): the f32 lse is good to 2^-24 |lse| + 2^-21
        np.testing.assert_allclose(w[b], np.broadcast_to(seen, w[b].shape), rtol=2.0 ** -18, atol=0)
