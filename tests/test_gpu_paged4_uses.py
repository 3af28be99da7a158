"""Uses of the 4-bit paged cache and of the page calls that their documentation allows, next to the
plain ones of test_gpu_paged4.py: a whole run of them, captured steps whose caches grow under them,
calls from several host threads, pools past 2^32 bytes, tables far wider than the lengths. Tolerances
are those derived there."""
import threading

import numpy as np
import pytest
import torch

from oracle import paged4_oracle as p4
from sliding_window_gqa_prep_gb300 import _abi
import sliding_window_gqa_prep_gb300 as swa
from test_gpu_paged4 import BF, E4, HF, U8, Batch4, bits, dev, f64, zero

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test collected on a machine without a GPU")
    yield


def cache4(pages, nk, page, hd):
    """Empty pools: codes anything, scales NaN."""
    return [x for _ in range(2) for x in (torch.full((pages, nk, page, hd // 2), 0x5a, dtype=U8, device="cuda"),
                                          torch.full((pages, nk, page, hd // 16), 127, dtype=U8, device="cuda").view(E4))]


class Request:
    """What a test's program knows of a sequence: its keys and values as they were stored."""

    def __init__(self, k=None, v=None):
        self.k, self.v = list(k or []), list(v or [])

    def copy(self):
        return Request(self.k, self.v)


@pytest.mark.parametrize("hd,window,sinks", [(64, 0, 0), (128, 24, 2), (256, 0, 0)])
def test_a_run_of_prompts_branches_and_compaction(hd, window, sinks):
    """Prompts enter, branch, decode, end and begin; pages are shared, copied, freed and moved. After every
    step the attention and what is read back are those of the sequences' own keys."""
    nh, nk, page, width, pages = 4, 2, 16, 8, 40
    exps = {"exp_k": 0, "exp_v": -2}
    rng, g = np.random.default_rng(hd), torch.Generator().manual_seed(hd)
    pools = cache4(pages, nk, page, hd)
    turns = swa.rotary_turns(hd)
    table, lens, refs = dev(np.full((2, width), -1)), dev([0, 0]), dev([0] * pages)
    seqs = [Request(), Request()]

    def step(parent, rows):
        """The next batch: sequences of `parent`, and `rows` new rows for each."""
        nonlocal table, lens, refs, seqs
        err = zero()
        table, lens, refs, left = swa.paged_fork(pools, table, lens, refs, dev(parent), page, room=dev(rows), err=err)
        assert left.item() >= 0 and int(err.item()) == 0
        assert left.item() == int((refs == 0).sum())
        seqs = [seqs[p].copy() if p >= 0 else Request() for p in parent]
        assert lens.tolist() == [len(x.k) for x in seqs]
        lens = lens + dev(rows)
        T = sum(rows)
        x = torch.randn(T, nh + 2 * nk, hd, generator=g).to(BF)
        pos = dev([len(s.k) + i for s, r in zip(seqs, rows) for i in range(r)])
        start = dev(np.concatenate([[0], np.cumsum(rows)]))
        cache = (*pools, table, start, lens)
        xc = x.cuda()
        q = swa.paged4_append(xc[:, nh:nh + nk], xc[:, nh + nk:], pos, *cache, q=xc[:, :nh], turns=turns, err=err, **exps)
        k, v = swa.paged4_read(*cache, T=T, err=err, **exps)
        at = 0
        for s, r in zip(seqs, rows):
            s.k += list(f64(k[at:at + r]))
            s.v += list(f64(v[at:at + r]))
            at += r
        # what was stored is near what entered: half a step of the largest of 16, and the scale's rounding
        assert (np.abs(f64(v) - f64(x[:, nh + nk:])) <= np.abs(f64(x[:, nh + nk:])).max() * (1 / 6 + 1 / 16)).all()
        check(q, start, rows, err)

    def check(q, start, rows, err):
        cache = (*pools, table, start, lens)
        lse = torch.empty(q.shape[0], nh, device="cuda")
        out = swa.paged4_attend(q, *cache, hd ** -0.5, max_rows=max(rows), window=window, sinks=sinks, lse=lse, err=err, **exps)
        whole = dev(np.concatenate([[0], np.cumsum(lens.tolist())]))
        k, v = swa.paged4_read(*pools, table, whole, lens, T=int(whole[-1].item()), err=err, **exps)
        assert int(err.item()) == 0
        at, row = 0, 0
        for s, r in zip(seqs, rows):
            n = len(s.k)
            assert (f64(k[at:at + n]) == np.array(s.k).reshape(n, nk, hd)).all()
            assert (f64(v[at:at + n]) == np.array(s.v).reshape(n, nk, hd)).all()
            for i in range(r):
                see = p4.visible(n, n - r + i, window, sinks)
                for h in range(nh):
                    kk, vv = np.array(s.k)[see, h // (nh // nk)], np.array(s.v)[see, h // (nh // nk)]
                    x = kk @ f64(q[row, h]) * hd ** -0.5
                    p = np.exp(x - x.max())
                    ref, av = p @ vv / p.sum(), p @ np.abs(vv) / p.sum()
                    d = hd * 2.0 ** -24 * (np.abs(kk) @ np.abs(f64(q[row, h]))).max() * hd ** -0.5
                    tol = (2.0 ** -11 + 2 * (d + 2.0 ** -19) + n * 2.0 ** -24) * av + n * 2.0 ** -36 * np.abs(vv).max() + 2.0 ** -8 * np.abs(ref)
                    assert (np.abs(f64(out[row, h]) - ref) <= tol + 1e-30).all()
                row += 1
            at += n

    step([0, 1], [37, 20])                                   # prompts
    step([0, 0, 1, 1], [1, 1, 1, 1])                         # branches: pages in common, the last one copied
    step([2, 0, 0, 3], [1, 1, 1, 1])                         # beams change places, one ends
    step([0, 1, 2, -1, 3], [3, 1, 2, 40, 1])                 # a prompt beside drafts and decode tokens
    step([0, 4, 3], [1, 5, 1])
    moved = swa.paged_compact(pools, table, refs)            # pages in use to the front
    table, refs = moved[0], moved[1]
    used = moved[3].item()
    assert int((refs[:used] > 0).sum()) == used and not refs[used:].any()
    pools = [x[:used + 8].contiguous() for x in pools]       # most of the rest is given back
    refs, pages = refs[:used + 8].contiguous(), used + 8
    step([0, 1, 2, 2], [1, 1, 1, 17])
    step([3, 0], [1, 1])


@pytest.mark.parametrize("hd,nh,nk", [(64, 4, 2), (128, 32, 8), (256, 8, 2)])
def test_a_captured_step_over_growing_caches(hd, nh, nk):
    """One graph of append, attend and a fork that gives room, replayed while lengths grow inside a table made
    for the longest: what the calls give one at a time, from a length of one on, across tiles and pages."""
    B, page, max_pages, pages = 3, 32, 40, 130
    g = torch.Generator().manual_seed(61)
    start, turns = dev(range(B + 1)), swa.rotary_turns(hd)
    x = torch.zeros(B, nh + 2 * nk, hd, dtype=BF, device="cuda")
    pos, parent, room = dev([0] * B), dev(range(B)), dev([1] * B)

    def state():
        return dict(pools=cache4(pages, nk, page, hd), table=dev(np.full((B, max_pages), -1)), other=dev(np.full((B, max_pages), -1)),
                    lens=dev([0] * B), refs=dev([0] * pages), left=dev([0]), out=torch.zeros(B, nh, hd, dtype=BF, device="cuda"),
                    lse=torch.zeros(B, nh, device="cuda"), same=dev([0] * B), err=zero())

    def step(s):
        # counts in place; the new table is made beside the old one and copied back
        swa.paged_fork(s["pools"], s["table"], s["lens"], s["refs"], parent, page, room=room, table_out=s["other"], lens_out=s["same"],
                       refs_out=s["refs"], left=s["left"], err=s["err"])
        s["table"].copy_(s["other"])
        s["lens"].add_(1)
        cache = (*s["pools"], s["table"], start, s["lens"])
        q = swa.paged4_append(x[:, nh:nh + nk], x[:, nh + nk:], pos, *cache, q=x[:, :nh], turns=turns, err=s["err"])
        swa.paged4_attend(q, *cache, hd ** -0.5, max_rows=1, out=s["out"], lse=s["lse"], err=s["err"])
    a, b, warm = state(), state(), state()
    step(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    assert not b["out"].any()                                # the capture ran nothing
    for it in range(150):
        x.copy_(torch.randn(B, nh + 2 * nk, hd, generator=g).to(BF))
        pos.fill_(it)
        torch.cuda.synchronize()
        step(a)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("out", "lse", "table", "refs", "lens", "left"):
            assert torch.equal(a[name], b[name]), (it, name)
    assert int(a["err"].item()) == 0 and int(b["err"].item()) == 0 and a["lens"].tolist() == [150] * B
    assert int(a["refs"].sum()) == B * 5 and a["left"].item() == pages - 15
    for y, z in zip(a["pools"], b["pools"]):
        assert torch.equal(y.view(U8), z.view(U8))


def test_calls_from_several_threads():
    """Host threads with a stream each, their first calls at the same time: the bits of the calls
    alone."""
    kinds = [dict(t=[1, 1], lens=[900, 1300], nh=8, nk=2, hd=64, page=16), dict(t=[90, 3], lens=[900, 300], nh=8, nk=2, hd=64, page=32),
             dict(t=[1, 1], lens=[700, 90], nh=8, nk=2, hd=256, page=64, window=100, sinks=3), dict(t=[70], lens=[700], nh=4, nk=2, hd=128, page=64)]
    batches = [Batch4(dtype=dt, seed=62 + i, **kw) for i, kw in enumerate(kinds) for dt in (BF, HF)]
    torch.cuda.synchronize()
    got, faults = [None] * len(batches), []
    gate = threading.Barrier(len(batches))

    def work(i):
        try:
            bt, s = batches[i], torch.cuda.Stream()
            gate.wait(60)
            for _ in range(20):
                lse = torch.empty(bt.T, bt.nh, device="cuda")
                s.wait_stream(torch.cuda.current_stream())
                o = swa.paged4_attend(bt.q, *bt.args, bt.scale, max_rows=max(bt.t), lse=lse, stream=s, **bt.mask)
                k, v = swa.paged4_read(*bt.args, T=bt.T, stream=s)
                f = swa.paged_fork([bt.k], bt.args[4], bt.args[6], dev([1] * bt.k.shape[0]), dev([0]), bt.page, stream=s)
                s.synchronize()
                if got[i] is None:
                    got[i] = (o, lse, k.view(torch.int16), v.view(torch.int16), *f)
                assert all(torch.equal(a, b) for a, b in zip(got[i], (o, lse, k.view(torch.int16), v.view(torch.int16), *f)))
        except BaseException as e:                           # noqa: BLE001 (told to the test's thread)
            faults.append((i, repr(e)))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(batches))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not faults, faults
    for bt, (o, lse, *_) in zip(batches, got):
        o1, l1, err = bt.attend()
        assert err == 0 and torch.equal(o, o1) and torch.equal(lse, l1)


@pytest.mark.parametrize("rows", [1, 40])
def test_pools_past_32_bits(rows):
    """Pages whose bytes lie past 2^32 in the codes: written, read and attended like the first ones, and
    copied by a fork and a compaction."""
    nk, page, hd, nh = 2, 256, 256, 8
    pages = (1 << 32) // (nk * page * hd // 2) + 40          # 4.3 GB of codes, twice
    pools = [x for _ in range(2) for x in (torch.zeros(pages, nk, page, hd // 2, dtype=U8, device="cuda"),
                                           torch.zeros(pages, nk, page, hd // 16, dtype=U8, device="cuda").view(E4))]
    n = 700
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(n, nk, hd, generator=g).to(BF).cuda() for _ in range(2))
    q = torch.randn(rows, nh, hd, generator=g).to(BF).cuda()
    got = []
    for table in ([[0, 1, 2]], [[pages - 1, pages - 3, pages - 2]]):
        where = (dev(table), dev([0, n]), dev([n]))
        swa.paged4_append(k, v, None, *pools, *where)
        a, b = swa.paged4_read(*pools, *where, T=n)
        got.append((a, b, swa.paged4_attend(q, *pools, where[0], dev([0, rows]), where[2], hd ** -0.5, max_rows=rows)))
    assert all(torch.equal(x, y) for x, y in zip(*got)) and got[0][0].abs().sum() > 0
    # the first three pages still hold it; 4 sequences of a table whose last page is copied to the lowest free ones
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[pages - 3:] = 1
    out, lens, refs2, left = swa.paged_fork(pools, dev([[pages - 1, pages - 3, pages - 2]]), dev([n]), refs, dev([0, 0]), page, room=dev([1, 1]))
    assert out.tolist() == [[pages - 1, pages - 3, pages - 2], [pages - 1, pages - 3, 0]] and left.item() == pages - 4
    c, used = swa.paged_compact(pools, out, refs2)[0], 4
    assert int(c.max()) < used
    a, b = swa.paged4_read(*pools, c, dev([0, n, 2 * n]), dev([n, n]), T=2 * n)
    assert torch.equal(a[:n], got[0][0]) and torch.equal(a[n:], got[0][0]) and torch.equal(b[n:], got[0][1])


@pytest.mark.parametrize("kw", [dict(t=[1, 1, 2], lens=[300, 1, 90], nh=8, nk=2, hd=128, page=16),
                                dict(t=[1], lens=[260], nh=32, nk=1, hd=256, page=64),        # one token of 32 heads: the chunk kernel
                                dict(t=[100, 1], lens=[300, 40], nh=4, nk=2, hd=64, page=32, window=60, sinks=5)])
def test_tables_far_wider_than_the_lengths(kw):
    """Rows in front of the first sequence and behind the last one, and a table of many more pages than are
    held: neither is touched."""
    bt = Batch4(seed=17, **kw)
    ref = bt.oracle()
    wide = torch.full((len(bt.t), 3000), -1, dtype=torch.int32, device="cuda")
    wide[:, :bt.max_pages] = bt.args[4]
    out, lse, err = bt.attend(args=(*bt.pools, wide, *bt.args[5:]))
    assert err == 0
    bt.check(out, lse, ref)
    q = torch.cat((torch.full_like(bt.q[:1], float("nan")), bt.q))
    o, l = torch.full((bt.T + 1, bt.nh, bt.hd), 5.0, dtype=BF, device="cuda"), torch.full((bt.T + 1, bt.nh), 77.0, device="cuda")
    swa.paged4_attend(q, *bt.pools, wide, bt.args[5] + 1, bt.args[6], bt.scale, max_rows=max(bt.t), out=o, lse=l, **bt.mask)
    assert (o[0] == 5.0).all() and (l[0] == 77.0).all()
    bt.check(o[1:], l[1:], ref)


def test_many_sequences_a_call():
    """More sequences than threads of a block, and than the chunk kernel sorts; some without rows."""
    rng = np.random.default_rng(4)
    for t in ([1] * 400, [int(x) for x in rng.integers(0, 3, 300)], [int(x) for x in rng.choice([0, 1, 70], 80)]):
        lens = [int(max(a, x)) for a, x in zip(t, rng.integers(1, 120, len(t)))]
        bt = Batch4(t=t, lens=lens, nh=2, nk=1, hd=64, page=16, seed=18)
        out, lse, err = bt.attend()
        assert err == 0
        bt.check(out, lse)


def test_scores_of_one_key_above_all_others():
    """Rows whose maximum comes late and rises far: the running maximum is raised in the last tiles, by more than
    weights may grow."""
    for kw in (dict(t=[1, 1], lens=[2000, 700], nh=8, nk=2, hd=128, page=16), dict(t=[140], lens=[900], nh=2, nk=1, hd=128, page=64),
               dict(t=[3], lens=[1500], nh=4, nk=1, hd=256, page=32), dict(t=[130], lens=[500], nh=2, nk=1, hd=256, page=32)):
        bt = Batch4(seed=19, sharp=12.0, **kw)
        ks = bt.ks.view(U8)
        for b in range(len(bt.t)):                           # scales rise along the sequence
            for j in range(bt.n[b]):
                ks[int(bt.table[b, j // bt.page]), :, j % bt.page] = 40 + 30 * j // bt.n[b]
        out, lse, err = bt.attend()
        assert err == 0
        bt.check(out, lse)


@pytest.mark.parametrize("hd,rot,interleaved", [(64, 64, False), (64, 10, True), (128, 128, False), (128, 44, False), (256, 256, False), (256, 20, False)])
@pytest.mark.parametrize("T", [3, 700])
def test_queries_rotated_in_place(hd, rot, interleaved, T):
    """q_out may be q: the same bits as apart, partners in the lane, in another one and in two."""
    bt = Batch4(t=[T], lens=[T + 5], nh=10, nk=2, hd=hd, page=16)
    k = torch.randn(T, 2, hd, device="cuda").to(BF)
    kw = dict(turns=swa.rotary_turns(rot), interleaved=interleaved)
    pos = dev(range(5, T + 5))
    apart = swa.paged4_append(k, k, pos, *bt.args, q=bt.q, **kw)
    own = bt.q.clone()
    assert swa.paged4_append(k, k, pos, *bt.args, q=own, q_out=own, **kw) is own
    assert torch.equal(own, apart) and not torch.equal(own, bt.q)


def test_calls_without_rows():
    """No rows: nothing is launched and nothing changes, in eager calls and in a captured one."""
    bt = Batch4(t=[0, 0], lens=[5, 0], nh=4, nk=2, hd=64, page=16)
    none, q = torch.empty(0, 2, 64, dtype=BF, device="cuda"), torch.empty(0, 4, 64, dtype=BF, device="cuda")
    before, err = [y.clone() for y in (bt.k, bt.ks.view(U8))], zero()

    def calls():
        return (swa.paged4_append(none, none, None, *bt.args, q=q, err=err), *swa.paged4_read(*bt.args, T=0, err=err),
                swa.paged4_attend(q, *bt.args, 0.1, max_rows=1, err=err))
    assert [y.shape[0] for y in calls()] == [0] * 4
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    graph.replay()
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(before[0], bt.k) and torch.equal(before[1], bt.ks.view(U8))
    out, lens, refs, left = swa.paged_fork([], bt.args[4], dev([5, 0]), dev([1] * bt.k.shape[0]), dev([-1]), 16)     # no pools: the tables alone
    assert out.tolist() == [[-1] * bt.max_pages] and lens.tolist() == [0] and left.item() == int((refs == 0).sum())


def test_refusals_of_the_binding():
    bt = Batch4(t=[2], lens=[20], nh=4, nk=2, hd=64, page=16)
    x = torch.randn(2, 2, 64, device="cuda").to(BF)
    bad = [lambda: swa.paged4_append(x, x[:1], None, *bt.args), lambda: swa.paged4_append(x.double(), x.double(), None, *bt.args),
           lambda: swa.paged4_append(x, x, None, *bt.args, q=bt.q, q_out=torch.empty_like(bt.q).float()),
           lambda: swa.paged4_append(x, x, None, *bt.args, q_out=torch.empty_like(bt.q)),
           lambda: swa.paged4_append(x, x, torch.zeros(2, dtype=torch.int32), *bt.args, turns=swa.rotary_turns(64)),
           lambda: swa.paged4_read(*bt.args), lambda: swa.paged4_read(*bt.args, k_out=x, T=3), lambda: swa.paged4_read(*bt.args, k_out=x, v_out=x.float()),
           lambda: swa.paged4_attend(bt.q.float(), *bt.args, 0.1, max_rows=2), lambda: swa.paged4_attend(bt.q[0], *bt.args, 0.1, max_rows=2),
           lambda: swa.paged4_attend(bt.q, bt.k, bt.ks.view(U8), *bt.args[2:], 0.1, max_rows=2),
           lambda: swa.paged4_attend(bt.q, *bt.args, 0.1, max_rows=2, out=bt.q[:1]),
           lambda: swa.paged_fork([bt.k], bt.args[4], bt.args[6], dev([0] * 3), dev([0]), 16),
           lambda: swa.paged_fork([bt.k.cpu()], bt.args[4], bt.args[6], dev([1] * bt.k.shape[0]), dev([0]), 16),
           lambda: swa.paged_compact([bt.k], bt.args[4].long(), dev([1] * bt.k.shape[0]))]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: swa.paged4_attend(bt.q, *bt.args, 0.1, max_rows=2, window=-1), lambda: swa.paged4_attend(bt.q, *bt.args, -0.1, max_rows=2),
              lambda: swa.paged4_append(x, x, None, *bt.args, exp_k=40), lambda: swa.paged4_read(*bt.args, T=2, exp_v=-40),
              lambda: swa.paged4_append(x, x, None, bt.k, bt.ks, bt.k, bt.ks, *bt.args[4:]),
              lambda: swa.paged_fork([bt.k], bt.args[4], bt.args[6], dev([1] * bt.k.shape[0]), dev([0]), 24),
              lambda: swa.paged_fork([bt.k], bt.args[4], bt.args[6], dev([1] * bt.k.shape[0]), dev([0]), 16, table_out=bt.args[4]),
              lambda: swa.paged_fork([bt.k, bt.k], bt.args[4], bt.args[6], dev([1] * bt.k.shape[0]), dev([0]), 16)):
        with pytest.raises(swa.SwaError) as e:
            f()
        assert e.value.status == _abi.SWA_E_SHAPE
