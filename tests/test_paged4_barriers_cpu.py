"""The barriers of the 4-bit attention kernels as a model, run in random orders (see
test_paged_barriers_cpu.py): a wait that ends must end on the phase it meant, a slot must hold what
its user expects, every role ends. Ring sizes and arrival counts are read from the kernels' source.
Two protocols that are known to be wrong have to fail: scores exchanged in one place, and, at two S buffers, no wait for
the last but one value product."""
import random
import re

import pytest

from test_paged_barriers_cpu import Alias, Bar, arrivals, constant, run_all, some_steps, source, split_run, wait


def test_split_kernel():
    text = source("swa_paged4.cu")
    assert arrivals(text) == {"b_full": "1", "b_empty": "kWarps4"}
    assert "kWarps4 = 4;" in text and re.search(r"ST = FIT < 8 \? FIT : 8;", text)
    for seed in range(60):
        rng = random.Random(seed)
        split_run(rng.randint(2, 8), 4, rng.randint(0, 30), seed)


def exchange_run(rounds, buffers, seed):
    """Two warps that add their parts of scores up: each writes its own, meets the other at a named barrier
    and reads the other's; `buffers` rounds have a place of their own."""
    rng, met = random.Random(seed), [0, 0]
    place = [[None] * buffers for _ in range(2)]

    def warp(w):
        for i in range(rounds):
            yield from some_steps(rng, 4)
            place[w][i % buffers] = i
            met[w] = i + 1
            while met[1 - w] < i + 1:
                yield
            yield from some_steps(rng, 4)
            assert place[1 - w][i % buffers] == i
    run_all([warp(0), warp(1)], rng)


def test_exchange_of_scores():
    text = source("swa_paged4.cu")
    assert "XB = FS > 1 ? 2 * kWarps4 * G * NV * 512" in text and "turn ^= kWarps4 * G * NV * 512;" in text
    for seed in range(100):
        exchange_run(20, 2, seed)
    with pytest.raises(AssertionError):
        for seed in range(100):
            exchange_run(20, 1, seed)


def chunk_run(NT, SB, RK, RV, mine, seed, last_but_one=True):
    """mine: key tiles that each query tile sees; the CTA's share n has the larger of them. With two query
    tiles their softmax warps convert (V: the first's, K: the second's), else warps of their own."""
    rng, n = random.Random(seed), max(mine)
    own = NT == 2
    raw, free = [Bar(1) for _ in range(RK + RV)], [Bar(1) for _ in range(RK + RV)]     # 4 warps: 1 here
    full, empty = [Bar(1) for _ in range(4)], [Bar(NT) for _ in range(4)]
    q = [Bar(1) for _ in range(NT)]
    s = [Bar(1) for _ in range(NT * SB)]
    p = [[Bar(1), Bar(1)] for _ in range(NT * SB)]
    pv, turn = [Bar(1) for _ in range(NT)], [Bar(1) for _ in range(NT)]
    codes, held = [None] * (RK + RV), [None] * 4

    def in_order():
        for x in range(-2, n):
            if x >= -1 and x + 1 < n:
                yield x + 1, True
            if x + 2 < n:
                yield x + 2, False

    def raw_of(x, is_v):
        """(slot, use): K's and V's own rings where different warps convert them, else one"""
        if not own:
            return (2 * x + is_v) % (RK + RV), (2 * x + is_v) // (RK + RV)
        return (RK + x % RV, x // RV) if is_v else (x % RK, x // RK)

    def loader():
        for x, is_v in in_order():
            slot, use = raw_of(x, is_v)
            if use > 0:
                yield from wait(free[slot], use - 1)
            codes[slot] = (x, is_v)
            yield from some_steps(rng, 5)
            raw[slot].arrive()

    def convert(x, is_v):
        r, use = raw_of(x, is_v)
        slot = (2 if is_v else 0) + (x & 1)
        yield from wait(raw[r], use)
        if x >= 2:
            yield from wait(empty[slot], (x >> 1) - 1)
        assert codes[r] == (x, is_v)
        yield from some_steps(rng, 6)
        assert codes[r] == (x, is_v)
        held[slot] = (x, is_v)
        free[r].arrive()
        full[slot].arrive()

    def converter():
        for x, is_v in in_order():
            yield from convert(x, is_v)

    def issuer(t):
        m, other = mine[t], mine[1 - t] if NT == 2 else 0

        def pass_turn():
            if NT == 2:
                turn[1 - t].arrive()

        def s_mma(j):
            yield from wait(full[j & 1], j >> 1)
            assert held[j & 1] == (j, False)
            if j > 0:
                pass_turn()
            s[t * SB + j % SB].arrive()

        def pv_mma(j):
            slot = 2 + (j & 1)
            yield from wait(full[slot], j >> 1)
            if NT == 2:
                if t == 0:
                    if j > 0 and other > 0:
                        yield from wait(turn[0], j - 1)
                elif j < other:
                    yield from wait(turn[1], j)
            for h in range(2):
                yield from wait(p[t * SB + j % SB][h], j // SB)
                assert held[slot] == (j, True)
                if h == 1 and j + 1 == m:
                    pass_turn()
                if h == 1:
                    pv[t].arrive()
                if h == 0:
                    empty[j & 1].arrive()

        def pv_done(j):
            yield from wait(pv[t], j)
            empty[2 + (j & 1)].arrive()
        if m > 0:
            yield from wait(q[t], 0)
            yield from s_mma(0)
        for j in range(m):
            if SB == 2 and j > 0:
                yield from pv_done(j - 1)
            if SB == 2 and j + 1 < m:
                yield from s_mma(j + 1)
            yield from pv_mma(j)
            if SB == 1:
                yield from pv_done(j)
                if j + 1 < m:
                    yield from s_mma(j + 1)
        for j in range(m, n):                               # the other tile's keys
            for slot in (j & 1, 2 + (j & 1)):
                yield from wait(full[slot], j >> 1)
                empty[slot].arrive()

    def softmax(t):
        m, ahead = mine[t], 1 if t == 0 else 2
        if m > 0:
            yield from some_steps(rng, 5)
            q[t].arrive()
        if own:
            for x in range(min(ahead, n)):
                yield from convert(x, t == 0)
        for j in range(m):
            yield from wait(s[t * SB + j % SB], j // SB)
            if j > 0 and SB == 2 and rng.random() < 0.4:    # the maximum is raised
                yield from wait(pv[t], j - 1)
            for h in range(2):
                yield from some_steps(rng, 6)
                if last_but_one and SB == 2 and h == 1 and j > 0 and j == m - 1:
                    yield from wait(pv[t], j - 1)
                p[t * SB + j % SB][h].arrive()
            if own and j + ahead < n:
                yield from convert(j + ahead, t == 0)
        if own:
            for x in range(m + ahead, n):
                yield from convert(x, t == 0)
        if m > 0:
            yield from wait(pv[t], m - 1)
    roles = [loader()] + [issuer(t) for t in range(NT)] + [softmax(t) for t in range(NT)]
    run_all(roles + ([] if own else [converter()]), rng)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_kernel(D):
    text, base = source("swa_paged4_chunk.cuh"), source("swa_paged_chunk.cu")
    assert "NT = ChunkCfg<D>::NT, SB = ChunkCfg<D>::SB" in text and "OWN = NT == 2;" in text
    NT, SB = (constant(base, x, D) for x in ("NT", "SB"))
    RK, RV = (constant(text, x, D) for x in ("RK", "RV"))
    assert arrivals(text) == {"b_raw": "1", "b_free": "C::CW", "b_full": "C::CW", "b_empty": "NT", "b_q": "128", "b_pv": "1", "b_fin": "1",
                              "b_turn": "1", "b_s": "1", "b_p": "128"}
    rng = random.Random(D)
    for seed in range(400):
        a = rng.randint(0, 12)
        # the second query tile's rows come later: they see as many keys or more, or there are none
        chunk_run(NT, SB, RK, RV, [a] if NT == 1 else [a, rng.choice([0, a, a + 1, a + 2])], seed)


def test_chunk_kernel_needs_its_wait_for_the_last_but_one_product():
    with pytest.raises(Alias):
        for seed in range(400):
            chunk_run(1, 2, 2, 1, [random.Random(seed).randint(0, 12)], seed, last_but_one=False)


def test_register_shares_of_the_chunk_kernel_are_checked():
    """As for the 16-bit kernel: the shares that setmaxnreg hands out stand against the launch's."""
    text = source("swa_paged4_chunk.cuh")
    assert re.search(r"static_assert\(NT \* 128 \* R_SOFT \+ \(THREADS - NT \* 128\) \* R_REST <= THREADS \* REGS", text)
    assert "regs_give<C::R_REST>()" in text and "regs_take<C::R_SOFT>()" in text
    assert re.search(r"allow_smem<paged4_chunk_kernel<D>>\([^;]*Chunk4Cfg<D>::REGS\)", text)


def test_tensor_memory_is_allocated_after_the_wait():
    text = source("swa_paged4_chunk.cuh")
    assert 0 <= text.find("pdl_wait();") < text.find("tc_alloc(")
