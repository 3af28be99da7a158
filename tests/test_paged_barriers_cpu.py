"""The barriers of the paged kernels as a model: every role of a CTA is a coroutine that waits and
arrives as the kernel does, run in random orders.

A wait on a barrier sees only the parity of its phase. One that comes two phases late or early takes
a stale phase for its own, so each role that waits on a barrier has to wait for each of its phases
(or know otherwise that it has passed). `Bar.test` asserts that: a wait that ends must end on the
phase it meant. The model also asserts what a slot holds when it is used, and that every role ends.

Ring sizes and arrival counts are read from the kernels' source, so that a change there without one
here shows up. Two protocols that are known to be wrong have to fail: one ring of K slots shared by
paged_weigh's two issuing warps, and the tensor-core kernel at two S buffers without its wait for the
last but one value product.
"""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sliding_window_gqa_prep_gb300", "csrc")


class Alias(AssertionError):
    pass


class Stuck(AssertionError):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.phase, self.left = count, 0, count

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.phase, self.left = self.phase + 1, self.count

    def test(self, phase):
        ended = (self.phase & 1) != (phase & 1)
        if ended and not self.phase > phase:
            raise Alias((self.phase, phase))
        return ended


def wait(bar, phase):
    while not bar.test(phase):
        yield


def some_steps(rng, most):
    for _ in range(rng.randint(0, most)):
        yield


def run_all(roles, rng, most=300_000):
    live = list(roles)
    for _ in range(most):
        if not live:
            return
        role = rng.choice(live)
        for _ in range(rng.choice([1, 1, 5, 200])):
            try:
                next(role)
            except StopIteration:
                live.remove(role)
                break
    raise Stuck([(r.__name__, r.gi_frame.f_locals) for r in live])


# ------------------------------------------------------------------ constants from the source
def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def constant(text, name, D):
    """`static constexpr int NAME = D == 64 ? 8 : 5` (possibly in a list of them) for a head width."""
    x = re.search(r"\b%s = ([^,;]+)[,;]" % name, text).group(1)
    while "?" in x:
        cond, rest = x.split("?", 1)
        a, b = rest.split(":", 1)
        x = a if eval(cond, {"D": D}) else b
    return int(x)


def arrivals(text):
    return dict(re.findall(r"mbar_init\(&(b_\w+)(?:\[\w+\])*, ([^)]+)\)", text))


# ------------------------------------------------------------------ the split kernel
def split_run(stages, warps, tiles, seed):
    rng = random.Random(seed)
    full, empty = [Bar(1) for _ in range(stages)], [Bar(warps) for _ in range(stages)]
    held = [None] * stages

    def copier():
        for it in range(tiles):
            st = it % stages
            if it >= stages:
                yield from wait(empty[st], it // stages - 1)
            held[st] = it
            yield from some_steps(rng, 5)
            full[st].arrive()

    def products():
        for it in range(tiles):
            st = it % stages
            yield from wait(full[st], it // stages)
            assert held[st] == it
            yield from some_steps(rng, 5)
            assert held[st] == it
            empty[st].arrive()
    run_all([copier()] + [products() for _ in range(warps)], rng)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_split_kernel(D):
    text = source("swa_paged.cu")
    ds = constant(text, "DS", D)
    assert arrivals(text) == {"b_full": "1", "b_empty": "4 * DS"}
    for seed in range(60):
        split_run(constant(text, "ST", D), 4 * ds, random.Random(seed).randint(0, 30), seed)


# ------------------------------------------------------------------ the tensor-core kernel
def pos_k(SB, j):
    return 2 * j if SB == 1 else (0 if j == 0 else 2 * j - 1)


def pos_v(SB, j, n):
    return 2 * j + 1 if SB == 1 else (2 * j + 2 if j < n - 1 else 2 * n - 1)


def chunk_run(NT, SB, NS, mine, seed, last_but_one=True):
    """mine: key tiles that each query tile sees; the CTA's share has the larger of them."""
    rng, n = random.Random(seed), max(mine)
    full, empty = [Bar(1) for _ in range(NS)], [Bar(NT) for _ in range(NS)]
    q = [Bar(1) for _ in range(NT)]                         # 128 threads of a softmax warpgroup: 1 here
    s = [Bar(1) for _ in range(NT * SB)]
    p = [[Bar(1), Bar(1)] for _ in range(NT * SB)]
    pv, turn = [Bar(1) for _ in range(NT)], [Bar(1) for _ in range(NT)]
    held = [None] * NS

    def loader():
        def load(pos, what):
            slot, use = pos % NS, pos // NS
            if use > 0:
                yield from wait(empty[slot], use - 1)
            held[slot] = what
            yield from some_steps(rng, 5)
            full[slot].arrive()
        for x in range(n):
            if SB == 1:
                yield from load(pos_k(SB, x), ("k", x))
                yield from load(pos_v(SB, x, n), ("v", x))
            else:
                if x == 0:
                    yield from load(0, ("k", 0))
                if x + 1 < n:
                    yield from load(pos_k(SB, x + 1), ("k", x + 1))
                yield from load(pos_v(SB, x, n), ("v", x))

    def issuer(t):
        m, other = mine[t], mine[1 - t] if NT == 2 else 0

        def pass_turn():
            if NT == 2:
                turn[1 - t].arrive()

        def s_mma(j):
            slot = pos_k(SB, j) % NS
            yield from wait(full[slot], pos_k(SB, j) // NS)
            assert held[slot] == ("k", j)
            if j > 0:
                pass_turn()
            s[t * SB + j % SB].arrive()

        def pv_mma(j):
            slot = pos_v(SB, j, n) % NS
            yield from wait(full[slot], pos_v(SB, j, n) // NS)
            if NT == 2:
                if t == 0:
                    if j > 0 and other > 0:
                        yield from wait(turn[0], j - 1)
                elif j < other:
                    yield from wait(turn[1], j)
            for h in range(2):
                yield from wait(p[t * SB + j % SB][h], j // SB)
                assert held[slot] == ("v", j)
                if h == 1 and j + 1 == m:
                    pass_turn()
                if h == 1:
                    pv[t].arrive()
                if h == 0:
                    empty[pos_k(SB, j) % NS].arrive()

        def pv_done(j):
            yield from wait(pv[t], j)
            empty[pos_v(SB, j, n) % NS].arrive()
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
            for pos in (pos_k(SB, j), pos_v(SB, j, n)):
                yield from wait(full[pos % NS], pos // NS)
                empty[pos % NS].arrive()

    def softmax(t):
        m = mine[t]
        if m > 0:
            yield from some_steps(rng, 5)
            q[t].arrive()
        for j in range(m):
            yield from wait(s[t * SB + j % SB], j // SB)
            if j > 0 and SB == 2 and rng.random() < 0.4:    # the maximum is raised
                yield from wait(pv[t], j - 1)
            for h in range(2):
                yield from some_steps(rng, 6)
                if last_but_one and SB == 2 and h == 1 and j > 0 and j == m - 1:
                    yield from wait(pv[t], j - 1)
                p[t * SB + j % SB][h].arrive()
        if m > 0:
            yield from wait(pv[t], m - 1)
    run_all([loader()] + [issuer(t) for t in range(NT)] + [softmax(t) for t in range(NT)], rng)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_kernel(D):
    text = source("swa_paged_chunk.cu")
    NT, SB, NS = (constant(text, x, D) for x in ("NT", "SB", "NS"))
    assert arrivals(text) == {"b_full": "1", "b_empty": "NT", "b_q": "128", "b_pv": "1", "b_fin": "1", "b_turn": "1",
                              "b_s": "1", "b_p": "128", "b_tail": "1"}
    rng = random.Random(D)
    for seed in range(400):
        a = rng.randint(0, 12)
        # the second query tile's rows come later: they see as many keys or more, or there are none
        chunk_run(NT, SB, NS, [a] if NT == 1 else [a, rng.choice([0, a, a + 1, a + 2])], seed)


def test_chunk_kernel_needs_its_wait_for_the_last_but_one_product():
    with pytest.raises(Alias):
        for seed in range(400):
            chunk_run(1, 2, 5, [random.Random(seed).randint(0, 12)], seed, last_but_one=False)


# ------------------------------------------------------------------ the weighing kernel
def weigh_run(units, NS, NOTE, seed, shared_ring=False):
    """units: (halves, first query tile, query tiles, head) of a CTA's share, in order."""
    rng, NSH = random.Random(seed), NS // 2
    k_full, k_empty = [Bar(1) for _ in range(NS)], [Bar(1) for _ in range(NS)]
    q_full, q_empty = [Bar(1) for _ in range(2)], [Bar(2) for _ in range(2)]
    n_full, n_empty = [Bar(1) for _ in range(NOTE)], [Bar(2) for _ in range(NOTE)]   # 8 warps: 2 here
    pair_bar, s, s_free = Bar(1), [Bar(1) for _ in range(4)], [Bar(1) for _ in range(4)]
    filled = Bar(2)                                         # the named barrier of the summing warps
    k_in, q_in, n_in = [None] * NS, [None] * 2, [None] * NOTE

    def moved(i):
        return i + 1 == len(units) or units[i + 1][3] != units[i][3]

    def pair(i):
        _, q0, nq, _ = units[i]
        return nq <= 2 and nq - q0 == 2

    def slot_of(h, count):
        """(slot, use) of the half's count-th K tile, or of the count-th of both in a shared ring."""
        return (count % NS, count // NS) if shared_ring else (h * NSH + count % NSH, count // NSH)

    def k_loader():
        kc, total = [0, 0], 0
        for i, (halves, q0, nq, _) in enumerate(units):
            if q0 >= nq:
                continue
            for h in range(halves):
                slot, use = slot_of(h, total if shared_ring else kc[h])
                if use > 0:
                    yield from wait(k_empty[slot], use - 1)
                k_in[slot] = (i, h)
                yield from some_steps(rng, 6)
                k_full[slot].arrive()
                kc[h] += 1
                total += 1
        if not shared_ring:
            for h in range(2):
                for u in range(max(0, kc[h] - NSH), kc[h]):
                    slot, use = slot_of(h, u)
                    yield from wait(k_empty[slot], use)

    def q_loader():
        qc, fresh, pending = 0, True, None

        def tell():
            nonlocal pending
            if pending is not None:
                q_full[pending & 1].arrive()
                pending = None

        def until_free(bar, use):
            if use > 0 and not bar.test(use - 1):
                tell()
                yield from wait(bar, use - 1)

        def load(tag):
            nonlocal qc, pending
            yield from until_free(q_empty[qc & 1], qc >> 1)
            q_in[qc & 1] = tag
            yield from some_steps(rng, 6)
            tell()
            if rng.random() < 0.5:
                q_full[qc & 1].arrive()                     # a whole tile, by TMA
            else:
                pending = qc
            q, qc = qc, qc + 1
            yield from until_free(n_empty[q % NOTE], q // NOTE)
            n_in[q % NOTE] = tag
            n_full[q % NOTE].arrive()
        for i, (_, q0, nq, head) in enumerate(units):
            if nq <= 2:
                if fresh and pair(i):
                    tell()
                    for q in (qc, qc + 1):
                        yield from until_free(q_empty[q & 1], q >> 1)
                        yield from until_free(n_empty[q % NOTE], q // NOTE)
                    pair_bar.arrive()
                    qc += 2
                elif fresh:
                    for qt in range(q0, nq):
                        yield from load((head, qt))
                    tell()
            else:
                for qt in range(q0, nq):
                    yield from load((i, qt))
            fresh = moved(i)
        tell()
        for q in range(max(0, qc - 2), qc):
            yield from wait(q_empty[q & 1], q >> 1)

    def issuer(h):
        kc = jc = qc = seen = 0
        base = units[0][1]
        for i, (halves, q0, nq, head) in enumerate(units):
            kept = nq <= 2
            for qt in range(q0, nq):
                qi = qc + qt - base if kept else qc
                if qi >= seen:
                    yield from wait(q_full[qi & 1], qi >> 1)
                    seen = qi + 1
                want = (head, qt) if kept else (i, qt)
                assert q_in[qi & 1] == want
                if h < halves:
                    slot, use = slot_of(h, kc + h if shared_ring else kc)
                    buf = 2 * h + (jc & 1)
                    if qt == q0:
                        yield from wait(k_full[slot], use)
                    if jc >= 2:
                        yield from wait(s_free[buf], (jc >> 1) - 1)
                    assert k_in[slot] == (i, h)
                    yield from some_steps(rng, 4)
                    assert q_in[qi & 1] == want and k_in[slot] == (i, h)
                    s[buf].arrive()
                    if qt == nq - 1:
                        k_empty[slot].arrive()
                    jc += 1
                if not kept:
                    q_empty[qi & 1].arrive()
                    qc += 1
            if q0 < nq:
                if shared_ring:
                    kc += halves
                elif h < halves:
                    kc += 1
            if moved(i) and kept:
                for t in range(base, nq):
                    q_empty[(qc + t - base) & 1].arrive()
                qc += nq - base
            if moved(i) and i + 1 < len(units):
                base = units[i + 1][1]

    def sums(h):
        jc = qc = seen = pairs = fills = 0
        base = units[0][1]

        def fill(i):
            nonlocal pairs, fills
            _, q0, nq, head = units[i]
            if not pair(i):
                return
            yield from wait(pair_bar, pairs)
            pairs += 1
            for k in range(2):
                q_in[(qc + k) & 1] = n_in[(qc + k) % NOTE] = (head, q0 + k)
                yield from some_steps(rng, 6)
            filled.arrive()
            fills += 1
            while filled.phase < fills:
                yield
            if h == 0:
                for k in range(2):
                    q_full[(qc + k) & 1].arrive()
                    n_full[(qc + k) % NOTE].arrive()
        yield from fill(0)
        for i, (halves, q0, nq, head) in enumerate(units):
            kept = nq <= 2
            for qt in range(q0, nq):
                qi = qc + qt - base if kept else qc
                if qi >= seen:
                    yield from wait(n_full[qi % NOTE], qi // NOTE)
                    seen = qi + 1
                want = (head, qt) if kept else (i, qt)
                assert n_in[qi % NOTE] == want
                if h < halves:
                    buf = 2 * h + (jc & 1)
                    yield from wait(s[buf], jc >> 1)
                    yield from some_steps(rng, 8)
                    assert n_in[qi % NOTE] == want
                    s_free[buf].arrive()
                    jc += 1
                if not kept:
                    n_empty[qi % NOTE].arrive()
                    qc += 1
            if moved(i) and kept:
                for t in range(base, nq):
                    n_empty[(qc + t - base) % NOTE].arrive()
                qc += nq - base
            if moved(i) and i + 1 < len(units):
                base = units[i + 1][1]
                yield from fill(i + 1)
    run_all([k_loader(), q_loader(), issuer(0), issuer(1), sums(0), sums(1)], rng)


def share(seed):
    """A CTA's units: heads of one to five units; the last of a head may have one half, later ones
    may leave out query tiles; heads without rows among them."""
    rng, units = random.Random(seed), []
    for head in range(rng.randint(1, 6)):
        nq, n = rng.choice([0, 1, 1, 2, 2, 3, 5, 9]), rng.randint(1, 5)
        q = rng.randint(0, max(0, nq - 1))
        for i in range(n):
            units.append((1 if i == n - 1 and rng.random() < 0.5 else 2, min(q, nq), nq, head))
            if nq > 1 and rng.random() < 0.3:
                q = min(nq - 1, q + 1)
    return units


@pytest.mark.parametrize("D", [64, 128, 256])
def test_weigh_kernel(D):
    text = source("swa_weigh.cu")
    NS, note = constant(text, "NS", D), constant(text, "kNote", D)
    assert arrivals(text) == {"b_kfull": "1", "b_kempty": "1", "b_qfull": "1", "b_qempty": "2", "b_fin": "1", "b_s": "1",
                              "b_sfree": "4", "b_nfull": "1", "b_nempty": "8", "b_pair": "1"}
    for seed in range(600):
        weigh_run(share(seed + 1000 * D), NS, note, seed)


def test_weigh_kernel_needs_a_ring_a_half():
    """Units of one half shift the slots of a shared ring: a warp meets a phase of a barrier that it
    has not waited for before."""
    with pytest.raises(Alias):
        for seed in range(600):
            weigh_run(share(seed), 2, 4, seed, shared_ring=True)
