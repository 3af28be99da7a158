"""What is measured of the 4-bit paged cache and of the calls that share its pages: paged4_append
(with paged4_read), paged4_read, paged4_attend, paged_fork and paged_compact, each beside its
plain form in elementary torch operations.

A case names its operator (``op``) and sizes. Lengths and parents follow from the case alone
(``mix`` numbers the mixture), the values of its tensors from the seed.

The 4-bit form: blocks of 16 features share a scale s in 8 bits (e4m3) and hold one of
0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign (e2m1) each; a value is code * s * 2^exp.
"""
from __future__ import annotations

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
WIDTH = {"bf16": 2, "f16": 2, "f32": 4}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode token of 64 young sequences enters the cache: latency
        {"name": "append4_tokens", "op": "append", "B": 64, "rows": 1, "nh": 16, "nk": 4, "d": 128, "rot": 128,
         "page": 16, "lo": 1, "hi": 64, "src": "bf16", "interleaved": False, "mix": 1},
        # ragged prompt chunks enter the cache from an f32 projection
        {"name": "append4_prompt", "op": "append", "B": 4, "rows": 2048, "nh": 32, "nk": 8, "d": 128, "rot": 128,
         "page": 64, "lo": 2048, "hi": 2560, "src": "f32", "interleaved": False, "mix": 2},
        # the last rows of a few short sequences, back in f32
        {"name": "read4_rows", "op": "read", "B": 4, "rows": 33, "nk": 2, "d": 64, "page": 16, "lo": 40, "hi": 133,
         "dtype": "f32", "mix": 3},
        # whole prefixes leave for a cache in 16 bits
        {"name": "read4_prefix", "op": "read", "B": 8, "rows": 8192, "nk": 8, "d": 128, "page": 64, "lo": 4096, "hi": 8192,
         "dtype": "bf16", "mix": 4},
        # one sequence's decode token over a short context: the smallest call
        {"name": "attend4_small", "op": "attend", "B": 1, "rows": 1, "nh": 8, "nk": 2, "d": 64, "page": 16,
         "lo": 133, "hi": 133, "window": 0, "sinks": 0, "dtype": "bf16", "mix": 5},
        # one decode token of a batch with ragged contexts
        {"name": "attend4_tokens", "op": "attend", "B": 64, "rows": 1, "nh": 32, "nk": 8, "d": 128, "page": 64,
         "lo": 1024, "hi": 8192, "window": 0, "sinks": 0, "dtype": "bf16", "mix": 6},
        # drafted tokens of a layer with a window and first tokens that stay, far into long contexts
        {"name": "attend4_window", "op": "attend", "B": 32, "rows": 4, "nh": 16, "nk": 4, "d": 256, "page": 128,
         "lo": 8192, "hi": 32768, "window": 4096, "sinks": 4, "dtype": "f16", "mix": 7},
        # prompt chunks behind earlier chunks: the largest call
        {"name": "attend4_chunk", "op": "attend", "B": 4, "rows": 2048, "nh": 32, "nk": 8, "d": 128, "page": 64,
         "lo": 2048, "hi": 16384, "window": 0, "sinks": 0, "dtype": "bf16", "mix": 8},
        # a step of a beam search: 16 requests of 4 beams
        {"name": "fork_beams", "op": "fork", "B": 64, "ways": 4, "out": 64, "nk": 4, "d": 128, "page": 16, "lo": 64, "hi": 1024,
         "dtype": "bf16", "mix": 9},
        # every prompt of a batch is continued eight ways
        {"name": "fork_prompts", "op": "fork", "B": 32, "ways": 1, "out": 256, "nk": 8, "d": 128, "page": 64, "lo": 1024, "hi": 4096,
         "dtype": "bf16", "mix": 10},
        # a small pool after some requests ended
        {"name": "compact_few", "op": "compact", "B": 16, "nk": 4, "d": 64, "page": 16, "lo": 16, "hi": 256, "pool": 600,
         "dtype": "f16", "mix": 11},
        # a large pool, a third in use, before part of it is given back
        {"name": "compact_pool", "op": "compact", "B": 64, "nk": 8, "d": 128, "page": 64, "lo": 256, "hi": 4096, "pool": 6000,
         "dtype": "bf16", "mix": 12},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "attend", "fork", "compact"])
    d, nk = rng.choice([64, 128, 256]), rng.choice([1, 2, 3, 4, 8])
    c = {"op": op, "d": d, "nk": nk, "page": rng.choice([16, 32, 64, 128, 256]), "mix": rng.randrange(1 << 30)}
    if op == "append":
        rows = _log(rng, 1, 2048)
        c.update(B=max(1, min(_log(rng, 1, 64), 8192 * 128 // (rows * d))), rows=rows, nh=nk * rng.choice([1, 2, 3, 4]),
                 rot=rng.choice([d, d // 2, d // 2 + 2 * rng.randint(0, 9)]), src=rng.choice(["bf16", "f16", "f32"]),
                 interleaved=rng.random() < 0.5, lo=1, hi=rows + _log(rng, 1, 512))
    elif op == "read":
        rows = _log(rng, 1, 8192)
        c.update(B=max(1, min(_log(rng, 1, 64), 65536 * 128 // (rows * d))), rows=rows, lo=1, hi=rows + _log(rng, 1, 512),
                 dtype=rng.choice(["bf16", "f16", "f32"]))
    elif op == "attend":
        rows = 1 if rng.random() < 0.4 else _log(rng, 1, 2048)
        hi, nh = _log(rng, 16, 32768), nk * rng.choice([1, 2, 3, 4, 5, 8])
        while rows * hi * nh * d > 1 << 37:
            rows = (rows + 1) // 2
        most = min(64, max(1, (1 << 37) // (rows * hi * nh * d)), max(1, (1 << 29) // (hi * nk * d)), max(1, (1 << 32) // (rows * hi * nh)))
        c.update(B=_log(rng, 1, most), rows=rows, nh=nh, lo=_log(rng, 1, hi), hi=max(hi, rows), window=0, sinks=0,
                 dtype=rng.choice(["bf16", "f16"]))
        if rng.random() < 0.5:
            c.update(window=_log(rng, 1, hi), sinks=rng.choice([0, 1, 4, 100]))
    else:
        hi = _log(rng, 16, 8192)
        b = _log(rng, 1, max(1, min(64, (1 << 27) // (hi * nk * d))))
        c.update(B=b, lo=_log(rng, 1, hi), hi=hi, dtype=rng.choice(["bf16", "f16"]))
        if op == "fork":
            c.update(ways=rng.choice([w for w in (1, 2, 4, 8) if w <= b]),
                     out=_log(rng, 1, max(1, min(256, (1 << 26) // (c["page"] * nk * d)))))
        else:
            c.update(pool=b * -(-hi // c["page"]) + _log(rng, 1, 2000))
            while c["pool"] * c["page"] * nk * d > 1 << 29:
                c["nk"] = nk = max(1, nk // 2)
                c["pool"] = b * -(-hi // c["page"]) + (c["pool"] - b * -(-hi // c["page"]) + 1) // 2
    return c


def _lengths(c):
    """Rows t_b and cached keys len_b (the chunk's rows among them) of every sequence."""
    rng = random.Random(c["mix"])
    t, n = [], []
    for _ in range(c["B"]):
        rows = c.get("rows", 0)
        if rows > 1 and c["op"] != "read":
            rows = rng.randint((rows + 1) // 2, rows)
        length = max(1, rng.randint(c["lo"], c["hi"]))
        if c["op"] == "read":
            rows = min(rows, length)
        t.append(rows)
        n.append(max(rows, length))
    return t, n


def _parents(c):
    """The old sequence that each new one continues (-1: none) and the slots each has to have
    room for behind its length."""
    rng = random.Random(c["mix"] + 1)
    if c["out"] == c["B"]:                 # beams: a parent among the own request's, some requests end
        w, par = c["ways"], []
        for r in range(c["out"]):
            par.append(r // w * w + rng.randrange(min(w, c["B"] - r // w * w)))
        ends = {r // w for r in range(c["out"]) if rng.random() < 0.03}
        par = [-1 if r // w in ends else p for r, p in enumerate(par)]
    else:
        par = [min(c["B"] - 1, r * c["B"] // c["out"]) for r in range(c["out"])]
    return par, [1 if p >= 0 else rng.randint(1, c["hi"]) for p in par]


# --------------------------------------------------------------------------- the 4-bit form
def _rotate(x, pos, freqs, interleaved):
    rot = 2 * freqs.shape[0]
    a = pos.to(torch.float64)[:, None] * freqs[None, :]
    cos, sin = torch.cos(a)[:, None, :], torch.sin(a)[:, None, :]
    y = x.to(torch.float64)
    if interleaved:
        u, v = y[..., 0:rot:2], y[..., 1:rot:2]
        r = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
    else:
        u, v = y[..., :rot // 2], y[..., rot // 2:rot]
        r = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
    return torch.cat((r, y[..., rot:]), -1)


def _two_to(e):
    """2^e of whole numbers from -20 to 20, to the last bit."""
    return torch.tensor([2.0 ** i for i in range(-20, 21)], dtype=torch.float64, device=e.device)[e.long() + 20]


def _quantise(x, exp):
    """Codes [..][hd / 2] (the lower half of a byte is the even feature) and scales [..][hd / 16]:
    a block's scale is its largest value / 6 in e4m3, a code the nearest level, ties to even."""
    b = x.unflatten(-1, (-1, 16))
    m = b.abs()
    s = (m.amax(-1).double() * 2.0 ** -exp / 6.0).clamp(max=448.0)
    k = torch.frexp(s.clamp(min=2.0 ** -6)).exponent - 4      # three bits behind the leading one
    s = (torch.round(s * _two_to(-k)) * _two_to(k)).float().to(torch.float8_e4m3fn)
    u = (s.to(x.dtype) * 2.0 ** exp)[..., None]
    c = (m > 0.25 * u).to(torch.uint8)
    c += m >= 0.75 * u
    c += m > 1.25 * u
    c += m >= 1.75 * u
    c += m > 2.5 * u
    c += m >= 3.5 * u
    c += m > 5.0 * u
    c += 8 * (b < 0)
    c = c.flatten(-2)
    return c[..., 0::2] + 16 * c[..., 1::2], s


def _values(codes, scales, exp):
    """What codes and scales stand for, in f32 (exact)."""
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = table[c.int()].unflatten(-1, (-1, 16))
    return (v * (scales.float() * 2.0 ** exp)[..., None]).flatten(-2)


# --------------------------------------------------------------------------- inputs
def _freqs(rot, theta=10000.0):
    return [theta ** (-2.0 * e / rot) for e in range(rot // 2)]


def _turns(freqs):
    """Turns per position as 64-bit fixed point: whole turns drop out of pos * turns."""
    out = []
    for f in freqs:
        v = int((f / (2.0 * math.pi)) % 1.0 * 2.0 ** 64) % (1 << 64)
        out.append(v - (1 << 64) if v >= 1 << 63 else v)
    return out


def _tables(s, c, t, n, g):
    """Pages in a shuffled order, some of the pool unused, and the batch's row starts."""
    page = c["page"]
    need = [-(-x // page) for x in n]
    wide, used = max(need), sum(need)
    pool = used + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + need[:-1], device="cuda").cumsum(0)
    col = torch.arange(wide, device="cuda")
    idx = (first[:, None] + col[None, :]).clamp(max=pool - 1)
    held = col[None, :] < torch.tensor(need, device="cuda")[:, None]
    s["table"] = torch.where(held, order[idx], torch.full_like(order[idx], -1)).contiguous()
    s["lens"] = torch.tensor(n, dtype=torch.int32, device="cuda")
    start = [0]
    for x in t:
        start.append(start[-1] + x)
    s["row_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    return pool, start[-1]


def _pool4(pool, c, g, spread):
    """One cache of quantised normal values whose heads differ in size by up to `spread`."""
    nk, page, d = c["nk"], c["page"], c["d"]
    size = torch.linspace(1.0, spread, nk, device="cuda")[None, :, None, None]
    return _quantise(torch.randn(pool, nk, page, d, generator=g, device="cuda") * size, 0)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    nk, d, page = c["nk"], c["d"], c["page"]
    t, n = _lengths(c)
    if c["op"] in ("fork", "compact"):
        dt = TYPES[c["dtype"]]
        if c["op"] == "fork":
            par, room = _parents(c)
            # beams of a request share the pages of their common prefix
            w = c["ways"]
            n = [n[b // w * w] for b in range(c["B"])]
            shared = [0 if b % w == 0 else n[b] // page * 3 // 4 for b in range(c["B"])]
            need = [-(-x // page) for x in n]
            fresh = [a - b for a, b in zip(need, shared)]
            more = sum(-(-r // page) + 1 for r in room)
            pool, wide = sum(fresh) + more, max(need + [-(-(r + (n[p] if p >= 0 else 0)) // page) for p, r in zip(par, room)])
            s["parent"] = torch.tensor(par, dtype=torch.int32, device="cuda")
            s["room"] = torch.tensor(room, dtype=torch.int32, device="cuda")
        else:
            need = [-(-x // page) for x in n]
            shared, fresh, pool, wide, w = [0] * c["B"], need, c["pool"], max(need), 1
        order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32).tolist()
        rows, at = [], 0
        for b in range(c["B"]):
            mine = rows[b // w * w][:shared[b]] if shared[b] else []
            mine = mine + order[at:at + fresh[b]]
            at += fresh[b]
            rows.append(mine + [-1] * (wide - len(mine)))
        s["table"] = torch.tensor(rows, dtype=torch.int32, device="cuda")
        s["lens"] = torch.tensor(n, dtype=torch.int32, device="cuda")
        held = s["table"][s["table"] >= 0].long()
        s["refs"] = torch.bincount(held, minlength=pool).to(torch.int32)
        s["pools"] = [torch.randn(pool, nk, page, d, generator=g, device="cuda", dtype=dt) for _ in range(2)]
        return s
    pool, T = _tables(s, c, t, n, g)
    s["T"] = T
    s["exp_k"], s["exp_v"] = 0, -6         # values are smaller than keys
    (s["k"], s["ks"]), (s["v"], s["vs"]) = _pool4(pool, c, g, 3.0), _pool4(pool, c, g, 1.5)
    if c["op"] == "read":
        s["k_out"] = torch.empty(T, nk, d, device="cuda", dtype=TYPES[c["dtype"]])
        s["v_out"] = torch.empty_like(s["k_out"])
        return s
    if c["op"] == "append":
        src = TYPES[c["src"]]
        s["q_in"] = torch.randn(T, c["nh"], d, generator=g, device="cuda").to(src)
        s["k_in"] = (4.0 * torch.randn(T, nk, d, generator=g, device="cuda")).to(src)
        s["v_in"] = (0.1 * torch.randn(T, nk, d, generator=g, device="cuda")).to(src)
        seq, i = _row_seq(s)
        s["pos"] = (s["lens"][seq] - (s["row_start"][seq + 1] - s["row_start"][seq]) + i).to(torch.int32)
        f = _freqs(c["rot"])
        s["freqs"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        s["turns"] = torch.tensor(_turns(f), dtype=torch.int64, device="cuda")
        s["q_out"] = torch.empty(T, c["nh"], d, device="cuda", dtype=torch.float16 if c["src"] == "f16" else torch.bfloat16)
        # the whole of every sequence, to read it back
        s["all_start"] = torch.cat((torch.zeros(1, dtype=torch.int32, device="cuda"), s["lens"].cumsum(0).to(torch.int32)))
        s["k_out"] = torch.empty(sum(n), nk, d, device="cuda", dtype=torch.bfloat16)
        s["v_out"] = torch.empty_like(s["k_out"])
        return s
    s["q"] = torch.randn(T, c["nh"], d, generator=g, device="cuda").to(TYPES[c["dtype"]])
    s["scale"] = d ** -0.5
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(T, c["nh"], device="cuda", dtype=torch.float32)
    return s


def _row_seq(s):
    """The sequence of every packed row, and the row's number in it."""
    r = torch.arange(s["T"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["row_start"], r, right=True) - 1
    return seq, r - s["row_start"][seq]


# --------------------------------------------------------------------------- plain forms
def _slots(s, starts, total):
    """Page and place in it of packed rows: the last rows of every sequence."""
    r = torch.arange(total, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(starts, r, right=True) - 1
    slot = (s["lens"][seq] - starts[seq + 1] + r).long()
    page = s["case"]["page"]
    return s["table"][seq, slot // page].long(), slot % page


def _plain_read(s, starts, like):
    page, at = _slots(s, starts, like.shape[0])
    return tuple(_values(s[a][page, :, at], s[b][page, :, at], s["exp_" + a]).to(like.dtype) for a, b in (("k", "ks"), ("v", "vs")))


def _plain_append(s):
    c = s["case"]
    page, at = _slots(s, s["row_start"], s["T"])
    q = _rotate(s["q_in"], s["pos"], s["freqs"], c["interleaved"]).to(s["q_out"].dtype)
    k, ks = _quantise(_rotate(s["k_in"], s["pos"], s["freqs"], c["interleaved"]), s["exp_k"])
    v, vs = _quantise(s["v_in"].float(), s["exp_v"])
    s["k"][page, :, at], s["v"][page, :, at] = k, v
    s["ks"].view(torch.uint8)[page, :, at], s["vs"].view(torch.uint8)[page, :, at] = ks.view(torch.uint8), vs.view(torch.uint8)
    return (q,) + _plain_read(s, s["all_start"], s["k_out"])


def _plain_attend(s):
    c = s["case"]
    nk, d, page, rows, B = c["nk"], c["d"], c["page"], c["rows"], c["B"]
    hpg = c["nh"] // nk
    tab = s["table"].long().clamp(min=0)
    cap = tab.shape[1] * page
    k, v = (_values(s[a][tab], s[b][tab], s["exp_" + a]).transpose(1, 2).reshape(B, nk, cap, d) for a, b in (("k", "ks"), ("v", "vs")))
    start, t = s["row_start"][:-1].long(), (s["row_start"][1:] - s["row_start"][:-1]).long()
    i = torch.arange(rows, device="cuda")
    r = (start[:, None] + i[None, :]).clamp(max=s["T"] - 1)
    q = s["q"][r].float().view(B, rows, nk, hpg, d).permute(0, 2, 1, 3, 4).reshape(B, nk, rows * hpg, d)
    limit = s["lens"].long()[:, None] - t[:, None] + i[None, :] + 1
    limit = torch.where(i[None, :] < t[:, None], limit, torch.zeros_like(limit))[:, :, None]
    j = torch.arange(cap, device="cuda")[None, None, :]
    seen = j < limit
    if c["window"]:
        seen &= (j >= limit - c["window"]) | (j < c["sinks"])
    seen = seen[:, None, :, None, :]
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    x.view(B, nk, rows, hpg, cap).masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = x.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / z.clamp(min=1e-38)
    lse = (m + z.log()).view(B, nk, rows, hpg).permute(0, 2, 1, 3).reshape(B, rows, nk * hpg)
    o = o.view(B, nk, rows, hpg, d).permute(0, 2, 1, 3, 4).reshape(B, rows, nk * hpg, d)
    seq, i = _row_seq(s)
    return o[seq, i.long()].to(s["q"].dtype), lse[seq, i.long()]


def _plain_fork(s):
    c = s["case"]
    page, table, lens = c["page"], s["table"].long(), s["lens"].long()
    par, room, pool = s["parent"].long(), s["room"].long(), s["refs"].shape[0]
    R, wide = par.shape[0], table.shape[1]
    r, col = torch.arange(R, device="cuda"), torch.arange(wide, device="cuda")
    lives, p0 = par >= 0, par.clamp(min=0)
    new_len = torch.where(lives, lens[p0], 0)
    taken = (new_len + page - 1) // page
    out = torch.where(col[None, :] < taken[:, None], table[p0], -1)
    # all old tables let go of their pages, the new ones hold theirs
    refs = s["refs"].long() - torch.bincount(table[table >= 0], minlength=pool) + torch.bincount(out[out >= 0], minlength=pool)
    # a page that is written next has one holder: the others get a copy
    at = (new_len // page).clamp(max=wide - 1)
    half = new_len % page != 0
    mine = torch.where(half, out[r, at], 0)
    opens = torch.bincount(mine[half], minlength=pool)
    first = torch.full((pool,), R, device="cuda").scatter_reduce(0, mine, torch.where(half, r, R), "amin")
    copy = half & (refs[mine] > 1) & ~((opens[mine] == refs[mine]) & (first[mine] == r))
    refs = refs - torch.bincount(mine[copy], minlength=pool)
    free = torch.nonzero(refs == 0)[:, 0]
    grow = (new_len + room + page - 1) // page - taken
    need = grow + copy
    base = need.cumsum(0) - need
    src, dst = mine[copy], free[base[copy]]
    out[r[copy], at[copy]] = dst
    fresh = (col[None, :] >= taken[:, None]) & (col[None, :] < (taken + grow)[:, None])
    which = (base + copy)[:, None] + col[None, :] - taken[:, None]
    out = torch.where(fresh, free[which.clamp(min=0, max=free.shape[0] - 1)], out)
    refs[free[:int(need.sum())]] = 1
    for p in s["pools"]:
        p[dst] = p[src]
    left = (free.shape[0] - need.sum()).to(torch.int32).view(1)
    return out.to(torch.int32), new_len.to(torch.int32), refs.to(torch.int32), left, s["pools"]


def _plain_compact(s):
    refs, table = s["refs"], s["table"].long()
    used = refs > 0
    count = used.sum()
    page = torch.arange(refs.shape[0], device="cuda")
    src, dst = torch.nonzero(used & (page >= count))[:, 0], torch.nonzero(~used & (page < count))[:, 0]
    moved = torch.where(used, page, -1)
    moved[src] = dst
    out = torch.where(table >= 0, moved[table.clamp(min=0)], table)
    new = torch.zeros_like(refs)
    new[moved[used]] = refs[used]
    for p in s["pools"]:
        p[dst] = p[src]
    return out.to(torch.int32), new, moved.to(torch.int32), count.to(torch.int32).view(1), s["pools"]


# --------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "append":
            return _plain_append(s)
        if op == "read":
            return _plain_read(s, s["row_start"], s["k_out"])
        if op == "attend":
            return _plain_attend(s)
        return _plain_fork(s) if op == "fork" else _plain_compact(s)
    import sliding_window_gqa_prep_gb300 as swa
    if op == "fork":
        table, lens, refs, left = swa.paged_fork(s["pools"], s["table"], s["lens"], s["refs"], s["parent"], c["page"], room=s["room"])
        return table, lens, refs, left, s["pools"]
    if op == "compact":
        table, refs, moved, used = swa.paged_compact(s["pools"], s["table"], s["refs"])
        return table, refs, moved, used, s["pools"]
    cache, exps = (s["k"], s["ks"], s["v"], s["vs"], s["table"]), {"exp_k": s["exp_k"], "exp_v": s["exp_v"]}
    if op == "append":
        swa.paged4_append(s["k_in"], s["v_in"], s["pos"], *cache, s["row_start"], s["lens"], q=s["q_in"], q_out=s["q_out"],
                          turns=s["turns"], interleaved=c["interleaved"], **exps)
        swa.paged4_read(*cache, s["all_start"], s["lens"], k_out=s["k_out"], v_out=s["v_out"], **exps)
        return s["q_out"], s["k_out"], s["v_out"]
    if op == "read":
        return swa.paged4_read(*cache, s["row_start"], s["lens"], k_out=s["k_out"], v_out=s["v_out"], **exps)
    swa.paged4_attend(s["q"], *cache, s["row_start"], s["lens"], s["scale"], max_rows=c["rows"], window=c["window"],
                      sinks=c["sinks"], out=s["out"], lse=s["lse"], **exps)
    return s["out"], s["lse"]


# --------------------------------------------------------------------------- exact values
def _stored(x, exp):
    """The values of x's blocks after quantisation, by distance to the levels, in 64 bits."""
    y = x.to(torch.float64).unflatten(-1, (-1, 16)) / 2.0 ** exp
    top = y.abs().amax(-1, keepdim=True)
    # every e4m3 number, and the nearest of them; of two as near the one with the even mantissa
    e4m3 = torch.tensor([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127],
                        dtype=torch.float64, device=x.device)
    want = (top / 6.0).clamp(max=448.0)
    low = (torch.searchsorted(e4m3, want, right=True) - 1).clamp(max=125)
    up = (want - e4m3[low]) - (e4m3[low + 1] - want)
    s = e4m3[torch.where((up > 0) | ((up == 0) & (low % 2 == 1)), low + 1, low)]
    z = y.abs() / s.clamp(min=2.0 ** -20)
    even_first = torch.tensor([LEVELS[i] for i in (0, 2, 4, 6, 1, 3, 5, 7)], dtype=torch.float64, device=x.device)
    level = even_first[(z[..., None] - even_first).abs().argmin(-1)]
    return (torch.sign(y) * level * s * 2.0 ** exp).flatten(-2)


def _decoded(codes, scales, exp):
    """The values of codes by the bits of the two formats, in 64 bits."""
    c = torch.stack((codes % 16, codes // 16), -1).flatten(-2).to(torch.int64)
    sign, e, m = c // 8, c // 2 % 4, c % 2
    v = torch.where(e > 0, (1.0 + 0.5 * m.double()) * _two_to(e - 1), 0.5 * m.double())
    b = scales.view(torch.uint8).to(torch.int64)
    e, m = b // 8, (b % 8).double()
    u = torch.where(e > 0, (1.0 + m / 8.0) * _two_to(e - 7), m * 2.0 ** -9)
    return v * (1 - 2 * sign) * u.repeat_interleave(16, -1) * 2.0 ** exp


def exact(case, seed):
    """The operators from their definitions in 64 bits, one sequence and head at a time."""
    c = case
    f64 = torch.float64
    if c["op"] == "attend" and sum(x * y for x, y in zip(*_lengths(c))) * c["nh"] * c["d"] > 4e12:
        return None
    s = prepare(case, seed)
    if c["op"] == "fork":
        return _exact_fork(s)
    if c["op"] == "compact":
        return _exact_compact(s)
    t, n = _lengths(c)
    page, nk, d = c["page"], c["nk"], c["d"]

    def held(b, j0, j1):
        j = torch.arange(j0, j1, device="cuda")
        at = s["table"][b].long()[j // page], slice(None), j % page
        return _decoded(s["k"][at], s["ks"][at], s["exp_k"]), _decoded(s["v"][at], s["vs"][at], s["exp_v"])

    if c["op"] == "read":
        both = [held(b, n[b] - t[b], n[b]) for b in range(c["B"])]
        return torch.cat([x for x, _ in both]), torch.cat([x for _, x in both])
    if c["op"] == "append":
        def turn(x):
            ang = torch.outer(s["pos"].to(f64), s["freqs"])
            z = torch.polar(torch.ones_like(ang), ang)[:, None, :]
            rot, y = c["rot"], x.to(f64).clone()
            at = (slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
            w = torch.complex(y[..., at[0]].contiguous(), y[..., at[1]].contiguous()) * z
            y[..., at[0]], y[..., at[1]] = w.real, w.imag
            return y
        k, v, row, ks, vs = _stored(turn(s["k_in"]), s["exp_k"]), _stored(s["v_in"], s["exp_v"]), 0, [], []
        for b in range(c["B"]):
            a, z = held(b, 0, n[b] - t[b])
            ks += [a, k[row:row + t[b]]]
            vs += [z, v[row:row + t[b]]]
            row += t[b]
        return turn(s["q_in"]), torch.cat(ks), torch.cat(vs)
    hpg = c["nh"] // nk
    out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=f64, device="cuda")
    row = 0
    for b in range(c["B"]):
        kb, vb = held(b, 0, n[b])
        idx = torch.arange(n[b], device="cuda")
        step = max(1, (1 << 27) // (hpg * n[b]))        # rows in slices, so that a slice's scores stay small
        for h in range(nk):
            for i0 in range(0, t[b], step):
                i1 = min(t[b], i0 + step)
                at, hs = slice(row + i0, row + i1), slice(h * hpg, (h + 1) * hpg)
                x = torch.einsum("rhd,kd->rhk", s["q"][at, hs].to(f64), kb[:, h]) * s["scale"]
                own_slot = n[b] - t[b] + torch.arange(i0, i1, device="cuda")[:, None, None]
                hidden = idx > own_slot
                if c["window"]:
                    hidden |= (own_slot - idx >= c["window"]) & (idx >= c["sinks"])
                x = x.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[at, hs] = z
                out[at, hs] = torch.einsum("rhk,kd->rhd", torch.exp(x - z[..., None]), vb[:, h])
        row += t[b]
    return out, lse


def _exact_fork(s):
    """By lists on the host: who holds what, then page after page from the lowest free one."""
    page, table, lens = s["case"]["page"], s["table"].tolist(), s["lens"].tolist()
    par, room, refs = s["parent"].tolist(), s["room"].tolist(), s["refs"].tolist()
    wide = len(table[0])
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] -= 1
    rows, new_len = [], []
    for p in par:
        n = lens[p] if p >= 0 else 0
        rows.append(table[p][:-(-n // page)] if n else [])
        new_len.append(n)
        for q in rows[-1]:
            refs[q] += 1
    writers = {}
    for r, n in enumerate(new_len):
        if n % page:
            writers.setdefault(rows[r][n // page], []).append(r)
    copies = []
    leave = {r for p, w in writers.items() if refs[p] > 1 for r in (w[1:] if len(w) == refs[p] else w)}
    for r in leave:
        refs[rows[r][-1]] -= 1
    free = iter([p for p, k in enumerate(refs) if k == 0])
    for r, n in enumerate(new_len):
        if r in leave:
            copies.append((rows[r][-1], next(free)))
            rows[r][-1] = copies[-1][1]
            refs[rows[r][-1]] = 1
        while len(rows[r]) < -(-(n + room[r]) // page):
            rows[r].append(next(free))
            refs[rows[r][-1]] = 1
    for src, dst in copies:
        for p in s["pools"]:
            p[dst] = p[src]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return i32([r + [-1] * (wide - len(r)) for r in rows]), i32(new_len), i32(refs), i32([sum(k == 0 for k in refs)]), s["pools"]


def _exact_compact(s):
    refs, table = s["refs"].tolist(), s["table"].tolist()
    count = sum(k > 0 for k in refs)
    holes = iter([p for p in range(count) if refs[p] == 0])
    moved = [(-1 if k == 0 else p if p < count else next(holes)) for p, k in enumerate(refs)]
    new = [0] * len(refs)
    for p, q in enumerate(moved):
        if q >= 0:
            new[q] = refs[p]
            if q != p:
                for x in s["pools"]:
                    x[q] = x[p]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return i32([[moved[p] if p >= 0 else p for p in row] for row in table]), i32(new), i32(moved), i32([count]), s["pools"]


# --------------------------------------------------------------------------- work
def work(case):
    c = case
    t, n = _lengths(c)
    d, nk, B, page = c["d"], c["nk"], c["B"], c["page"]
    key = nk * (d // 2 + d // 16)          # a key or a value of all heads
    if c["op"] == "read":
        return {"bytes": sum(t) * (2 * key + 2 * nk * d * WIDTH[c["dtype"]]) + 8 * B, "flops": 2 * sum(t) * nk * d}
    if c["op"] == "append":
        # in: the chunk; out: the rotated q and the codes; then every key is read and written in 16 bits
        T = sum(t)
        size = T * (c["nh"] + 2 * nk) * d * WIDTH[c["src"]] + T * c["nh"] * d * 2 + 2 * T * key + 4 * T
        return {"bytes": size + sum(n) * (2 * key + 4 * nk * d), "flops": 3 * T * (c["nh"] + nk) * c["rot"]}
    if c["op"] == "attend":
        size, pairs = 0, 0
        for rows, length in zip(t, n):
            base, w, k = length - rows, c["window"] or length, c["sinks"] if c["window"] else 0
            first = max(0, base + 1 - w)   # the first key in the first row's window
            size += 2 * key * (length - first + min(first, k))
            for i in range(rows):
                lo = max(0, base + i + 1 - w)
                pairs += base + i + 1 - lo + min(lo, k)
        T = sum(t)
        return {"bytes": size + 4 * T * c["nh"] * d + 4 * T * c["nh"], "flops": 4 * pairs * c["nh"] * d}
    whole = 2 * nk * page * d * 2          # a page of keys and of values, 16 bits
    if c["op"] == "fork":
        par, room = _parents(c)
        w = c["ways"]
        n = [n[b // w * w] for b in range(B)]
        times = [par.count(b) for b in range(B)]
        copies = sum(k - 1 for k, x in zip(times, n) if k > 1 and x % page)
        wide = max([-(-x // page) for x in n] + [-(-(r + (n[p] if p >= 0 else 0)) // page) for p, r in zip(par, room)])
        return {"bytes": 2 * copies * whole + 4 * (B + c["out"]) * wide, "flops": 0}
    used = sum(-(-x // page) for x in n)
    moves = used * (c["pool"] - used) // c["pool"]
    return {"bytes": int(2 * moves * whole + 8 * c["pool"]), "flops": 0}
