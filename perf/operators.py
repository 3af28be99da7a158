"""What is measured of the paged-cache operators: rotary, paged_append, paged_attend,
paged_weigh and paged_evict, each beside its plain form in elementary torch operations.

A case names its operator (``op``) and sizes. The lengths of its sequences follow from the
case alone (``mix`` numbers the mixture), the values of its tensors from the seed.
"""
from __future__ import annotations

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
WIDTH = {"bf16": 2, "f16": 2, "f32": 4}


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's q and k heads of a batch: latency
        {"name": "rotary_tokens", "op": "rotary", "T": 64, "H": 40, "d": 128, "rot": 128,
         "interleaved": False, "inverse": False, "dtype": "bf16", "far": 20000},
        # the gradient of the rotation over a long packed prompt in f32: half of each head,
        # interleaved pairs, positions far beyond the trained length
        {"name": "rotary_prompt", "op": "rotary", "T": 16383, "H": 40, "d": 128, "rot": 64,
         "interleaved": True, "inverse": True, "dtype": "f32", "far": 1000000},
        # one decode token of 64 sequences enters the cache
        {"name": "append_tokens", "op": "append", "B": 64, "rows": 1, "nh": 16, "nk": 4, "d": 128, "rot": 128,
         "page": 16, "lo": 1, "hi": 1024, "dtype": "bf16", "src": "bf16", "interleaved": False, "mix": 1},
        # ragged prompt chunks enter the cache from an f32 projection
        {"name": "append_prompt", "op": "append", "B": 4, "rows": 2048, "nh": 32, "nk": 8, "d": 128, "rot": 128,
         "page": 64, "lo": 2048, "hi": 8192, "dtype": "bf16", "src": "f32", "interleaved": False, "mix": 2},
        # one sequence's decode token over a short context: the smallest call
        {"name": "attend_small", "op": "attend", "B": 1, "rows": 1, "nh": 8, "nk": 2, "d": 64, "page": 16,
         "lo": 133, "hi": 133, "dtype": "bf16", "mix": 3},
        # one decode token of a batch with ragged contexts
        {"name": "attend_tokens", "op": "attend", "B": 64, "rows": 1, "nh": 16, "nk": 4, "d": 128, "page": 64,
         "lo": 1024, "hi": 8192, "dtype": "bf16", "mix": 4},
        # decode over long contexts with wide heads
        {"name": "attend_long", "op": "attend", "B": 16, "rows": 1, "nh": 8, "nk": 2, "d": 256, "page": 128,
         "lo": 32768, "hi": 131072, "dtype": "f16", "mix": 5},
        # prompt chunks behind earlier chunks: the largest call
        {"name": "attend_chunk", "op": "attend", "B": 4, "rows": 2048, "nh": 32, "nk": 8, "d": 128, "page": 64,
         "lo": 2048, "hi": 16384, "dtype": "bf16", "mix": 6},
        # each decode step adds its weights
        {"name": "weigh_tokens", "op": "weigh", "B": 64, "rows": 1, "nh": 16, "nk": 4, "d": 128, "page": 64,
         "lo": 2048, "hi": 4160, "dtype": "bf16", "mix": 7},
        # a prompt's keys weighed by its last rows
        {"name": "weigh_prompt", "op": "weigh", "B": 4, "rows": 64, "nh": 32, "nk": 8, "d": 128, "page": 64,
         "lo": 16384, "hi": 32768, "dtype": "f16", "mix": 8},
        # every 64 tokens a batch's caches go back to their budget
        {"name": "evict_tokens", "op": "evict", "B": 32, "nk": 8, "d": 128, "page": 64, "lo": 2112, "hi": 2112,
         "keep": 2048, "recent": 256, "sinks": 4, "dtype": "bf16", "mix": 9},
        # a long prompt's cache is cut down to its budget before decoding
        {"name": "evict_prompt", "op": "evict", "B": 4, "nk": 8, "d": 128, "page": 64, "lo": 16384, "hi": 32768,
         "keep": 4096, "recent": 512, "sinks": 4, "dtype": "f16", "mix": 10},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attend", "attend", "weigh", "evict"])
    d = rng.choice([64, 128, 256])
    c = {"op": op, "d": d, "dtype": rng.choice(["bf16", "f16"])}
    if op == "rotary":
        rot = rng.choice([d, d // 2, d // 4, d // 2 + 2 * rng.randint(0, 9)])
        c.update(T=_log(rng, 1, 16384), H=rng.randint(1, 48) if d < 256 else rng.randint(1, 20), rot=rot,
                 interleaved=rng.random() < 0.5, inverse=rng.random() < 0.3,
                 dtype=rng.choice(["bf16", "f16", "f32"]), far=_log(rng, 100, 1000000))
        return c
    nk = rng.choice([1, 2, 3, 4, 8])
    hpg = rng.choice([1, 2, 3, 4, 5, 8])
    c.update(nk=nk, nh=nk * hpg, page=rng.choice([16, 32, 64, 128]), mix=rng.randrange(1 << 30))
    if op == "append":
        rows = _log(rng, 1, 2048)
        c.update(B=max(1, min(_log(rng, 1, 64), 8192 // rows)), rows=rows, rot=rng.choice([d, d // 2]),
                 src=rng.choice([c["dtype"], "f32"]), interleaved=rng.random() < 0.5, lo=1, hi=rows + _log(rng, 1, 2048))
    elif op in ("attend", "weigh"):
        rows = 1 if rng.random() < 0.4 else _log(rng, 1, 2048)
        hi = _log(rng, 16, 32768)
        while rows * hi * c["nh"] * d > 1 << 37:
            rows = (rows + 1) // 2
        most = min(64, max(1, (1 << 36) // (rows * hi * c["nh"] * d)), max(1, (1 << 29) // (hi * nk * d)))
        c.update(B=_log(rng, 1, most), rows=rows, lo=_log(rng, 1, hi), hi=max(hi, rows))
    else:
        hi = _log(rng, 16, 32768)
        c.update(B=_log(rng, 1, min(64, max(1, (1 << 28) // (hi * nk * d)))), lo=_log(rng, 1, hi), hi=hi,
                 keep=_log(rng, 8, hi), recent=_log(rng, 1, 512), sinks=rng.choice([0, 1, 4]))
        del c["nh"]
    return c


def _lengths(c):
    """Rows t_b and cached keys len_b (the chunk's rows among them) of every sequence."""
    rng = random.Random(c["mix"])
    t, n = [], []
    for _ in range(c["B"]):
        rows = c.get("rows", 0)
        if rows > 1:
            rows = rng.randint((rows + 1) // 2, rows)
        t.append(rows)
        n.append(max(rows, rng.randint(c["lo"], c["hi"])))
    return t, n


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


def _plan(s, rot):
    f = _freqs(rot)
    s["freqs"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    s["turns"] = torch.tensor(_turns(f), dtype=torch.int64, device="cuda")


def _cache(s, c, t, n, g):
    """Pages in a shuffled order, some of the pool unused, and the batch's row starts."""
    B, nk, d, page, dt = c["B"], c["nk"], c["d"], c["page"], TYPES[c["dtype"]]
    need = [-(-x // page) for x in n]
    wide, used = max(need), sum(need)
    pool = used + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + need[:-1], device="cuda").cumsum(0)
    col = torch.arange(wide, device="cuda")
    idx = (first[:, None] + col[None, :]).clamp(max=pool - 1)
    held = col[None, :] < torch.tensor(need, device="cuda")[:, None]
    s["table"] = torch.where(held, order[idx], torch.zeros_like(order[idx])).contiguous()
    s["cache_k"] = torch.randn(pool, nk, page, d, generator=g, device="cuda", dtype=dt)
    s["cache_v"] = torch.randn(pool, nk, page, d, generator=g, device="cuda", dtype=dt)
    s["lens"] = torch.tensor(n, dtype=torch.int32, device="cuda")
    start = [0]
    for x in t:
        start.append(start[-1] + x)
    s["row_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    return start[-1]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = TYPES[c["dtype"]]
    s = {"case": c}
    d = c["d"]
    if c["op"] == "rotary":
        s["x"] = torch.randn(c["T"], c["H"], d, generator=g, device="cuda").to(dt)
        s["pos"] = torch.randint(0, c["far"], (c["T"],), generator=g, device="cuda", dtype=torch.int32)
        s["out"] = torch.empty_like(s["x"])
        _plan(s, c["rot"])
        return s
    t, n = _lengths(c)
    T = _cache(s, c, t, n, g)
    B, nk, page = c["B"], c["nk"], c["page"]
    cap = s["table"].shape[1] * page
    if c["op"] == "evict":
        # accumulated weights have a long tail; tokens no row has weighed yet tie at zero
        w = torch.exp(2.0 * torch.randn(B, nk, cap, generator=g, device="cuda"))
        s["weight"] = torch.where(torch.rand(B, nk, cap, generator=g, device="cuda") < 0.02, torch.zeros_like(w), w)
        # an earlier eviction left the positions out of order
        far = 2 * cap
        s["slot_pos"] = torch.rand(B, nk, far, generator=g, device="cuda").argsort(-1)[..., :cap].to(torch.int32).contiguous()
        s["recent_from"] = torch.full((B,), far - c["recent"], dtype=torch.int32, device="cuda")
        s["weight_out"] = torch.zeros_like(s["weight"])
        s["slot_pos_out"] = torch.zeros_like(s["slot_pos"])
        s["lens_out"] = torch.zeros_like(s["lens"])
        return s
    src = TYPES[c.get("src", c["dtype"])]
    s["q"] = torch.randn(T, c["nh"], d, generator=g, device="cuda").to(src)
    s["scale"] = d ** -0.5
    if c["op"] == "append":
        s["k"] = torch.randn(T, nk, d, generator=g, device="cuda").to(src)
        s["v"] = torch.randn(T, nk, d, generator=g, device="cuda").to(src)
        seq, i = _row_seq(s)
        s["pos"] = (s["lens"][seq] - (s["row_start"][seq + 1] - s["row_start"][seq]) + i).to(torch.int32)
        s["q_out"] = torch.empty(T, c["nh"], d, device="cuda", dtype=dt)
        _plan(s, c["rot"])
    elif c["op"] == "attend":
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(T, c["nh"], device="cuda", dtype=torch.float32)
    else:
        s["weight"] = torch.rand(B, nk, cap, generator=g, device="cuda")
        s["weight_out"] = torch.zeros_like(s["weight"])
        s["lse"] = _plain_attend(s, values=False)[1]
    return s


def _row_seq(s):
    """The sequence of every packed row, and the row's number in it."""
    T = s["q"].shape[0]
    r = torch.arange(T, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["row_start"], r, right=True) - 1
    return seq, r - s["row_start"][seq]


# --------------------------------------------------------------------------- plain forms
def _rotate(x, pos, freqs, interleaved, inverse):
    rot = 2 * freqs.shape[0]
    a = pos.to(torch.float64)[:, None] * freqs[None, :]
    cos, sin = torch.cos(a).float()[:, None, :], torch.sin(a).float()[:, None, :]
    if inverse:
        sin = -sin
    y = x.float()
    if interleaved:
        u, v = y[..., 0:rot:2], y[..., 1:rot:2]
        r = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
    else:
        u, v = y[..., :rot // 2], y[..., rot // 2:rot]
        r = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
    return torch.cat((r, y[..., rot:]), -1)


def _plain_append(s):
    c = s["case"]
    dt = TYPES[c["dtype"]]
    seq, i = _row_seq(s)
    slot = (s["lens"][seq] - (s["row_start"][seq + 1] - s["row_start"][seq]) + i).long()
    page = s["table"][seq, slot // c["page"]].long()
    q = _rotate(s["q"], s["pos"], s["freqs"], c["interleaved"], False).to(dt)
    k = _rotate(s["k"], s["pos"], s["freqs"], c["interleaved"], False).to(dt)
    s["cache_k"][page, :, slot % c["page"]] = k
    s["cache_v"][page, :, slot % c["page"]] = s["v"].to(dt)
    return q, s["cache_k"], s["cache_v"]


def _groups(c, cap):
    """Sequences taken together, so that their scores stay below 2^30 values."""
    step = max(1, (1 << 30) // max(c["nh"] * c["rows"] * cap, c["nk"] * cap * c["d"]))
    return [(b, min(c["B"], b + step)) for b in range(0, c["B"], step)]


def _scores(s, b0, b1):
    """Masked scores [b][nk][rows * hpg][cap] of some sequences, rows padded."""
    c = s["case"]
    nk, d, page, rows = c["nk"], c["d"], c["page"], c["rows"]
    hpg = c["nh"] // nk
    tab = s["table"][b0:b1].long()
    nb, cap = b1 - b0, tab.shape[1] * page
    k = s["cache_k"][tab].transpose(1, 2).reshape(nb, nk, cap, d).float()
    start, t = s["row_start"][b0:b1].long(), (s["row_start"][b0 + 1:b1 + 1] - s["row_start"][b0:b1]).long()
    i = torch.arange(rows, device="cuda")
    r = (start[:, None] + i[None, :]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][r].float().view(nb, rows, nk, hpg, d).permute(0, 2, 1, 3, 4).reshape(nb, nk, rows * hpg, d)
    limit = s["lens"][b0:b1].long()[:, None] - t[:, None] + i[None, :] + 1
    limit = torch.where(i[None, :] < t[:, None], limit, torch.zeros_like(limit))
    seen = torch.arange(cap, device="cuda")[None, None, :] < limit[:, :, None]
    seen = seen[:, None, :, None, :].expand(nb, 1, rows, hpg, cap).reshape(nb, 1, rows * hpg, cap)
    sc = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    return sc.masked_fill_(~seen, -math.inf), tab, cap


def _plain_attend(s, values=True):
    c = s["case"]
    nk, d, rows = c["nk"], c["d"], c["rows"]
    hpg = c["nh"] // nk
    outs, lses = [], []
    for b0, b1 in _groups(c, s["table"].shape[1] * c["page"]):
        sc, tab, cap = _scores(s, b0, b1)
        nb = b1 - b0
        m = sc.amax(-1, keepdim=True).clamp(min=-3e38)
        p = sc.sub_(m).exp_()
        l = p.sum(-1, keepdim=True)
        lses.append((m + l.log()).view(nb, nk, rows, hpg).permute(0, 2, 1, 3).reshape(nb, rows, nk * hpg))
        if values:
            v = s["cache_v"][tab].transpose(1, 2).reshape(nb, nk, cap, d).float()
            o = torch.matmul(p, v) / l.clamp(min=1e-38)
            outs.append(o.view(nb, nk, rows, hpg, d).permute(0, 2, 1, 3, 4).reshape(nb, rows, nk * hpg, d))
    seq, i = _row_seq(s)
    lse = torch.cat(lses)[seq, i.long()]
    return (torch.cat(outs)[seq, i.long()].to(s["q"].dtype) if values else None), lse


def _plain_weigh(s):
    c = s["case"]
    nk, rows = c["nk"], c["rows"]
    hpg = c["nh"] // nk
    for b0, b1 in _groups(c, s["table"].shape[1] * c["page"]):
        sc, _, cap = _scores(s, b0, b1)
        nb = b1 - b0
        start = s["row_start"][b0:b1].long()
        r = (start[:, None] + torch.arange(rows, device="cuda")[None, :]).clamp(max=s["q"].shape[0] - 1)
        lse = s["lse"][r].view(nb, rows, nk, hpg).permute(0, 2, 1, 3).reshape(nb, nk, rows * hpg, 1)
        w = s["weight"][b0:b1] + sc.sub_(lse).exp_().sum(2)
        held = torch.arange(cap, device="cuda")[None, None, :] < s["lens"][b0:b1][:, None, None]
        s["weight_out"][b0:b1] = torch.where(held, w, s["weight_out"][b0:b1])
    return s["weight_out"]


def _plain_evict(s):
    c = s["case"]
    B, nk, page, keep, d = c["B"], c["nk"], c["page"], c["keep"], c["d"]
    w, pos, n = s["weight"], s["slot_pos"], s["lens"].long()
    cap = w.shape[2]
    slot = torch.arange(cap, device="cuda")
    held = slot[None, None, :] < n[:, None, None]
    safe = (pos < c["sinks"]) | (pos >= s["recent_from"][:, None, None])
    rank = torch.where(safe, torch.full_like(w, math.inf), w)
    rank = torch.where(held, rank, torch.full_like(w, -math.inf))
    order = rank.sort(dim=-1, descending=True, stable=True).indices
    new = n.clamp(max=keep)
    kept = torch.zeros_like(w, dtype=torch.bool)
    kept.scatter_(2, order, (slot < keep).expand(B, nk, cap))
    kept &= held
    front = slot[None, None, :] < new[:, None, None]
    freed, moved = front & ~kept, kept & ~front
    # the i-th freed slot takes the i-th moved one: both lists in slot order, the rest stays
    to = torch.argsort(~freed, dim=-1, stable=True)
    by = torch.argsort(~moved, dim=-1, stable=True)
    count = freed.sum(-1, keepdim=True)
    live = slot[None, None, :] < count
    b, g, j = torch.nonzero(live, as_tuple=True)
    to, by = to[b, g, j], by[b, g, j]
    tab = s["table"].long()
    at, of = (tab[b, to // page], g, to % page), (tab[b, by // page], g, by % page)
    s["cache_k"][at] = s["cache_k"][of]
    s["cache_v"][at] = s["cache_v"][of]
    wo, po = w.clone(), pos.clone()
    wo[b, g, to], po[b, g, to] = w[b, g, by], pos[b, g, by]
    s["weight_out"].copy_(torch.where(front, wo, s["weight_out"]))
    s["slot_pos_out"].copy_(torch.where(front, po, s["slot_pos_out"]))
    s["lens_out"].copy_(new)
    return s["lens_out"], s["slot_pos_out"], s["weight_out"], s["cache_k"], s["cache_v"]


# --------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "rotary":
            y = _rotate(s["x"], s["pos"], s["freqs"], c["interleaved"], c["inverse"])
            return y.to(s["x"].dtype)
        if op == "append":
            return _plain_append(s)
        if op == "attend":
            return _plain_attend(s)
        if op == "weigh":
            return _plain_weigh(s)
        return _plain_evict(s)
    import sliding_window_gqa_prep_gb300 as swa
    if op == "rotary":
        return swa.rotary(s["x"], s["pos"], s["turns"], interleaved=c["interleaved"], inverse=c["inverse"], out=s["out"])
    if op == "append":
        swa.paged_append(s["k"], s["v"], s["pos"], s["cache_k"], s["cache_v"], s["table"], s["row_start"], s["lens"],
                         q=s["q"], q_out=s["q_out"], turns=s["turns"], interleaved=c["interleaved"])
        return s["q_out"], s["cache_k"], s["cache_v"]
    if op == "attend":
        swa.paged_attend(s["q"], s["cache_k"], s["cache_v"], s["table"], s["row_start"], s["lens"], s["scale"],
                         max_rows=c["rows"], out=s["out"], lse=s["lse"])
        return s["out"], s["lse"]
    if op == "weigh":
        return swa.paged_weigh(s["q"], s["lse"], s["cache_k"], s["table"], s["row_start"], s["lens"], s["scale"],
                               max_rows=c["rows"], weight=s["weight"], out=s["weight_out"])
    swa.paged_evict(s["cache_k"], s["cache_v"], s["table"], s["lens"], s["weight"], s["slot_pos"], c["keep"],
                    recent_from=s["recent_from"], sinks=c["sinks"], weight_out=s["weight_out"],
                    slot_pos_out=s["slot_pos_out"], lens_out=s["lens_out"])
    return s["lens_out"], s["slot_pos_out"], s["weight_out"], s["cache_k"], s["cache_v"]


# --------------------------------------------------------------------------- exact values
def exact(case, seed):
    """The operators from their definitions in 64 bits, one sequence and head at a time."""
    c = case
    f64 = torch.float64
    if c["op"] in ("attend", "weigh"):
        if sum(x * y for x, y in zip(*_lengths(c))) * c["nh"] * c["d"] > 4e12:
            return None
    s = prepare(case, seed)
    if c["op"] == "rotary" or c["op"] == "append":
        def turn(x, inverse):
            ang = torch.outer(s["pos"].to(f64), s["freqs"]) * (-1.0 if inverse else 1.0)
            z = torch.polar(torch.ones_like(ang), ang)[:, None, :]
            rot, y = c["rot"], x.to(f64).clone()
            at = (slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
            w = torch.complex(y[..., at[0]].contiguous(), y[..., at[1]].contiguous()) * z
            y[..., at[0]], y[..., at[1]] = w.real, w.imag
            return y
        if c["op"] == "rotary":
            return turn(s["x"], c["inverse"])
        q, k, v = turn(s["q"], False), turn(s["k"], False), s["v"].to(f64)
        ck, cv = s["cache_k"].to(f64), s["cache_v"].to(f64)
        t, n = _lengths(c)
        row = 0
        for b in range(c["B"]):
            slots = torch.arange(n[b] - t[b], n[b], device="cuda")
            pages = s["table"][b].long()[slots // c["page"]]
            ck[pages, :, slots % c["page"]] = k[row:row + t[b]]
            cv[pages, :, slots % c["page"]] = v[row:row + t[b]]
            row += t[b]
        return q, ck, cv
    t, n = _lengths(c)
    if c["op"] in ("attend", "weigh"):
        nk, d, page = c["nk"], c["d"], c["page"]
        hpg = c["nh"] // nk
        out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
        lse = torch.zeros(s["lse"].shape, dtype=f64, device="cuda")
        wo = s["weight_out"].to(f64) if c["op"] == "weigh" else None
        row = 0
        for b in range(c["B"]):
            idx = torch.arange(n[b], device="cuda")
            pages, off = s["table"][b].long()[idx // page], idx % page
            # rows in slices, so that a slice's scores stay small
            step = max(1, (1 << 27) // (hpg * n[b]))
            for h in range(nk):
                k = s["cache_k"][pages, h, off].to(f64)
                v = s["cache_v"][pages, h, off].to(f64)
                if wo is not None:
                    wo[b, h, :n[b]] = s["weight"][b, h, :n[b]].to(f64)
                for i0 in range(0, t[b], step):
                    i1 = min(t[b], i0 + step)
                    at = slice(row + i0, row + i1)
                    hs = slice(h * hpg, (h + 1) * hpg)
                    x = torch.einsum("rhd,kd->rhk", s["q"][at, hs].to(f64), k) * s["scale"]
                    last = n[b] - t[b] + torch.arange(i0, i1, device="cuda")
                    x = x.masked_fill(idx[None, None, :] > last[:, None, None], -math.inf)
                    if wo is not None:
                        wo[b, h, :n[b]] += torch.exp(x - s["lse"][at, hs].to(f64)[..., None]).sum((0, 1))
                    else:
                        z = torch.logsumexp(x, -1)
                        lse[at, hs] = z
                        out[at, hs] = torch.einsum("rhk,kd->rhd", torch.exp(x - z[..., None]), v)
            row += t[b]
        return wo if wo is not None else (out, lse)
    # evict: a host loop over sequences and heads
    w, pos = s["weight"].cpu(), s["slot_pos"].cpu()
    wo, po = s["weight_out"].cpu().to(f64), s["slot_pos_out"].cpu()
    tab, line = s["table"].cpu(), int(s["recent_from"][0])
    ck, cv = s["cache_k"].to(f64), s["cache_v"].to(f64)
    lens = []
    for b in range(c["B"]):
        new = min(n[b], c["keep"])
        lens.append(new)
        for h in range(c["nk"]):
            wl, pl = w[b, h, :n[b]].tolist(), pos[b, h, :n[b]].tolist()
            best = sorted(range(n[b]), key=lambda j: (not (pl[j] < c["sinks"] or pl[j] >= line), 0.0
                          if (pl[j] < c["sinks"] or pl[j] >= line) else -wl[j], j))[:new]
            stay = set(best)
            src = [j for j in sorted(best) if j >= new]
            dst = [j for j in range(new) if j not in stay]
            for a, z in zip(dst, src):
                wl[a], pl[a] = wl[z], pl[z]
            wo[b, h, :new] = torch.tensor(wl[:new], dtype=f64)
            po[b, h, :new] = torch.tensor(pl[:new], dtype=po.dtype)
            if dst:
                a, z = torch.tensor(dst), torch.tensor(src)
                pa, pz = tab[b][a // c["page"]].long().cuda(), tab[b][z // c["page"]].long().cuda()
                a, z = (a % c["page"]).cuda(), (z % c["page"]).cuda()
                ck[pa, h, a] = ck[pz, h, z]
                cv[pa, h, a] = cv[pz, h, z]
    return torch.tensor(lens, dtype=torch.int32), po, wo, ck, cv


# --------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["T"] * c["H"]
        return {"bytes": 2 * n * c["d"] * WIDTH[c["dtype"]] + 4 * c["T"] + 4 * c["rot"], "flops": 3 * n * c["rot"]}
    t, n = _lengths(c)
    d, nk, B = c["d"], c["nk"], c["B"]
    if c["op"] == "evict":
        # weights and positions in and out; a freed slot in front for every kept one behind
        # the budget: the unprotected share of the budget, times the share of slots behind it
        size, ops = 0, 0
        for x in n:
            new = min(x, c["keep"])
            moved = new * (x - new) / x
            size += nk * (8 * x + 8 * new + moved * 2 * 2 * d * 2)
            ops += nk * x
        return {"bytes": int(size) + 8 * B, "flops": int(ops)}
    nh, T = c["nh"], sum(t)
    if c["op"] == "append":
        size = (T * (nh + 2 * nk) * d) * (WIDTH[c["src"]] + 2) + 4 * T
        return {"bytes": size, "flops": 3 * T * (nh + nk) * c["rot"]}
    pairs = sum(x * (y - x) + x * (x + 1) // 2 for x, y in zip(t, n))
    if c["op"] == "attend":
        return {"bytes": 4 * sum(n) * nk * d + 4 * T * nh * d + 4 * T * nh, "flops": 4 * pairs * nh * d}
    return {"bytes": 2 * sum(n) * nk * d + 2 * T * nh * d + 4 * T * nh + 8 * sum(n) * nk, "flops": 2 * pairs * nh * d}
