"""Plain float64 restatement of the 4-bit paged cache (include/swa.h: swa_paged4_append,
swa_paged4_read, swa_paged4_attend) and of the calls that share pages (swa_paged_fork,
swa_paged_compact). Shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np

from .paged_oracle import gather, rows

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# every e4m3 number without sign, by its bits (0x7f is NaN)
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)])
E4M3[127] = np.nan


def nearest(x, grid):
    """Index of the nearest grid value (ascending), the even index of two as near."""
    i = min(int(np.searchsorted(grid, x)), len(grid) - 1)
    if i == 0:
        return 0
    lo, hi = x - grid[i - 1], grid[i] - x
    return i if hi < lo or (hi == lo and i % 2 == 0) else i - 1


def encode_block(x, exp):
    """(codes [16], scale bits) of 16 values."""
    x = np.asarray(x, np.float64)
    if not np.isfinite(x).all():
        return np.zeros(16, np.int64), 127
    s = nearest(min(np.abs(x).max() * 2.0 ** -exp / 6.0, 448.0), E4M3[:127])
    if s == 0:
        return np.zeros(16, np.int64), 0
    u = E4M3[s] * 2.0 ** exp
    c = [nearest(abs(v) / u, LEVELS) for v in x]
    return np.array([i + 8 if i and v < 0 else i for i, v in zip(c, x)]), s


def encode(x, exp):
    """Rows [..][hd] -> (bytes [..][hd / 2], scale bits [..][hd / 16])."""
    x = np.asarray(x, np.float64)
    c, s = np.zeros(x.shape, np.uint8), np.zeros(x.shape[:-1] + (x.shape[-1] // 16,), np.uint8)
    for at in np.ndindex(*s.shape):
        block = slice(16 * at[-1], 16 * at[-1] + 16)
        c[at[:-1]][block], s[at] = encode_block(x[at[:-1]][block], exp)
    return c[..., 0::2] | (c[..., 1::2] << 4), s


def decode(codes, scales, exp):
    """(bytes, scale bits) -> values."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (-1,))
    v = np.where(c & 8, -1.0, 1.0) * LEVELS[c & 7]
    return v * np.repeat(E4M3[scales & 127], 16, -1) * 2.0 ** exp


def visible(n, own, window, sinks):
    """Which of n slots the row of slot `own` sees."""
    j = np.arange(n)
    seen = j <= own
    if window > 0:
        seen &= (j > own - window) | (j < sinks)
    return seen


def attend(q, ck, cv, table, row_start, lens, scale, window=0, sinks=0):
    """(out, lse, mean of |v| under the same weights, largest sum |q_i k_i| * scale) of values
    ck, cv [num_pages][nk][page][hd]."""
    T, nh, hd = q.shape
    nk = ck.shape[1]
    hpg = nh // nk
    out, lse = np.zeros((T, nh, hd)), np.full((T, nh), -np.inf)
    absv, sabs = np.zeros((T, nh, hd)), np.zeros((T, nh))
    for b in range(len(lens)):
        r0, r1 = rows(row_start, b)
        n = int(lens[b])
        for g in range(nk):
            k, v = gather(ck, table, b, g, n), gather(cv, table, b, g, n)
            for r in range(r0, r1):
                see = visible(n, n - (r1 - r0) + (r - r0), window, sinks)
                if not see.any():
                    continue
                kk, vv = k[see], v[see]
                for h in range(g * hpg, (g + 1) * hpg):
                    s = kk @ q[r, h] * scale
                    m = s.max()
                    p = np.exp(s - m)
                    out[r, h] = p @ vv / p.sum()
                    absv[r, h] = p @ np.abs(vv) / p.sum()
                    lse[r, h] = m + np.log(p.sum())
                    sabs[r, h] = (np.abs(kk) @ np.abs(q[r, h])).max() * scale
    return out, lse, absv, sabs


def fork(table, lens, refs, parent, room, page, num_pages):
    """(table, lens, refs, left, [(from, to)]) of the next batch, by lists."""
    width = len(table[0])
    refs = list(refs)
    held = lambda p: 0 <= p < num_pages
    for row in table:
        for p in row:
            if held(p):
                refs[p] -= 1
    out, new = [], []
    for q in parent:
        n = min(max(lens[q], 0), width * page) if 0 <= q < len(table) else 0
        row = [p if held(p) else -1 for p in table[q][:-(-n // page)]] if n else []
        out.append(row)
        new.append(n)
        for p in row:
            if p >= 0:
                refs[p] += 1
    writers = {}
    for r, n in enumerate(new):
        if n % page and out[r][-1] >= 0:
            writers.setdefault(out[r][-1], []).append(r)
    leave = set()
    for p, w in writers.items():
        if refs[p] > 1:
            leave |= set(w[1:] if len(w) == refs[p] else w)
    free = [p for p in range(num_pages) if refs[p] == 0]
    need, copies = 0, []

    def take():
        nonlocal need
        need += 1
        if need > len(free):
            return -1
        refs[free[need - 1]] = 1
        return free[need - 1]
    for r, n in enumerate(new):
        if r in leave:
            src, dst = out[r][-1], take()
            refs[src] -= 1
            out[r][-1] = dst
            if dst >= 0:
                copies.append((src, dst))
        extra = min(max(room[r], 0), width * page - n) if room is not None else 0
        for _ in range(-(-(n + extra) // page) - -(-n // page)):
            out[r].append(take())
    return [row + [-1] * (width - len(row)) for row in out], new, refs, len(free) - need, copies


def compact(table, refs, num_pages):
    """(table, refs, moved, used, [(from, to)])."""
    used = sum(k != 0 for k in refs)
    holes = [p for p in range(used) if refs[p] == 0]
    moved, new, copies = [-1] * num_pages, [0] * num_pages, []
    for p in range(num_pages):
        if refs[p] != 0:
            moved[p] = p if p < used else holes[len(copies)]
            new[moved[p]] = refs[p]
            if moved[p] != p:
                copies.append((p, moved[p]))
    return [[moved[p] if 0 <= p < num_pages else p for p in row] for row in table], new, moved, used, copies
