"""Plain float64 restatement of the paged-cache operators (include/swa.h: swa_rotary,
swa_paged_append, swa_paged_attend, swa_paged_weigh, swa_paged_evict), one row, head
and sequence at a time. Shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np


def rotary(x, pos, freqs, interleaved=False, inverse=False, mag=1.0):
    """x [T][H][hd], pos [T], freqs [rot/2] in radians per position."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    rot = 2 * len(freqs)
    for r in range(x.shape[0]):
        for e, f in enumerate(freqs):
            a = float(int(pos[r])) * float(f) * (-1.0 if inverse else 1.0)
            c, s = np.cos(a) * mag, np.sin(a) * mag
            i, j = (2 * e, 2 * e + 1) if interleaved else (e, rot // 2 + e)
            y[r, :, i] = x[r, :, i] * c - x[r, :, j] * s
            y[r, :, j] = x[r, :, j] * c + x[r, :, i] * s
    return y


def freqs(rot, theta, kind="plain", factor=1.0, orig_len=0.0, low=1.0, high=32.0):
    out = []
    for e in range(rot // 2):
        th = theta * factor ** (rot / (rot - 2)) if kind == "base" else theta
        f = th ** (-2.0 * e / rot)
        if kind == "linear":
            f /= factor
        elif kind == "parts":
            turns = orig_len * f / (2 * np.pi)
            if turns <= low:
                f = f / factor
            elif turns < high:
                k = (turns - low) / (high - low)
                f = k * f + (1 - k) * f / factor
        out.append(f)
    return np.array(out)


def rows(row_start, b):
    return int(row_start[b]), int(row_start[b + 1])


def gather(pages, table, b, g, n):
    """Rows [n][hd] of sequence b, KV head g; zeros where a page is out of range."""
    page = pages.shape[2]
    out = np.zeros((n, pages.shape[3]))
    for j in range(n):
        p = int(table[b][j // page])
        if 0 <= p < pages.shape[0]:
            out[j] = pages[p, g, j % page]
    return out


def attend(q, ck, cv, table, row_start, lens, scale):
    """(out, lse, mean of |v| under the same weights, largest sum |q_i k_i| * scale) in float64."""
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
                lim = n - (r1 - r0) + (r - r0) + 1
                if lim <= 0:
                    continue
                for h in range(g * hpg, (g + 1) * hpg):
                    s = k[:lim] @ q[r, h] * scale
                    m = s.max()
                    p = np.exp(s - m)
                    out[r, h] = p @ v[:lim] / p.sum()
                    absv[r, h] = p @ np.abs(v[:lim]) / p.sum()
                    lse[r, h] = m + np.log(p.sum())
                    sabs[r, h] = (np.abs(k[:lim]) @ np.abs(q[r, h])).max() * scale
    return out, lse, absv, sabs


def weigh(q, lse, ck, table, row_start, lens, scale, weight):
    """The weights after the chunk: [B][nk][cap], entries from lens on as given."""
    nh, nk = q.shape[1], ck.shape[1]
    hpg = nh // nk
    out = np.array(weight, np.float64)
    for b in range(len(lens)):
        r0, r1 = rows(row_start, b)
        n = int(lens[b])
        for g in range(nk):
            k = gather(ck, table, b, g, n)
            for r in range(r0, r1):
                lim = n - (r1 - r0) + (r - r0) + 1
                for h in range(g * hpg, (g + 1) * hpg):
                    if lim > 0:
                        out[b, g, :lim] += np.exp(k[:lim] @ q[r, h] * scale - lse[r, h])
    return out


def evict_order(weight, pos, n, sinks, recent):
    """Slots of one (sequence, KV head) in the order in which they stay."""
    def rank(j):
        if pos[j] < sinks or (recent is not None and pos[j] >= recent):
            return (0, 0.0, j)
        if np.isnan(weight[j]):
            return (1, 0.0, j)
        return (2, -float(weight[j]) + 0.0, j)
    return sorted(range(n), key=rank)


def evict(weight, pos, n, keep, sinks, recent):
    """Slots that move: (new length, [(to, from)]) of one (sequence, KV head)."""
    new = min(n, keep)
    stay = set(evict_order(weight, pos, n, sinks, recent)[:new])
    freed = [j for j in range(new) if j not in stay]
    moved = [j for j in range(new, n) if j in stay]
    return new, list(zip(freed, moved))
