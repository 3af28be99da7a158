"""The 4-bit paged cache in 64 bits on the GPU, for batches that are too large for the oracle's loops:
the encoding and the attention of oracle/paged4_oracle.py over whole tensors, and a batch of random keys.
Shares no code with the CUDA path."""
import math

import torch

from oracle import paged4_oracle as p4

U8, E4 = torch.uint8, torch.float8_e4m3fn


def _grid(g, device):
    return torch.tensor(g, dtype=torch.float64, device=device)


def nearest(x, grid):
    """Index of the nearest grid value (ascending), the even index of two as near."""
    i = torch.searchsorted(grid, x).clamp(max=len(grid) - 1)
    lo = (i - 1).clamp(min=0)
    below, above = x - grid[lo], grid[i] - x
    up = (i == 0) | (above < below) | ((above == below) & (i % 2 == 0))
    return torch.where(up, i, lo)


def encode(x, exp):
    """f64 rows [..][hd] -> (bytes [..][hd / 2], scale bits [..][hd / 16])."""
    e4m3, levels = _grid(p4.E4M3[:127], x.device), _grid(p4.LEVELS, x.device)
    b = x.unflatten(-1, (-1, 16))
    fine = b.isfinite().all(-1)
    b = torch.where(fine[..., None], b, 0.0)
    s = nearest((b.abs().amax(-1) * 2.0 ** -exp / 6.0).clamp(max=448.0), e4m3)
    u = (e4m3[s] * 2.0 ** exp)[..., None]
    c = torch.where(u > 0, nearest(b.abs() / torch.where(u > 0, u, 1.0), levels), 0)
    c = c + 8 * ((c > 0) & (b < 0))
    c = torch.where(fine[..., None], c, 0).flatten(-2)
    return (c[..., 0::2] + 16 * c[..., 1::2]).to(U8), torch.where(fine, s, 127).to(U8)


def decode(codes, scales, exp):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = _grid(p4.LEVELS, codes.device)[c & 7] * (1 - 2 * (c >> 3))
    return v * (_grid(p4.E4M3, codes.device)[scales.view(U8).long()] * 2.0 ** exp).repeat_interleave(16, -1)


def rotate(x, pos, turns, interleaved=False, mag=1.0):
    """The rotary positions of rows [T][H][hd] in f64, by turns [rot / 2] (64-bit fixed point, whole ones drop out)."""
    x = x.double()
    rot = 2 * len(turns)
    a = (pos.long()[:, None, None] * turns).double() * (2.0 ** -63 * math.pi)
    c, s = a.cos() * mag, a.sin() * mag
    at = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    u, v = x[..., at[0]], x[..., at[1]]
    y = x.clone()
    y[..., at[0]], y[..., at[1]] = u * c - v * s, v * c + u * s
    return y


class Cache:
    """A ragged batch over random codes with scales 2^-3 .. 1; slots that no sequence holds have scale NaN."""

    def __init__(self, t, lens, nk, hd, page, seed=0, pad=0, wide=0, exps=(0, 0)):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.t, self.n, self.nk, self.hd, self.page, self.exps = list(t), list(lens), nk, hd, page, exps
        need = [max(1, -(-x // page)) for x in self.n]
        width, pool = max(need + [wide]), sum(need) + 2
        order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        first = torch.tensor([0] + need, device="cuda").cumsum(0)[:-1]
        col = torch.arange(width, device="cuda")
        held = col < torch.tensor(need, device="cuda")[:, None]
        self.table = torch.where(held, order[(first[:, None] + col).clamp(max=pool - 1)], -1).to(torch.int32).contiguous()
        pools = []
        lens_d = torch.tensor(self.n, device="cuda")
        j = torch.arange(width * page, device="cuda")
        live = (j < lens_d[:, None]).view(len(self.n), width, page)
        where = live.nonzero(as_tuple=True)
        at = self.table[where[0], where[1]].long()
        for _ in range(2):
            codes = torch.randint(0, 256, (pool, nk, page, hd // 2), generator=g, device="cuda", dtype=torch.int32).to(U8)
            scales = torch.full((pool, nk, page, hd // 16), 127, dtype=U8, device="cuda")
            scales[at, :, where[2]] = torch.randint(32, 57, (at.numel(), nk, hd // 16), generator=g, device="cuda", dtype=torch.int32).to(U8)
            pools += [codes, scales.view(E4)]
        self.pools = pools
        start = [0]
        for x in self.t:
            start.append(start[-1] + x)
        self.start, self.live, self.T = start, start[-1], start[-1] + pad
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
        self.args = (*pools, self.table, i32(start), i32(self.n))
        self.exp = {"exp_k": exps[0], "exp_v": exps[1]}

    def keys(self, b):
        """(K, V) [n][nk][hd] of sequence b in f64."""
        j = torch.arange(self.n[b], device="cuda")
        at = self.table[b].long()[j // self.page], slice(None), j % self.page
        k, ks, v, vs = self.pools
        return decode(k[at], ks.view(U8)[at], self.exps[0]), decode(v[at], vs.view(U8)[at], self.exps[1])

    def attend(self, q, scale, window=0, sinks=0):
        """(out, lse, mean of |v| under the same weights, largest sum |q_i k_i| * scale) in f64."""
        nh = q.shape[1]
        hpg = nh // self.nk
        q = q.double()
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        absv, lse = torch.zeros_like(out), torch.full(q.shape[:2], -float("inf"), dtype=torch.float64, device="cuda")
        sabs = torch.zeros_like(lse)
        for b, (t, n) in enumerate(zip(self.t, self.n)):
            if t == 0 or n == 0:
                continue
            k, v = (x.repeat_interleave(hpg, 1).transpose(0, 1) for x in self.keys(b))      # [nh][n][hd]
            rows = slice(self.start[b], self.start[b + 1])
            x = torch.einsum("thd,hnd->thn", q[rows], k) * scale
            own = (n - t + torch.arange(t, device="cuda"))[:, None, None]
            j = torch.arange(n, device="cuda")
            hidden = j > own
            if window:
                hidden = hidden | ((j <= own - window) & (j >= sinks))
            x = x.masked_fill(hidden, -float("inf"))
            m = x.amax(-1, keepdim=True)
            p = torch.where(m.isneginf(), 0.0, (x - m).exp())
            z = p.sum(-1)
            some = z > 0
            w = p / torch.where(some, z, 1.0)[..., None]
            out[rows], absv[rows] = torch.einsum("thn,hnd->thd", w, v), torch.einsum("thn,hnd->thd", w, v.abs())
            lse[rows] = torch.where(some, m[..., 0] + z.log(), -float("inf"))
            s = torch.einsum("thd,hnd->thn", q[rows].abs(), k.abs()).masked_fill(hidden, 0.0) * scale
            sabs[rows] = s.amax(-1)
        return out, lse, absv, sabs
