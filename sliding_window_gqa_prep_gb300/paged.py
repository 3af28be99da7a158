"""Python binding of the rotary and paged-cache entry points (include/swa.h).

Beside the sliding-window path, for the layers that keep every key:
  rotary_turns(rot, theta, ...)                  -> turns [rot/2] (the schedule, once)
  rotary(x, pos, turns, ...)                     -> rotated rows (inverse: the gradient)
  paged_append(k, v, pos, cache_k, cache_v, ...) -> q_out; k and v enter the pages
  paged_attend(q, cache_k, cache_v, ...)         -> out [T][nh][hd]
  paged_weigh(q, lse, cache_k, ...)              -> weight each cached key received
  paged_evict(cache_k, cache_v, ...)             -> (lens, weights, positions) after
One step of a layer is append, attend and, where the cache has a budget, weigh and
now and then evict. Tensors of a call lie on one CUDA device; the call runs on that
device's current stream, or on ``stream`` (a stream of that device), where outputs
and workspaces that the caller does not pass are allocated too.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Tuple

import torch

from . import _abi

__all__ = ["rotary_freqs", "rotary_turns", "rotary", "paged_append", "paged_attend",
           "paged_attend_workspace_size", "paged_weigh", "paged_evict", "paged_evict_workspace_size"]

_TYPES = {torch.float32: _abi.SWA_F32, torch.bfloat16: _abi.SWA_BF16, torch.float16: _abi.SWA_F16}
_KINDS = {"plain": 0, "linear": 1, "base": 2, "parts": 3}
_I32, _F32 = torch.int32, torch.float32


def _arg(x, name, dev, shape=None, dtype=None, dense=True) -> int:
    """Device address of a checked tensor."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.device != dev:
        raise ValueError(f"{name} is on {x.device}, expected {dev}")
    if dtype is not None and x.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")
    if shape is not None and tuple(x.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected {shape}")
    if dense and not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return x.data_ptr()


def _opt(x, name, dev, shape=None, dtype=None) -> int:
    return 0 if x is None else _arg(x, name, dev, shape, dtype)


def _rows(x, name, dev, dtype) -> Tuple[int, int]:
    """Address and row stride of packed rows [T][heads][hd] with dense heads."""
    ptr = _arg(x, name, dev, dtype=dtype, dense=False)
    T, H, hd = x.shape
    if (x.stride(2) != 1 and hd > 1) or (x.stride(1) != hd and H > 1):
        raise ValueError(f"{name}: the heads of a row must be dense")
    return ptr, (x.stride(0) if T > 1 else H * hd)


@contextlib.contextmanager
def _place(dev, stream):
    """The call's device and stream as the current ones; yields the stream's handle."""
    if stream is not None and stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {dev}")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        yield torch.cuda.current_stream(dev).cuda_stream


def _lib():
    return _abi.load()


def _schedule(rot, theta, schedule, factor, orig_len, low, high):
    if schedule not in _KINDS:
        raise ValueError(f"schedule must be one of {sorted(_KINDS)}, got {schedule!r}")
    s = _abi.RotarySchedule()
    s.kind, s.rot, s.theta, s.factor = _KINDS[schedule], int(rot), float(theta), float(factor)
    s.orig_len, s.low, s.high = float(orig_len), float(low), float(high)
    if not 2 <= s.rot <= 1024:
        raise ValueError(f"rot must be even, 2 to 1024, got {rot}")
    f, t = (ctypes.c_double * (s.rot // 2))(), (ctypes.c_uint64 * (s.rot // 2))()
    _abi.check(_lib().swa_rotary_turns(ctypes.byref(s), f, t), "swa_rotary_turns")
    return list(f), list(t)


def rotary_freqs(rot, theta=10000.0, *, schedule="plain", factor=1.0, orig_len=0.0, low=1.0, high=32.0):
    """Frequencies [rot/2] in radians per position (f64, CPU) of a schedule: "plain",
    "linear" (positions divided by factor), "base" (theta raised so that the slowest pair
    turns factor times slower) or "parts" (pairs with at least `high` turns over orig_len
    positions as they are, with at most `low` divided by factor, mixed in between)."""
    return torch.tensor(_schedule(rot, theta, schedule, factor, orig_len, low, high)[0], dtype=torch.float64)


def rotary_turns(rot, theta=10000.0, *, schedule="plain", factor=1.0, orig_len=0.0, low=1.0, high=32.0,
                 device="cuda"):
    """The same schedule as the kernels take it: turns per position as 64-bit fixed point,
    an int64 tensor [rot/2] on the device. Make it once and keep it."""
    t = _schedule(rot, theta, schedule, factor, orig_len, low, high)[1]
    return torch.tensor([v - (1 << 64) if v >> 63 else v for v in t], dtype=torch.int64).to(device)


def rotary(x, pos, turns, *, interleaved: bool = False, inverse: bool = False, mag: float = 1.0, out=None,
           stream=None):
    """Rotary positions of packed rows x [T][H][hd] (f32, bf16 or f16; any row and head
    strides at multiples of 16 bytes): the first 2 * len(turns) features of every head turn
    by pos[row], the others are copied. inverse=True is the gradient of the call. out may
    be x."""
    if x.dim() != 3 or x.dtype not in _TYPES:
        raise ValueError("x must be [T][H][hd] in float32, bfloat16 or float16")
    T, H, hd = x.shape
    dev = x.device
    with _place(dev, stream) as handle:
        if out is None:
            out = torch.empty(T, H, hd, device=dev, dtype=x.dtype)
        a = _abi.RotaryArgs()
        a.x, a.out = _arg(x, "x", dev, dense=False), _arg(out, "out", dev, (T, H, hd), x.dtype, dense=False)
        for y, name in ((x, "x"), (out, "out")):
            if hd > 1 and y.stride(2) != 1:
                raise ValueError(f"{name}: the features of a head must be dense")
        a.T, a.H, a.hd, a.rot, a.dtype = T, H, hd, 2 * turns.numel(), _TYPES[x.dtype]
        # a stride along a dimension of one is free: the dense one then
        a.x_head, a.out_head = (x.stride(1), out.stride(1)) if H > 1 else (hd, hd)
        a.x_row, a.out_row = (x.stride(0), out.stride(0)) if T > 1 else (H * a.x_head, H * a.out_head)
        a.interleaved, a.inverse, a.mag = int(interleaved), int(inverse), float(mag)
        a.pos = _arg(pos, "pos", dev, (T,), _I32)
        a.turns = _arg(turns, "turns", dev, (turns.numel(),), torch.int64)
        _abi.check(_lib().swa_rotary(ctypes.byref(a), handle), "swa_rotary")
    return out


def _cache(c, cache_k, cache_v, page_table, row_start, lens, dev) -> None:
    if cache_k.dim() != 4 or cache_k.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("cache_k must be [num_pages][nk][page][hd] in bfloat16 or float16")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B][max_pages]")
    B = page_table.shape[0]
    c.k = _arg(cache_k, "cache_k", dev)
    c.v = c.k if cache_v is None else _arg(cache_v, "cache_v", dev, tuple(cache_k.shape), cache_k.dtype)
    c.num_pages, c.nk, c.page, c.hd = cache_k.shape
    c.B, c.max_pages, c.dtype = B, page_table.shape[1], _TYPES[cache_k.dtype]
    c.table = _arg(page_table, "page_table", dev, dtype=_I32)
    c.row_start = _opt(row_start, "row_start", dev, (B + 1,), _I32)
    c.lens = _arg(lens, "lens", dev, (B,), _I32)


def paged_append(k, v, pos, cache_k, cache_v, page_table, row_start, lens, *, q=None, q_out=None, turns=None,
                 interleaved: bool = False, mag: float = 1.0, slot_pos=None, weight=None, err=None, stream=None):
    """A chunk's rows enter the cache: k [T][nk][hd] rotated by pos (when turns is given) and
    v, rounded to the cache's type, go to the slots lens[b] - t_b + i of their sequence;
    lens counts the chunk's rows. q [T][nh][hd] is rotated and rounded into q_out, which is
    returned (None without q). slot_pos and weight [B][nk][cap], when given, get the new
    slots' positions and weight 0."""
    dev = cache_k.device
    with _place(dev, stream) as handle:
        a = _abi.PagedAppendArgs()
        _cache(a.cache, cache_k, cache_v, page_table, row_start, lens, dev)
        if row_start is None:
            raise ValueError("row_start is required")
        nk, hd, cap = a.cache.nk, a.cache.hd, a.cache.max_pages * a.cache.page
        if k.dtype not in _TYPES:
            raise ValueError("k must be float32, bfloat16 or float16")
        T = k.shape[0]
        if tuple(k.shape) != (T, nk, hd) or tuple(v.shape) != (T, nk, hd):
            raise ValueError(f"k and v must be [T][{nk}][{hd}]")
        a.T, a.src, a.interleaved, a.mag = T, _TYPES[k.dtype], int(interleaved), float(mag)
        a.k, a.k_row = _rows(k, "k", dev, k.dtype)
        a.v, a.v_row = _rows(v, "v", dev, k.dtype)
        if q is not None:
            if q.dim() != 3 or q.shape[0] != T or q.shape[2] != hd:
                raise ValueError(f"q must be [{T}][nh][{hd}]")
            a.nh = q.shape[1]
            a.q, a.q_row = _rows(q, "q", dev, k.dtype)
            if q_out is None:
                q_out = torch.empty(T, a.nh, hd, device=dev, dtype=cache_k.dtype)
            a.q_out = _arg(q_out, "q_out", dev, (T, a.nh, hd), cache_k.dtype)
        elif q_out is not None:
            raise ValueError("q_out without q")
        a.pos = _opt(pos, "pos", dev, (T,), _I32)
        if turns is not None:
            a.turns, a.rot = _arg(turns, "turns", dev, (turns.numel(),), torch.int64), 2 * turns.numel()
        a.slot_pos = _opt(slot_pos, "slot_pos", dev, (a.cache.B, nk, cap), _I32)
        a.weight = _opt(weight, "weight", dev, (a.cache.B, nk, cap), _F32)
        a.err = _opt(err, "err", dev, (1,), _I32)
        _abi.check(_lib().swa_paged_append(ctypes.byref(a), handle), "swa_paged_append")
    return q_out


def _sizes(a, B, T, nh, nk, hd, page, max_pages, max_rows, dtype):
    c = a.cache
    c.B, c.nk, c.hd, c.page, c.max_pages, c.dtype = B, nk, hd, page, max_pages, _TYPES[dtype]
    a.T, a.nh, a.max_rows = T, nh, max_rows


def paged_attend_workspace_size(B, T, nh, nk, hd, page, max_pages, max_rows, dtype=torch.bfloat16) -> int:
    """Workspace bytes of paged_attend on the current device."""
    a = _abi.PagedAttendArgs()
    _sizes(a, B, T, nh, nk, hd, page, max_pages, max_rows, dtype)
    n = int(_lib().swa_paged_attend_workspace_size(ctypes.byref(a)))
    if n == 0:
        raise _abi.SwaError(_abi.SWA_E_SHAPE, "swa_paged_attend_workspace_size")
    return n


def paged_attend(q, cache_k, cache_v, page_table, row_start, lens, scale: float, *, max_rows: int, out=None,
                 lse=None, workspace=None, err=None, ev_start=None, ev_stop=None, stream=None):
    """Causal attention of a chunk's rows q [T][nh][hd] (the cache's type) over the paged
    cache, their own keys already appended: row i of sequence b sees the slots below
    lens[b] - t_b + i + 1. max_rows bounds the rows of a sequence. out [T][nh][hd] in the
    cache's type or float32; lse [T][nh] f32, when given, gets log sum exp of the scores.
    Rows of no sequence are left as they were (zeros in a new out)."""
    dev = q.device
    with _place(dev, stream) as handle:
        a = _abi.PagedAttendArgs()
        _cache(a.cache, cache_k, cache_v, page_table, row_start, lens, dev)
        if row_start is None:
            raise ValueError("row_start is required")
        if q.dim() != 3 or q.shape[2] != a.cache.hd:
            raise ValueError(f"q must be [T][nh][{a.cache.hd}]")
        T, nh, hd = q.shape
        a.T, a.nh, a.max_rows, a.scale = T, nh, int(max_rows), float(scale)
        a.q, a.q_row = _rows(q, "q", dev, cache_k.dtype)
        if out is None:
            out = torch.zeros(T, nh, hd, device=dev, dtype=q.dtype)
        if out.dtype not in (q.dtype, _F32):
            raise ValueError(f"out must be {q.dtype} or float32")
        a.out, a.out_f32 = _arg(out, "out", dev, (T, nh, hd)), int(out.dtype == _F32)
        a.lse = _opt(lse, "lse", dev, (T, nh), _F32)
        if workspace is None:
            need = int(_lib().swa_paged_attend_workspace_size(ctypes.byref(a)))
            workspace = torch.empty(max(need, 1), device=dev, dtype=torch.uint8)
        a.workspace, a.workspace_bytes = _arg(workspace, "workspace", dev, dtype=torch.uint8), workspace.numel()
        a.err = _opt(err, "err", dev, (1,), _I32)
        a.ev_start = ev_start.cuda_event if ev_start is not None else None
        a.ev_stop = ev_stop.cuda_event if ev_stop is not None else None
        _abi.check(_lib().swa_paged_attend(ctypes.byref(a), handle), "swa_paged_attend")
    return out


def paged_weigh(q, lse, cache_k, page_table, row_start, lens, scale: float, *, max_rows: int, weight=None, out=None,
                err=None, stream=None):
    """The attention weight every cached key received from the rows q, added to weight
    [B][nk][cap] (None: zeros): out[b][g][j] = weight[b][g][j] + sum over rows that see slot j
    and heads of g of exp(scale <q, k_j> - lse). lse [T][nh] is paged_attend's for the same
    rows. out may be weight; entries from lens[b] on are left as they were (zeros in a new
    out)."""
    dev = q.device
    with _place(dev, stream) as handle:
        a = _abi.PagedWeighArgs()
        _cache(a.cache, cache_k, None, page_table, row_start, lens, dev)
        if row_start is None:
            raise ValueError("row_start is required")
        if q.dim() != 3 or q.shape[2] != a.cache.hd:
            raise ValueError(f"q must be [T][nh][{a.cache.hd}]")
        T, nh, _ = q.shape
        shape = (a.cache.B, a.cache.nk, a.cache.max_pages * a.cache.page)
        a.T, a.nh, a.max_rows, a.scale = T, nh, int(max_rows), float(scale)
        a.q, a.q_row = _rows(q, "q", dev, cache_k.dtype)
        a.lse = _arg(lse, "lse", dev, (T, nh), _F32)
        a.weight = _opt(weight, "weight", dev, shape, _F32)
        if out is None:
            out = torch.zeros(shape, device=dev, dtype=_F32)
        a.out = _arg(out, "out", dev, shape, _F32)
        a.err = _opt(err, "err", dev, (1,), _I32)
        _abi.check(_lib().swa_paged_weigh(ctypes.byref(a), handle), "swa_paged_weigh")
    return out


def paged_evict_workspace_size(B, nk, page, max_pages, keep) -> int:
    """Workspace bytes of paged_evict."""
    a = _abi.PagedEvictArgs()
    c = a.cache
    c.B, c.nk, c.page, c.max_pages, a.keep = B, nk, page, max_pages, int(keep)
    n = int(_lib().swa_paged_evict_workspace_size(ctypes.byref(a)))
    if n == 0:
        raise _abi.SwaError(_abi.SWA_E_SHAPE, "swa_paged_evict_workspace_size")
    return n


def paged_evict(cache_k, cache_v, page_table, lens, weight, slot_pos, keep: int, *, recent_from=None, sinks: int = 0,
                weight_out=None, slot_pos_out=None, lens_out=None, workspace=None, err=None, stream=None):
    """Cut every sequence's cache to at most `keep` keys per KV head: those at positions
    below sinks or from recent_from[b] on first, then by weight. Kept keys behind the new
    length move into the freed slots (within the pages, in place); weight and slot_pos
    [B][nk][cap] are read, their new values and the new lengths written to the outputs.
    Returns (lens_out, weight_out, slot_pos_out)."""
    dev = cache_k.device
    with _place(dev, stream) as handle:
        a = _abi.PagedEvictArgs()
        _cache(a.cache, cache_k, cache_v, page_table, None, lens, dev)
        B, shape = a.cache.B, (a.cache.B, a.cache.nk, a.cache.max_pages * a.cache.page)
        a.keep, a.sinks = int(keep), int(sinks)
        a.weight, a.slot_pos = _arg(weight, "weight", dev, shape, _F32), _arg(slot_pos, "slot_pos", dev, shape, _I32)
        a.recent_from = _opt(recent_from, "recent_from", dev, (B,), _I32)
        if weight_out is None:
            weight_out = torch.zeros_like(weight)
        if slot_pos_out is None:
            slot_pos_out = torch.zeros_like(slot_pos)
        if lens_out is None:
            lens_out = torch.empty_like(lens)
        a.weight_out = _arg(weight_out, "weight_out", dev, shape, _F32)
        a.slot_pos_out = _arg(slot_pos_out, "slot_pos_out", dev, shape, _I32)
        a.lens_out = _arg(lens_out, "lens_out", dev, (B,), _I32)
        if workspace is None:
            need = int(_lib().swa_paged_evict_workspace_size(ctypes.byref(a)))
            workspace = torch.empty(max(need, 1), device=dev, dtype=torch.uint8)
        a.workspace, a.workspace_bytes = _arg(workspace, "workspace", dev, dtype=torch.uint8), workspace.numel()
        a.err = _opt(err, "err", dev, (1,), _I32)
        _abi.check(_lib().swa_paged_evict(ctypes.byref(a), handle), "swa_paged_evict")
    return lens_out, weight_out, slot_pos_out
