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

import ctypes
import functools
import struct
from typing import Tuple

import torch

from . import _abi

__all__ = ["rotary_freqs", "rotary_turns", "rotary", "paged_append", "paged_attend",
           "paged_attend_workspace_size", "paged_weigh", "paged_evict", "paged_evict_workspace_size"]

_TYPES = {torch.float32: _abi.SWA_F32, torch.bfloat16: _abi.SWA_BF16, torch.float16: _abi.SWA_F16}
_TYPES16 = {torch.bfloat16: _abi.SWA_BF16, torch.float16: _abi.SWA_F16}
_KINDS = {"plain": 0, "linear": 1, "base": 2, "parts": 3}
_I32, _I64, _F32, _U8 = torch.int32, torch.int64, torch.float32, torch.uint8

# The argument structs of include/swa.h as struct formats (native alignment): one pack
# call costs a decode step less host time than setting a ctypes field at a time.
_CACHE = "7i5P"                                        # swa_paged_cache
_ROTARY = struct.Struct("@7ifP2qP2q2P")                # swa_rotary_args
_APPEND = struct.Struct("@" + _CACHE + "5if3P3q6P")    # swa_paged_append_args
_ATTEND = struct.Struct("@" + _CACHE + "4ifPq3PN3P")   # swa_paged_attend_args
_WEIGH = struct.Struct("@" + _CACHE + "3ifPq4P")       # swa_paged_weigh_args
_EVICT = struct.Struct("@" + _CACHE + "2i7PNP")        # swa_paged_evict_args


def _complain(x, name, dev, dtype, shape):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.get_device() != dev:
        raise ValueError(f"{name} is on {x.device}, expected cuda:{dev}")
    if x.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")
    if shape is not None and tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _arg(x, name, dev, dtype, shape=None) -> int:
    """Device address of a checked dense tensor. (Half of a small call's host time is spent
    here: no more is asked than what has to be.)"""
    try:
        if x.get_device() == dev and x.dtype is dtype and (shape is None or x.shape == shape) and x.is_contiguous():
            return x.data_ptr()
    except AttributeError:
        pass
    _complain(x, name, dev, dtype, shape)


def _opt(x, name, dev, dtype, shape=None) -> int:
    return 0 if x is None else _arg(x, name, dev, dtype, shape)


def _rows(x, name, dev, dtype, shape) -> Tuple[int, int]:
    """Address and row stride of packed rows [T][heads][hd] with dense heads."""
    try:
        if x.get_device() == dev and x.dtype is dtype and x.shape == shape:
            T, H, hd = shape
            if x.is_contiguous():
                return x.data_ptr(), H * hd
            row, head, one = x.stride()
            if one != 1 or (head != hd and H > 1):
                raise ValueError(f"{name}: the heads of a row must be dense")
            return x.data_ptr(), (row if T > 1 else H * hd)
    except AttributeError:
        pass
    _complain(x, name, dev, dtype, shape)


_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _place(x, name, stream):
    """The device of a call's first tensor and the handle of the stream it runs on: the current
    one. No handle where another device or `stream` has to become current first (_there)."""
    dev = x.get_device() if isinstance(x, torch.Tensor) else -1
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if stream is None and _current_device() == dev:
        return dev, _current_stream(dev)
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors are on cuda:{dev}")
    return dev, None


def _there(fn, args):
    """The call fn(**args) on the device args["dev"] and on args["stream"]."""
    dev, stream, _ = args.pop("dev"), args.pop("stream"), args.pop("on")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        return fn(**args)


_lib = _abi.load


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


def rotary(x, pos, turns, *, interleaved: bool = False, inverse: bool = False, mag: float = 1.0, out=None, stream=None):
    """Rotary positions of packed rows x [T][H][hd] (f32, bf16 or f16; any row and head
    strides at multiples of 16 bytes): the first 2 * len(turns) features of every head turn
    by pos[row], the others are copied. inverse=True is the gradient of the call. out may
    be x."""
    dev, on = _place(x, "x", stream)
    if on is None:
        return _there(rotary, locals())
    if x.dim() != 3 or x.dtype not in _TYPES:
        raise ValueError("x must be [T][H][hd] in float32, bfloat16 or float16")
    T, H, hd = x.shape
    if out is None:
        out = torch.empty(T, H, hd, device=x.device, dtype=x.dtype)
    elif out.get_device() != dev or out.dtype != x.dtype or out.shape != x.shape:
        _complain(out, "out", dev, x.dtype, x.shape)
    x_row, x_head, x_one = x.stride()
    o_row, o_head, o_one = out.stride()
    if (x_one != 1 or o_one != 1) and hd > 1:
        raise ValueError("x and out: the features of a head must be dense")
    # a stride along a dimension of one is free: the dense one then
    if H <= 1:
        x_head = o_head = hd
    if T <= 1:
        x_row, o_row = H * x_head, H * o_head
    n = turns.numel()
    a = _ROTARY.pack(T, H, hd, 2 * n, _TYPES[x.dtype], bool(interleaved), bool(inverse), mag,
                     x.data_ptr(), x_row, x_head, out.data_ptr(), o_row, o_head,
                     _arg(pos, "pos", dev, _I32, (T,)), _arg(turns, "turns", dev, _I64, (n,)))
    _abi.check(_lib().swa_rotary(a, on), "swa_rotary")
    return out


def _cache(cache_k, cache_v, page_table, row_start, lens, dev):
    """The fields of a swa_paged_cache and the capacity of a sequence. (cache_v is cache_k where
    the call reads no values.)"""
    try:
        dtype, shape, pages = cache_k.dtype, cache_k.shape, page_table.shape
    except AttributeError:
        raise ValueError("cache_k and page_table must be CUDA tensors") from None
    if len(shape) != 4 or dtype not in _TYPES16:
        raise ValueError("cache_k must be [num_pages][nk][page][hd] in bfloat16 or float16")
    if len(pages) != 2:
        raise ValueError("page_table must be [B][max_pages]")
    num_pages, nk, page, hd = shape
    B, max_pages = pages
    k = _arg(cache_k, "cache_k", dev, dtype)
    v = k if cache_v is cache_k else _arg(cache_v, "cache_v", dev, dtype, shape)
    return (B, nk, hd, page, num_pages, max_pages, _TYPES16[dtype], k, v,
            _arg(page_table, "page_table", dev, _I32),
            0 if row_start is None else _arg(row_start, "row_start", dev, _I32, (B + 1,)),
            _arg(lens, "lens", dev, _I32, (B,))), max_pages * page


def paged_append(k, v, pos, cache_k, cache_v, page_table, row_start, lens, *, q=None, q_out=None, turns=None,
                 interleaved: bool = False, mag: float = 1.0, slot_pos=None, weight=None, err=None,
                 stream=None):
    """A chunk's rows enter the cache: k [T][nk][hd] rotated by pos (when turns is given) and
    v, rounded to the cache's type, go to the slots lens[b] - t_b + i of their sequence;
    lens counts the chunk's rows. q [T][nh][hd] is rotated and rounded into q_out, which is
    returned (None without q). slot_pos and weight [B][nk][cap], when given, get the new
    slots' positions and weight 0."""
    dev, on = _place(k, "k", stream)
    if on is None:
        return _there(paged_append, locals())
    cache, cap = _cache(cache_k, cache_v, page_table, row_start, lens, dev)
    B, nk, hd = cache[:3]
    if row_start is None:
        raise ValueError("row_start is required")
    if k.dtype not in _TYPES:
        raise ValueError("k must be float32, bfloat16 or float16")
    T = k.shape[0]
    kp, k_row = _rows(k, "k", dev, k.dtype, (T, nk, hd))
    vp, v_row = _rows(v, "v", dev, k.dtype, (T, nk, hd))
    nh = qp = q_row = qo = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError(f"q must be [{T}][nh][{hd}]")
        nh = q.shape[1]
        qp, q_row = _rows(q, "q", dev, k.dtype, (T, nh, hd))
        if q_out is None:
            q_out = torch.empty(T, nh, hd, device=q.device, dtype=cache_k.dtype)
        qo = _arg(q_out, "q_out", dev, cache_k.dtype, (T, nh, hd))
    elif q_out is not None:
        raise ValueError("q_out without q")
    n = 0 if turns is None else turns.numel()
    a = _APPEND.pack(*cache, T, nh, 2 * n, _TYPES[k.dtype], bool(interleaved), mag, qp, kp, vp, q_row, k_row, v_row,
                     qo, _opt(pos, "pos", dev, _I32, (T,)), _opt(turns, "turns", dev, _I64, (n,)),
                     _opt(slot_pos, "slot_pos", dev, _I32, (B, nk, cap)), _opt(weight, "weight", dev, _F32, (B, nk, cap)),
                     _opt(err, "err", dev, _I32, (1,)))
    _abi.check(_lib().swa_paged_append(a, on), "swa_paged_append")
    return q_out


def paged_attend_workspace_size(B, T, nh, nk, hd, page, max_pages, max_rows, dtype=torch.bfloat16) -> int:
    """Workspace bytes of paged_attend on the current device (1: none is needed)."""
    a = _ATTEND.pack(B, nk, hd, page, 0, max_pages, _TYPES[dtype], 0, 0, 0, 0, 0, T, nh, max_rows, 0, 0.0, 0, 0, 0, 0,
                     0, 0, 0, 0, 0)
    n = int(_lib().swa_paged_attend_workspace_size(a))
    if n == 0:
        raise _abi.SwaError(_abi.SWA_E_SHAPE, "swa_paged_attend_workspace_size")
    return n


@functools.lru_cache(maxsize=1024)
def _attend_need(dev, B, T, nh, nk, hd, page, max_pages, max_rows, dtype) -> int:
    """paged_attend_workspace_size for device dev (the current one); 0 for sizes it refuses."""
    a = _ATTEND.pack(B, nk, hd, page, 0, max_pages, _TYPES[dtype], 0, 0, 0, 0, 0, T, nh, max_rows, 0, 0.0, 0, 0, 0, 0,
                     0, 0, 0, 0, 0)
    return int(_lib().swa_paged_attend_workspace_size(a))


def paged_attend(q, cache_k, cache_v, page_table, row_start, lens, scale: float, *, max_rows: int, out=None,
                 lse=None, workspace=None, err=None, ev_start=None, ev_stop=None, stream=None):
    """Causal attention of a chunk's rows q [T][nh][hd] (the cache's type) over the paged
    cache, their own keys already appended: row i of sequence b sees the slots below
    lens[b] - t_b + i + 1. max_rows bounds the rows of a sequence. out [T][nh][hd] in the
    cache's type or float32; lse [T][nh] f32, when given, gets log sum exp of the scores.
    Rows of no sequence are left as they were (zeros in a new out)."""
    dev, on = _place(q, "q", stream)
    if on is None:
        return _there(paged_attend, locals())
    cache, _ = _cache(cache_k, cache_v, page_table, row_start, lens, dev)
    B, nk, hd, page, _, max_pages = cache[:6]
    if row_start is None:
        raise ValueError("row_start is required")
    if q.dim() != 3:
        raise ValueError(f"q must be [T][nh][{hd}]")
    T, nh = q.shape[:2]
    qp, q_row = _rows(q, "q", dev, cache_k.dtype, (T, nh, hd))
    if out is None:
        out = torch.zeros(T, nh, hd, device=q.device, dtype=q.dtype)
    wide = out.dtype == _F32
    op = _arg(out, "out", dev, _F32 if wide else q.dtype, (T, nh, hd))
    ws = size = 0
    if workspace is not None:
        ws, size = _arg(workspace, "workspace", dev, _U8), workspace.numel()
    else:
        size = _attend_need(dev, B, T, nh, nk, hd, page, max_pages, max_rows, cache_k.dtype)
        if size > 1:
            workspace = torch.empty(size, device=q.device, dtype=_U8)
            ws = workspace.data_ptr()
    a = _ATTEND.pack(*cache, T, nh, max_rows, wide, scale, qp, q_row, op, _opt(lse, "lse", dev, _F32, (T, nh)),
                     ws, size, _opt(err, "err", dev, _I32, (1,)),
                     ev_start.cuda_event if ev_start is not None else 0, ev_stop.cuda_event if ev_stop is not None else 0)
    _abi.check(_lib().swa_paged_attend(a, on), "swa_paged_attend")
    return out


def paged_weigh(q, lse, cache_k, page_table, row_start, lens, scale: float, *, max_rows: int, weight=None, out=None,
                err=None, stream=None):
    """The attention weight every cached key received from the rows q, added to weight
    [B][nk][cap] (None: zeros): out[b][g][j] = weight[b][g][j] + sum over rows that see slot j
    and heads of g of exp(scale <q, k_j> - lse). lse [T][nh] is paged_attend's for the same
    rows. out may be weight; entries from lens[b] on are left as they were (zeros in a new
    out)."""
    dev, on = _place(q, "q", stream)
    if on is None:
        return _there(paged_weigh, locals())
    cache, cap = _cache(cache_k, cache_k, page_table, row_start, lens, dev)
    B, nk, hd = cache[:3]
    if row_start is None:
        raise ValueError("row_start is required")
    if q.dim() != 3:
        raise ValueError(f"q must be [T][nh][{hd}]")
    T, nh = q.shape[:2]
    qp, q_row = _rows(q, "q", dev, cache_k.dtype, (T, nh, hd))
    if out is None:
        out = torch.zeros(B, nk, cap, device=q.device, dtype=_F32)
    a = _WEIGH.pack(*cache, T, nh, max_rows, scale, qp, q_row, _arg(lse, "lse", dev, _F32, (T, nh)),
                    _opt(weight, "weight", dev, _F32, (B, nk, cap)), _arg(out, "out", dev, _F32, (B, nk, cap)),
                    _opt(err, "err", dev, _I32, (1,)))
    _abi.check(_lib().swa_paged_weigh(a, on), "swa_paged_weigh")
    return out


def paged_evict_workspace_size(B, nk, page, max_pages, keep) -> int:
    """Workspace bytes of paged_evict."""
    n = _evict_need(B, nk, page, max_pages, int(keep))
    if n == 0:
        raise _abi.SwaError(_abi.SWA_E_SHAPE, "swa_paged_evict_workspace_size")
    return n


@functools.lru_cache(maxsize=1024)
def _evict_need(B, nk, page, max_pages, keep) -> int:
    return int(_lib().swa_paged_evict_workspace_size(
        _EVICT.pack(B, nk, 0, page, 0, max_pages, 0, 0, 0, 0, 0, 0, keep, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)))


def paged_evict(cache_k, cache_v, page_table, lens, weight, slot_pos, keep: int, *, recent_from=None, sinks: int = 0,
                weight_out=None, slot_pos_out=None, lens_out=None, workspace=None, err=None, stream=None):
    """Cut every sequence's cache to at most `keep` keys per KV head: those at positions
    below sinks or from recent_from[b] on first, then by weight. Kept keys behind the new
    length move into the freed slots (within the pages, in place); weight and slot_pos
    [B][nk][cap] are read, their new values and the new lengths written to the outputs.
    Returns (lens_out, weight_out, slot_pos_out)."""
    dev, on = _place(cache_k, "cache_k", stream)
    if on is None:
        return _there(paged_evict, locals())
    cache, cap = _cache(cache_k, cache_v, page_table, None, lens, dev)
    B, nk = cache[:2]
    shape = (B, nk, cap)
    wp, pp = _arg(weight, "weight", dev, _F32, shape), _arg(slot_pos, "slot_pos", dev, _I32, shape)
    if weight_out is None:
        weight_out = torch.zeros_like(weight)
    if slot_pos_out is None:
        slot_pos_out = torch.zeros_like(slot_pos)
    if lens_out is None:
        lens_out = torch.empty_like(lens)
    if workspace is None:
        size = max(_evict_need(B, nk, cache[3], cache[5], keep), 1)
        workspace = torch.empty(size, device=cache_k.device, dtype=_U8)
        ws = workspace.data_ptr()
    else:
        ws, size = _arg(workspace, "workspace", dev, _U8), workspace.numel()
    a = _EVICT.pack(*cache, keep, sinks, wp, pp, _opt(recent_from, "recent_from", dev, _I32, (B,)),
                    _arg(weight_out, "weight_out", dev, _F32, shape), _arg(slot_pos_out, "slot_pos_out", dev, _I32, shape),
                    _arg(lens_out, "lens_out", dev, _I32, (B,)), ws, size, _opt(err, "err", dev, _I32, (1,)))
    _abi.check(_lib().swa_paged_evict(a, on), "swa_paged_evict")
    return lens_out, weight_out, slot_pos_out
