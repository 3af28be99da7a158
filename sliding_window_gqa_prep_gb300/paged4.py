"""Python binding of the 4-bit paged cache and of the calls that share pages (include/swa.h).

The paged cache of paged.py in 4.5 bits a feature: blocks of 16 features hold a scale
(float8_e4m3fn) and 16 codes (e2m1, two a byte), value = code * scale * 2^exp.
  paged4_append(k, v, pos, cache_k, scale_k, ...)  -> q_out; k and v enter the pages
  paged4_read(cache_k, scale_k, ...)               -> (k, v) rows as the cache holds them
  paged4_attend(q, cache_k, scale_k, ...)          -> out [T][nh][hd], window and sinks
A cache is four pools: cache_k, cache_v uint8 [num_pages][nk][page][hd / 2] and scale_k, scale_v
float8_e4m3fn [num_pages][nk][page][hd / 16]; exp_k and exp_v are the same in every call of it.
For the pools of any paged cache, in 4 or in 16 bits:
  paged_fork(pools, table, lens, refs, parent, page, ...)  -> the next batch's tables
  paged_compact(pools, table, refs, ...)                   -> pages in use to the front
Tensors of a call lie on one CUDA device; the call runs on that device's current stream, or on
``stream`` (a stream of that device), where outputs and workspaces that the caller does not
pass are allocated too.
"""
from __future__ import annotations

import functools
import struct

import torch

from . import _abi
from .paged import (_F32, _I32, _I64, _TYPES, _TYPES16, _U8, _arg, _complain, _lib, _opt, _place, _rows, _there)

__all__ = ["paged4_append", "paged4_read", "paged4_attend", "paged4_attend_workspace_size", "paged_fork",
           "paged_fork_workspace_size", "paged_compact", "paged_compact_workspace_size"]

_E4M3 = torch.float8_e4m3fn
_CACHE = "8i7P"                                        # swa_paged4_cache
_APPEND = struct.Struct("@" + _CACHE + "6if3P3q4P")    # swa_paged4_append_args
_READ = struct.Struct("@" + _CACHE + "2i3P")           # swa_paged4_read_args
_ATTEND = struct.Struct("@" + _CACHE + "7ifPq3PN3P")   # swa_paged4_attend_args
_POOLS = "2i%dP%dq" % (_abi.SWA_MAX_POOLS, _abi.SWA_MAX_POOLS)   # swa_page_pools
_FORK = struct.Struct("@" + _POOLS + "4i10PNP")        # swa_paged_fork_args
_COMPACT = struct.Struct("@" + _POOLS + "2i7PNP")      # swa_paged_compact_args


def _cache4(cache_k, scale_k, cache_v, scale_v, page_table, row_start, lens, exp_k, exp_v, dev):
    """The fields of a swa_paged4_cache. (Checked in one expression first: seven calls of _arg take a
    microsecond longer, and name what is wrong.)"""
    try:
        shape, pages = cache_k.shape, page_table.shape
    except AttributeError:
        raise ValueError("cache_k and page_table must be CUDA tensors") from None
    if len(shape) != 4:
        raise ValueError("cache_k must be [num_pages][nk][page][hd / 2]")
    if len(pages) != 2:
        raise ValueError("page_table must be [B][max_pages]")
    num_pages, nk, page, bytes_ = shape
    hd = 2 * bytes_
    scales = (num_pages, nk, page, hd // 16)
    B, max_pages = pages
    try:
        if (cache_k.dtype is _U8 and cache_v.dtype is _U8 and scale_k.dtype is _E4M3 and scale_v.dtype is _E4M3
                and page_table.dtype is _I32 and row_start.dtype is _I32 and lens.dtype is _I32
                and cache_v.shape == shape and scale_k.shape == scales and scale_v.shape == scales
                and row_start.shape == (B + 1,) and lens.shape == (B,)
                and dev == cache_k.get_device() == cache_v.get_device() == scale_k.get_device() == scale_v.get_device()
                == page_table.get_device() == row_start.get_device() == lens.get_device()
                and cache_k.is_contiguous() and cache_v.is_contiguous() and scale_k.is_contiguous() and scale_v.is_contiguous()
                and page_table.is_contiguous() and row_start.is_contiguous() and lens.is_contiguous()):
            return (B, nk, hd, page, num_pages, max_pages, exp_k, exp_v, cache_k.data_ptr(), scale_k.data_ptr(),
                    cache_v.data_ptr(), scale_v.data_ptr(), page_table.data_ptr(), row_start.data_ptr(), lens.data_ptr())
    except AttributeError:
        pass
    return (B, nk, hd, page, num_pages, max_pages, exp_k, exp_v,
            _arg(cache_k, "cache_k", dev, _U8), _arg(scale_k, "scale_k", dev, _E4M3, scales),
            _arg(cache_v, "cache_v", dev, _U8, shape), _arg(scale_v, "scale_v", dev, _E4M3, scales),
            _arg(page_table, "page_table", dev, _I32), _arg(row_start, "row_start", dev, _I32, (B + 1,)),
            _arg(lens, "lens", dev, _I32, (B,)))


def paged4_append(k, v, pos, cache_k, scale_k, cache_v, scale_v, page_table, row_start, lens, *, exp_k: int = 0,
                  exp_v: int = 0, q=None, q_out=None, turns=None, interleaved: bool = False, mag: float = 1.0, err=None,
                  stream=None):
    """A chunk's rows enter the 4-bit cache: k [T][nk][hd] rotated by pos (when turns is given)
    and v, both encoded, go to the slots lens[b] - t_b + i of their sequence; lens counts the
    chunk's rows. q [T][nh][hd] is rotated and rounded into q_out (bfloat16 or float16; a new
    one has q's type, bfloat16 for float32), which is returned (None without q)."""
    dev, on = _place(k, "k", stream)
    if on is None:
        return _there(paged4_append, locals())
    cache = _cache4(cache_k, scale_k, cache_v, scale_v, page_table, row_start, lens, exp_k, exp_v, dev)
    nk, hd = cache[1:3]
    if k.dtype not in _TYPES or k.dim() != 3:
        raise ValueError("k must be [T][nk][hd] in float32, bfloat16 or float16")
    T = k.shape[0]
    kp, k_row = _rows(k, "k", dev, k.dtype, (T, nk, hd))
    vp, v_row = _rows(v, "v", dev, k.dtype, (T, nk, hd))
    nh = qp = q_row = qo = q_type = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError(f"q must be [{T}][nh][{hd}]")
        nh = q.shape[1]
        qp, q_row = _rows(q, "q", dev, k.dtype, (T, nh, hd))
        if q_out is None:
            q_out = torch.empty(T, nh, hd, device=q.device, dtype=q.dtype if q.dtype in _TYPES16 else torch.bfloat16)
        if q_out.dtype not in _TYPES16:
            raise ValueError("q_out must be bfloat16 or float16")
        qo, q_type = _arg(q_out, "q_out", dev, q_out.dtype, (T, nh, hd)), _TYPES16[q_out.dtype]
    elif q_out is not None:
        raise ValueError("q_out without q")
    n = 0 if turns is None else turns.numel()
    a = _APPEND.pack(*cache, T, nh, 2 * n, _TYPES[k.dtype], q_type, bool(interleaved), mag, qp, kp, vp, q_row, k_row, v_row,
                     qo, _opt(pos, "pos", dev, _I32, (T,)), _opt(turns, "turns", dev, _I64, (n,)),
                     _opt(err, "err", dev, _I32, (1,)))
    _abi.check(_lib().swa_paged4_append(a, on), "swa_paged4_append")
    return q_out


def paged4_read(cache_k, scale_k, cache_v, scale_v, page_table, row_start, lens, *, T=None, exp_k: int = 0, exp_v: int = 0,
                dtype=torch.bfloat16, k_out=None, v_out=None, err=None, stream=None):
    """The last rows of every sequence as the 4-bit cache holds them: packed row i of the t_b
    rows of sequence b gets the values of slot lens[b] - t_b + i. Returns (k_out, v_out), each
    [T][nk][hd]; of outputs that are not given both are made (T rows of dtype, zeros in rows of
    no sequence), or only the given one is written."""
    dev, on = _place(cache_k, "cache_k", stream)
    if on is None:
        return _there(paged4_read, locals())
    cache = _cache4(cache_k, scale_k, cache_v, scale_v, page_table, row_start, lens, exp_k, exp_v, dev)
    nk, hd = cache[1:3]
    if k_out is None and v_out is None:
        if T is None:
            raise ValueError("T (the packed rows) is required without k_out and v_out")
        k_out, v_out = (torch.zeros(T, nk, hd, device=cache_k.device, dtype=dtype) for _ in range(2))
    first = k_out if k_out is not None else v_out
    if not isinstance(first, torch.Tensor) or first.dim() != 3 or first.dtype not in _TYPES:
        raise ValueError("k_out and v_out must be [T][nk][hd] in float32, bfloat16 or float16")
    n = first.shape[0]
    if T is not None and T != n:
        raise ValueError(f"k_out and v_out have {n} rows, expected T = {T}")
    a = _READ.pack(*cache, n, _TYPES[first.dtype], _opt(k_out, "k_out", dev, first.dtype, (n, nk, hd)),
                   _opt(v_out, "v_out", dev, first.dtype, (n, nk, hd)), _opt(err, "err", dev, _I32, (1,)))
    _abi.check(_lib().swa_paged4_read(a, on), "swa_paged4_read")
    return k_out, v_out


def _attend4_sizes(B, T, nh, nk, hd, page, max_pages, max_rows, window, sinks) -> bytes:
    return _ATTEND.pack(B, nk, hd, page, 0, max_pages, 0, 0, 0, 0, 0, 0, 0, 0, 0, T, nh, max_rows, window, sinks,
                        _abi.SWA_BF16, 0, 0.0, 0, 0, 0, 0, 0, 0, 0, 0, 0)


def paged4_attend_workspace_size(B, T, nh, nk, hd, page, max_pages, max_rows, window: int = 0, sinks: int = 0) -> int:
    """Workspace bytes of paged4_attend on the current device (1: none is needed)."""
    n = int(_lib().swa_paged4_attend_workspace_size(_attend4_sizes(B, T, nh, nk, hd, page, max_pages, max_rows, window, sinks)))
    if n == 0:
        raise _abi.SwaError(_abi.SWA_E_SHAPE, "swa_paged4_attend_workspace_size")
    return n


@functools.lru_cache(maxsize=1024)
def _attend4_need(dev, *sizes) -> int:
    """The workspace's bytes for device dev (the current one); 0 for sizes it refuses."""
    return int(_lib().swa_paged4_attend_workspace_size(_attend4_sizes(*sizes)))


def paged4_attend(q, cache_k, scale_k, cache_v, scale_v, page_table, row_start, lens, scale: float, *, max_rows: int,
                  exp_k: int = 0, exp_v: int = 0, window: int = 0, sinks: int = 0, out=None, lse=None, workspace=None,
                  err=None, ev_start=None, ev_stop=None, stream=None):
    """Causal attention of a chunk's rows q [T][nh][hd] (bfloat16 or float16) over the 4-bit
    cache, their own keys already appended: row i of sequence b, whose slot is p = lens[b] - t_b
    + i, sees the slots up to p; with window > 0 of these the last `window` (its own among them)
    and the first `sinks` of the sequence. max_rows bounds the rows of a sequence. out
    [T][nh][hd] in q's type or float32; lse [T][nh] f32, when given, gets log sum exp of the
    scores. Rows of no sequence are left as they were (zeros in a new out)."""
    dev, on = _place(q, "q", stream)
    if on is None:
        return _there(paged4_attend, locals())
    cache = _cache4(cache_k, scale_k, cache_v, scale_v, page_table, row_start, lens, exp_k, exp_v, dev)
    B, nk, hd, page, _, max_pages = cache[:6]
    if q.dim() != 3 or q.dtype not in _TYPES16:
        raise ValueError(f"q must be [T][nh][{hd}] in bfloat16 or float16")
    T, nh = q.shape[:2]
    qp, q_row = _rows(q, "q", dev, q.dtype, (T, nh, hd))
    if out is None:
        out = torch.zeros(T, nh, hd, device=q.device, dtype=q.dtype)
    wide = out.dtype == _F32
    op = _arg(out, "out", dev, _F32 if wide else q.dtype, (T, nh, hd))
    ws = size = 0
    if workspace is not None:
        ws, size = _arg(workspace, "workspace", dev, _U8), workspace.numel()
    else:
        size = _attend4_need(dev, B, T, nh, nk, hd, page, max_pages, max_rows, window, sinks)
        if size > 1:
            workspace = torch.empty(size, device=q.device, dtype=_U8)
            ws = workspace.data_ptr()
    a = _ATTEND.pack(*cache, T, nh, max_rows, window, sinks, _TYPES16[q.dtype], wide, scale, qp, q_row, op,
                     _opt(lse, "lse", dev, _F32, (T, nh)), ws, size, _opt(err, "err", dev, _I32, (1,)),
                     ev_start.cuda_event if ev_start is not None else 0, ev_stop.cuda_event if ev_stop is not None else 0)
    _abi.check(_lib().swa_paged4_attend(a, on), "swa_paged4_attend")
    return out


# ------------------------------------------------------------------ pages
def _pools(pools, num_pages, dev):
    """The fields of a swa_page_pools: contiguous tensors whose first dimension is the page."""
    n = len(pools)
    if n > _abi.SWA_MAX_POOLS:
        raise ValueError(f"at most {_abi.SWA_MAX_POOLS} pools, got {n}")
    base, size = [], []
    for p in pools:
        if not isinstance(p, torch.Tensor) or p.dim() < 2 or p.shape[0] != num_pages:
            raise ValueError(f"pools[{len(base)}] must be a CUDA tensor [{num_pages}][..]")
        if p.get_device() != dev or not p.is_contiguous():
            _complain(p, f"pools[{len(base)}]", dev, p.dtype, None)
        base.append(p.data_ptr())
        size.append(p.nbytes // max(num_pages, 1))           # (the call refuses pools without pages)
    rest = [0] * (_abi.SWA_MAX_POOLS - n)
    return (num_pages, n, *base, *rest, *size, *rest)


def _table(page_table, dev):
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be a CUDA tensor [B][max_pages]")
    return _arg(page_table, "page_table", dev, _I32), *page_table.shape


def _pages(refs, dev):
    if not isinstance(refs, torch.Tensor) or refs.dim() != 1:
        raise ValueError("refs must be a CUDA tensor [num_pages]")
    return _arg(refs, "refs", dev, _I32), refs.shape[0]


def _made(given, name, dev, shape, device):
    """An int32 output and its address: the caller's, checked, or a new one."""
    if given is not None:
        return given, _arg(given, name, dev, _I32, shape)
    new = torch.empty(shape, device=device, dtype=_I32)
    return new, new.data_ptr()


def _workspace(given, need, dev, device):
    """Address and bytes of a workspace of `need` bytes (1: none), and what keeps it."""
    if given is not None:
        return _arg(given, "workspace", dev, _U8), given.numel(), given
    if need <= 1:
        return 0, 0, None
    new = torch.empty(need, device=device, dtype=_U8)
    return new.data_ptr(), need, new


@functools.lru_cache(maxsize=256)
def _fork_need(num_pages, B, R, page, max_pages) -> int:
    z = [0] * _abi.SWA_MAX_POOLS
    return int(_lib().swa_paged_fork_workspace_size(_FORK.pack(num_pages, 0, *z, *z, B, R, page, max_pages, *[0] * 12)))


def paged_fork_workspace_size(num_pages, B, R, page, max_pages) -> int:
    """Workspace bytes of paged_fork from a batch of B sequences to one of R (1: none is needed)."""
    n = _fork_need(num_pages, B, R, page, max_pages)
    if n == 0:
        raise _abi.SwaError(_abi.SWA_E_SHAPE, "swa_paged_fork_workspace_size")
    return n


def paged_fork(pools, page_table, lens, refs, parent, page: int, *, room=None, table_out=None, lens_out=None, refs_out=None,
               left=None, workspace=None, err=None, stream=None):
    """From one batch's tables to the next one's. New sequence r continues old sequence
    parent[r] (a beam, a branch, the same request), or starts empty (-1); old sequences that no
    one continues let go of their pages. Pages of common keys are shared; one that a sequence
    writes next and that others hold too is copied in all pools; room[r] slots behind the length
    are given pages. page_table [B][max_pages] and lens [B] are the old batch, refs [num_pages]
    counts the holders of each page (0: free), page is the slots of a page; all int32. pools: up
    to 8 contiguous tensors [num_pages][..]. Returns (table_out, lens_out, refs_out, left):
    left [1] is the number of free pages, below 0 that of the pages that were lacking (their
    entries are -1). refs_out may be refs."""
    dev, on = _place(page_table, "page_table", stream)
    if on is None:
        return _there(paged_fork, locals())
    tp, B, max_pages = _table(page_table, dev)
    rp, num_pages = _pages(refs, dev)
    packed = _pools(pools, num_pages, dev)
    if not isinstance(parent, torch.Tensor) or parent.dim() != 1:
        raise ValueError("parent must be a CUDA tensor [R]")
    R = parent.shape[0]
    where = page_table.device
    table_out, to = _made(table_out, "table_out", dev, (R, max_pages), where)
    lens_out, lo = _made(lens_out, "lens_out", dev, (R,), where)
    refs_out, ro = _made(refs_out, "refs_out", dev, (num_pages,), where)
    left, fo = _made(left, "left", dev, (1,), where)
    ws = _workspace(workspace, _fork_need(num_pages, B, R, page, max_pages), dev, where)
    a = _FORK.pack(*packed, B, R, page, max_pages, tp, _arg(lens, "lens", dev, _I32, (B,)), _arg(parent, "parent", dev, _I32),
                   _opt(room, "room", dev, _I32, (R,)), rp, to, lo, ro, fo, ws[0], ws[1], _opt(err, "err", dev, _I32, (1,)))
    _abi.check(_lib().swa_paged_fork(a, on), "swa_paged_fork")
    return table_out, lens_out, refs_out, left


@functools.lru_cache(maxsize=256)
def _compact_need(num_pages, B, max_pages) -> int:
    z = [0] * _abi.SWA_MAX_POOLS
    return int(_lib().swa_paged_compact_workspace_size(_COMPACT.pack(num_pages, 0, *z, *z, B, max_pages, *[0] * 9)))


def paged_compact_workspace_size(num_pages, B, max_pages) -> int:
    """Workspace bytes of paged_compact (1: none is needed)."""
    n = _compact_need(num_pages, B, max_pages)
    if n == 0:
        raise _abi.SwaError(_abi.SWA_E_SHAPE, "swa_paged_compact_workspace_size")
    return n


def paged_compact(pools, page_table, refs, *, table_out=None, refs_out=None, moved=None, used=None, workspace=None, err=None,
                  stream=None):
    """The pages in use (refs > 0) move to the front of all pools (contiguous tensors
    [num_pages][..], up to 8), into the free pages there. Returns (table_out, refs_out, moved,
    used): the new table and counts (each may be the old one), every page's new place (-1: it
    was free) and the number of pages in use, from which on the pools may be given back."""
    dev, on = _place(page_table, "page_table", stream)
    if on is None:
        return _there(paged_compact, locals())
    tp, B, max_pages = _table(page_table, dev)
    rp, num_pages = _pages(refs, dev)
    packed = _pools(pools, num_pages, dev)
    where = page_table.device
    table_out, to = _made(table_out, "table_out", dev, (B, max_pages), where)
    refs_out, ro = _made(refs_out, "refs_out", dev, (num_pages,), where)
    moved, mo = _made(moved, "moved", dev, (num_pages,), where)
    used, uo = _made(used, "used", dev, (1,), where)
    ws = _workspace(workspace, _compact_need(num_pages, B, max_pages), dev, where)
    a = _COMPACT.pack(*packed, B, max_pages, tp, rp, to, ro, mo, uo, ws[0], ws[1], _opt(err, "err", dev, _I32, (1,)))
    _abi.check(_lib().swa_paged_compact(a, on), "swa_paged_compact")
    return table_out, refs_out, moved, used
