"""The 4-bit paged cache and the page calls without a GPU: the oracle against closed forms,
the packed structs, and every refusal (arguments are checked before any CUDA call)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged4_oracle as p4
from sliding_window_gqa_prep_gb300 import _abi, paged4
import sliding_window_gqa_prep_gb300 as swa

FAKE = 0x10000   # an aligned address that is never dereferenced: checks fail first
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


# ------------------------------------------------------------------ oracle pins
def test_oracle_formats():
    assert p4.E4M3[126] == 448 and p4.E4M3[8] == 2.0 ** -6 and p4.E4M3[1] == 2.0 ** -9
    x = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert (x == p4.E4M3[:127]).all()
    c, s = p4.encode(np.array([0.25, 0.2500001, -0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.1, 0, -6, 6, 1, 2, 3, 4]), 0)
    assert s.tolist() == [56]                                # scale 1
    # ties to the even code; the lower half of a byte is the even feature
    codes = np.stack((c & 15, c >> 4), -1).reshape(-1).tolist()
    assert codes == [0, 1, 8 + 2, 2, 4, 4, 6, 6, 8 + 7, 0, 8 + 7, 7, 2, 4, 5, 6]
    assert p4.decode(c, s, 3).tolist() == [0, 4, -8, 8, 16, 16, 32, 32, -48, 0, -48, 48, 8, 16, 24, 32]
    assert p4.encode_block(np.full(16, 1e9), 0)[1] == 126 and p4.encode_block(np.full(16, 1e-9), 0)[1] == 0
    assert p4.encode_block([np.nan] + [1.0] * 15, 0)[1] == 127


def test_oracle_rounding_is_at_most_half_a_step():
    rng = np.random.default_rng(0)
    for exp in (-4, 0, 5):
        x = rng.standard_normal((50, 32)) * 2.0 ** exp * 3
        c, s = p4.encode(x, exp)
        y = p4.decode(c, s, exp)
        u = np.repeat(p4.E4M3[s], 16, -1) * 2.0 ** exp
        # the widest step is 2 units, and a scale rounded down leaves 6 units 1/16 short at most
        assert (np.abs(y - x) <= u * (1 + 6 / 16)).all()
        assert np.abs(y - x).mean() < 0.15 * np.abs(x).mean()


def test_oracle_visible():
    assert p4.visible(6, 3, 0, 9).tolist() == [True] * 4 + [False] * 2
    assert p4.visible(6, 4, 2, 1).tolist() == [True, False, False, True, True, False]
    assert not p4.visible(4, -1, 2, 2).any()


def test_oracle_fork_and_compact():
    # two sequences of 20 keys in pages of 16: one branches, one ends
    table, refs = [[5, 3, -1], [4, 1, -1]], [0, 1, 0, 1, 1, 1, 0]
    out, lens, new, left, copies = p4.fork(table, [20, 20], refs, [0, 0], [1, 20], 16, 7)
    assert out == [[5, 3, -1], [5, 0, 1]] and lens == [20, 20] and copies == [(3, 0)]
    assert new == [1, 1, 0, 1, 0, 2, 0] and left == 3
    out, new, moved, used, copies = p4.compact(out, new, 7)
    assert used == 4 and moved == [0, 1, -1, 3, -1, 2, -1] and copies == [(5, 2)]
    assert out == [[2, 3, -1], [2, 0, 1]] and new == [1, 1, 2, 1, 0, 0, 0]


# ------------------------------------------------------------------ refusals
def _cache(c, **kw):
    c.B, c.nk, c.hd, c.page, c.num_pages, c.max_pages, c.k_exp, c.v_exp = 2, 2, 128, 16, 8, 4, 0, -3
    for i, f in enumerate(("k", "k_scale", "v", "v_scale", "table", "row_start", "lens")):
        setattr(c, f, FAKE + i * MB)
    for k, v in kw.items():
        setattr(c, k, v)


CACHE_BAD = [(dict([(f, None)]), _abi.SWA_E_NULL) for f in ("k", "k_scale", "v", "v_scale", "table", "lens", "row_start")] + [
    (dict(B=0), _abi.SWA_E_SHAPE), (dict(B=65536), _abi.SWA_E_SHAPE), (dict(nk=0), _abi.SWA_E_SHAPE),
    (dict(hd=96), _abi.SWA_E_SHAPE), (dict(page=8), _abi.SWA_E_SHAPE), (dict(page=48), _abi.SWA_E_SHAPE),
    (dict(page=512), _abi.SWA_E_SHAPE), (dict(num_pages=0), _abi.SWA_E_SHAPE), (dict(num_pages=1 << 27), _abi.SWA_E_SHAPE),
    (dict(max_pages=0), _abi.SWA_E_SHAPE), (dict(max_pages=(1 << 26) + 1), _abi.SWA_E_SHAPE),
    (dict(k_exp=33), _abi.SWA_E_SHAPE), (dict(v_exp=-33), _abi.SWA_E_SHAPE),
    (dict(k=FAKE + 8), _abi.SWA_E_ALIGN), (dict(v_scale=FAKE + 4), _abi.SWA_E_ALIGN), (dict(table=FAKE + 2), _abi.SWA_E_ALIGN),
    (dict(row_start=FAKE + 1), _abi.SWA_E_ALIGN),
]
FAR = FAKE + 16 * MB


def _append(cache=None, **kw):
    a = _abi.Paged4AppendArgs()
    _cache(a.cache, **(cache or {}))
    a.T, a.nh, a.rot, a.src, a.q_dtype, a.mag = 4, 4, 128, _abi.SWA_BF16, _abi.SWA_BF16, 1.0
    a.q, a.k, a.v, a.pos, a.turns, a.q_out = (FAR + i * MB for i in range(6))
    a.q_row, a.k_row, a.v_row = 512, 256, 256
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_append_refusals(lib):
    call = lambda a: lib.swa_paged4_append(ctypes.byref(a), None)
    assert lib.swa_paged4_append(None, None) == _abi.SWA_E_NULL
    for kw, rc in CACHE_BAD:
        assert call(_append(cache=kw)) == rc, kw
    for kw in (dict(k=None), dict(v=None), dict(q=None), dict(q_out=None), dict(pos=None), dict(turns=None)):
        assert call(_append(**kw)) == _abi.SWA_E_NULL, kw
    for kw in (dict(T=-1), dict(rot=3), dict(rot=130), dict(src=3), dict(q_dtype=_abi.SWA_F32), dict(q_dtype=5), dict(nh=0),
               dict(nh=-1), dict(mag=float("nan")), dict(k_row=128), dict(v_row=0), dict(q_row=504), dict(q_out=FAR + 16),
               dict(q_out=FAR, q_row=520), dict(q_out=FAR, src=_abi.SWA_F16), dict(q_out=FAR + MB), dict(q_out=FAR + 2 * MB),
               dict(T=1 << 30, nh=1 << 19), dict(T=1 << 28, nh=1, q_row=1 << 39), dict(T=1 << 28, nh=1, v_row=1 << 39)):
        assert call(_append(**kw)) == _abi.SWA_E_SHAPE, kw
    for kw in (dict(k=FAR + 2), dict(q_out=FAR + 5 * MB + 8), dict(k_row=258), dict(src=_abi.SWA_F32, v_row=258), dict(pos=FAR + 1),
               dict(turns=FAR + 4)):
        assert call(_append(**kw)) == _abi.SWA_E_ALIGN, kw
    # pools of 8 pages of 2 heads of 16 keys: codes 16384 bytes, scales 2048
    for kw in (dict(v=FAKE + 16368), dict(k_scale=FAKE + 16), dict(v_scale=FAKE + MB + 2032)):
        assert call(_append(cache=kw)) == _abi.SWA_E_SHAPE, kw
    assert call(_append(T=0)) == _abi.SWA_OK


def _read(cache=None, **kw):
    a = _abi.Paged4ReadArgs()
    _cache(a.cache, **(cache or {}))
    a.T, a.dtype, a.k_out, a.v_out = 4, _abi.SWA_F32, FAR, FAR + MB
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_read_refusals(lib):
    call = lambda a: lib.swa_paged4_read(ctypes.byref(a), None)
    assert lib.swa_paged4_read(None, None) == _abi.SWA_E_NULL
    for kw, rc in CACHE_BAD:
        assert call(_read(cache=kw)) == rc, kw
    assert call(_read(k_out=None, v_out=None)) == _abi.SWA_E_NULL
    # 4 rows of 2 heads of 128 in f32: 4096 bytes
    for kw in (dict(T=-1), dict(dtype=3), dict(T=1 << 31 - 1, cache=dict(nk=65535, B=1)), dict(v_out=FAR + 4080), dict(k_out=FAKE),
               dict(v_out=FAKE + 3 * MB - 4080)):
        assert call(_read(**kw)) == _abi.SWA_E_SHAPE, kw
    for kw in (dict(k_out=FAR + 8), dict(v_out=FAR + MB + 2)):
        assert call(_read(**kw)) == _abi.SWA_E_ALIGN, kw
    assert call(_read(T=0)) == _abi.SWA_OK


def _attend(cache=None, **kw):
    a = _abi.Paged4AttendArgs()
    _cache(a.cache, **(cache or {}))
    a.T, a.nh, a.max_rows, a.scale, a.q_row, a.q_dtype = 4, 4, 2, 0.1, 512, _abi.SWA_BF16
    a.q, a.out, a.workspace, a.workspace_bytes = FAR, FAR + MB, FAR + 2 * MB, 1 << 40
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_attend_refusals(lib):
    call = lambda a: lib.swa_paged4_attend(ctypes.byref(a), None)
    size = lambda a: lib.swa_paged4_attend_workspace_size(ctypes.byref(a))
    assert lib.swa_paged4_attend(None, None) == _abi.SWA_E_NULL
    for kw, rc in CACHE_BAD:
        assert call(_attend(cache=kw)) == rc, kw
    for kw in (dict(q=None), dict(out=None)):
        assert call(_attend(**kw)) == _abi.SWA_E_NULL, kw
    bad = (dict(T=-1), dict(max_rows=0), dict(nh=5), dict(nh=0), dict(nh=66), dict(T=1 << 30), dict(window=-1), dict(sinks=-1),
           dict(q_dtype=_abi.SWA_F32), dict(q_dtype=3))
    for kw in bad + (dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q_row=500),
                     dict(T=1 << 28, q_row=1 << 39)):
        assert call(_attend(**kw)) == _abi.SWA_E_SHAPE, kw
    for kw in (dict(q=FAR + 8), dict(out=FAR + MB + 4), dict(q_row=516), dict(lse=FAR + 2), dict(workspace=FAR + 16)):
        assert call(_attend(**kw)) == _abi.SWA_E_ALIGN, kw
    # q, out and lse may not share a byte: 4 rows of 4 heads of 128 are 4096 bytes, of lse 64
    for kw in (dict(out=FAR), dict(out=FAR + 4080), dict(lse=FAR + 4092), dict(lse=FAR + MB + 4092),
               dict(lse=FAR + MB + 8188, out_f32=1)):
        assert call(_attend(**kw)) == _abi.SWA_E_SHAPE, kw
    assert call(_attend(T=0)) == _abi.SWA_OK
    assert lib.swa_paged4_attend_workspace_size(None) == 0 and size(_attend()) > 0
    for kw in bad:
        assert size(_attend(**kw)) == 0, kw
    assert size(_attend(cache=dict(page=48))) == 0


def _fork(pools=2, page_bytes=64, num_pages=10, **kw):
    a = _abi.PagedForkArgs()
    a.pools.num_pages, a.pools.pools = num_pages, pools
    for i in range(min(max(pools, 0), 8)):
        a.pools.base[i], a.pools.page_bytes[i] = FAKE + i * MB, page_bytes
    a.B, a.R, a.page, a.max_pages = 2, 3, 16, 4
    names = ("table", "lens", "parent", "room", "refs", "table_out", "lens_out", "refs_out", "left", "workspace")
    for i, f in enumerate(names):
        setattr(a, f, FAR + i * MB)
    a.workspace_bytes = 1 << 19
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_fork_refusals(lib):
    call = lambda a: lib.swa_paged_fork(ctypes.byref(a), None)
    size = lambda a: lib.swa_paged_fork_workspace_size(ctypes.byref(a))
    assert lib.swa_paged_fork(None, None) == _abi.SWA_E_NULL
    for f in ("table", "lens", "parent", "refs", "table_out", "lens_out", "refs_out", "left"):
        assert call(_fork(**{f: None})) == _abi.SWA_E_NULL, f
    bad = (dict(pools=-1), dict(pools=9), dict(num_pages=0), dict(num_pages=1 << 30), dict(B=0), dict(R=0), dict(B=65536), dict(R=65536),
           dict(page=8), dict(page=24), dict(page=512), dict(max_pages=0), dict(max_pages=(1 << 26) + 1),
           dict(R=65535, max_pages=(1 << 15) + 1), dict(B=65535, max_pages=(1 << 15) + 1))
    for kw in bad:
        assert size(_fork(**kw)) == 0, kw
        assert call(_fork(**kw)) == _abi.SWA_E_SHAPE, kw
    for kw in (dict(page_bytes=0), dict(page_bytes=-16), dict(page_bytes=1 << 46)):
        assert call(_fork(**kw)) == _abi.SWA_E_SHAPE, kw
    a = _fork()
    a.pools.base[1] = None
    assert call(a) == _abi.SWA_E_NULL
    for at, off in ((1, 8), (0, 2)):
        a = _fork()
        a.pools.base[at] += off
        assert call(a) == _abi.SWA_E_ALIGN
    assert call(_fork(page_bytes=24)) == _abi.SWA_E_ALIGN
    for kw in (dict(table=FAR + 2), dict(left=FAR + 8 * MB + 1), dict(workspace=FAR + 9 * MB + 128)):
        assert call(_fork(**kw)) == _abi.SWA_E_ALIGN, kw
    assert size(_fork()) == 1                                # few pages and entries: one launch, no workspace
    for kw in (dict(workspace=None), dict(workspace_bytes=size(_fork(num_pages=10000)) - 1)):
        assert call(_fork(num_pages=10000, **kw)) == _abi.SWA_E_WORKSPACE, kw
    a = _fork()
    a.pools.base[1] = FAKE + 639 // 16 * 16                   # 10 pages of 64 bytes each
    assert call(a) == _abi.SWA_E_SHAPE
    # outputs on inputs (48 bytes of table_out, 40 of refs_out), on each other, on pools and the workspace
    for kw in (dict(table_out=FAR), dict(table_out=FAR - 44), dict(lens_out=FAR + MB + 4), dict(refs_out=FAR + 2 * MB - 36), dict(left=FAR + 3 * MB + 8),
               dict(refs_out=FAR + 4 * MB + 4), dict(left=FAR + 5 * MB + 44), dict(lens_out=FAKE + 636), dict(room=FAR + 7 * MB)):
        assert call(_fork(**kw)) == _abi.SWA_E_SHAPE, kw
    for kw in (dict(refs_out=FAR + 9 * MB), dict(table=FAR + 9 * MB)):
        assert call(_fork(num_pages=10000, **kw)) == _abi.SWA_E_SHAPE, kw


def _compact(pools=2, page_bytes=64, num_pages=10, **kw):
    a = _abi.PagedCompactArgs()
    a.pools.num_pages, a.pools.pools = num_pages, pools
    for i in range(min(max(pools, 0), 8)):
        a.pools.base[i], a.pools.page_bytes[i] = FAKE + i * MB, page_bytes
    a.B, a.max_pages = 2, 4
    for i, f in enumerate(("table", "refs", "table_out", "refs_out", "moved", "used", "workspace")):
        setattr(a, f, FAR + i * MB)
    a.workspace_bytes = 1 << 19
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_compact_refusals(lib):
    call = lambda a: lib.swa_paged_compact(ctypes.byref(a), None)
    size = lambda a: lib.swa_paged_compact_workspace_size(ctypes.byref(a))
    assert lib.swa_paged_compact(None, None) == _abi.SWA_E_NULL
    for f in ("table", "refs", "table_out", "refs_out", "moved", "used"):
        assert call(_compact(**{f: None})) == _abi.SWA_E_NULL, f
    for kw in (dict(pools=-1), dict(pools=9), dict(num_pages=0), dict(num_pages=1 << 30), dict(B=0), dict(B=65536), dict(max_pages=0),
               dict(max_pages=(1 << 26) + 1), dict(B=65535, max_pages=(1 << 15) + 1)):
        assert size(_compact(**kw)) == 0, kw
        assert call(_compact(**kw)) == _abi.SWA_E_SHAPE, kw
    assert call(_compact(page_bytes=0)) == _abi.SWA_E_SHAPE and call(_compact(page_bytes=8 * 3)) == _abi.SWA_E_ALIGN
    for kw in (dict(moved=FAR + 2), dict(workspace=FAR + 6 * MB + 16)):
        assert call(_compact(**kw)) == _abi.SWA_E_ALIGN, kw
    assert size(_compact()) == 1
    for kw in (dict(workspace=None), dict(workspace_bytes=size(_compact(num_pages=10000)) - 1)):
        assert call(_compact(num_pages=10000, **kw)) == _abi.SWA_E_WORKSPACE, kw
    for kw in (dict(table_out=FAR + 4), dict(refs_out=FAR + MB - 4), dict(moved=FAR + MB), dict(used=FAR), dict(moved=FAR + 3 * MB + 36),
               dict(used=FAKE)):
        assert call(_compact(**kw)) == _abi.SWA_E_SHAPE, kw
    assert call(_compact(num_pages=10000, moved=FAR + 6 * MB)) == _abi.SWA_E_SHAPE


# ------------------------------------------------------------------ the binding
def test_packed_structs_match_the_abi(lib):
    for fmt, cls in ((paged4._APPEND, _abi.Paged4AppendArgs), (paged4._READ, _abi.Paged4ReadArgs), (paged4._ATTEND, _abi.Paged4AttendArgs),
                     (paged4._FORK, _abi.PagedForkArgs), (paged4._COMPACT, _abi.PagedCompactArgs)):
        assert fmt.size == ctypes.sizeof(cls)
        fields = []
        for name, kind in cls._fields_:
            if kind is _abi.Paged4Cache:
                fields += [(name, sub, None) for sub, _ in kind._fields_]
            elif kind is _abi.PagePools:
                fields += [(name, "num_pages", None), (name, "pools", None)]
                fields += [(name, sub, i) for sub in ("base", "page_bytes") for i in range(_abi.SWA_MAX_POOLS)]
            else:
                fields.append((name, None, None))
        values = [float(i + 1) if getattr(dict(cls._fields_)[f[0]], "_type_", "") == "f" else i + 1 for i, f in enumerate(fields)]
        a = cls.from_buffer_copy(fmt.pack(*values))
        for (name, sub, i), want in zip(fields, values):
            x = getattr(a, name)
            x = getattr(x, sub) if sub else x
            assert (x if i is None else x[i]) == want, (cls, name, sub, i)


def parts():
    """A cache on the CPU, whose device number is -1."""
    k, ks = torch.zeros(4, 2, 16, 32, dtype=torch.uint8), torch.zeros(4, 2, 16, 4, dtype=torch.float8_e4m3fn)
    table = torch.zeros(1, 3, dtype=torch.int32)
    return [k, ks, k.clone(), ks.clone(), table, torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)]


def test_cache_fields():
    p = parts()
    f = paged4._cache4(*p, 1, -2, -1)
    assert f[:8] == (1, 2, 64, 16, 4, 3, 1, -2) and f[8:] == tuple(x.data_ptr() for x in p)


@pytest.mark.parametrize("which", range(7))
def test_what_is_no_part_of_a_cache_is_refused(which):
    for other in (None, 5, torch.zeros(3, dtype=torch.int64)):
        p = parts()
        p[which] = other
        with pytest.raises(ValueError):
            paged4._cache4(*p, 0, 0, -1)


def test_pools_of_the_page_calls():
    a, b = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(4, 3, 16, dtype=torch.uint8)
    f = paged4._pools([a, b], 4, -1)
    assert f[:4] == (4, 2, a.data_ptr(), b.data_ptr()) and f[10:12] == (2 * 16 * 64 * 2, 48)
    for bad in ([a[:3]], [a.transpose(1, 2)], [a] * 9, [None], [torch.zeros(4)]):
        with pytest.raises(ValueError):
            paged4._pools(bad, 4, -1)


def test_workspace_sizes():
    assert swa.paged_fork_workspace_size(100000, 4, 8, 16, 10) > 100000 * 12
    assert swa.paged_compact_workspace_size(100000, 4, 10) > 100000 * 12
    assert swa.paged_fork_workspace_size(1000, 4, 8, 16, 10) == swa.paged_compact_workspace_size(1000, 4, 10) == 1
    for fn, a in ((swa.paged_fork_workspace_size, (1000, 4, 8, 17, 10)), (swa.paged_compact_workspace_size, (0, 4, 10)),
                  (swa.paged4_attend_workspace_size, (1, 4, 4, 3, 128, 16, 4, 4))):
        with pytest.raises(swa.SwaError):
            fn(*a)
