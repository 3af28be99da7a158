"""Rotary and paged-cache entry points without a GPU: the frequency schedules (host code
of the library) against their formulas, the oracle against closed forms, and every
refusal (arguments are checked before any CUDA call)."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import paged_oracle as po
from sliding_window_gqa_prep_gb300 import _abi
import sliding_window_gqa_prep_gb300 as swa

FAKE = 0x10000   # an aligned address that is never dereferenced: checks fail first
BIG = 1 << 44    # another one, far from it


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


# ------------------------------------------------------------------ schedules
SCHEDULES = [
    dict(rot=64, theta=10000.0),
    dict(rot=2, theta=500000.0),
    dict(rot=20, theta=1e6, schedule="linear", factor=4.0),
    dict(rot=128, theta=10000.0, schedule="base", factor=8.0),
    dict(rot=128, theta=10000.0, schedule="parts", factor=16.0, orig_len=4096, low=1.0, high=32.0),
    dict(rot=64, theta=500000.0, schedule="parts", factor=8.0, orig_len=8192, low=1.0, high=4.0),
]


@pytest.mark.parametrize("kw", SCHEDULES)
def test_rotary_schedules(kw):
    f = swa.rotary_freqs(**kw).numpy()
    ref = po.freqs(kw["rot"], kw["theta"], kw.get("schedule", "plain"), kw.get("factor", 1.0),
                   kw.get("orig_len", 0.0), kw.get("low", 1.0), kw.get("high", 32.0))
    # pow and a handful of f64 operations, each within a few ulp
    np.testing.assert_allclose(f, ref, rtol=1e-14)
    t = swa.rotary_turns(device="cpu", **kw).numpy()
    for e in range(kw["rot"] // 2):
        got = Fraction(int(t[e]) % (1 << 64), 1 << 64)
        want = Fraction(float(f[e])) / Fraction(2 * math.pi) % 1
        # one f64 division: relative 2^-53 of f / 2 pi, plus the cut at 2^-64
        d = abs(got - want)
        assert min(d, 1 - d) <= Fraction(float(f[e])) * Fraction(1, 1 << 52) + Fraction(1, 1 << 63)


def test_schedule_ends():
    plain = swa.rotary_freqs(64).numpy()
    base = swa.rotary_freqs(64, schedule="base", factor=4.0).numpy()
    assert base[0] == plain[0] and abs(base[-1] * 4.0 / plain[-1] - 1) < 1e-13
    parts = swa.rotary_freqs(64, schedule="parts", factor=4.0, orig_len=2048).numpy()
    turns = 2048 * plain / (2 * np.pi)
    assert np.allclose(parts[turns >= 32], plain[turns >= 32], rtol=1e-15)
    assert np.allclose(parts[turns <= 1], plain[turns <= 1] / 4, rtol=1e-15)


def test_schedule_refusals(lib):
    def call(**kw):
        s = _abi.RotarySchedule()
        s.kind, s.rot, s.theta, s.factor, s.orig_len, s.low, s.high = 0, 8, 1e4, 2.0, 100.0, 1.0, 32.0
        for k, v in kw.items():
            setattr(s, k, v)
        f = (ctypes.c_double * 512)()
        return lib.swa_rotary_turns(ctypes.byref(s), f, None)
    assert lib.swa_rotary_turns(None, None, None) == _abi.SWA_E_NULL
    assert call() == _abi.SWA_OK
    for kw in (dict(kind=4), dict(kind=-1), dict(rot=7), dict(rot=0), dict(rot=1026), dict(theta=0.0),
               dict(theta=float("nan")), dict(kind=1, factor=0.5), dict(kind=2, rot=2),
               dict(kind=3, orig_len=0.0), dict(kind=3, low=32.0), dict(kind=3, high=float("inf")),
               dict(kind=1, factor=float("inf"))):
        assert call(**kw) == _abi.SWA_E_SHAPE, kw
    with pytest.raises(ValueError):
        swa.rotary_freqs(8, schedule="other")
    with pytest.raises(ValueError):
        swa.rotary_freqs(4096)


# ------------------------------------------------------------------ oracle pins
def test_oracle_rotary():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 16))
    f = po.freqs(12, 100.0)
    pos = np.array([0, 1, 7, -3, 1 << 30])
    for inter in (False, True):
        y = po.rotary(x, pos, f, inter)
        np.testing.assert_array_equal(y[0], x[0])                       # position 0
        np.testing.assert_array_equal(y[..., 12:], x[..., 12:])         # behind rot
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1))  # a rotation
        np.testing.assert_allclose(po.rotary(y, pos, f, inter, True), x, atol=1e-12)
    # relative positions: <R(a) q, R(b) k> depends on a - b alone
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    d = [float((po.rotary(q, [a], f) * po.rotary(k, [a - 5], f)).sum()) for a in (5, 9, 1000)]
    assert max(d) - min(d) < 1e-11


def test_oracle_attend_and_weigh():
    rng = np.random.default_rng(1)
    ck, cv = rng.standard_normal((6, 2, 16, 8)), rng.standard_normal((6, 2, 16, 8))
    table = np.array([[3, 1, 5], [0, 2, 4]])
    row_start, lens = np.array([0, 3, 4]), np.array([20, 33])
    q = rng.standard_normal((5, 4, 8))
    out, lse, absv, _ = po.attend(q, ck, cv, table, row_start, lens, 0.3)
    assert not out[4].any() and np.isneginf(lse[4]).all()               # a row of no sequence
    k0 = np.concatenate([ck[p, 1] for p in (3, 1, 5)])[:19]             # row 1 of sequence 0 sees 19
    v0 = np.concatenate([cv[p, 1] for p in (3, 1, 5)])[:19]
    p = np.exp(0.3 * k0 @ q[1, 3])
    np.testing.assert_allclose(out[1, 3], p @ v0 / p.sum())
    np.testing.assert_allclose(lse[1, 3], np.log(p.sum()))
    w = po.weigh(q, lse, ck, table, row_start, lens, 0.3, np.zeros((2, 2, 48)))
    # every row and head gives weight 1 in all
    np.testing.assert_allclose(w.sum(-1), [[3 * 2, 3 * 2], [1 * 2, 1 * 2]])
    assert not w[0, :, 20:].any()


def test_oracle_evict():
    w = np.array([5.0, 1.0, np.nan, 1.0, -0.0, 0.0, 7.0, 2.0])
    pos = np.array([10, 11, 12, 13, 14, 15, 0, 17])
    assert po.evict_order(w, pos, 8, 1, 17) == [6, 7, 2, 0, 1, 3, 4, 5]
    assert po.evict(w, pos, 8, 4, 1, 17) == (4, [(1, 6), (3, 7)])
    assert po.evict(w, pos, 8, 9, 1, 17) == (8, [])
    assert po.evict(w, pos, 8, 1, 0, None) == (1, [(0, 2)])


# ------------------------------------------------------------------ refusals
def _cache(c, **kw):
    c.B, c.nk, c.hd, c.page, c.num_pages, c.max_pages, c.dtype = 2, 2, 128, 16, 8, 4, _abi.SWA_BF16
    for f in ("k", "v", "table", "row_start", "lens"):
        setattr(c, f, FAKE)
    for k, v in kw.items():
        setattr(c, k, v)


CACHE_BAD = [
    (dict(k=None), _abi.SWA_E_NULL), (dict(v=None), _abi.SWA_E_NULL), (dict(table=None), _abi.SWA_E_NULL),
    (dict(lens=None), _abi.SWA_E_NULL), (dict(row_start=None), _abi.SWA_E_NULL),
    (dict(B=0), _abi.SWA_E_SHAPE), (dict(B=65536), _abi.SWA_E_SHAPE), (dict(nk=0), _abi.SWA_E_SHAPE),
    (dict(hd=96), _abi.SWA_E_SHAPE), (dict(page=8), _abi.SWA_E_SHAPE), (dict(page=48), _abi.SWA_E_SHAPE),
    (dict(page=512), _abi.SWA_E_SHAPE), (dict(num_pages=0), _abi.SWA_E_SHAPE),
    (dict(num_pages=1 << 27), _abi.SWA_E_SHAPE),          # 2^27 * 2 * 16 rows = 2^32
    (dict(max_pages=0), _abi.SWA_E_SHAPE), (dict(max_pages=(1 << 26) + 1), _abi.SWA_E_SHAPE),
    (dict(dtype=_abi.SWA_F32), _abi.SWA_E_SHAPE), (dict(dtype=7), _abi.SWA_E_SHAPE),
    (dict(k=FAKE + 8), _abi.SWA_E_ALIGN), (dict(v=FAKE + 2), _abi.SWA_E_ALIGN),
    (dict(table=FAKE + 2), _abi.SWA_E_ALIGN), (dict(lens=FAKE + 1), _abi.SWA_E_ALIGN),
]


def _rotary(**kw):
    a = _abi.RotaryArgs()
    a.T, a.H, a.hd, a.rot, a.dtype, a.mag = 4, 3, 64, 64, _abi.SWA_BF16, 1.0
    a.x, a.out, a.pos, a.turns = FAKE, BIG, FAKE, FAKE
    a.x_row, a.x_head, a.out_row, a.out_head = 192, 64, 192, 64
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_rotary_refusals(lib):
    call = lambda a: lib.swa_rotary(ctypes.byref(a), None)
    assert lib.swa_rotary(None, None) == _abi.SWA_E_NULL
    for f in ("x", "out", "pos", "turns"):
        assert call(_rotary(**{f: None})) == _abi.SWA_E_NULL
    for kw in (dict(T=-1), dict(H=0), dict(hd=60), dict(hd=1032), dict(rot=0), dict(rot=65), dict(rot=66),
               dict(dtype=3), dict(mag=float("inf")), dict(x_head=32), dict(x_row=128), dict(out_row=100),
               dict(out_head=-64), dict(T=1 << 30, H=1 << 20), dict(out=FAKE + 64),
               dict(out=FAKE, out_row=256)):
        assert call(_rotary(**kw)) == _abi.SWA_E_SHAPE, kw
    for kw in (dict(x=FAKE + 8), dict(out=BIG + 2), dict(x_row=196), dict(out_head=66, out_row=200),
               dict(pos=FAKE + 2), dict(turns=FAKE + 4)):
        assert call(_rotary(**kw)) == _abi.SWA_E_ALIGN, kw
    assert call(_rotary(T=0, x=None)) == _abi.SWA_OK                    # nothing to do
    # strides whose offsets would pass 64 bits
    for kw in (dict(T=1 << 30, H=1, x_row=1 << 39, out_row=1 << 39), dict(H=1 << 20, x_head=1 << 39, out_head=1 << 39),
               dict(T=1, H=1, x_row=(1 << 40) + 8), dict(T=1 << 20, H=1, hd=8, rot=8, out_row=1 << 25)):
        assert call(_rotary(**kw)) == _abi.SWA_E_SHAPE, kw


def _append(cache=None, **kw):
    a = _abi.PagedAppendArgs()
    _cache(a.cache, **(cache or {}))
    a.T, a.nh, a.rot, a.src, a.mag = 4, 4, 128, _abi.SWA_BF16, 1.0
    for f in ("q", "k", "v", "pos", "turns"):
        setattr(a, f, FAKE)
    a.q_out = BIG
    a.q_row, a.k_row, a.v_row = 512, 256, 256
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_append_refusals(lib):
    call = lambda a: lib.swa_paged_append(ctypes.byref(a), None)
    assert lib.swa_paged_append(None, None) == _abi.SWA_E_NULL
    for kw, rc in CACHE_BAD:
        assert call(_append(cache=kw)) == rc, kw
    for kw in (dict(k=None), dict(v=None), dict(q=None), dict(q_out=None), dict(pos=None), dict(turns=None),
               dict(rot=0, turns=None, pos=None, slot_pos=FAKE)):
        assert call(_append(**kw)) == _abi.SWA_E_NULL, kw
    for kw in (dict(T=-1), dict(rot=3), dict(rot=130), dict(src=_abi.SWA_F16), dict(src=5), dict(nh=0),
               dict(mag=float("nan")), dict(k_row=128), dict(v_row=0), dict(q_row=504), dict(q_out=FAKE + 16),
               dict(q_out=FAKE, q_row=520)):
        assert call(_append(**kw)) == _abi.SWA_E_SHAPE, kw
    for kw in (dict(k=FAKE + 2), dict(q_out=BIG + 8), dict(k_row=258), dict(pos=FAKE + 1), dict(turns=FAKE + 4),
               dict(slot_pos=FAKE + 2), dict(weight=FAKE + 3)):
        assert call(_append(**kw)) == _abi.SWA_E_ALIGN, kw
    assert call(_append(T=0)) == _abi.SWA_OK
    apart = dict(cache=dict(v=BIG << 1))
    # q_out over k's or v's rows; one pool for both; row offsets that would pass 64 bits
    for kw in (dict(k=BIG + 1024, **apart), dict(v=BIG - 1024, **apart), dict(), dict(cache=dict(v=FAKE + 65520)),
               dict(T=1 << 28, nh=1, q_row=1 << 39, **apart), dict(T=1 << 28, nh=1, k_row=1 << 39, **apart),
               dict(T=1 << 28, nh=1, v_row=1 << 39, **apart)):
        assert call(_append(**kw)) == _abi.SWA_E_SHAPE, kw


def _attend(cache=None, **kw):
    a = _abi.PagedAttendArgs()
    _cache(a.cache, **(cache or {}))
    a.T, a.nh, a.max_rows, a.scale, a.q_row = 4, 4, 2, 0.1, 512
    a.q, a.out, a.workspace, a.workspace_bytes = FAKE, FAKE, FAKE, 1 << 40
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_attend_refusals(lib):
    call = lambda a: lib.swa_paged_attend(ctypes.byref(a), None)
    assert lib.swa_paged_attend(None, None) == _abi.SWA_E_NULL
    for kw, rc in CACHE_BAD:
        assert call(_attend(cache=kw)) == rc, kw
    for kw in (dict(q=None), dict(out=None)):
        assert call(_attend(**kw)) == _abi.SWA_E_NULL, kw
    for kw in (dict(T=-1), dict(max_rows=0), dict(nh=5), dict(nh=0), dict(nh=66), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(T=1 << 30), dict(q_row=500)):
        assert call(_attend(**kw)) == _abi.SWA_E_SHAPE, kw
    for kw in (dict(q=FAKE + 8), dict(out=FAKE + 4), dict(q_row=516), dict(lse=FAKE + 2), dict(workspace=FAKE + 16)):
        assert call(_attend(**kw)) == _abi.SWA_E_ALIGN, kw
    # contexts of more than 512 keys are split and need one
    for kw in (dict(workspace=None), dict(workspace_bytes=64)):
        assert call(_attend(cache=dict(max_pages=64), **kw)) == _abi.SWA_E_WORKSPACE, kw
    assert call(_attend(T=0)) == _abi.SWA_OK
    # q, out and lse may not share a byte: 4 rows of 4 heads of 128 in bf16 are 4096 bytes, of lse 64
    for kw in (dict(), dict(out=FAKE + 4080), dict(out=BIG, lse=FAKE + 4092), dict(out=BIG, lse=BIG + 4092),
               dict(out=BIG, lse=BIG + 8188, out_f32=1), dict(out=BIG, T=1 << 28, q_row=1 << 39)):
        assert call(_attend(**kw)) == _abi.SWA_E_SHAPE, kw
    assert lib.swa_paged_attend_workspace_size(ctypes.byref(_attend(cache=dict(page=48)))) == 0
    assert lib.swa_paged_attend_workspace_size(None) == 0
    assert lib.swa_paged_attend_workspace_size(ctypes.byref(_attend(nh=5))) == 0
    assert lib.swa_paged_attend_workspace_size(ctypes.byref(_attend())) > 0


def _weigh(cache=None, **kw):
    a = _abi.PagedWeighArgs()
    _cache(a.cache, **(cache or {}))
    a.T, a.nh, a.max_rows, a.scale, a.q_row = 4, 4, 2, 0.1, 512
    a.q, a.lse, a.weight, a.out = FAKE, FAKE, FAKE, BIG
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_weigh_refusals(lib):
    call = lambda a: lib.swa_paged_weigh(ctypes.byref(a), None)
    assert lib.swa_paged_weigh(None, None) == _abi.SWA_E_NULL
    for kw, rc in CACHE_BAD:
        assert call(_weigh(cache=kw)) == rc, kw
    for kw in (dict(q=None), dict(lse=None), dict(out=None)):
        assert call(_weigh(**kw)) == _abi.SWA_E_NULL, kw
    for kw in (dict(T=-1), dict(max_rows=0), dict(T=1 << 30), dict(nh=5), dict(nh=66), dict(scale=-1.0),
               dict(scale=float("inf")), dict(q_row=8), dict(out=FAKE + 4)):
        assert call(_weigh(**kw)) == _abi.SWA_E_SHAPE, kw
    for kw in (dict(q=FAKE + 8), dict(q_row=514), dict(lse=FAKE + 2), dict(weight=FAKE + 1), dict(out=BIG + 2)):
        assert call(_weigh(**kw)) == _abi.SWA_E_ALIGN, kw
    # out (1024 bytes) over q or lse; row offsets that would pass 64 bits
    for kw in (dict(out=FAKE), dict(q=BIG + 1008), dict(lse=BIG + 1020), dict(lse=BIG - 60), dict(T=1 << 28, q_row=1 << 39)):
        assert call(_weigh(**kw)) == _abi.SWA_E_SHAPE, kw


def _evict(cache=None, **kw):
    a = _abi.PagedEvictArgs()
    _cache(a.cache, **(cache or {}))
    a.keep, a.sinks = 8, 0
    a.weight, a.slot_pos, a.weight_out, a.slot_pos_out, a.lens_out = FAKE, FAKE + 4096, BIG, BIG + 4096, BIG + 8192
    a.workspace, a.workspace_bytes = FAKE, 1 << 30
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_evict_refusals(lib):
    call = lambda a: lib.swa_paged_evict(ctypes.byref(a), None)
    assert lib.swa_paged_evict(None, None) == _abi.SWA_E_NULL
    for kw, rc in CACHE_BAD:
        if "row_start" not in kw:
            assert call(_evict(cache=kw)) == rc, kw
    for f in ("weight", "slot_pos", "weight_out", "slot_pos_out", "lens_out"):
        assert call(_evict(**{f: None})) == _abi.SWA_E_NULL
    # 2 * 2 * 64 entries of 4 bytes = 1024 bytes an array
    for kw in (dict(keep=0), dict(sinks=-1), dict(weight_out=FAKE), dict(slot_pos_out=FAKE + 4096 + 1020),
               dict(lens_out=FAKE), dict(weight_out=BIG + 4096), dict(recent_from=BIG), dict(lens_out=BIG + 1020)):
        assert call(_evict(**kw)) == _abi.SWA_E_SHAPE, kw
    for kw in (dict(weight=FAKE + 2), dict(lens_out=BIG + 8193), dict(workspace=FAKE + 128)):
        assert call(_evict(**kw)) == _abi.SWA_E_ALIGN, kw
    for kw in (dict(workspace=None), dict(workspace_bytes=100)):
        assert call(_evict(**kw)) == _abi.SWA_E_WORKSPACE, kw
    assert lib.swa_paged_evict_workspace_size(None) == 0
    assert lib.swa_paged_evict_workspace_size(ctypes.byref(_evict(keep=0))) == 0


def test_packed_structs_match_the_abi(lib):
    """The binding packs the argument structs by format strings: the same sizes and field
    offsets as the ctypes declarations."""
    from sliding_window_gqa_prep_gb300 import paged
    for fmt, cls in ((paged._ROTARY, _abi.RotaryArgs), (paged._APPEND, _abi.PagedAppendArgs),
                     (paged._ATTEND, _abi.PagedAttendArgs), (paged._WEIGH, _abi.PagedWeighArgs),
                     (paged._EVICT, _abi.PagedEvictArgs)):
        assert fmt.size == ctypes.sizeof(cls)
        fields = []
        for name, kind in cls._fields_:
            if kind is _abi.PagedCache:
                fields += [(name, sub) for sub, _ in kind._fields_]
            else:
                fields.append((name, None))
        values = [float(i + 1) if getattr(dict(cls._fields_)[f[0]], "_type_", "") == "f" else i + 1
                  for i, f in enumerate(fields)]
        a = cls.from_buffer_copy(fmt.pack(*values))
        for (name, sub), want in zip(fields, values):
            x = getattr(a, name)
            assert (getattr(x, sub) if sub else x) == want, (cls, name, sub)


def test_binding_wants_cuda_tensors():
    import torch
    x = torch.zeros(2, 3, 64)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        swa.rotary(x, torch.zeros(2, dtype=torch.int32), swa.rotary_turns(64, device="cpu"))
