"""The bound behind the encoding of rotated keys (swa_paged4_append): where f32 leaves a scale or a code open the
kernel takes the angles again in f64, and `kTol` says how far f32 may be off. Here by arithmetic, and on a model of
the kernel's f32 operations whose table of sines is as far off as CUDA grants it."""
import os
import re

import numpy as np
import pytest

from oracle import paged4_oracle as p4

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sliding_window_gqa_prep_gb300", "csrc", "swa_paged4_rows.cu")
U = 2.0 ** -24                                               # a rounding in f32, relative


@pytest.fixture(scope="module")
def source():
    with open(SOURCE) as h:
        return h.read()


@pytest.fixture(scope="module")
def tol(source):
    return float.fromhex(re.search(r"constexpr float kTol = (0x[0-9a-f.p+-]+)f;", source).group(1))


def test_the_bound_by_arithmetic(tol):
    """Every rounding at its largest, in units of |u| + |v| times mag (|cos| and the result below that)."""
    # sincospif: an ulp of a number below 1; the step that adds what the angle's f32 lacks: half an ulp
    table = 1.0 + 0.5
    # the table times mag; the product with x; the fused sum (of the result)
    rotated = table + 1.0 + 1.0 + 1.0
    # codes: the quotient, correctly rounded, and y +- d, which has to pass the border by an ulp of it (two halves)
    code = rotated + 1.0 + 2.0
    # scales: top +- tol, 1/6 in f32, the product with it, which has to pass the border by an ulp
    scale = rotated + 1.0 + 1.0 + 1.0 + 2.0
    # the tolerance itself is rounded four times
    assert tol * (1 - 4 * U) > max(code, scale) * U


@pytest.mark.parametrize("mag", [1.0, 1.25, 0.7071067690849304, 3.1830987930297852, 1.9999])
def test_scales_that_f32_leaves_open_are_seen(source, tol, mag):
    """Features next to the border between two scales, small partners: wherever f32 gives another scale than f64, the
    two ends of the kernel's interval differ too."""
    assert "f32_e4m3((s.top - tol_top) * (1.f / 6.f)) != f32_e4m3((s.top + tol_top) * (1.f / 6.f))" in source
    f, rng = np.float32, np.random.default_rng(5)
    grid = p4.E4M3[:127]

    def e4m3(x):
        x = np.clip(x.astype(np.float64), 0.0, 448.0)
        i = np.minimum(np.searchsorted(grid, x), 126)
        lo = np.maximum(i - 1, 0)
        a, b = x - grid[lo], grid[i] - x
        return np.where((i == 0) | (b < a) | ((a == b) & (i % 2 == 0)), i, lo)
    wrong = 0
    for _ in range(5):
        n = 1000000
        mg = f(mag)
        # cosines from 0.8 to 1, below 0: the angles whose f32 lacks most
        turn, low = rng.integers(1700000000, 2 ** 31, n) * rng.choice([-1, 1], n), rng.integers(0, 2 ** 32, n)
        angle = (turn + low * 2.0 ** -32) * 2.0 ** -31 * np.pi
        t = turn.astype(f)
        exact = np.cos(t.astype(np.float64) * 2.0 ** -31 * np.pi)
        cos = exact.astype(f)
        # the neighbour on the other side of the exact value: less than an ulp off
        away = np.where(cos.astype(np.float64) < exact, np.nextafter(cos, f(2)), np.nextafter(cos, f(-2)))
        cos = np.clip(away, -1, 1).astype(f)
        sin = np.sin(t.astype(np.float64) * 2.0 ** -31 * np.pi).astype(f)
        rest = (((turn - t.astype(np.int64)).astype(np.float64) + low * 2.0 ** -32) * 2.0 ** -31 * np.pi).astype(f)
        # products of two f32 are exact in f64, so a fused operation is one in f64, rounded
        c = ((cos.astype(np.float64) - sin.astype(np.float64) * rest).astype(f) * mg).astype(f)
        s = ((sin.astype(np.float64) + cos.astype(np.float64) * rest).astype(f) * mg).astype(f)
        k = rng.integers(60, 100, n)
        border = 3 * (grid[k] + grid[k + 1])
        v = (rng.standard_normal(n) * 2.0 ** -rng.integers(6, 14, n) * border).astype(f)
        cs, sn = np.cos(angle) * float(mg), np.sin(angle) * float(mg)
        some = np.abs(cs) > 0.02
        u = ((border + v * sn) / np.where(some, cs, 1.0)).astype(f)
        u = (u.view(np.int32) + rng.integers(-2, 3, n).astype(np.int32)).view(f)
        y = (-v.astype(np.float64) * s + (u * c).astype(f)).astype(f)
        top = np.abs(y)
        d = ((np.abs(u) + np.abs(v)).astype(f) * (f(tol) * mg)).astype(f)
        lo, hi = (e4m3(((x).astype(f) * f(1 / 6)).astype(f)) for x in (top - d, top + d))
        true = e4m3(np.abs(u.astype(np.float64) * cs - v.astype(np.float64) * sn) / 6)
        assert not ((lo == hi) & (lo != true) & some).any(), int(((lo == hi) & (lo != true) & some).sum())
        wrong += int(((e4m3((top * f(1 / 6)).astype(f)) != true) & some).sum())
    assert wrong > 1000                                      # the samples do come near borders
