"""The codes that paged4_append stores, for equality with the encoding in float64 (paged4_f64.py): of prompts, whose
blocks take several rows and all heads, and of rotated keys at the edges of the encoding. The tolerance of q is that of
test_gpu_paged4.py."""
import pytest
import torch

from oracle import paged4_oracle as p4
import sliding_window_gqa_prep_gb300 as swa
import paged4_f64 as ref4
from paged4_f64 import Cache, U8

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test collected on a machine without a GPU")
    yield


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def zero():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def tiny(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def rows_of(T, nh, nk, hd, src, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    proj = torch.randn(T, (nh + 2 * nk) * hd + 8, generator=g, device="cuda")
    proj *= torch.exp2(torch.randint(-12, 5, (T, 1), generator=g, device="cuda").float())
    proj[torch.rand(proj.shape, generator=g, device="cuda") < 0.05] = 0
    proj = proj.to(src)
    return (proj[:, :nh * hd].unflatten(1, (nh, hd)), proj[:, nh * hd:(nh + nk) * hd].unflatten(1, (nk, hd)),
            proj[:, (nh + nk) * hd:(nh + 2 * nk) * hd].unflatten(1, (nk, hd)))


def stored(bt, k, v):
    """The pools after rows k, v (f64) entered."""
    want = [x.view(U8).clone() for x in bt.pools]
    for b, (t, n) in enumerate(zip(bt.t, bt.n)):
        j = torch.arange(n - t, n, device="cuda")
        at = bt.table[b].long()[j // bt.page], slice(None), j % bt.page
        for i, x in ((0, k), (2, v)):
            want[i][at], want[i + 1][at] = ref4.encode(x[bt.start[b]:bt.start[b + 1]], bt.exps[i // 2])
    return want


def append_and_check(bt, nh, src, rot, inter, mag, dtype, pos, qkv):
    q, k, v = qkv
    err = zero()
    q_out = torch.full((bt.T, nh, bt.hd), 5.0, dtype=dtype, device="cuda") if nh else None
    turns = swa.rotary_turns(rot) if rot else None
    turn = (lambda x: ref4.rotate(x, pos, turns, inter, mag)) if rot else (lambda x: x.double())   # noqa: E731
    want = stored(bt, turn(k), v.double())
    swa.paged4_append(k, v, pos, *bt.args, q=q if nh else None, q_out=q_out, turns=turns, interleaved=inter, mag=mag, err=err, **bt.exp)
    assert int(err.item()) == 0
    for name, got, w in zip(("k", "k scale", "v", "v scale"), bt.pools, want):
        bad = (got.view(U8) != w).nonzero()
        assert not len(bad), (name, len(bad), bad[:4].tolist())
    if not nh:
        return
    live, rq, a = bt.live, turn(q), q.double().abs()
    other, h = a.clone(), rot // 2
    if inter:
        other[..., 0:rot:2], other[..., 1:rot:2] = a[..., 1:rot:2], a[..., 0:rot:2]
    elif rot:
        other[..., :h], other[..., h:rot] = a[..., h:rot], a[..., :h]
    tol = (8 * 2.0 ** -24 + 2.0 ** -21) * mag * (a + other) + torch.finfo(dtype).eps / 2 * rq.abs() + tiny(dtype)
    assert ((q_out.double() - rq).abs() <= tol)[:live].all() and (q_out[live:] == 5.0).all()


@pytest.mark.parametrize("src,dtype", [(FP, BF), (BF, BF), (HF, HF)])
@pytest.mark.parametrize("rot,inter", [("all", False), ("all", True), ("some", False), (0, False)])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_append_of_prompts(hd, rot, inter, src, dtype):
    """Rows from which a block takes all heads, and several rows a warp: exact codes of prompts, from
    halves in one lane and in two, and pairs side by side."""
    most, a_warp = (8, 4) if hd == 64 else (4, 2) if hd == 128 else (4, 1)
    rot = hd if rot == "all" else 20 if rot == "some" else 0
    for T in (4 * sms() * most + 3, 4 * sms() * a_warp + 1):
        nh, nk = 5, 3
        t = [T - T // 3, 0, T // 3 - 1, 1]
        bt = Cache(t, [t[0] + 40, 9, t[2], 130], nk, hd, 32, seed=24, pad=1, exps=(1, -3))
        g = torch.Generator(device="cuda").manual_seed(25)
        pos = torch.randint(0, 100000, (bt.T,), generator=g, device="cuda", dtype=torch.int32)
        append_and_check(bt, nh, src, rot, inter, 1.25 if rot == 20 else 1.0, dtype, pos, rows_of(bt.T, nh, nk, hd, src, 26))


def test_the_encoding_here_is_the_oracle_s():
    g = torch.Generator().manual_seed(27)
    x = torch.randn(40, 2, 64, generator=g, dtype=torch.float64) * torch.exp2(torch.randint(-14, 14, (40, 1, 1), generator=g).double())
    x[0, 0, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 2).double()
    x[1, 0, 3], x[1, 1] = float("inf"), 0.0
    c, s = ref4.encode(x.cuda(), -2)
    wc, ws = p4.encode(x.numpy(), -2)
    assert (c.cpu().numpy() == wc).all() and (s.cpu().numpy() == ws).all()
    assert (ref4.decode(c[2:], s[2:], -2).cpu().numpy() == p4.decode(wc[2:], ws[2:], -2)).all()


@pytest.mark.parametrize("mag", [1.0, 1.25, 0.7071067690849304, 3.1830987930297852])
@pytest.mark.parametrize("inter", [False, True])
def test_append_rotated_next_to_borders_of_scales_and_codes(inter, mag):
    """Large features next to small partners whose rotation ends next to a border, between two scales (a block's
    largest value) and between two codes, found in f64: where f32 angles, a magnitude that is no power of two and three
    roundings could all fall the same way."""
    hd = rot = 64
    T = 20000
    mag = float(torch.tensor(mag))                           # as f32 has it
    g = torch.Generator(device="cuda").manual_seed(28)
    pos = torch.randint(1, 60000, (T,), generator=g, device="cuda", dtype=torch.int32)
    freqs = swa.rotary_freqs(rot).cuda()
    e4m3 = torch.tensor(p4.E4M3[:127], device="cuda")
    s = torch.randint(20, 100, (T, 1, hd // 16), generator=g, device="cuda")
    scale = e4m3[s]
    want = scale[..., None] * torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda", dtype=torch.float64)[
        torch.randint(0, 7, (T, 1, hd // 16, 16), generator=g, device="cuda")]
    want[..., 0] = 3 * (scale + e4m3[s + 1])                 # 6 times the middle of two scales
    want = (want * torch.where(torch.rand(want.shape, generator=g, device="cuda") < 0.5, -1.0, 1.0)).flatten(-2)
    # a pair's second feature is small: the first then is the border over the cosine
    a = pos.double()[:, None, None] * freqs
    c, sn = a.cos() * mag, a.sin() * mag
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    k = torch.zeros(T, 1, hd, device="cuda")
    small = (torch.randn(T, 1, rot // 2, generator=g, device="cuda") * 2.0 ** -10).double()
    k[..., second] = small.float()
    safe = torch.where(c.abs() < 0.05, 1.0, c)
    k[..., first] = ((want[..., first] + k[..., second].double() * sn) / safe).float()
    bt = Cache([T], [T], 1, hd, 64, seed=29)
    append_and_check(bt, 0, FP, rot, inter, mag, BF, pos, (None, k, k))


@pytest.mark.parametrize("src", [FP, BF])
def test_append_of_finite_keys_near_the_largest(src):
    """Finite keys and values near the type's largest: a rotation whose f32 result passes the range is no
    infinity, it takes the largest scale. An infinity or NaN still makes its pair's blocks NaN."""
    hd = rot = 64
    T = 300
    g = torch.Generator(device="cuda").manual_seed(30)
    big = float(torch.finfo(src).max)
    k = (torch.rand(T, 2, hd, generator=g, device="cuda") * 2 - 1) * big
    k[:100] = big
    k[100:200] = torch.where(torch.rand(100, 2, hd, generator=g, device="cuda") < 0.5, -big, big)
    k[200:, :, :20] *= 1e-30
    k = k.to(src).clamp(-big, big)
    pos = torch.randint(0, 60000, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[::7] = 0
    for inter, mag in ((False, 1.0), (True, 1.0), (False, 1.5), (True, 2.0 ** 100)):
        bt = Cache([T], [T + 3], 2, hd, 64, seed=31, exps=(20, 32))
        append_and_check(bt, 0, src, rot, inter, mag, BF, pos, (None, k, k))
        assert not (bt.pools[1].view(U8)[bt.table[0].long()[:4]] == 127).any()
    k[5, 0, 3], k[6, 1, 40], k[250, 0, 63] = float("inf"), float("nan"), float("-inf")
    bt = Cache([T], [T], 2, hd, 64, seed=31, exps=(20, 32))
    append_and_check(bt, 0, src, rot, False, 1.0, BF, pos, (None, k, k))
