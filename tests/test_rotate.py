"""medusa_qk_norm_rotate: norms of queries and keys by head and their rotation by position, against float64."""
import ctypes
import math

import pytest
import torch

from medusa_speculative_decoding_heads_gb300 import _build, binding as mb
from oracle import medusa_oracle as MO, serving_oracle as SO

from _helpers import gpu_ready
from _serving import assert_within, cfg_for, i32

BF16, F32 = torch.bfloat16, torch.float32
KINDS = [(BF16, 128), (BF16, 64), (F32, 64), (F32, 128)]


def freqs(rot, dev, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().to(dev)


def bound(x, y, M, f, pos, rot, normed):
    """Largest error of each value, in units of the arithmetic.

    The norm: D squares and their sum are off by D 2^-24, half of that behind the square root, whose reciprocal
    adds 2 units of 2^-23 and the two products 2^-24 each. The angle's remainder is off by pi 2^-27 (rounded to
    float32 within an eighth of a turn) and (pi / 4) 2^-24 (its product with pi), the series by less than 2^-24
    and five roundings of at most 2^-25 each: 2^-22 for sine and cosine together covers them. pos f / 2 pi comes
    from a float64 product (2^-52 of it). Turning adds two products and a sum, 3 of 2^-24."""
    D = x.shape[-1]
    e = (3 * 2.0 ** -24 + 2.0 ** -22) + ((D / 2 + 8) * 2.0 ** -24 if normed else 0.0)
    far = float((pos.double().abs().max() * f.double().abs().max())) * 2.0 ** -51 if rot else 0.0
    half = {BF16: 2.0 ** -8, F32: 2.0 ** -24}[x.dtype]
    return M * (e + far) * (1 + half) + y.abs() * half + 1e-37


def check(q, k, qw, kw, eps, f, rot, pairs, pos, qo, ko, what=""):
    for x, w, out, name in ((q, qw, qo, "queries"), (k, kw, ko, "keys")):
        y, M = SO.norm_rotate(x, w, eps, f, rot, pairs, pos)
        assert_within(out, y, bound(x, y, M, f, pos, rot, w is not None), f"{what} {name}")


def make(T, Hq, Hkv, D, dtype, dev, seed=0, fused=False, far=5000):
    gen = torch.Generator(device=dev).manual_seed(seed)
    new = lambda *s: torch.randn(s, generator=gen, device=dev).to(dtype)
    if fused:
        x = new(T, Hq + 2 * Hkv, D)
        q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    else:
        q, k = new(T, Hq, D), new(T, Hkv, D)
    pos = torch.randint(0, far, (T,), generator=gen, device=dev).int()
    return q, k, 1 + new(D) / 4, 1 + new(D) / 4, pos


def call(q, k, qw, kw, eps, f, rot, pairs, pos, qo=None, ko=None, stream=None):
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    qo = torch.full((T, Hq, D), 7.0, dtype=q.dtype, device=q.device) if qo is None else qo
    ko = torch.full((T, Hkv, D), 7.0, dtype=q.dtype, device=q.device) if ko is None else ko
    mb.qk_norm_rotate(cfg_for(1, Hq, Hkv, D, q.dtype), q, k, T, q.stride(0), k.stride(0), qw, kw, eps, f, rot,
                      mb.ROTATE_PAIRS if pairs else mb.ROTATE_HALVES, pos, qo, ko, qo.stride(0), ko.stride(0), stream)
    return qo, ko


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("rot", [0, 8, 24, 64, -1])
def test_rotated_dims(rot, pairs, dtype, D):
    dev = gpu_ready()
    rot = D if rot < 0 else rot
    f = freqs(rot, dev)
    for T, fused in ((1, False), (37, True), (200, False)):
        q, k, qw, kw, pos = make(T, 6, 2, D, dtype, dev, seed=T + rot, fused=fused)
        for a, b in ((qw, kw), (None, kw), (qw, None), (None, None)):
            check(q, k, a, b, 1e-6, f, rot, pairs, pos, *call(q, k, a, b, 1e-6, f, rot, pairs, pos))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 8), (9, 9), (16, 1), (14, 2), (40, 40), (71, 1)])
def test_heads(Hq, Hkv, dtype, D):
    dev = gpu_ready()
    q, k, qw, kw, pos = make(19, Hq, Hkv, D, dtype, dev, seed=Hq, fused=True)
    f = freqs(D, dev)
    check(q, k, qw, kw, 1e-5, f, D, False, pos, *call(q, k, qw, kw, 1e-5, f, D, False, pos))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("pairs", [False, True])
def test_far_positions(pairs, dtype, D):
    """Angles of many turns, at the ends of the positions' range, and frequencies of a turn and more."""
    dev = gpu_ready()
    q, k, qw, kw, _ = make(9, 4, 2, D, dtype, dev, seed=3)
    pos = i32([0, 1, -1, 131071, 1000003, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 77777777], dev)
    for f in (freqs(D, dev), torch.linspace(0.0, 7.0, D // 2, device=dev), -freqs(D, dev, 500.0)):
        check(q, k, qw, kw, 1e-6, f, D, pairs, pos, *call(q, k, qw, kw, 1e-6, f, D, pairs, pos))


@pytest.mark.gpu
@pytest.mark.parametrize("pairs", [False, True])
def test_sines_all_the_way_round(pairs):
    """Vectors (1, 0) turn into (cos, sin): a position's angle anywhere on the circle, without a norm."""
    dev = gpu_ready()
    T = 4096
    q = torch.zeros((T, 1, 64), device=dev)
    q[:, :, 0:64:2] = 1.0
    if not pairs:
        q[:] = 0
        q[:, :, :32] = 1.0
    pos = torch.arange(-T // 2, T // 2, device=dev).int()
    f = torch.linspace(1e-4, math.pi, 32, device=dev)
    check(q, q, None, None, 0.0, f, 64, pairs, pos, *call(q, q.clone(), None, None, 0.0, f, 64, pairs, pos))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
def test_in_place_and_rows_left_alone(dtype, D):
    """In place inside a fused projection's output: values and everything else keep what they held."""
    dev = gpu_ready()
    q, k, qw, kw, pos = make(61, 6, 2, D, dtype, dev, seed=8, fused=True)
    before = q._base.clone() if q._base is not None else None
    q0, k0 = q.clone(), k.clone()
    f = freqs(D, dev)
    T = 50
    call(q[:T], k[:T], qw, kw, 1e-6, f, D, False, pos[:T].contiguous(), q[:T], k[:T])
    check(q0[:T], k0[:T], qw, kw, 1e-6, f, D, False, pos[:T], q[:T], k[:T], "in place")
    assert torch.equal(q[T:], q0[T:]) and torch.equal(k[T:], k0[T:])
    assert before is not None and torch.equal(q._base[:, 8:], before[:, 8:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("branching", [(2, 2), (4, 3, 2, 1)])
def test_trees(branching, dtype, D):
    """Positions as medusa_tree_build gives them, keys into the staged layout."""
    dev = gpu_ready()
    B, Hq, Hkv = 3, 8, 2
    tree = MO.tree_layout(branching)
    N = len(tree["parent"])
    q, k, qw, kw, _ = make(B * N, Hq, Hkv, D, dtype, dev, seed=N, fused=True)
    depth = torch.tensor([int(d) for d in tree["depth"]], device=dev)
    pos = (torch.tensor([0, 900, 16000], device=dev)[:, None] + depth[None]).int().contiguous()
    cfg = cfg_for(B, Hq, Hkv, D, dtype, 16384 + N, branching)
    assert mb.node_count(cfg) == N
    f = freqs(D, dev)
    qo = torch.full((B, N, Hq, D), 7.0, dtype=dtype, device=dev)
    ko = torch.full((B, Hkv, N, D), 7.0, dtype=dtype, device=dev)
    mb.qk_norm_rotate(cfg, q, k, B * N, q.stride(0), k.stride(0), qw, kw, 1e-6, f, D, mb.ROTATE_HALVES, pos, qo, ko, Hq * D, 0)
    check(q, k, qw, kw, 1e-6, f, D, False, pos.flatten(), qo.view(B * N, Hq, D), ko.transpose(1, 2).reshape(B * N, Hkv, D))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
def test_zeros_and_non_finite_values(dtype, D):
    """A head of zeros stays zero (eps > 0) or is 0 / 0 (eps = 0); what is no number stays in its own head."""
    dev = gpu_ready()
    q, k, qw, kw, pos = make(5, 4, 2, D, dtype, dev, seed=4)
    f = freqs(D, dev)
    q[1, 2] = 0
    clean = call(q, k, qw, kw, 1e-6, f, D, False, pos)
    assert bool((clean[0][1, 2] == 0).all())
    assert bool(call(q, k, qw, kw, 0.0, f, D, False, pos)[0][1, 2].isnan().all())
    bad = q.clone()
    bad[3, 1, 5], bad[0, 0, 0] = float("nan"), float("inf")
    qo, ko = call(bad, k, qw, kw, 1e-6, f, D, False, pos)
    assert bool(qo[3, 1].isnan().all()) and torch.equal(ko, clean[1])
    keep = torch.ones((5, 4), dtype=torch.bool, device=dev)
    keep[3, 1] = keep[0, 0] = False
    assert torch.equal(qo[keep], clean[0][keep])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
def test_frequencies_that_are_no_number(dtype, D):
    dev = gpu_ready()
    q, k, qw, kw, pos = make(3, 2, 2, D, dtype, dev, seed=6)
    f = freqs(D, dev)
    clean = call(q, k, qw, kw, 1e-6, f, D, True, pos)[0]
    f[1], f[3] = float("inf"), float("nan")
    got = call(q, k, qw, kw, 1e-6, f, D, True, pos)[0]
    dead = torch.zeros(D, dtype=torch.bool, device=dev)
    dead[[2, 3, 6, 7]] = True
    assert bool(got[..., dead].isnan().all()) and torch.equal(got[..., ~dead], clean[..., ~dead])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_offsets_past_32_bits(dtype, D):
    dev = gpu_ready()
    stride = 1 << 20
    T = 2200 if dtype == BF16 else 2150
    view = torch.empty(T * stride, dtype=dtype, device=dev).view(T, stride)
    rows = view[:, :8 * D].unflatten(1, (8, D))
    gen = torch.Generator(device=dev).manual_seed(1)
    rows.copy_(torch.randn((T, 8, D), generator=gen, device=dev))
    q, k = rows[:, :6], rows[:, 6:]
    q0, k0 = q.clone(), k.clone()
    pos = torch.arange(T, device=dev).int()
    f = freqs(D, dev)
    call(q, k, None, None, 0.0, f, D, False, pos, q, k)
    check(q0, k0, None, None, 0.0, f, D, False, pos, q, k)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_streams_and_graph(dtype, D):
    """Calls at once on two streams; a captured call replayed on changed inputs and positions; equal bits."""
    dev = gpu_ready()
    sets = [make(700, 8, 2, D, dtype, dev, seed=s) for s in (1, 2)]
    f = freqs(D, dev)
    want = [call(*s[:4], 1e-6, f, D, False, s[4]) for s in sets]
    outs = [tuple(torch.zeros_like(x) for x in w) for w in want]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, st in zip(sets, outs, streams):
            call(*s[:4], 1e-6, f, D, False, s[4], *o, st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    q, k, qw, kw, pos = (x.clone() for x in sets[0])
    o = tuple(torch.zeros_like(x) for x in want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(q, k, qw, kw, 1e-6, f, D, False, pos, *o)
    for x, y in zip((q, k, qw, kw, pos), sets[1]):
        x.copy_(y)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o[0], want[1][0]) and torch.equal(o[1], want[1][1])


# ----------------------------------------------------------------------------- the oracle (no GPU)
def test_oracle_turns_complex_numbers():
    gen = torch.Generator().manual_seed(2)
    x = torch.randn((7, 3, 16), generator=gen)
    pos, f = torch.arange(7) * 13, freqs(8, "cpu")
    for pairs in (False, True):
        y, M = SO.norm_rotate(x, None, 0.0, f, 8, pairs, pos)
        z = x.double()[..., :8]
        z = torch.complex(z[..., 0::2], z[..., 1::2]) if pairs else torch.complex(z[..., :4].contiguous(), z[..., 4:].contiguous())
        z = z * torch.exp(1j * (pos.double()[:, None] * f.double()))[:, None]
        want = torch.stack([z.real, z.imag], -1).flatten(-2) if pairs else torch.cat([z.real, z.imag], -1)
        assert (y[..., :8] - want).abs().max() < 1e-12 and torch.equal(y[..., 8:], x.double()[..., 8:])
        assert bool((M >= y.abs() - 1e-12).all())
    y, _ = SO.norm_rotate(x, torch.full((16,), 2.0), 0.0, f, 0, False, pos)
    assert ((y * y).mean(-1) - 4.0).abs().max() < 1e-12


# ----------------------------------------------------------------------------- refusals (no GPU)
def status(T=8, q_stride=None, k_stride=None, qo_stride=None, ko_stride=None, q=4096, k=8192, qw=256, kw=256, eps=1e-6, f=512,
           rot=None, pairing=0, pos=4, qo=12288, ko=16384, dtype=BF16, D=128, Hq=4, Hkv=2, B=1, branching=(1,)):
    _build.build()
    cfg = cfg_for(B, 4, 2, D, dtype, branching=branching)
    cfg.Hq, cfg.Hkv = Hq, Hkv
    ptr = lambda x: ctypes.c_void_p(x) if x else None
    or_ = lambda x, y: y if x is None else x
    return mb.load().medusa_qk_norm_rotate(
        ctypes.byref(cfg), ptr(q), ptr(k), T, or_(q_stride, Hq * D), or_(k_stride, Hkv * D), ptr(qw), ptr(kw), eps, ptr(f),
        or_(rot, D), pairing, ptr(pos), ptr(qo), ptr(ko), or_(qo_stride, Hq * D), or_(ko_stride, Hkv * D), None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), -1), (dict(q=0), -1), (dict(k=0), -1), (dict(qo=0), -1), (dict(ko=0), -1), (dict(f=0), -1), (dict(pos=0), -1),
    (dict(q=4104), -1), (dict(k=8200), -1), (dict(qo=12290), -1), (dict(ko=16392), -1), (dict(qw=264), -1), (dict(kw=8), -1),
    (dict(f=516), -1), (dict(eps=-1e-6), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
    (dict(rot=-8), -1), (dict(rot=136), -1), (dict(rot=12), -2), (dict(rot=2), -2), (dict(pairing=2), -1), (dict(pairing=-1), -1),
    (dict(q_stride=511), -1), (dict(q_stride=516), -1), (dict(k_stride=248), -1), (dict(qo_stride=0), -1), (dict(ko_stride=-256), -1),
    (dict(dtype=F32, q_stride=514), -1), (dict(D=96), -2), (dict(Hkv=3), -2),
    (dict(q=4096, qo=4096, q_stride=1024), -1), (dict(k=8192, ko=8192, k_stride=512), -1),
    (dict(ko_stride=0), -1), (dict(ko_stride=0, T=1, ko=8192), -1), (dict(ko_stride=0, T=14, B=2, branching=(2, 2), ko=8192), -1),
    (dict(T=2 ** 31 - 1), -2), (dict(T=2 ** 24, Hq=1024, Hkv=2), -2),
    (dict(T=0, q=0, k=0, qo=0, ko=0, f=0, pos=0), 0),
])
def test_refusals(kw, want):
    assert status(**kw) == want
