"""medusa_prompt_attention: causal attention over packed prompts, against float64."""
import ctypes

import pytest
import torch

from medusa_speculative_decoding_heads_gb300 import _build, binding as mb
from oracle import serving_oracle as SO

from _helpers import gpu_ready
from _serving import assert_within, cfg_for, i32, offsets, tolerance

BF16, F32 = torch.bfloat16, torch.float32


def make(lens, Hq, Hkv, D, dtype, dev, seed=0, pad=0, first=0, fused=False):
    gen = torch.Generator(device=dev).manual_seed(seed)
    cu = offsets(lens, first)
    T = cu[-1] + pad
    if fused:
        x = torch.randn((T, Hq + 2 * Hkv, D), generator=gen, device=dev).to(dtype)
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cu
    new = lambda h: torch.randn((T, h, D), generator=gen, device=dev).to(dtype)
    return new(Hq) * 2, new(Hkv), new(Hkv), cu


def call(q, k, v, cu, O=None, stream=None):
    T, Hq, D = q.shape
    O = torch.full((T, Hq, D), 7.0, dtype=q.dtype, device=q.device) if O is None else O
    cfg = cfg_for(len(cu) - 1, Hq, k.shape[1], D, q.dtype)
    cu = cu if isinstance(cu, torch.Tensor) else i32(cu, q.device)
    mb.prompt_attention(cfg, q, k, v, T, q.stride(0), k.stride(0), v.stride(0), cu, O, stream)
    return O


def check(q, k, v, cu, O, what=""):
    """Owned rows against float64; the others still hold what they held (7)."""
    ref, A, S = SO.prompt_attention(q, k, v, cu)
    owned = torch.zeros(q.shape[0], dtype=torch.bool, device=q.device)
    for a, e in zip(cu[:-1], cu[1:]):
        if 0 <= a <= e <= q.shape[0]:
            owned[a:e] = True
    keys = max([e - a for a, e in zip(cu[:-1], cu[1:])] + [1])
    assert_within(O[owned], ref[owned], tolerance(q.dtype, ref, A, S, keys)[owned], what or "prompt attention")
    assert bool((O[~owned] == 7.0).all()), f"{what}: rows that no sequence owns were written"
    assert mb.poll_errors() == (0, 0, 0)


LENS = [[1], [0, 1, 2, 0, 3], [31, 32, 33], [127, 128, 129], [255, 256, 257], [300, 0, 65, 1], [700], [0]]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_lengths(lens, dtype, D):
    dev = gpu_ready()
    q, k, v, cu = make(lens, 4, 2, D, dtype, dev, seed=len(lens), pad=5)
    check(q, k, v, cu, call(q, k, v, cu))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (4, 1), (6, 2), (8, 8), (16, 1), (14, 2), (32, 1), (12, 3), (40, 40)])
def test_heads(Hq, Hkv, dtype, D):
    dev = gpu_ready()
    q, k, v, cu = make([150, 1, 0, 290], Hq, Hkv, D, dtype, dev, seed=Hq, fused=True)
    check(q, k, v, cu, call(q, k, v, cu))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_long_and_many(dtype, D):
    """One prompt of several thousand rows, then a hundred short ones."""
    dev = gpu_ready()
    q, k, v, cu = make([3001], 2, 1, D, dtype, dev, seed=3)
    check(q, k, v, cu, call(q, k, v, cu))
    q, k, v, cu = make([(7 * i) % 41 for i in range(100)] + [513], 4, 4, D, dtype, dev, seed=4, first=3, pad=2)
    check(q, k, v, cu, call(q, k, v, cu))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 128)])
def test_many_sequences(dtype, D):
    """More sequences than any per-thread table would hold."""
    dev = gpu_ready()
    lens = [1 + (i % 3) for i in range(1500)]
    lens[700], lens[1499] = 400, 270
    q, k, v, cu = make(lens, 2, 1, D, dtype, dev, seed=9)
    check(q, k, v, cu, call(q, k, v, cu))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_non_finite_values_stay_in_their_sequence(dtype, D):
    """Neighbours and padding full of NaN and infinities do not reach a sequence's rows."""
    dev = gpu_ready()
    lens = [70, 130, 1, 200, 65]
    q, k, v, cu = make(lens, 4, 2, D, dtype, dev, seed=5, first=9, pad=40)
    ref_q, ref_k, ref_v = q.clone(), k.clone(), v.clone()
    for a, e in ((0, 9), (cu[1], cu[2]), (cu[3], cu[4]), (cu[5], q.shape[0])):
        q[a:e], k[a:e] = float("nan"), float("inf")
        v[a:e:2], v[a + 1:e:2] = float("nan"), float("-inf")
    O = call(q, k, v, cu)
    ref, A, S = SO.prompt_attention(ref_q, ref_k, ref_v, cu)
    tol = tolerance(dtype, ref, A, S, max(lens))
    for s in (0, 2, 4):
        rows = slice(cu[s], cu[s + 1])
        assert_within(O[rows], ref[rows], tol[rows], f"sequence {s}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_growing_scores(dtype, D):
    """Keys whose scores grow by hundreds along the prompt (the running maximum moves at every tile),
    then ones that fall; and equal scores everywhere."""
    dev = gpu_ready()
    n = 700
    q, k, v, cu = make([n, n, n], 2, 1, D, dtype, dev, seed=8)
    ramp = torch.linspace(0, 30, n, device=dev)[:, None, None]
    q[:] = 0
    q[:, :, 0] = 80.0
    k[:n, :, :1] = ramp.to(dtype)
    k[n:2 * n, :, :1] = (30 - ramp).to(dtype)
    k[2 * n:] = 1.0
    check(q, k, v, cu, call(q, k, v, cu))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_bad_offsets_are_skipped(dtype, D):
    """Sequences whose bounds decrease or leave [0, T] write nothing; the others are right."""
    dev = gpu_ready()
    q, k, v, _ = make([200], 4, 2, D, dtype, dev, seed=6)
    for cu in ([0, 60, 250], [-5, 60, 130], [0, 50, 40, 140][:2] + [200, 190]):
        O = call(q, k, v, cu)
        good = [(a, e) for a, e in zip(cu[:-1], cu[1:]) if 0 <= a <= e <= 200]
        ref, A, S = SO.prompt_attention(q, k, v, cu)
        tol = tolerance(dtype, ref, A, S, 200)
        written = torch.zeros(200, dtype=torch.bool, device=dev)
        for a, e in good:
            assert_within(O[a:e], ref[a:e], tol[a:e], str(cu))
            written[a:e] = True
        assert bool((O[~written] == 7.0).all()), cu


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_offsets_past_32_bits(dtype, D):
    """Rows so far apart that their element offsets pass 2^31."""
    dev = gpu_ready()
    stride = 1 << 20
    T = 2200 if dtype == BF16 else 2150
    x = torch.empty(T * stride, dtype=dtype, device=dev)
    view = x.view(T, stride)
    gen = torch.Generator(device=dev).manual_seed(1)
    Hq, Hkv = 4, 2
    view[:, :(Hq + 2 * Hkv) * D] = torch.randn((T, (Hq + 2 * Hkv) * D), generator=gen, device=dev).to(dtype)
    part = lambda h0, h: view[:, h0 * D:(h0 + h) * D].unflatten(1, (h, D))
    q, k, v = part(0, Hq), part(Hq, Hkv), part(Hq + Hkv, Hkv)
    cu = [T - 300, T - 100, T]
    check(q, k, v, cu, call(q, k, v, cu))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_streams_and_graph(dtype, D):
    """Two calls at once on two streams, and a captured call replayed on changed inputs and lengths."""
    dev = gpu_ready()
    sets = [make([500, 33, 260], 8, 2, D, dtype, dev, seed=s) for s in (1, 2)]
    want = [call(*s) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.full_like(w, 7.0) for w in want]
    cus = [i32(s[3], dev) for s in sets]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, o, c, st in zip(sets, outs, cus, streams):
            call(s[0], s[1], s[2], c, o, st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    q, k, v, cu = sets[0]
    q, k, v, cu_d, O = q.clone(), k.clone(), v.clone(), cus[0].clone(), torch.full_like(want[0], 7.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(q, k, v, cu_d, O)
    q.copy_(sets[1][0]), k.copy_(sets[1][1]), v.copy_(sets[1][2])
    new_cu = [0, 100, 790, 793]
    cu_d.copy_(i32(new_cu, dev))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    check(q, k, v, new_cu, O, "replayed")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_same_inputs_same_bits(dtype, D):
    dev = gpu_ready()
    q, k, v, cu = make([900, 17, 400], 8, 2, D, dtype, dev, seed=2)
    first = call(q, k, v, cu)
    for _ in range(3):
        assert torch.equal(call(q, k, v, cu), first)


# ----------------------------------------------------------------------------- the oracle (no GPU)
def test_oracle_is_causal_attention():
    """Against torch's attention in float64, each sequence on its own; rows outside stay 0."""
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((60, h, 64), generator=gen) for h in (6, 2, 2))
    cu = [5, 5, 25, 26, 55]
    O, A, S = SO.prompt_attention(q, k, v, cu)
    for a, e in zip(cu[:-1], cu[1:]):
        if e == a:
            continue
        t = lambda x: x[a:e].double().transpose(0, 1)
        want = torch.nn.functional.scaled_dot_product_attention(t(q), t(k).repeat_interleave(3, 0), t(v).repeat_interleave(3, 0),
                                                                is_causal=True).transpose(0, 1)
        assert (O[a:e] - want).abs().max() < 1e-12
    assert bool((O[:5] == 0).all()) and bool((O[55:] == 0).all())
    assert bool((A >= O.abs() - 1e-12).all()) and bool((S[5:55] > 0).all())


# ----------------------------------------------------------------------------- refusals (no GPU)
def status(T=8, B=2, q_stride=None, k_stride=None, v_stride=None, q=4096, k=4096, v=4096, cu=4096, o=4096, dtype=BF16, D=128,
           Hq=4, Hkv=2, **kw):
    _build.build()
    cfg = cfg_for(2, 4, 2, D, dtype)
    cfg.B, cfg.Hq, cfg.Hkv = B, Hq, Hkv
    ptr = lambda x: ctypes.c_void_p(x) if x else None
    return mb.load().medusa_prompt_attention(
        ctypes.byref(cfg), ptr(q), ptr(k), ptr(v), T, q_stride if q_stride is not None else Hq * D,
        k_stride if k_stride is not None else Hkv * D, v_stride if v_stride is not None else Hkv * D, ptr(cu), ptr(o), None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), -1), (dict(q=0), -1), (dict(k=0), -1), (dict(v=0), -1), (dict(cu=0), -1), (dict(o=0), -1),
    (dict(q=4104), -1), (dict(k=4098), -1), (dict(v=4104), -1), (dict(o=4104), -1),
    (dict(q_stride=511), -1), (dict(q_stride=516), -1), (dict(k_stride=255), -1), (dict(v_stride=-256), -1),
    (dict(v_stride=0), -1), (dict(dtype=F32, q_stride=514), -1), (dict(D=96), -2), (dict(Hkv=3), -2),
    (dict(T=0, q=0, k=0, v=0, o=0, cu=0), 0),
])
def test_refusals(kw, want):
    assert status(**kw) == want


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_units_than_blocks_is_refused(dtype):
    assert status(B=2 ** 27, Hq=32, dtype=dtype) == -2
    assert status(B=2 ** 31 - 1, Hq=32, dtype=dtype) == -2
    assert status(T=2 ** 31 - 1, Hq=128, dtype=dtype) == -2
