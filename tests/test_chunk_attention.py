"""medusa_chunk_attention_paged and medusa_window_attention_paged: new tokens over a paged cache, against float64."""
import ctypes

import pytest
import torch

from medusa_speculative_decoding_heads_gb300 import _build, binding as mb
from oracle import serving_oracle as SO

from _helpers import gpu_ready
from _serving import assert_within, cfg_for, i32, offsets, tolerance

BF16, F32 = torch.bfloat16, torch.float32
KINDS = [(BF16, 128), (BF16, 64), (F32, 64), (F32, 128)]
BAD_PAGES = [-1, -7, 1 << 30, 2 ** 31 - 1]   # what block-table entries that are not read may hold


class Case:
    """New rows of some sequences, their pages, and a cache that is full of what is no number where no row may look."""

    def __init__(self, rows, start, Hq, Hkv, D, dtype, dev, seed=0, P=128, pad=0, first=0, window=None, sinks=0, fused=False,
                 spare=3, extra_cap=0):
        gen = torch.Generator(device=dev).manual_seed(seed)
        cpu = torch.Generator().manual_seed(seed)
        self.dev, self.dtype, self.P, self.window, self.sinks, self.start = dev, dtype, P, window, sinks, list(start)
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.cu = offsets(rows, first)
        self.T = self.cu[-1] + pad
        B = len(rows)
        width = max([-(-(s + n) // P) for s, n in zip(start, rows)] + [1]) + extra_cap
        self.L_cap = width * P
        held = [-(-(s + n) // P) if n else 0 for s, n in zip(start, rows)]
        self.num = sum(held) + spare
        ids = torch.randperm(self.num, generator=cpu).tolist()
        nan = float("nan")
        self.Kp, self.Vp = (torch.full((self.num, Hkv, P, D), nan, dtype=dtype, device=dev) for _ in range(2))
        self.table, at = [[BAD_PAGES[(b + i) % 4] for i in range(width)] for b in range(B)], 0
        for b, (n, s) in enumerate(zip(rows, start)):
            if n == 0:
                continue
            end = s + n
            K, V = (torch.full((held[b] * P, Hkv, D), nan, dtype=dtype, device=dev) for _ in range(2))
            j = torch.arange(end, device=dev)
            seen = (j < sinks) | (j > s - window) if window is not None else j >= 0
            for X in (K, V):
                X[:end][seen] = torch.randn((int(seen.sum()), Hkv, D), generator=gen, device=dev).to(dtype)
            live = seen.nonzero().flatten() // P
            for i in set(live.tolist()):
                page = ids[at]
                at += 1
                self.table[b][i] = page
                self.Kp[page], self.Vp[page] = (X[i * P:(i + 1) * P].transpose(0, 1) for X in (K, V))
        heads = Hq + 2 * Hkv if fused else Hq
        self.q = (2 * torch.randn((self.T, heads, D), generator=gen, device=dev)).to(dtype)[:, :Hq]
        self.cfg = cfg_for(B, Hq, Hkv, D, dtype, self.L_cap)
        self.table_d, self.cu_d, self.start_d = i32(self.table, dev), i32(self.cu, dev), i32(self.start, dev)

    def workspace(self):
        return torch.full((mb.chunk_workspace_size(self.cfg, self.T) // 4,), float("nan"), device=self.dev)   # 256-byte aligned

    def call(self, O=None, ws=None, stream=None, start="own"):
        O = torch.full((self.T, self.Hq, self.D), 7.0, dtype=self.dtype, device=self.dev) if O is None else O
        ws = self.workspace() if ws is None else ws
        head = (self.cfg, self.q, self.T, self.q.stride(0), self.cu_d, self.start_d if start == "own" else start, self.Kp, self.Vp,
                self.num, self.P, self.table_d)
        if self.window is None:
            mb.chunk_attention_paged(*head, O, ws if ws.numel() else None, stream)
        else:
            mb.window_attention_paged(*head, self.window, self.sinks, O, ws if ws.numel() else None, stream)
        return O

    def check(self, O, what="", start="own"):
        ref, A, S, owned = SO.chunk_attention(self.q, self.Kp, self.Vp, self.P, self.table, self.cu,
                                              self.start if start == "own" else start, self.L_cap, self.window, self.sinks)
        tol = tolerance(self.dtype, ref, A, S, self.L_cap)
        assert_within(O[owned], ref[owned], tol[owned], what or "chunk attention")
        assert bool((O[~owned] == 7.0).all()), f"{what}: rows that are not computed were written"
        assert mb.poll_errors() == (0, 0, 0)


SHAPES = [([1], [0]), ([1], [127]), ([1], [128]), ([1, 1, 1], [0, 255, 256]), ([2, 0, 3], [126, 5, 127]), ([31, 33], [97, 0]),
          ([128, 129, 127], [0, 128, 1]), ([255, 257], [256, 130]), ([300, 1, 0, 65, 1], [0, 900, 10, 333, 2]), ([700], [0]),
          ([513, 1], [640, 1151]), ([0], [0]), ([0, 0], [5, 0])]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("rows,start", SHAPES, ids=str)
def test_lengths(rows, start, dtype, D):
    dev = gpu_ready()
    for P in (128, 384):
        c = Case(rows, start, 4, 2, D, dtype, dev, seed=len(rows), pad=5, P=P)
        c.check(c.call())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (4, 1), (6, 2), (8, 8), (16, 1), (14, 2), (32, 1), (12, 3), (40, 40), (96, 1)])
def test_heads(Hq, Hkv, dtype, D):
    dev = gpu_ready()
    c = Case([150, 1, 0, 5], [290, 600, 3, 100], Hq, Hkv, D, dtype, dev, seed=Hq, fused=True)
    c.check(c.call())
    c = Case([1, 1, 1], [600, 3, 100], Hq, Hkv, D, dtype, dev, seed=Hq, fused=True)
    c.check(c.call())


WINDOWS = [(1, 0), (1, 1), (1, 4), (2, 300), (64, 0), (127, 1), (128, 0), (128, 128), (129, 4), (200, 127), (257, 129), (384, 256),
           (1000, 4), (2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (300, 2 ** 31 - 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_windows(window, sinks, dtype, D):
    """Windows that end inside pages, at their ends, reach into the first rows or past everything."""
    dev = gpu_ready()
    for rows, start, P in (([1, 1, 1, 1], [0, 383, 384, 1000], 128), ([130, 1, 0, 300, 20], [500, 640, 9, 0, 371], 256),
                           ([513], [300], 128)):
        c = Case(rows, start, 4, 2, D, dtype, dev, seed=window % 97, pad=2, P=P, window=window, sinks=sinks)
        c.check(c.call(), f"window {window}, sinks {sinks}, rows {rows}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
def test_long_caches(dtype, D):
    """Single tokens and short chunks over thousands of rows (work split over the keys), one sequence and several."""
    dev = gpu_ready()
    for rows, start in (([1], [9000]), ([3], [5117]), ([1, 1, 70, 1], [4000, 0, 6001, 11111]), ([200], [7000])):
        for window in (None, 2500):
            c = Case(rows, start, 8, 2, D, dtype, dev, seed=sum(rows), window=window, sinks=5 if window else 0)
            c.check(c.call(), f"{rows} after {start}")


def patterns(B):
    gen = torch.Generator().manual_seed(B)
    r = lambda hi: int(torch.randint(0, hi, (1,), generator=gen))
    yield "single tokens", [1] * B, [r(400) for _ in range(B)]
    yield "random, zeros among them", [[0, 1, 1, r(40), r(300)][r(5)] for _ in range(B)], [r(300) for _ in range(B)]
    yield "a long one last", [r(3) for _ in range(B - 1)] + [700], [r(100) for _ in range(B - 1)] + [200]
    yield "a long one first", [700] + [r(3) for _ in range(B - 1)], [200] + [r(100) for _ in range(B - 1)]
    yield "empty but for two", [0] * (B - 2) + [130, 1], [0] * (B - 1) + [4]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,Hq,Hkv", [(BF16, 128, 3, 3), (BF16, 64, 4, 1), (F32, 64, 4, 2), (F32, 128, 3, 1)])
@pytest.mark.parametrize("B", [31, 32, 33, 65, 333])
def test_many_sequences(B, dtype, D, Hq, Hkv):
    dev = gpu_ready()
    for name, rows, start in patterns(B):
        c = Case(rows, start, Hq, Hkv, D, dtype, dev, seed=B, pad=3, first=2)
        c.check(c.call(), name)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("B,at", [(40, 3), (70, 31), (70, 32), (70, 33), (200, 150), (33, 0)])
def test_many_sequences_ahead_of_a_decrease(B, at, dtype, D):
    """Offsets that fall somewhere among more sequences than a warp has lanes: those ahead are right, none behind is computed."""
    dev = gpu_ready()
    c = Case([1 + b % 3 for b in range(B)], [(37 * b) % 300 for b in range(B)], 4, 2, D, dtype, dev, seed=B, pad=2)
    cu = list(c.cu)
    cu[at + 1] = cu[at] - 1
    c.cu_d, c.cu = i32(cu, dev), cu
    c.check(c.call(), f"{at} of {B}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_thousands_of_sequences(dtype, D):
    """Single tokens and a few longer ones among 3000 sequences; finding whose work is whose stays cheap beside it."""
    dev = gpu_ready()
    B = 3000
    rows = [1] * B
    rows[17], rows[1500], rows[2999], rows[40] = 300, 2, 150, 0
    c = Case(rows, [b % 140 for b in range(B)], 2, 1, D, dtype, dev, seed=1)
    c.check(c.call())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
def test_no_start_is_zero(dtype, D):
    """A prompt in one piece: start may be NULL, and the rows are those of medusa_prompt_attention's formula."""
    dev = gpu_ready()
    c = Case([333, 0, 65], [0, 0, 0], 4, 2, D, dtype, dev, seed=1)
    O = c.call(start=None)
    c.check(O, start=None)
    assert torch.equal(O, c.call())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
def test_sequences_that_are_skipped(dtype, D):
    """Starts and offsets that leave the cache, the rows, or decrease: their rows stay as they are, the others are right."""
    dev = gpu_ready()
    good = Case([40, 1, 130, 7], [100, 300, 0, 249], 4, 2, D, dtype, dev, seed=3, pad=20)
    for b, s in ((0, -1), (1, -2 ** 31), (2, 2 ** 31 - 1), (3, good.L_cap - 6), (2, good.L_cap - 129)):
        good.start_d = i32([s if i == b else x for i, x in enumerate(good.start)], dev)
        keep, good.start = good.start, good.start_d.tolist()
        good.check(good.call(), f"start {s}")
        good.start = keep
    good.start_d = i32(good.start, dev)
    for cu in ([0, 40, 41, 171, 900], [-3, 40, 41, 171, 178], [0, 40, 30, 171, 178], [5, 4, 41, 171, 178], [0, 40, 41, 171, 170],
               [0, 40, 41, 2 ** 31 - 1, 178]):
        good.cu_d, good.cu = i32(cu, dev), cu
        good.check(good.call(), f"offsets {cu}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("page", [-1, -2 ** 31, "num", 2 ** 31 - 1])
def test_pages_outside_the_pool_are_zeros(page, dtype, D):
    dev = gpu_ready()
    for rows, start in (([1, 1], [700, 300]), ([140, 1], [300, 500])):
        c = Case(rows, start, 4, 2, D, dtype, dev, seed=5)
        c.table[0][1] = c.table[1][0] = c.num if page == "num" else page
        c.table_d = i32(c.table, dev)
        O = c.call()
        c.check(O, f"page {page}")
        assert mb.poll_checks() == ((-6, mb.CHECK_PAGE) if mb.checked_build() else (0, 0))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
def test_growing_and_equal_scores(dtype, D):
    """Keys whose scores grow by hundreds along the cache, ones that fall, and equal scores everywhere."""
    dev = gpu_ready()
    for n, s in ((1, 1500), (300, 900)):
        c = Case([n, n, n], [s, s, s], 2, 1, D, dtype, dev, seed=8)
        ramp = torch.linspace(0, 30, n + s, device=dev)
        c.q[:] = 0
        c.q[:, :, 0] = 80.0
        for b, keys in enumerate((ramp, 30 - ramp, torch.ones_like(ramp))):
            for i in range(0, n + s, 128):
                part = keys[i:i + 128]
                c.Kp[c.table[b][i // 128], :, :part.numel(), 0] = part.to(dtype)
                if b == 2:
                    c.Kp[c.table[b][i // 128], :, :part.numel()] = 1.0
        c.check(c.call())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
def test_infinite_scores(dtype, D):
    """Keys that score -inf weigh nothing; a row that sees only such is no number; nor is one that sees +inf."""
    dev = gpu_ready()
    for rows, start in (([1, 1, 1], [200, 0, 1500]), ([20, 140], [190, 0])):
        c = Case(rows, start, 4, 2, D, dtype, dev, seed=9)
        c.q[..., 0] = c.q[..., 0].abs() + 0.5
        clean = c.Kp.clone()
        dead = 150
        for b in range(len(rows)):
            for i in (0, 1):
                if c.table[b][i] in range(c.num):
                    c.Kp[c.table[b][i], :, :max(0, min(128, dead - 128 * i)), 0] = float("-inf")
        O = c.call()
        window, sinks = c.window, c.sinks
        for b, (a, e) in enumerate(zip(c.cu[:-1], c.cu[1:])):
            s = c.start[b]
            n = max(0, min(e - a, dead - s))   # rows without a finite score
            assert bool(O[a:a + n].isnan().all())
            if n == e - a:
                continue
            j = torch.arange(dead, s + e - a, device=dev)
            pages = torch.tensor([c.table[b][int(x) // 128] for x in j], device=dev)
            p = torch.arange(s + n, s + e - a, device=dev)[:, None]
            ref, A, S = SO.attend(c.q[a + n:e], clean[pages, :, j % 128], c.Vp[pages, :, j % 128], j <= p)
            assert_within(O[a + n:e], ref, tolerance(dtype, ref, A, S, c.L_cap), "behind the dead rows")
        c.Kp.copy_(clean)
        b = len(rows) - 1
        c.Kp[c.table[b][0], :, 100, 0] = float("inf")
        O = c.call()
        a, e = c.cu[b], c.cu[b + 1]
        first = max(0, 100 - c.start[b])
        assert bool(O[a + first:e].isnan().all()) and bool(torch.isfinite(O[:a + first]).all())
        assert (window, sinks) == (None, 0)
        assert mb.poll_errors() == (0, 0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_far_pages_and_rows(dtype, D):
    """A pool whose far pages lie past 2^31 elements, and packed rows past that, too."""
    dev = gpu_ready()
    Hkv, P = 2, 128
    num = (2 ** 31 + 2 ** 26) // (Hkv * P * D)
    c = Case([1, 140], [300, 200], 4, Hkv, D, dtype, dev, seed=4)
    Kp, Vp = (torch.empty((num, Hkv, P, D), dtype=dtype, device=dev) for _ in range(2))
    for b, row in enumerate(c.table):
        for i, page in enumerate(row):
            if 0 <= page < c.num:
                far = num - 1 - 3 * b - i
                Kp[far], Vp[far] = c.Kp[page], c.Vp[page]
                c.table[b][i] = far
    c.Kp, c.Vp, c.num, c.table_d = Kp, Vp, num, i32(c.table, dev)
    stride = 1 << 24
    T = c.T
    q = torch.empty(T * stride, dtype=dtype, device=dev).view(T, stride)[:, :4 * D].unflatten(1, (4, D))
    q.copy_(c.q)
    c.q = q
    c.check(c.call())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_streams_graphs_and_workspaces(dtype, D):
    """Two calls at once with a workspace each; a captured call replayed on changed rows, lengths, starts and tables; two
    graphs that share a workspace, one after the other; equal bits every time."""
    dev = gpu_ready()
    cases = [Case([1, 200, 1, 0, 33], [3000, 500, 0, 9, 4000], 8, 2, D, dtype, dev, seed=s, extra_cap=2) for s in (1, 2)]
    want = [c.call() for c in cases]
    for c, w in zip(cases, want):
        c.check(w)
    outs, spaces = [torch.full_like(w, 7.0) for w in want], [c.workspace() for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, o, w, st in zip(cases, outs, spaces, streams):
            c.call(o, w, st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    graphs, shared = [], spaces[0]
    for c, o in zip(cases, outs):
        o.fill_(7.0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(o, shared)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    c, other = cases
    T = c.T
    c.q.copy_(other.q)
    new_rows = [100, 1, 130, 2, 1]
    new = Case(new_rows, [900, 4000, 300, 0, 2000], 8, 2, D, dtype, dev, seed=11, extra_cap=0)
    assert new.T <= T
    c.cu_d.copy_(new.cu_d), c.start_d.copy_(new.start_d)
    c.cu, c.start = new.cu, new.start
    Kp, Vp, num = new.Kp, new.Vp, new.num
    table = [[(x if 0 <= x < num else -1) % c.num if 0 <= x < num else -1 for x in row] + [-1] * 99 for row in new.table]
    c.table = [row[:c.L_cap // 128] for row in table]
    c.table_d.copy_(i32(c.table, dev))
    c.Kp.zero_(), c.Vp.zero_()
    m = min(c.num, num)
    c.Kp[:m], c.Vp[:m] = torch.nan_to_num(Kp[:m]), torch.nan_to_num(Vp[:m])
    outs[0].fill_(7.0)
    for _ in range(3):
        graphs[0].replay()
    torch.cuda.synchronize()
    c.check(outs[0], "replayed on other rows")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
def test_same_inputs_same_bits(dtype, D):
    dev = gpu_ready()
    c = Case([1, 300, 1, 1], [5000, 200, 17, 1000], 8, 2, D, dtype, dev, seed=2)
    first = c.call()
    for _ in range(4):
        assert torch.equal(c.call(), first)


# ----------------------------------------------------------------------------- the oracle (no GPU)
def test_oracle_is_masked_attention():
    """Chunks of one sequence against torch's attention in float64 over the whole of it, with and without a window."""
    gen = torch.Generator().manual_seed(3)
    n, P, Hq, Hkv, D = 300, 128, 4, 2, 64
    q, k, v = (torch.randn((n, h, D), generator=gen) for h in (Hq, Hkv, Hkv))
    pool = [torch.zeros((4, Hkv, P, D)) for _ in range(2)]
    table = [[2, 0, 3]]
    for i in range(3):
        for p, x in zip(pool, (k, v)):
            p[table[0][i], :, :min(P, n - i * P)] = x[i * P:(i + 1) * P].transpose(0, 1)
    t = lambda x, g: x.double().transpose(0, 1).repeat_interleave(g, 0)
    i = torch.arange(n)
    for window, sinks in ((None, 0), (50, 3), (1, 0), (200, 140)):
        see = i[None] <= i[:, None]
        if window:
            see &= (i[None] > i[:, None] - window) | (i[None] < sinks)
        want = torch.nn.functional.scaled_dot_product_attention(t(q, 1), t(k, 2), t(v, 2), attn_mask=see).transpose(0, 1)
        for a, e in ((0, 1), (0, 300), (127, 130), (299, 300)):
            O, A, S, owned = SO.chunk_attention(q[a:e], *pool, P, table, [0, e - a], [a], 384, window, sinks)
            assert (O - want[a:e]).abs().max() < 1e-12 and bool(owned.all())
    O, _, _, owned = SO.chunk_attention(q[:9], *pool, P, table * 3, [0, 3, 6, 9], [-1, 382, 381], 384)
    assert owned.tolist() == [False] * 6 + [True] * 3


# ----------------------------------------------------------------------------- refusals (no GPU)
def status(window_call=False, T=8, q_stride=None, q=4096, kp=4096, vp=4096, cu=4, start=0, table=4, o=4096, ws=4096, num=9, P=128,
           window=5, sinks=0, dtype=BF16, D=128, Hq=4, Hkv=2, cap=1024):
    _build.build()
    cfg = cfg_for(2, 4, 2, D, dtype, cap)
    cfg.Hq, cfg.Hkv = Hq, Hkv
    ptr = lambda x: ctypes.c_void_p(x) if x else None
    head = (ctypes.byref(cfg), ptr(q), T, Hq * D if q_stride is None else q_stride, ptr(cu), ptr(start), ptr(kp), ptr(vp), num, P,
            ptr(table))
    if window_call:
        return mb.load().medusa_window_attention_paged(*head, window, sinks, ptr(o), ptr(ws), None)
    return mb.load().medusa_chunk_attention_paged(*head, ptr(o), ptr(ws), None)


@pytest.mark.parametrize("window_call", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), -1), (dict(q=0), -1), (dict(kp=0), -1), (dict(vp=0), -1), (dict(cu=0), -1), (dict(table=0), -1), (dict(o=0), -1),
    (dict(q=4104), -1), (dict(kp=4098), -1), (dict(vp=4104), -1), (dict(o=4104), -1), (dict(ws=4112), -1), (dict(ws=0), -1),
    (dict(q_stride=511), -1), (dict(q_stride=516), -1), (dict(q_stride=-512), -1), (dict(dtype=F32, q_stride=514), -1),
    (dict(num=0), -1), (dict(P=64), -2), (dict(P=192), -2), (dict(P=384), -2), (dict(cap=1000), -2), (dict(P=0), -2),
    (dict(num=2 ** 30), -2), (dict(T=2 ** 30, cap=2 ** 20), -2), (dict(D=96), -2), (dict(Hkv=3), -2),
    (dict(T=0, q=0, kp=0, vp=0, cu=0, table=0, o=0, ws=0), 0),
])
def test_refusals(kw, want, window_call):
    assert status(window_call, **kw) == want


@pytest.mark.parametrize("kw", [dict(window=0), dict(window=-3), dict(window=-2 ** 31), dict(sinks=-1)])
def test_window_refusals(kw):
    assert status(True, **kw) == -1


def test_workspace_refusals():
    _build.build()
    cfg = cfg_for(2, 4, 2, 128, BF16)
    n = ctypes.c_size_t()
    f = mb.load().medusa_chunk_workspace_size
    assert f(ctypes.byref(cfg), 0, ctypes.byref(n)) == 0 and n.value == 0
    assert f(ctypes.byref(cfg), -1, ctypes.byref(n)) == -1 and f(ctypes.byref(cfg), 1, None) == -1
    cfg.D = 80
    assert f(ctypes.byref(cfg), 1, ctypes.byref(n)) == -2
    assert f(None, 1, ctypes.byref(n)) == -1
