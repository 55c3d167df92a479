"""Attention of new tokens with a window where several edges meet: many sequences, skipped ones, pages outside the
pool, infinite scores; and the two float32 kernels on the same prompts."""
import pytest
import torch

from medusa_speculative_decoding_heads_gb300 import binding as mb
from oracle import serving_oracle as SO

from _helpers import gpu_ready
from _serving import assert_within, i32, tolerance
from test_chunk_attention import BF16, F32, KINDS, Case, patterns

WINDOWS = [(1, 0), (100, 4), (130, 0), (300, 200)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,Hq,Hkv", [(BF16, 128, 3, 3), (BF16, 64, 4, 1), (F32, 64, 4, 2), (F32, 128, 3, 1)])
@pytest.mark.parametrize("B", [31, 32, 33, 65, 333])
def test_windows_of_many_sequences(B, dtype, D, Hq, Hkv):
    """More sequences than a warp has lanes: the schedule reads their bounds again for each group of 32."""
    dev = gpu_ready()
    for x, (name, rows, start) in enumerate(patterns(B)):
        window, sinks = WINDOWS[x % len(WINDOWS)]
        c = Case(rows, start, Hq, Hkv, D, dtype, dev, seed=B, pad=3, first=2, window=window, sinks=sinks)
        c.check(c.call(), f"{name}, window {window}, sinks {sinks}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("B,at", [(5, 2), (33, 0), (70, 31), (70, 32), (200, 150)])
def test_windows_ahead_of_a_decrease(B, at, dtype, D):
    dev = gpu_ready()
    for window, sinks in WINDOWS[:2]:
        c = Case([1 + 40 * (b % 3) for b in range(B)], [(37 * b) % 300 for b in range(B)], 4, 2, D, dtype, dev, seed=B, pad=2,
                 window=window, sinks=sinks)
        cu = list(c.cu)
        cu[at + 1] = cu[at] - 1
        c.cu_d, c.cu = i32(cu, dev), cu
        c.check(c.call(), f"{at} of {B}, window {window}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
def test_windows_of_sequences_that_are_skipped(dtype, D):
    dev = gpu_ready()
    for window, sinks in WINDOWS:
        c = Case([40, 1, 130, 7], [100, 300, 0, 249], 4, 2, D, dtype, dev, seed=3, pad=20, window=window, sinks=sinks)
        own = list(c.start)
        for b, s in ((0, -1), (1, -2 ** 31), (2, 2 ** 31 - 1), (3, c.L_cap - 6)):
            c.start = [s if i == b else x for i, x in enumerate(own)]
            c.start_d = i32(c.start, dev)
            c.check(c.call(), f"start {s}, window {window}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("page", [-1, "num", 2 ** 31 - 1])
def test_window_pages_outside_the_pool_are_zeros(page, dtype, D):
    """In the window, among the first rows, and both."""
    dev = gpu_ready()
    for rows, start, where in (([1, 1], [700, 300], ((0, 5), (1, 0))), ([140, 1], [300, 500], ((0, 2), (1, 0), (1, 3)))):
        c = Case(rows, start, 4, 2, D, dtype, dev, seed=5, window=150, sinks=5)
        for b, i in where:
            assert 0 <= c.table[b][i] < c.num   # (a page that is looked up)
            c.table[b][i] = c.num if page == "num" else page
        c.table_d = i32(c.table, dev)
        c.check(c.call(), f"page {page}")
        assert mb.poll_checks() == ((-6, mb.CHECK_PAGE) if mb.checked_build() else (0, 0))


# Keys that score -inf: all of what a window leaves, but the first rows; the first rows; what only earlier rows see.
DEAD = {"all but the first rows": (4, 150), "from the first row on": (0, 150), "far behind": (30, 60), "a long run": (4, 1400),
        "none": (0, 0)}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("window,sinks", [(100, 0), (100, 4), (17, 1), (260, 140), (2 ** 31 - 1, 0)])
@pytest.mark.parametrize("dead", list(DEAD), ids=list(DEAD))
def test_infinite_scores_in_windows(dead, window, sinks, dtype, D):
    """Such keys weigh nothing; a row that sees only such is no number, whatever the rows beside it see."""
    dev = gpu_ready()
    low, high = DEAD[dead]
    for rows, start in (([1, 1, 1, 1], [200, 149, 1500, 3]), ([20, 140, 1], [140, 0, 1399]), ([300], [100])):
        c = Case(rows, start, 4, 2, D, dtype, dev, seed=9, window=window, sinks=sinks)
        c.q[..., 0] = c.q[..., 0].abs() + 0.5
        clean = c.Kp.clone()
        for row in c.table:
            for i, page in enumerate(row):
                a, e = max(0, low - 128 * i), min(128, high - 128 * i)
                if 0 <= page < c.num and a < e:   # (rows that nobody sees hold NaN before and need not after)
                    c.Kp[page, :, a:e, 0] = float("-inf")
        O = c.call()
        for b, (a, e) in enumerate(zip(c.cu[:-1], c.cu[1:])):
            s, n = c.start[b], e - a
            p, j = torch.arange(s, s + n, device=dev)[:, None], torch.arange(s + n, device=dev)
            see = (j <= p) & ((j > p - window) | (j < sinks)) & ((j < low) | (j >= high))
            some = see.any(1)
            assert bool(O[a:e][~some].isnan().all()), "rows without a finite score"
            if not bool(some.any()):
                continue
            held = see.any(0).nonzero().flatten()
            pages = torch.tensor([c.table[b][int(x) // 128] for x in held], device=dev)
            k, v = (pool[pages, :, held % 128] for pool in (clean, c.Vp))
            ref, A, S = SO.attend(c.q[a:e], k, v, see[:, held])
            tol = tolerance(dtype, ref, A, S, c.L_cap)
            assert_within(O[a:e][some], ref[some], tol[some], f"{dead}, window {window}, sinks {sinks}, rows {rows}")
        assert mb.poll_errors() == (0, 0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_float32_prompts_and_chunks_agree(D):
    """Whole prompts and chunks have float32 kernels of their own: on the same rows each keeps to the same bound."""
    dev = gpu_ready()
    rows = [333, 2, 65, 1, 700]
    c = Case(rows, [0] * len(rows), 6, 3, D, F32, dev, seed=4)
    K, V = (torch.empty((c.T, c.Hkv, D), device=dev) for _ in range(2))
    for b, (a, e) in enumerate(zip(c.cu[:-1], c.cu[1:])):
        for i in range(0, e - a, 128):
            n = min(128, e - a - i)
            for x, pool in ((K, c.Kp), (V, c.Vp)):
                x[a + i:a + i + n] = pool[c.table[b][i // 128], :, :n].transpose(0, 1)
    O, P = c.call(), torch.full((c.T, c.Hq, D), 7.0, device=dev)
    mb.prompt_attention(c.cfg, c.q, K, V, c.T, c.q.stride(0), K.stride(0), V.stride(0), c.cu_d, P)
    ref, A, S = SO.prompt_attention(c.q, K, V, c.cu)
    tol = tolerance(F32, ref, A, S, max(rows))
    assert_within(O, ref, tol, "chunks")
    assert_within(P, ref, tol, "prompts")
