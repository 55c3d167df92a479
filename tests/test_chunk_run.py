"""Requests on their way: prompts taken in chunks beside single tokens, each step's queries and keys normed and turned,
keys and values stored in their pages, attention taken over the cache; then a tree verified behind them."""
import os
import subprocess
import sys

import pytest
import torch

from medusa_speculative_decoding_heads_gb300 import binding as mb
from oracle import medusa_oracle as MO, serving_oracle as SO

from _helpers import gpu_ready
from _serving import ancestor_bits, assert_within, cfg_for, i32, offsets, tolerance
from test_rotate import check as check_rotated, freqs

BF16, F32 = torch.bfloat16, torch.float32
HERE = os.path.dirname(os.path.abspath(__file__))
# rows of each of four sequences in each step: a prompt in chunks, a short prompt and its tokens, one that comes later
STEPS = [[200, 65, 0, 1], [200, 1, 0, 1], [137, 1, 300, 1], [1, 1, 129, 1], [1, 0, 1, 1], [1, 1, 1, 1]]


class Requests:
    def __init__(self, dev, dtype, D, window=None, sinks=0, Hq=8, Hkv=2, P=128, width=6, seed=0, branching=(3, 2, 2)):
        self.dev, self.dtype, self.D, self.Hq, self.Hkv, self.P, self.window, self.sinks = dev, dtype, D, Hq, Hkv, P, window, sinks
        self.B, self.num = 4, 4 * width + 2
        self.gen = torch.Generator(device=dev).manual_seed(seed)
        self.mask, self.bits = ancestor_bits(branching, dev)
        self.N, self.tree = self.mask.shape[0], MO.tree_layout(branching)
        self.branching = branching
        self.cfg = cfg_for(self.B, Hq, Hkv, D, dtype, width * P, branching)
        self.Kp, self.Vp = (torch.full((self.num, Hkv, P, D), float("nan"), dtype=dtype, device=dev) for _ in range(2))
        self.table, self.refs, self.L = i32([[-1] * width] * self.B, dev), i32([0] * self.num, dev), [0] * self.B
        self.ws = torch.empty(mb.pages_workspace_size(self.cfg, self.num), dtype=torch.uint8, device=dev)
        self.flags = torch.zeros(self.B, dtype=torch.int32, device=dev)
        self.qw, self.kw = (1 + torch.randn(D, generator=self.gen, device=dev).to(dtype) / 4 for _ in range(2))
        self.f = freqs(D, dev)
        self.rows = [([], []) for _ in range(self.B)]   # what each sequence's cache must hold

    def projection(self, T):
        return torch.randn((T, self.Hq + 2 * self.Hkv, self.D), generator=self.gen, device=self.dev).to(self.dtype)

    def step(self, rows):
        cu, start = offsets(rows), i32(self.L, self.dev)
        T = cu[-1]
        mb.pages_reserve(self.cfg, self.num, self.P, i32([s + n for s, n in zip(self.L, rows)], self.dev), self.table, self.refs,
                         self.flags, self.ws)
        assert self.flags.tolist() == [0] * self.B
        x = self.projection(T)
        raw = x.clone()
        q, k, v = x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]
        s = x.stride(0)
        pos = i32([a + i for a, n in zip(self.L, rows) for i in range(n)], self.dev)
        mb.qk_norm_rotate(self.cfg, q, k, T, s, s, self.qw, self.kw, 1e-6, self.f, self.D, mb.ROTATE_HALVES, pos, q, k, s, s)
        check_rotated(raw[:, :self.Hq], raw[:, self.Hq:self.Hq + self.Hkv], self.qw, self.kw, 1e-6, self.f, self.D, False, pos, q, k)
        cu_d = i32(cu, self.dev)
        mb.kv_store_paged(self.cfg, k, v, T, s, s, cu_d, start, self.Kp, self.Vp, self.num, self.P, self.table)
        O = torch.full((T, self.Hq, self.D), 7.0, dtype=self.dtype, device=self.dev)
        ws = torch.empty(max(1, mb.chunk_workspace_size(self.cfg, T)), dtype=torch.uint8, device=self.dev)
        head = (self.cfg, q, T, s, cu_d, start, self.Kp, self.Vp, self.num, self.P, self.table)
        if self.window is None:
            mb.chunk_attention_paged(*head, O, ws)
        else:
            mb.window_attention_paged(*head, self.window, self.sinks, O, ws)
        for b, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
            self.rows[b][0].append(k[a:e])
            self.rows[b][1].append(v[a:e])
            self.L[b] += e - a
            if e == a:
                continue
            K, V = torch.cat(self.rows[b][0]), torch.cat(self.rows[b][1])
            j = torch.arange(self.L[b], device=self.dev)[None]
            p = torch.arange(self.L[b] - (e - a), self.L[b], device=self.dev)[:, None]
            see = j <= p
            if self.window is not None:
                see = see & ((j > p - self.window) | (j < self.sinks))
            ref, A, S = SO.attend(q[a:e], K, V, see)
            assert_within(O[a:e], ref, tolerance(self.dtype, ref, A, S, self.L[b]), f"sequence {b}, {self.L[b]} rows")

    def verify(self):
        """The trees' queries and keys at the positions that the tree build gives, then tree attention over the pages."""
        N, B = self.N, self.B
        out = lambda *s, t=torch.int32: torch.empty(s, dtype=t, device=self.dev)
        pos = out(B, N)
        topk = torch.zeros((B, len(self.branching), max(self.branching)), dtype=torch.int32, device=self.dev)
        L = i32(self.L, self.dev)
        mb.tree_build(self.cfg, i32([0] * B, self.dev), topk, L, out(N), out(N), out(N), out(N, N, t=torch.uint8), out(N, 2, t=torch.int64),
                      out(B, N), pos, None)
        assert pos.tolist() == [[n + int(d) for d in self.tree["depth"]] for n in self.L]
        x = self.projection(B * N)
        q, k, v = x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]
        Q = out(B, N, self.Hq, self.D, t=self.dtype)
        Kt = out(B, self.Hkv, N, self.D, t=self.dtype)
        s = x.stride(0)
        mb.qk_norm_rotate(self.cfg, q, k, B * N, s, s, self.qw, self.kw, 1e-6, self.f, self.D, mb.ROTATE_HALVES, pos, Q, Kt,
                          self.Hq * self.D, 0)
        check_rotated(q, k, self.qw, self.kw, 1e-6, self.f, self.D, False, pos.flatten(), Q.view(B * N, self.Hq, self.D),
                      Kt.transpose(1, 2).reshape(B * N, self.Hkv, self.D), "tree")
        Vt = v.reshape(B, N, self.Hkv, self.D).transpose(1, 2).contiguous()
        O = torch.empty_like(Q)
        ws = torch.empty(max(1, mb.prefix_workspace_size(self.cfg, 0)), dtype=torch.uint8, device=self.dev)
        mb.tree_attention_prefix(self.cfg, Q, self.Kp, self.Vp, self.num, self.P, None, 0, self.table, Kt, Vt, L, self.bits, O, ws)
        for b in range(B):
            K = torch.cat(self.rows[b][0] + [Kt[b].transpose(0, 1)])
            V = torch.cat(self.rows[b][1] + [Vt[b].transpose(0, 1)])
            see = torch.cat([torch.ones((N, self.L[b]), dtype=torch.bool), self.mask], 1).to(self.dev)
            ref, A, S = SO.attend(Q[b], K, V, see)
            assert_within(O[b], ref, tolerance(self.dtype, ref, A, S, K.shape[0]), f"tree of sequence {b}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (150, 4), (64, 0)])
def test_chunks_beside_single_tokens(window, sinks, dtype, D):
    dev = gpu_ready()
    r = Requests(dev, dtype, D, window, sinks, seed=D)
    for rows in STEPS:
        r.step(rows)
    if window is None and dtype == BF16 and D == 128:
        r.verify()
    assert mb.poll_errors() == (0, 0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(None, 0), (200, 4)])
def test_pieces_of_a_prompt_give_the_prompt(window, sinks):
    """The rows of a prompt are the same however it is cut: a whole one, chunks, single tokens (each within the
    bounds of its own rounding, so two of them within twice that)."""
    dev = gpu_ready()
    n, P, Hq, Hkv, D = 390, 128, 4, 2, 128
    gen = torch.Generator(device=dev).manual_seed(1)
    q, k, v = (torch.randn((n, h, D), generator=gen, device=dev).to(BF16) for h in (Hq, Hkv, Hkv))
    cfg = cfg_for(1, Hq, Hkv, D, BF16, 512)
    Kp, Vp = (torch.zeros((4, Hkv, P, D), dtype=BF16, device=dev) for _ in range(2))
    table = i32([[2, 0, 3, 1]], dev)
    mb.kv_store_paged(cfg, k, v, n, Hkv * D, Hkv * D, i32([0, n], dev), None, Kp, Vp, 4, P, table)
    ws = torch.empty(mb.chunk_workspace_size(cfg, n), dtype=torch.uint8, device=dev)
    ref, A, S, _ = SO.chunk_attention(q, Kp, Vp, P, table.tolist(), [0, n], [0], 512, window, sinks)
    tol = tolerance(BF16, ref, A, S, n)
    for size in (n, 133, 64, 1):
        O = torch.empty((n, Hq, D), dtype=BF16, device=dev)
        for a in range(0, n, size):
            m = min(size, n - a)
            head = (cfg, q[a:a + m], m, Hq * D, i32([0, m], dev), i32([a], dev), Kp, Vp, 4, P, table)
            if window is None:
                mb.chunk_attention_paged(*head, O[a:a + m], ws)
            else:
                mb.window_attention_paged(*head, window, sinks, O[a:a + m], ws)
        assert_within(O, ref, tol, f"chunks of {size}")


@pytest.mark.gpu
def test_checked_build_runs_them():
    """The range-checked library gives the same results, and reports a page outside the pool."""
    gpu_ready()
    env = dict(os.environ, MEDUSA_CHECKED="1")
    files = [os.path.join(HERE, f) for f in ("test_chunk_run.py", "test_chunk_attention.py", "test_rotate.py")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "-k",
                        "beside or lengths or outside or long_caches or rotated_dims", *files], env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
