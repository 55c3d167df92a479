"""A prompt's way through the cache: its pages reserved, its keys and values stored, its attention taken,
the sequence forked, the forks' trees attended behind the shared prompt, their accepted paths committed,
some of them freed, the pages compacted, and the next trees attended on what is left."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from medusa_speculative_decoding_heads_gb300 import binding as mb
from oracle import medusa_oracle as O, serving_oracle as SO

from _helpers import gpu_ready
from _serving import ancestor_bits, assert_within, cfg_for, i32, offsets, tolerance

BF16 = torch.bfloat16
HERE = os.path.dirname(os.path.abspath(__file__))


class Run:
    """Two layers' pools and the tables of a batch, with the rows each sequence must hold kept aside."""

    def __init__(self, dev, B=6, Hq=8, Hkv=2, P=128, width=8, num=40, branching=(3, 2, 2), layers=2, seed=0):
        self.dev, self.B, self.Hq, self.Hkv, self.P, self.num, self.layers, self.K = dev, B, Hq, Hkv, P, num, layers, len(branching)
        self.gen = torch.Generator(device=dev).manual_seed(seed)
        self.mask, self.bits = ancestor_bits(branching, dev)
        self.N, self.tree = self.mask.shape[0], O.tree_layout(branching)
        self.cfg = cfg_for(B, Hq, Hkv, 128, BF16, width * P, branching)
        self.Kp, self.Vp = (torch.full((layers, num, Hkv, P, 128), float("nan"), dtype=BF16, device=dev) for _ in range(2))
        self.table, self.refs, self.L = i32([[-1] * width] * B, dev), i32([0] * num, dev), i32([0] * B, dev)
        self.ws = torch.empty(mb.pages_workspace_size(self.cfg, num), dtype=torch.uint8, device=dev)
        self.rows = [[[] for _ in range(layers)] for _ in range(B)]   # (k, v) pieces [n][Hkv][128] per layer
        self.flags = torch.zeros(B, dtype=torch.int32, device=dev)

    def rnd(self, *shape):
        return torch.randn(shape, generator=self.gen, device=self.dev).to(BF16)

    def reserve(self, rows):
        mb.pages_reserve(self.cfg, self.num, self.P, i32(rows, self.dev), self.table, self.refs, self.flags, self.ws)
        assert self.flags.tolist() == [0] * self.B

    def prefill(self, lens):
        """Prompts of every layer: attention on the packed rows, keys and values into the pages."""
        self.reserve([n + self.N if n else 0 for n in lens])
        cu = offsets(lens)
        for layer in range(self.layers):
            qkv = self.rnd(cu[-1], self.Hq + 2 * self.Hkv, 128)   # one projection's output
            q, k, v = qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.Hkv], qkv[:, self.Hq + self.Hkv:]
            out = torch.empty((cu[-1], self.Hq, 128), dtype=BF16, device=self.dev)
            s = qkv.stride(0)
            mb.prompt_attention(self.cfg, q, k, v, cu[-1], s, s, s, i32(cu, self.dev), out)
            mb.kv_store_paged(self.cfg, k, v, cu[-1], s, s, i32(cu, self.dev), None, self.Kp[layer], self.Vp[layer], self.num,
                              self.P, self.table)
            ref, A, S = SO.prompt_attention(q, k, v, cu)
            assert_within(out, ref, tolerance(BF16, ref, A, S, max(lens)), f"prompt attention, layer {layer}")
            for b, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
                self.rows[b][layer].append((k[a:e], v[a:e]))
        self.L.copy_(i32(lens, self.dev))

    def fork(self, src, dst):
        mb.pages_fork(self.cfg, self.Kp, self.Vp, self.num, self.P, self.layers, self.Kp.stride(0), len(src), i32(src, self.dev),
                      i32(dst, self.dev), self.table, self.L, self.refs, self.flags, self.ws)
        assert self.flags.tolist()[:len(src)] == [0] * len(src)
        for s, d in zip(src, dst):
            self.rows[d] = [list(pieces) for pieces in self.rows[s]]

    def logical(self, b, layer):
        k, v = zip(*self.rows[b][layer])
        return torch.cat(k), torch.cat(v)

    def attend(self, staged, shared):
        """Every layer's tree attention behind `shared` rows, against the rows kept aside; returns the outputs."""
        ws = torch.empty(mb.prefix_workspace_size(self.cfg, shared), dtype=torch.uint8, device=self.dev)
        L, outs = self.L.tolist(), []
        live = [b for b in range(self.B) if L[b] > 0]
        prefix = self.table[live[0], :-(-shared // self.P)].contiguous() if shared else None
        for layer, (Q, Kt, Vt) in enumerate(staged):
            out = torch.empty_like(Q)
            mb.tree_attention_prefix(self.cfg, Q, self.Kp[layer], self.Vp[layer], self.num, self.P, prefix, shared, self.table,
                                     Kt, Vt, self.L, self.bits, out, ws)
            for b in live:
                k, v = self.logical(b, layer)
                assert k.shape[0] == L[b]
                k, v = torch.cat([k, Kt[b].transpose(0, 1)]), torch.cat([v, Vt[b].transpose(0, 1)])
                see = torch.cat([torch.ones((self.N, L[b]), dtype=torch.bool), self.mask], 1).to(self.dev)
                ref, A, S = SO.attend(Q[b], k, v, see)
                assert_within(out[b], ref, tolerance(BF16, ref, A, S, k.shape[0]), f"layer {layer}, sequence {b}")
            outs.append(out)
        return outs

    def commit(self, staged, rng):
        """A random accepted path per sequence, in every layer."""
        acc = [int(rng.integers(0, self.K + 1)) for _ in range(self.B)]
        path = np.full((self.B, self.K + 1), -1, dtype=np.int32)
        for b in range(self.B):
            cur = path[b, 0] = 0
            for r in range(1, acc[b] + 1):
                kids = O.children_of(self.tree["parent"], cur)
                cur = path[b, r] = kids[int(rng.integers(len(kids)))]
        Kt, Vt = (torch.stack([s[i] for s in staged]) for i in (1, 2))
        held = self.L.clone()
        mb.kv_commit_paged(self.cfg, self.Kp, self.Vp, self.P, self.table, Kt, Vt, self.layers, self.Kp.stride(0), Kt.stride(0),
                           self.L, i32(acc, self.dev), torch.from_numpy(path).to(self.dev),
                           torch.empty((self.B, self.K + 1), dtype=torch.int32, device=self.dev))
        for b, n in enumerate(held.tolist()):
            if n == 0:   # an empty sequence stays empty (its rows went to no page)
                continue
            nodes = path[b, :acc[b] + 1].tolist()
            for layer, (_, kt, vt) in enumerate(staged):
                self.rows[b][layer].append((kt[b][:, nodes].transpose(0, 1), vt[b][:, nodes].transpose(0, 1)))
        self.L[held == 0] = 0


@pytest.mark.gpu
@pytest.mark.parametrize("prompt,branching", [(400, (3, 2, 2)), (256, (4, 3, 2, 1)), (129, (2, 2))])
def test_prompt_fork_verify_free_compact(prompt, branching):
    dev = gpu_ready()
    r = Run(dev, branching=branching, seed=prompt)
    rng = np.random.default_rng(prompt)
    r.prefill([prompt, 0, 70, 0, 0, 0])
    r.fork([0, 0, 0], [1, 3, 4])
    r.reserve([n + r.N if n else 0 for n in r.L.tolist()])
    shared = prompt // 128 * 128
    stage = lambda: [(r.rnd(r.B, r.N, r.Hq, 128), r.rnd(r.B, r.Hkv, r.N, 128), r.rnd(r.B, r.Hkv, r.N, 128)) for _ in range(r.layers)]
    staged = stage()
    # sequence 2 has another prompt: it attends on its own, the others behind the shared one
    alone = r.L.clone()
    alone[2], kept = 0, r.L
    r.L, rows2 = alone, r.rows[2]
    r.attend(staged, shared)
    r.L = kept
    r.attend(staged, 0)
    r.commit(staged, rng)
    mb.pages_free(r.cfg, r.num, r.P, 2, i32([2, 1], dev), r.table, r.L, r.refs)
    r.rows[1], r.rows[2] = [[], []], [[], []]
    staged = stage()
    before = r.attend(staged, shared)
    page_map, n_live = i32([0] * r.num, dev), i32([0], dev)
    mb.pages_compact(r.cfg, r.Kp, r.Vp, r.num, r.P, r.layers, r.Kp.stride(0), r.table, r.refs, page_map, n_live, r.ws)
    live = n_live.item()
    table = r.table.cpu()
    assert int(table.max()) == live - 1 and int((r.refs > 0).sum()) == live and bool((r.refs[:live] > 0).all())
    for old, new in zip(before, r.attend(staged, shared)):   # the same rows, from other pages
        for b in (0, 3, 4):
            assert torch.equal(old[b], new[b])
    assert mb.poll_errors() == (0, 0, 0)


@pytest.mark.gpu
def test_checked_build_runs_them():
    """The range-checked library gives the same results, and reports a page outside the pool."""
    gpu_ready()
    env = dict(os.environ, MEDUSA_CHECKED="1")
    files = [os.path.join(HERE, f) for f in ("test_serving_run.py", "test_prefix_attention.py", "test_pages.py")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "-k",
                        "free_compact or lengths or invalid or few_rows or checked_pages or store", *files],
                       env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]


@pytest.mark.gpu
def test_checked_pages():
    """In the checked build a page id outside the pool is reported by each call that meets one; in the
    normal build nothing is, and in both it reads and writes nothing outside the pool."""
    dev = gpu_ready()
    r = Run(dev, seed=5)
    r.prefill([300, 140, 0, 0, 0, 0])
    mb.poll_checks()
    want = (-6, mb.CHECK_PAGE) if mb.checked_build() else (0, 0)
    r.table[1, 1] = r.num + 3
    q, kt, vt = r.rnd(r.B, r.N, r.Hq, 128), r.rnd(r.B, r.Hkv, r.N, 128), r.rnd(r.B, r.Hkv, r.N, 128)
    ws = torch.empty(mb.prefix_workspace_size(r.cfg, 0), dtype=torch.uint8, device=dev)
    mb.tree_attention_prefix(r.cfg, q, r.Kp[0], r.Vp[0], r.num, r.P, None, 0, r.table, kt, vt, r.L, r.bits, torch.empty_like(q), ws)
    assert mb.poll_checks() == want
    k = r.rnd(200, r.Hkv, 128)
    mb.kv_store_paged(r.cfg, k, k, 200, 256, 256, i32([0, 0, 200, 200, 200, 200, 200], dev), None, r.Kp[0], r.Vp[0], r.num, r.P, r.table)
    assert mb.poll_checks() == want
    mb.pages_free(r.cfg, r.num, r.P, 1, i32([1], dev), r.table, r.L, r.refs)
    assert mb.poll_checks() == want
