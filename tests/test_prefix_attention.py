"""medusa_tree_attention_prefix: tree attention of a batch behind one shared prefix, against float64."""
import ctypes

import numpy as np
import pytest
import torch

from medusa_speculative_decoding_heads_gb300 import _build, binding as mb, configs
from oracle import medusa_oracle as O, serving_oracle as SO

from _helpers import gpu_ready
from _serving import ancestor_bits, assert_within, cfg_for, i32, tolerance

BF16 = torch.bfloat16


class Case:
    """A shuffled pool: `shared` rows in pages of their own, each sequence's rows behind them in its own pages."""

    def __init__(self, L, shared, P, Hq, Hkv, branching, dev, seed=0, poison=False, L_cap=None):
        gen = torch.Generator(device=dev).manual_seed(seed)
        cpu = torch.Generator().manual_seed(seed)
        self.mask, self.bits = ancestor_bits(branching, dev)
        self.N, self.B, self.P, self.shared, self.dev = self.mask.shape[0], len(L), P, shared, dev
        most = max([shared] + list(L)) + self.N
        self.L_cap = L_cap or -(-most // P) * P
        width = self.L_cap // P
        first = -(-shared // P)
        num = first + self.B * width + 2
        ids = torch.randperm(num, generator=cpu).tolist()
        self.num, self.prefix, at = num, ids[:first], first
        self.table = []
        for n in L:
            row = [-1] * width
            for i in range(shared // P, -(-min(max(n, 0), self.L_cap) // P)):
                row[i], at = ids[at], at + 1
            self.table.append(row)
        rnd = lambda *s: torch.randn(s, generator=gen, device=dev).to(BF16)
        self.Q = rnd(self.B, self.N, Hq, 128) * 2
        self.Kp, self.Vp = rnd(num, Hkv, P, 128), rnd(num, Hkv, P, 128)
        self.Kt, self.Vt = rnd(self.B, Hkv, self.N, 128), rnd(self.B, Hkv, self.N, 128)
        if poison:   # whatever no sequence may read: pages in nobody's hands, rows past each length
            used = torch.zeros((num, P), dtype=torch.bool, device=dev)
            for i in range(shared):
                used[self.prefix[i // P], i % P] = True
            for b, n in enumerate(L):
                for i in range(shared, max(n, 0)):
                    if n + self.N <= self.L_cap:
                        used[self.table[b][i // P], i % P] = True
            bad = ~used
            self.Kp.transpose(1, 2)[bad] = float("nan")
            self.Vp.transpose(1, 2)[bad] = float("nan")
        self.L, self.Hq, self.Hkv, self.branching = list(L), Hq, Hkv, branching
        self.cfg = cfg_for(self.B, Hq, Hkv, 128, BF16, self.L_cap, branching)
        self.ws = None if dev == "cpu" else torch.full((max(mb.prefix_workspace_size(self.cfg, shared), 256),), 255,
                                                       dtype=torch.uint8, device=dev)

    def call(self, O=None, stream=None, shared=None):
        O = torch.full_like(self.Q, 7.0) if O is None else O
        if not hasattr(self, "dtable"):
            self.dtable, self.dprefix, self.dL = i32(self.table, self.dev), i32(self.prefix, self.dev), i32(self.L, self.dev)
        mb.tree_attention_prefix(self.cfg, self.Q, self.Kp, self.Vp, self.num, self.P,
                                 self.dprefix if self.prefix else None, self.shared, self.dtable, self.Kt, self.Vt, self.dL,
                                 self.bits, O, self.ws, stream)
        return O

    def check(self, O, what="prefix attention", rows=slice(None)):
        ref, A, S = SO.prefix_attention(self.Q, self.Kp, self.Vp, self.P, self.prefix, self.shared, self.table, self.Kt,
                                        self.Vt, self.L, self.mask, self.L_cap)
        tol = tolerance(BF16, ref, A, S, max(max(self.L), 1) + self.N)
        assert_within(O[rows], ref[rows], tol[rows], what)
        assert mb.poll_errors() == (0, 0, 0)


TREES = [(1,), (2, 2), (3, 2, 2), (4, 3, 2, 1), (5, 3, 2, 1, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("branching", TREES, ids=str)
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 2), (6, 1), (14, 2), (16, 1), (3, 1)])
def test_trees_and_heads(branching, Hq, Hkv):
    dev = gpu_ready()
    c = Case([400, 256, 257, 511, 384], 256, 128, Hq, Hkv, branching, dev, seed=Hq, poison=True)
    c.check(c.call())


@pytest.mark.gpu
@pytest.mark.parametrize("P", [128, 256])
@pytest.mark.parametrize("shared", [0, 128, 384, 1024])
@pytest.mark.parametrize("branching", [(1,), (3, 2, 2), (4, 3, 2, 1)], ids=str)
def test_lengths(shared, P, branching):
    """Lengths below, at and past the shared rows, zero, and page borders on either side."""
    dev = gpu_ready()
    L = sorted({0, 1, 127, 128, 129, max(shared - 1, 0), shared, shared + 1, shared + 127, shared + 128, shared + 129,
                shared + 300})
    c = Case(L, shared, P, 8, 2, branching, dev, seed=shared + P, poison=True)
    c.check(c.call())


@pytest.mark.gpu
@pytest.mark.parametrize("branching", [(1,), (4, 3, 2, 1)], ids=str)
def test_invalid_sequences_get_zeros(branching):
    """A negative length, and one without room for the tree: zeros, the others right."""
    dev = gpu_ready()
    c = Case([300, -1, 512, 260, -2 ** 31], 256, 128, 8, 2, branching, dev, seed=3, poison=True, L_cap=512)
    O = c.call()
    for b in (1, 2, 4):
        assert bool((O[b] == 0).all()), b
    c.check(O)


@pytest.mark.gpu
@pytest.mark.parametrize("B,branching,Hq,Hkv", [(1, (1,), 4, 4), (1, (4, 3, 2, 1), 8, 2), (33, (1,), 8, 1), (70, (2, 2), 4, 2)])
def test_batches(B, branching, Hq, Hkv):
    """One sequence (the prefix alone is split over the GPU) up to many; a prefix of thousands of rows."""
    dev = gpu_ready()
    L = [2048 + (37 * b) % 300 for b in range(B)]
    c = Case(L, 2048, 256, Hq, Hkv, branching, dev, seed=B)
    c.check(c.call())


@pytest.mark.gpu
@pytest.mark.parametrize("branching,Hq,Hkv", [((1,), 8, 8), ((1,), 16, 8), ((1,), 24, 8), ((1,), 64, 8), ((2, 2), 8, 8),
                                              ((3, 2, 2), 8, 8)])
@pytest.mark.parametrize("shared", [0, 512])
def test_few_rows_many_sequences(shared, branching, Hq, Hkv):
    """Single tokens and small trees of enough sequences to fill the GPU (lengths on both sides of the
    shared rows, invalid ones among them, pages that no sequence may read poisoned)."""
    dev = gpu_ready()
    L = [(shared - 3 + 29 * b) if b % 7 else 29 * b for b in range(25)]
    L[3], L[11], L[12] = -1, shared, 10 ** 6
    c = Case([min(n, 5000) for n in L], shared, 128, Hq, Hkv, branching, dev, seed=Hq + shared, poison=True, L_cap=1536)
    O = c.call()
    assert bool((O[3] == 0).all()) and bool((O[12] == 0).all())
    c.check(O)


@pytest.mark.gpu
@pytest.mark.parametrize("branching", [(1,), (4, 3, 2, 1)], ids=str)
def test_page_ids_outside_the_pool(branching):
    """A table entry outside the pool reads no memory outside it; the other sequences are right."""
    dev = gpu_ready()
    c = Case([400, 400, 400], 256, 128, 8, 2, branching, dev, seed=4)
    c.table[1][2], c.table[1][3] = c.num + 5, -3
    O = c.call()
    c.table[1] = c.table[0]   # sequence 1 is not compared
    for b in (0, 2):
        c.check(O, rows=slice(b, b + 1))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq", [8, 16])
def test_page_ids_outside_the_pool_of_many_sequences(Hq):
    """The same for single tokens of enough sequences to fill the GPU."""
    dev = gpu_ready()
    c = Case([256 + 13 * b for b in range(24)], 256, 128, Hq, 8, (1,), dev, seed=14)
    c.table[3][2], c.table[20][2], c.table[20][3] = -1, c.num, 2 ** 31 - 1
    O = c.call()
    c.table[3] = c.table[20] = c.table[23]   # these two are not compared
    for rows in (slice(0, 3), slice(4, 20), slice(21, 24)):
        c.check(O, rows=rows)


@pytest.mark.gpu
def test_single_tokens_streams_and_graph():
    """Two calls at once with workspaces of their own; a captured call replayed with other lengths."""
    dev = gpu_ready()
    cs = [Case([256 + 17 * b for b in range(24)], 256, 128, 8, 8, (1,), dev, seed=s) for s in (15, 16)]
    want = [c.call() for c in cs]
    outs, streams = [torch.full_like(w, 7.0) for w in want], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, o, st in zip(cs, outs, streams):
            c.call(o, st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    c, O = cs[0], torch.full_like(want[0], 7.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(O)
        c.call(O)
    c.L = [0, 100] + [256 + 11 * b for b in range(22)]
    c.dL.copy_(i32(c.L, dev))
    for _ in range(3):
        g.replay()
    c.check(O, "replayed")


@pytest.mark.gpu
def test_streams_graph_and_workspace():
    """Two calls at once with workspaces of their own; a captured call replayed with other lengths;
    two calls of different sizes that take turns with one workspace."""
    dev = gpu_ready()
    cs = [Case([300, 700, 256], 256, 128, 8, 2, (4, 3, 2, 1), dev, seed=s) for s in (1, 2)]
    want = [c.call() for c in cs]
    outs, streams = [torch.full_like(w, 7.0) for w in want], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, o, st in zip(cs, outs, streams):
            c.call(o, st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    c, O = cs[0], torch.full_like(want[0], 7.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(O)
    c.L = [256, 301, 100]
    c.dL.copy_(i32(c.L, dev))
    for _ in range(3):
        g.replay()
    c.check(O, "replayed")
    small = Case([130], 128, 128, 8, 2, (1,), dev, seed=5)
    small.ws = c.ws
    for _ in range(2):
        small.check(small.call(), "small call in the same workspace")
        c.check(c.call(), "large call in the same workspace")


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 2), (8, 1)])
@pytest.mark.parametrize("count", [64, 128])
def test_pruned_trees_up_to_the_limit(count, Hq, Hkv):
    """Trees of 64 and of 128 nodes (the most there may be), given by their rank paths."""
    dev = gpu_ready()
    paths = configs.pruned_paths(5, 8, count - 1)
    branching = tuple(1 + max(p[d] for p in paths if len(p) > d) for d in range(5))
    w = configs.scaled(configs.get("vicuna7b_b1"), branching=branching, tree_paths=paths)
    c = Case([300, 256, 0, 700], 256, 128, Hq, Hkv, (2, 2), dev, seed=count, poison=False, L_cap=1024)
    c.mask = torch.from_numpy(O.ancestor_mask(np.array(w.tree_nodes[0])).astype(bool))
    c.bits = torch.from_numpy(O.mask_bits(c.mask.numpy().astype(np.uint8)).view(np.int64)).to(dev)
    c.N, c.cfg = count, cfg_for(4, Hq, Hkv, 128, BF16, 1024, branching, tree_nodes=w.tree_nodes)
    gen = torch.Generator(device=dev).manual_seed(count)
    rnd = lambda *s: torch.randn(s, generator=gen, device=dev).to(BF16)
    c.Q, c.Kt, c.Vt = rnd(4, count, Hq, 128), rnd(4, Hkv, count, 128), rnd(4, Hkv, count, 128)
    c.ws = torch.empty(mb.prefix_workspace_size(c.cfg, 256), dtype=torch.uint8, device=dev)
    c.check(c.call())


@pytest.mark.gpu
@pytest.mark.parametrize("shared", [0, 256])
def test_two_nodes_a_head_for_each_query(shared):
    """A root and its child (the root does not see the child), many sequences; lengths around each step of the keys."""
    dev = gpu_ready()
    L = [shared + n for n in (0, 1, 30, 31, 32, 33, 62, 63, 64, 65, 95, 96, 97, 126, 127, 128, 129, 159, 160, 200)]
    c = Case(L, shared, 128, 8, 8, (1,), dev, seed=shared + 1, poison=True, L_cap=shared + 256)
    c.N, c.mask = 2, torch.tensor([[True, False], [True, True]])
    c.bits = torch.tensor([[1, 0], [3, 0]], dtype=torch.int64, device=dev)
    gen = torch.Generator(device=dev).manual_seed(12)
    rnd = lambda *s: torch.randn(s, generator=gen, device=dev).to(BF16)
    c.Q, c.Kt, c.Vt = rnd(20, 2, 8, 128) * 2, rnd(20, 8, 2, 128), rnd(20, 8, 2, 128)
    c.cfg = cfg_for(20, 8, 8, 128, BF16, shared + 256, (1,), tree_nodes=([-1, 0], [0, 0]))
    c.ws = torch.full((mb.prefix_workspace_size(c.cfg, shared),), 255, dtype=torch.uint8, device=dev)
    c.check(c.call())


@pytest.mark.gpu
@pytest.mark.parametrize("branching", [(1,), (2, 2)], ids=str)
def test_everything_shared(branching):
    """As many shared rows as the cache has: no sequence has rows of its own."""
    dev = gpu_ready()
    c = Case([0, 100, 500, 512 - (1 if branching == (1,) else 7)], 512, 128, 4, 2, branching, dev, seed=7, L_cap=512)
    c.check(c.call())


@pytest.mark.gpu
def test_one_sequence_behind_a_very_long_prefix():
    """The most key splits there are (32), and their merge."""
    dev = gpu_ready()
    c = Case([20000], 16384, 256, 2, 1, (1,), dev, seed=8)
    c.check(c.call())


@pytest.mark.gpu
@pytest.mark.parametrize("P", [384, 1024])
def test_page_sizes(P):
    dev = gpu_ready()
    c = Case([P + 5, 1300, 640, 2000], 640, P, 8, 2, (3, 2, 2), dev, seed=P, poison=True, L_cap=3 * P if P > 900 else 6 * P)
    c.check(c.call())


@pytest.mark.gpu
@pytest.mark.parametrize("B,branching", [(3, (3, 2, 2)), (20, (1,))])
def test_pages_past_32_bit_offsets(B, branching):
    """Pools of more than 2^31 elements, the pages in use at their far end."""
    dev = gpu_ready()
    c = Case([300 + 31 * b for b in range(B)], 256, 128, 16, 8, branching, dev, seed=11)
    first = 17000 - c.num
    far = lambda pool: torch.cat([torch.zeros((first, 8, 128, 128), dtype=BF16, device=dev), pool])
    c.Kp, c.Vp = far(c.Kp), far(c.Vp)
    c.prefix = [p + first for p in c.prefix]
    c.table = [[p + first if p >= 0 else p for p in row] for row in c.table]
    c.num = 17000
    assert c.Kp.numel() > 2 ** 31
    c.check(c.call())


# ----------------------------------------------------------------------------- the oracle (no GPU)
def test_oracle_is_the_paged_oracle():
    """Where every sequence's own table names the shared pages, the plain paged tree attention is the same."""
    c = Case([300, 256, 0, 411], 256, 128, 4, 2, (3, 2, 2), "cpu", seed=9, L_cap=640)
    got, A, S = SO.prefix_attention(c.Q, c.Kp, c.Vp, 128, c.prefix, 256, c.table, c.Kt, c.Vt, c.L, c.mask, c.L_cap)
    full = np.array([c.prefix + row[2:] for row in c.table])
    f64 = lambda t: t.float().numpy().astype(np.float64)
    want = O.tree_attention_paged(f64(c.Q), f64(c.Kp), f64(c.Vp), np.maximum(full, 0), 128, f64(c.Kt), f64(c.Vt), np.array(c.L),
                                  c.mask.numpy().astype(np.uint8), 4, 2)
    assert np.abs(got.numpy() - want).max() < 1e-12
    assert bool((A >= got.abs() - 1e-12).all()) and bool((S >= 0).all())


# ----------------------------------------------------------------------------- refusals (no GPU)
def status(num_pages=9, P=128, shared=256, L_cap=1024, dtype=BF16, D=128, drop=None, off=None):
    _build.build()
    cfg = cfg_for(2, 4, 2, D, dtype, L_cap)
    at = {n: 4096 for n in ("Q", "Kp", "Vp", "prefix", "table", "Kt", "Vt", "L", "bits", "O", "ws")}
    if drop:
        at[drop] = 0
    if off:
        at[off] += 8
    p = {n: ctypes.c_void_p(x) if x else None for n, x in at.items()}
    return mb.load().medusa_tree_attention_prefix(ctypes.byref(cfg), p["Q"], p["Kp"], p["Vp"], num_pages, P, p["prefix"], shared,
                                                  p["table"], p["Kt"], p["Vt"], p["L"], p["bits"], p["O"], p["ws"], None)


@pytest.mark.parametrize("kw,want", [
    *[(dict(drop=n), -1) for n in ("Q", "Kp", "Vp", "prefix", "table", "Kt", "Vt", "L", "bits", "O", "ws")],
    *[(dict(off=n), -1) for n in ("Q", "Kp", "Vp", "Kt", "Vt", "O", "ws")],
    (dict(num_pages=0), -1), (dict(P=64), -2), (dict(P=192), -2), (dict(P=384), -2), (dict(shared=-128), -1),
    (dict(shared=100), -2), (dict(shared=1152), -2), (dict(dtype=torch.float32), -2), (dict(D=64), -2),
])
def test_refusals(kw, want):
    assert status(**kw) == want


def test_workspace_size_refusals():
    _build.build()
    size = lambda cfg, s: mb.raw_call("medusa_prefix_workspace_size", ctypes.byref(cfg), s, ctypes.byref(ctypes.c_size_t()))
    good = cfg_for(2, 4, 2, 128, BF16)
    assert size(good, 256) == 0 and size(good, 0) == 0
    assert size(good, 100) == -2 and size(good, -1) == -1 and size(good, 2048) == -2
    assert size(cfg_for(2, 4, 2, 64, BF16), 256) == -2
    assert mb.raw_call("medusa_prefix_workspace_size", ctypes.byref(good), 256, None) == -1
