"""Tree attention (contiguous and paged) where the running maximum of some rows of a warp moves far at a
later key tile and that of others does not: short first tiles, scaled queries, planted scores."""
import os
import re

import numpy as np
import pytest
import torch

from medusa_speculative_decoding_heads_gb300 import binding as mb
from oracle import serving_oracle as SO

from _helpers import gpu_ready
from _serving import ancestor_bits, assert_within, cfg_for, i32, tolerance

BF16 = torch.bfloat16
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "medusa_speculative_decoding_heads_gb300", "csrc")


class Batch:
    """Committed rows and tree rows of a batch; laid out as one cache or as pages."""

    def __init__(self, L, Hq, Hkv, branching, dev, seed, scale=2.0, page=None):
        gen = torch.Generator(device=dev).manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device=dev)
        self.mask, self.bits = ancestor_bits(branching, dev)
        self.L, self.B, self.N, self.Hq, self.Hkv, self.dev = list(L), len(L), self.mask.shape[0], Hq, Hkv, dev
        self.P = page
        most = max(L) + self.N
        self.L_cap = -(-most // (page or 64)) * (page or 64)
        self.cfg = cfg_for(self.B, Hq, Hkv, 128, BF16, self.L_cap, branching)
        self.Q = (rnd(self.B, self.N, Hq, 128) * scale).to(BF16)
        self.K = [rnd(n, Hkv, 128).to(BF16) for n in L]
        self.V = [rnd(n, Hkv, 128).to(BF16) for n in L]
        self.Kt, self.Vt = rnd(self.B, Hkv, self.N, 128).to(BF16), rnd(self.B, Hkv, self.N, 128).to(BF16)

    def plant(self, jump):
        """Rows take turns (period 2 for the sign, 3 for whether it is there): the committed keys score +-jump
        with them, the tree's -+jump, so that half of a warp's maxima rise by 2 jump at the tree's tile."""
        row = torch.arange(self.N * self.Hq, device=self.dev).view(1, self.N, self.Hq)
        sign = (1.0 - 2.0 * (row % 2)) * (row % 3 > 0)
        self.Q[..., 0] = (sign * jump).to(BF16)
        for k in self.K:
            k[..., 0] = 11.0
        self.Kt[..., 0] = -11.0

    def call(self):
        O = torch.full_like(self.Q, 7.0)
        ws = torch.empty(max(mb.workspace_size(self.cfg), 256), dtype=torch.uint8, device=self.dev)
        L = i32(self.L, self.dev)
        if self.P is None:
            Kc, Vc = (torch.zeros((self.B, self.Hkv, self.L_cap, 128), dtype=BF16, device=self.dev) for _ in range(2))
            for b, n in enumerate(self.L):
                Kc[b, :, :n], Vc[b, :, :n] = self.K[b].transpose(0, 1), self.V[b].transpose(0, 1)
                Kc[b, :, n:n + self.N], Vc[b, :, n:n + self.N] = self.Kt[b], self.Vt[b]
            mb.tree_attention(self.cfg, self.Q, Kc, Vc, L, self.bits, O, ws)
            return O
        width = self.L_cap // self.P
        num = self.B * width + 1
        table = torch.randperm(num, generator=torch.Generator().manual_seed(1))[:self.B * width].view(self.B, width)
        Kp, Vp = (torch.zeros((num, self.Hkv, self.P, 128), dtype=BF16, device=self.dev) for _ in range(2))
        for b, n in enumerate(self.L):
            for i in range(0, n, self.P):
                m, page = min(self.P, n - i), int(table[b, i // self.P])
                Kp[page, :, :m], Vp[page, :, :m] = self.K[b][i:i + m].transpose(0, 1), self.V[b][i:i + m].transpose(0, 1)
        mb.tree_attention_paged(self.cfg, self.Q, Kp, Vp, num, self.P, table.int().to(self.dev), self.Kt, self.Vt, L, self.bits,
                                O, ws)
        return O

    def check(self, O, what):
        for b, n in enumerate(self.L):
            k = torch.cat([self.K[b], self.Kt[b].transpose(0, 1)])
            v = torch.cat([self.V[b], self.Vt[b].transpose(0, 1)])
            see = torch.cat([torch.ones((self.N, n), dtype=torch.bool), self.mask], 1).to(self.dev)
            ref, A, S = SO.attend(self.Q[b], k, v, see)
            assert_within(O[b], ref, tolerance(BF16, ref, A, S, n + self.N), f"{what}, sequence {b}")
        assert mb.poll_errors() == (0, 0, 0)


HEADS = [(2, 2), (8, 2), (10, 2), (16, 2)]   # 65-node tree: one ragged Q tile; two and leftover rows; three; four and leftover rows


@pytest.mark.gpu
@pytest.mark.parametrize("page", [None, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("L", [[1, 1], [2, 33], [0, 130, 1, 257]], ids=str)
def test_some_maxima_jump(L, Hq, Hkv, page):
    dev = gpu_ready()
    for scale in (1.0, 6.0):
        c = Batch(L, Hq, Hkv, (4, 3, 2, 1), dev, seed=Hq + len(L), scale=scale, page=page)
        c.check(c.call(), f"queries times {scale}")
    c.plant(30.0)
    c.check(c.call(), "planted")


@pytest.mark.gpu
def test_ragged_pages():
    """Nine sequences, 8 / 2 heads, 65 nodes, lengths 512 + 17 b: the last key ranges begin with a short tile."""
    dev = gpu_ready()
    for seed in range(3):
        c = Batch([512 + 17 * b for b in range(9)], 8, 2, (4, 3, 2, 1), dev, seed=seed, page=128)
        c.check(c.call(), f"seed {seed}")
        c.plant(30.0)
        c.check(c.call(), f"seed {seed}, planted")


def test_votes_do_not_hide_behind_a_short_circuit():
    """A warp's vote inside the argument of another one is skipped by the lanes whose left operand decides:
    the warp then stands at two different votes, and what follows runs on a part of it."""
    vote = re.compile(r"__(any|all|ballot)_sync\s*\(")
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name), encoding="utf-8") as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in vote.finditer(text):
            depth, end = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[end], 0)
                end += 1
            inner = text[m.end():end]
            at = vote.search(inner)
            assert at is None or not re.search(r"\|\||&&|\?", inner[:at.start()]), f"{name}: {inner.strip()}"
