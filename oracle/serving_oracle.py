"""Plain implementations of the prompt, shared-prefix and page operators (test infrastructure only).

Attention in float64 with torch (any device), one sequence at a time; page
bookkeeping with Python lists, one page at a time. Nothing here calls the library.
"""
from __future__ import annotations

import math
from typing import List, Sequence, Tuple

import torch

FLAG_CAPACITY, FLAG_PAGES = 4, 16


def attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, visible: torch.Tensor):
    """Rows q [R, Hq, D] over keys k, v [n, Hkv, D] where visible [R, n], in float64; KV head h // (Hq / Hkv).

    Returns (O, A, S): the result, the same weights applied to |v| and, per row and head, the
    largest sum of |q_d k_d| / sqrt(D) over the visible keys (what error bounds are made of). A row
    that sees nothing gives 0. Values at places that no row sees never enter."""
    R, Hq, D = q.shape
    seen, some = visible.any(0), visible.any(1)
    k, v, visible = k[seen], v[seen], visible[:, seen]
    G = Hq // k.shape[1]
    q = q.double().transpose(0, 1)                                          # [Hq, R, D]
    k, v = (x.double().transpose(0, 1).repeat_interleave(G, 0) for x in (k, v))   # [Hq, n, D]
    if k.shape[1] == 0:
        z = torch.zeros((R, Hq, D), dtype=torch.float64, device=q.device)
        return z, z, z[..., 0]
    scale = 1.0 / math.sqrt(D)
    s = (q @ k.transpose(1, 2) * scale).masked_fill(~visible, -math.inf)
    w = torch.exp(s - s.amax(2, keepdim=True))
    w = torch.where(some[:, None], w / w.sum(2, keepdim=True), 0.0)
    S = (q.abs() @ k.abs().transpose(1, 2) * scale).masked_fill(~visible, 0.0).amax(2)
    return (w @ v).transpose(0, 1), (w @ v.abs()).transpose(0, 1), S.transpose(0, 1)


def prompt_attention(Q, K, V, cu: Sequence[int]):
    """Causal attention of packed sequences, up to the first decrease of cu: (O, A, S) as ``attend``, [T][Hq][D] and
    [T][Hq]."""
    T, Hq, D = Q.shape
    O = torch.zeros((T, Hq, D), dtype=torch.float64, device=Q.device)
    A, S = torch.zeros_like(O), torch.zeros((T, Hq), dtype=torch.float64, device=Q.device)
    for a, e in zip(cu[:-1], cu[1:]):
        if e < a:
            break
        if a < 0 or e == a or e > T:
            continue
        i = torch.arange(e - a, device=Q.device)
        see = i[None, :] <= i[:, None]
        O[a:e], A[a:e], S[a:e] = attend(Q[a:e], K[a:e], V[a:e], see)
    return O, A, S


def prefix_attention(Q, Kp, Vp, P: int, prefix: Sequence[int], shared: int, table, Kt, Vt, L: Sequence[int], mask, L_cap: int):
    """Tree attention whose logical rows [0, shared) come from the pages `prefix`: (O, A, S)."""
    B, N, Hq, D = Q.shape
    O = torch.zeros(Q.shape, dtype=torch.float64, device=Q.device)
    A, S = torch.zeros_like(O), torch.zeros((B, N, Hq), dtype=torch.float64, device=Q.device)
    for b in range(B):
        n = int(L[b])
        if n < 0 or n + N > L_cap:
            continue
        rows = [(int(prefix[i // P]) if i < shared else int(table[b][i // P]), i % P) for i in range(n)]
        pages = torch.tensor([r[0] for r in rows], dtype=torch.long, device=Q.device)
        offs = torch.tensor([r[1] for r in rows], dtype=torch.long, device=Q.device)
        k = torch.cat([Kp[pages, :, offs], Kt[b].transpose(0, 1)], 0)   # [n + N, Hkv, D]
        v = torch.cat([Vp[pages, :, offs], Vt[b].transpose(0, 1)], 0)
        see = torch.cat([torch.ones((N, n), dtype=torch.bool, device=Q.device), mask.to(Q.device)], 1)
        O[b], A[b], S[b] = attend(Q[b], k, v, see)
    return O, A, S


class Pages:
    """Block tables, reference counts, lengths and (optionally) pools [layers][pages][Hkv][P][D]."""

    def __init__(self, table: List[List[int]], refs: List[int], L: List[int], P: int, pools=()):
        self.table, self.refs, self.L, self.P = [list(r) for r in table], list(refs), list(L), P
        self.pools = [p.clone() for p in pools]

    def _free(self) -> List[int]:
        return [p for p, n in enumerate(self.refs) if n <= 0]

    def reserve(self, rows: Sequence[int]) -> List[int]:
        free, wanted, flags = self._free(), 0, []
        width = len(self.table[0])
        for b, r in enumerate(rows):
            if r < 0 or r > width * self.P:
                flags.append(FLAG_CAPACITY)
                continue
            holes = [i for i in range(-(-r // self.P)) if self.table[b][i] < 0]
            first, wanted = wanted, wanted + len(holes)
            if holes and wanted > len(free):
                flags.append(FLAG_CAPACITY)
                continue
            for i, page in zip(holes, free[first:wanted]):
                self.table[b][i], self.refs[page] = page, 1
            flags.append(0)
        return flags

    def store(self, K, V, cu, start) -> None:
        """K, V [T][Hkv][D] into layer 0 of pools[0] (keys) and pools[1] (values)."""
        T, width, num = K.shape[0], len(self.table[0]), len(self.refs)
        for b, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
            if a < 0 or e < a or e > T:
                continue
            for r in range(e - a):
                i = (start[b] if start is not None else 0) + r
                if 0 <= i < width * self.P and 0 <= self.table[b][i // self.P] < num:
                    self.pools[0][0, self.table[b][i // self.P], :, i % self.P] = K[a + r]
                    self.pools[1][0, self.table[b][i // self.P], :, i % self.P] = V[a + r]

    def fork(self, src: Sequence[int], dst: Sequence[int]) -> List[int]:
        B, width, num = len(self.table), len(self.table[0]), len(self.refs)
        free, flags, wanted, todo = self._free(), [], 0, []
        for f, (s, d) in enumerate(zip(src, dst)):
            ok = 0 <= s < B and 0 <= d < B and 0 <= self.L[s] <= width * self.P
            ok = ok and d not in src and list(dst).count(d) == 1 and all(p < 0 for p in self.table[d])
            ok = ok and all(0 <= self.table[s][i] < num for i in range(-(-self.L[s] // self.P)))
            if not ok:
                flags.append(FLAG_PAGES)
                continue
            part = self.L[s] % self.P
            wanted += part > 0
            if part and wanted > len(free):
                flags.append(FLAG_CAPACITY)
                continue
            flags.append(0)
            todo.append((s, d, part, free[wanted - 1] if part else -1))
        for s, d, part, page in todo:
            full = self.L[s] // self.P
            for i in range(full):
                self.table[d][i] = self.table[s][i]
                self.refs[self.table[s][i]] += 1
            if part:
                old = self.table[s][full]
                self.table[d][full], self.refs[page] = page, 1
                for pool in self.pools:
                    pool[:, page, :, :part] = pool[:, old, :, :part]
            self.L[d] = self.L[s]
        return flags

    def free(self, seqs: Sequence[int]) -> None:
        for s in seqs:
            if 0 <= s < len(self.table):
                for i, page in enumerate(self.table[s]):
                    if 0 <= page < len(self.refs):
                        self.refs[page] -= 1
                    self.table[s][i] = -1
                self.L[s] = 0

    def compact(self) -> Tuple[List[int], int]:
        num = len(self.refs)
        live = sum(n > 0 for n in self.refs)
        page_map = [p if self.refs[p] > 0 else -1 for p in range(num)]
        holes = [p for p in range(live) if self.refs[p] <= 0]
        for p in range(live, num):
            if self.refs[p] > 0:
                to = holes.pop(0)
                page_map[p], self.refs[to], self.refs[p] = to, self.refs[p], 0
                for pool in self.pools:
                    pool[:, to] = pool[:, p]
        self.table = [[page_map[p] if 0 <= p < num else p for p in row] for row in self.table]
        return page_map, live
