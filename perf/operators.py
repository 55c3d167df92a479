"""Cases of the prompt, shared-prefix and page operators, with their plain forms.

Each case is one pass through an operator of the serving path around the verify step: attention over
packed prompts, storing a prompt's keys and values in the pages of a cache, tree attention of a batch
whose sequences share a long prefix, forking sequences that share pages, and freeing sequences with
compaction of the pages that are left. ``run`` computes a case in elementary torch operations, or with
``own`` through the library's binding.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BRANCH = {1: "", 7: "2,2", 22: "3,2,2", 65: "4,3,2,1", 111: "5,3,2,1,1"}   # nodes -> top-s per head


def _ints(text):
    return [int(x) for x in str(text).split(",") if x != ""]


def _text(values):
    return ",".join(str(int(v)) for v in values)


def _ragged(rng, count, lo, hi):
    """`count` lengths in [lo, hi], spread over their logarithm, odd ones among them."""
    return [max(lo, min(hi, int(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi + 1)))))) for _ in range(count)]


# ---------------------------------------------------------------------------------------------- cases
def listed():
    r = random.Random(20)
    return [
        # one user's question of a few dozen tokens: what counts is latency
        dict(name="prompt, 37 tokens", op="prompt", dtype="bf16", Hq=32, Hkv=32, D=128, lens="37", pad=0, fused=0),
        # a prefill batch of mixed requests, K/V heads shared by four, read from one fused projection, in a padded bucket
        dict(name="prompt, 16 mixed requests", op="prompt", dtype="bf16", Hq=32, Hkv=8, D=128,
             lens=_text([1, 0, 2047, 129] + _ragged(r, 12, 17, 4000)), pad=131, fused=1),
        # the longest cache of the grouped-head workload as one prompt
        dict(name="prompt, 16384 tokens", op="prompt", dtype="bf16", Hq=32, Hkv=8, D=128, lens="16384", pad=0, fused=0),
        # the small float32 shape (head dim 64), several prompts
        dict(name="prompt, float32", op="prompt", dtype="f32", Hq=8, Hkv=4, D=64, lens="700,1,129,1500", pad=0, fused=0),
        # a batch of answers to one long document, each verifying its 65-node tree (grouped heads)
        dict(name="prefix, 32 trees after 8192", op="prefix", Hq=32, Hkv=8, tree=65, shared=8192, P=128,
             own=_text(_ragged(r, 30, 17, 600) + [0, 128]), cap=9216),
        # the same without a tree: one token per sequence, a head for each query
        dict(name="prefix, 24 tokens after 4096", op="prefix", Hq=40, Hkv=40, tree=1, shared=4096, P=256,
             own=_text(_ragged(r, 24, 1, 300)), cap=5120),
        # one layer's keys and values of a prefill batch go into the pages just reserved for them
        dict(name="store, 8 prompts", op="store", dtype="bf16", Hkv=8, D=128, P=128, lens=_text(_ragged(r, 8, 300, 4000)),
             pad=77, used=100, cap=4096),
        # one short prompt, small float32 shape
        dict(name="store, 33 tokens", op="store", dtype="f32", Hkv=4, D=64, P=128, lens="33", pad=0, used=5, cap=256),
        # one prompt of the grouped-head workload split into 31 continuations, every layer's last page copied
        dict(name="fork, 31 of one", op="fork", dtype="bf16", Hkv=8, D=128, P=128, layers=32, B=32, sources="8269",
             forks=31, spare=9),
        # two of four short sequences doubled
        dict(name="fork, 2 of two", op="fork", dtype="bf16", Hkv=4, D=64, P=128, layers=2, B=4, sources="129,200", forks=2,
             spare=3),
        # a third of a full batch has finished: its pages go, the others move to the front of every layer's pool
        dict(name="free and compact, 48 sequences", op="compact", dtype="bf16", Hkv=8, D=128, P=128, layers=4,
             lens=_text(_ragged(r, 48, 300, 8000)), every=3, pool=2048, cap=8192),
        # the same for a handful of short ones
        dict(name="free and compact, 5 sequences", op="compact", dtype="f32", Hkv=2, D=64, P=128, layers=2,
             lens="130,257,1,500,384", every=2, pool=24, cap=512),
    ]


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "prefix", "prefix", "store", "fork", "compact"])
    P = rng.choice([128, 256])
    heads = rng.choice([(32, 32), (32, 8), (40, 40), (8, 4), (16, 2), (12, 4), (28, 4), (20, 4), (6, 1)])
    if op == "prompt":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        D = rng.choice([64, 128])
        most = 4000 if dtype == "bf16" else 900
        count = rng.choice([1, 1, 2, 3, 5, 9, 17])
        lens = _ragged(rng, count, 1, most)
        if count > 2:
            lens[rng.randrange(count)] = 0
        return dict(op=op, dtype=dtype, Hq=heads[0], Hkv=heads[1], D=D, lens=_text(lens), pad=rng.choice([0, 0, 1, 200]),
                    fused=rng.choice([0, 1]))
    if op == "prefix":
        B = rng.choice([1, 2, 3, 6, 11, 24, 32])
        tree = rng.choice(sorted(BRANCH))
        shared = 128 * max(1, int(math.exp(rng.uniform(0.0, math.log(64)))))
        rest = _ragged(rng, B, 1, 900)
        if B > 2:
            rest[rng.randrange(B)] = 0
        cap = -(-(shared + max(rest) + tree) // P) * P
        return dict(op=op, Hq=heads[0], Hkv=heads[1], tree=tree, shared=shared, P=P, own=_text(rest), cap=cap)
    dtype, D = rng.choice([("bf16", 128), ("bf16", 64), ("f32", 64), ("f32", 128)])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "store":
        lens = _ragged(rng, rng.choice([1, 2, 5, 12]), 1, 3500)
        return dict(op=op, dtype=dtype, Hkv=Hkv, D=D, P=P, lens=_text(lens), pad=rng.choice([0, 1, 60]),
                    used=rng.randrange(40), cap=-(-max(lens) // P) * P)
    if op == "fork":
        sources = _ragged(rng, rng.choice([1, 1, 2, 4]), 1, 6000)
        forks = rng.choice([1, 2, 5, 13, 28])
        return dict(op=op, dtype=dtype, Hkv=Hkv, D=D, P=P, layers=rng.choice([1, 2, 5, 16]), B=len(sources) + forks + 1,
                    sources=_text(sources), forks=forks, spare=rng.randrange(8))
    lens = _ragged(rng, rng.choice([3, 7, 20, 41]), 1, 5000)
    cap = -(-max(lens) // P) * P
    pool = sum(-(-n // P) for n in lens) + rng.randrange(1, 60)
    return dict(op=op, dtype=dtype, Hkv=Hkv, D=D, P=P, layers=rng.choice([1, 2, 3]), lens=_text(lens),
                every=rng.choice([2, 3, 4]), pool=pool, cap=cap)


# --------------------------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _normal(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(scale).to(dtype) if math.prod(shape) < 1 << 28 \
        else torch.randn(shape, generator=gen, device=DEV, dtype=dtype)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _tree_parents(branching):
    parent, level = [-1], [0]
    for s in branching:
        nxt = []
        for p in level:
            for _ in range(s):
                nxt.append(len(parent))
                parent.append(p)
        level = nxt
    return parent


def _ancestors(branching):
    """mask[i][j]: j is i or an ancestor of i."""
    parent = _tree_parents(branching)
    mask = np.zeros((len(parent), len(parent)), dtype=bool)
    for i in range(len(parent)):
        j = i
        while j >= 0:
            mask[i, j] = True
            j = parent[j]
    return mask


def _pages_for(rng, lens, P, width, pool):
    """A shuffled block table [B][width] for these lengths, -1 past them, and the pages' reference counts."""
    ids = list(range(pool))
    rng.shuffle(ids)
    table, at = np.full((len(lens), width), -1, dtype=np.int32), 0
    for b, n in enumerate(lens):
        k = -(-n // P)
        table[b, :k] = ids[at:at + k]
        at += k
    refs = np.zeros(pool, dtype=np.int32)
    refs[table[table >= 0]] = 1
    return table, refs


def _prefix_pages(case):
    rest = _ints(case["own"])
    return case["shared"] // case["P"] + (case["shared"] % case["P"] > 0), \
        sum(-(-(case["shared"] + n) // case["P"]) - case["shared"] // case["P"] for n in rest)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)
    op, st = case["op"], {"case": dict(case)}
    if op == "prompt":
        lens, dt = _ints(case["lens"]), _dtype(case)
        Hq, Hkv, D, T = case["Hq"], case["Hkv"], case["D"], sum(_ints(case["lens"])) + case["pad"]
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        if case["fused"]:   # one projection's output: a row holds its q, k and v heads
            qkv = _normal(gen, (T, Hq + 2 * Hkv, D), dt)
            qkv[:, :Hq] *= 2
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            q, k, v = _normal(gen, (T, Hq, D), dt, 2.0), _normal(gen, (T, Hkv, D), dt), _normal(gen, (T, Hkv, D), dt)
        st.update(lens=lens, q=q, k=k, v=v, cu=_i32(cu), O=torch.zeros((T, Hq, D), dtype=dt, device=DEV))
    elif op == "prefix":
        Hq, Hkv, D, N, S, P = case["Hq"], case["Hkv"], 128, case["tree"], case["shared"], case["P"]
        rest = _ints(case["own"])
        B, width = len(rest), case["cap"] // P
        first, more = _prefix_pages(case)
        pool = first + more + 3
        ids = list(range(pool))
        rng.shuffle(ids)
        table, at = np.full((B, width), -1, dtype=np.int32), first
        for b, n in enumerate(rest):   # whole pages of the prefix are shared, a sequence's own rows follow
            table[b, :S // P] = ids[:S // P]
            k = -(-(S + n) // P) - S // P
            table[b, S // P:S // P + k] = ids[at:at + k]
            at += k
        prefix = ids[:first]
        bf = torch.bfloat16
        Kp, Vp = _normal(gen, (pool, Hkv, P, D), bf), _normal(gen, (pool, Hkv, P, D), bf)
        table = torch.from_numpy(table).to(DEV)
        if S % P:   # the prefix ends inside a page: each sequence holds a copy of that page's first rows
            own_page = table[:, S // P].long().clamp(min=0)
            keep = (table[:, S // P] >= 0)
            Kp[own_page[keep], :, :S % P] = Kp[prefix[-1], :, :S % P].unsqueeze(0)
            Vp[own_page[keep], :, :S % P] = Vp[prefix[-1], :, :S % P].unsqueeze(0)
        mask = _ancestors(_ints(BRANCH[N]))
        bits = [[sum(1 << (j - 64 * w) for j in range(64 * w, min(N, 64 * w + 64)) if mask[i, j]) for w in (0, 1)]
                for i in range(N)]
        bits = np.array(bits, dtype=np.uint64).astype(np.int64)
        st.update(q=_normal(gen, (B, N, Hq, D), bf, 2.0), Kp=Kp, Vp=Vp, Kt=_normal(gen, (B, Hkv, N, D), bf),
                  Vt=_normal(gen, (B, Hkv, N, D), bf), table=table, prefix=_i32(prefix), L=_i32([S + n for n in rest]),
                  most=S + max(rest), mask=torch.from_numpy(mask).to(DEV), bits=torch.from_numpy(bits).to(DEV), pool=pool,
                  O=torch.zeros((B, N, Hq, D), dtype=bf, device=DEV))
    elif op == "store":
        lens, dt, P, Hkv, D = _ints(case["lens"]), _dtype(case), case["P"], case["Hkv"], case["D"]
        B, T, width = len(lens), sum(lens) + case["pad"], case["cap"] // P
        pool = case["used"] + sum(-(-n // P) for n in lens) + 2
        refs = np.zeros(pool, dtype=np.int32)
        refs[rng.sample(range(pool), case["used"])] = 1   # other sequences' pages
        kv = _normal(gen, (T, 2, Hkv, D), dt)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        st.update(lens=lens, k=kv[:, 0], v=kv[:, 1], cu=_i32(cu), rows=_i32(lens), pool=pool,
                  Kp=torch.zeros((pool, Hkv, P, D), dtype=dt, device=DEV), Vp=torch.zeros((pool, Hkv, P, D), dtype=dt, device=DEV),
                  table0=torch.full((B, width), -1, dtype=torch.int32, device=DEV), refs0=torch.from_numpy(refs).to(DEV),
                  flags=torch.zeros(B, dtype=torch.int32, device=DEV))
    elif op == "fork":
        src_len, dt, P, Hkv, D, n = _ints(case["sources"]), _dtype(case), case["P"], case["Hkv"], case["D"], case["forks"]
        B, width = case["B"], -(-(max(src_len) + 128) // P)
        pool = sum(-(-x // P) for x in src_len) + n + case["spare"]
        seqs = list(range(B))
        rng.shuffle(seqs)
        lens = [0] * B
        for b, x in zip(seqs, src_len):
            lens[b] = x
        table, refs = _pages_for(rng, lens, P, width, pool)
        st.update(src=_i32([seqs[i % len(src_len)] for i in range(n)]), dst=_i32(seqs[len(src_len):len(src_len) + n]),
                  Kp=_normal(gen, (case["layers"], pool, Hkv, P, D), dt), Vp=_normal(gen, (case["layers"], pool, Hkv, P, D), dt),
                  table0=torch.from_numpy(table).to(DEV), refs0=torch.from_numpy(refs).to(DEV), L0=_i32(lens), pool=pool,
                  flags=torch.zeros(n, dtype=torch.int32, device=DEV))
    else:
        lens, dt, P, Hkv, D = _ints(case["lens"]), _dtype(case), case["P"], case["Hkv"], case["D"]
        table, refs = _pages_for(rng, lens, P, case["cap"] // P, case["pool"])
        st.update(done=_i32(list(range(0, len(lens), case["every"]))), pool=case["pool"],
                  Kp=_normal(gen, (case["layers"], case["pool"], Hkv, P, D), dt),
                  Vp=_normal(gen, (case["layers"], case["pool"], Hkv, P, D), dt),
                  table0=torch.from_numpy(table).to(DEV), refs0=torch.from_numpy(refs).to(DEV), L0=_i32(lens),
                  page_map=torch.zeros(case["pool"], dtype=torch.int32, device=DEV),
                  n_live=torch.zeros(1, dtype=torch.int32, device=DEV))
    for name in ("table", "refs", "L"):   # the tables that a pass changes, beside what it begins with
        if name + "0" in st:
            st[name] = st[name + "0"].clone()
    return st


def _restore(st):
    for name in ("table", "refs", "L"):
        if name + "0" in st:
            st[name].copy_(st[name + "0"])


# ----------------------------------------------------------------------------------------- plain forms
def _softmax_products(q, k, v, visible):
    """softmax over the visible keys of q.k / sqrt(D), times v; float32, [..., rows, D] x [..., keys, D]."""
    s = (q * (1.0 / math.sqrt(q.shape[-1]))) @ k.transpose(-1, -2)
    s.masked_fill_(~visible, float("-inf"))
    s -= s.amax(-1, keepdim=True)
    s.exp_()
    return (s @ v) / s.sum(-1, keepdim=True)


def _plain_prompt(st):
    c, lens = st["case"], st["lens"]
    T, Hq, D = st["q"].shape
    Hkv, most = c["Hkv"], max(lens)
    i = torch.arange(most, device=DEV)
    at = st["cu"][:-1, None].long() + i                              # [B, most] packed row of a sequence's row i
    there = i < (st["cu"][1:] - st["cu"][:-1])[:, None]
    at = at.clamp(max=T - 1)
    q = st["q"][at].float().permute(0, 2, 1, 3).reshape(len(lens), Hkv, Hq // Hkv, most, D)
    k = st["k"][at].float().permute(0, 2, 1, 3).unsqueeze(2)
    v = st["v"][at].float().permute(0, 2, 1, 3).unsqueeze(2)
    o = _softmax_products(q, k, v, i[:, None] >= i[None, :])         # [B, Hkv, G, most, D]; rows past the end are dropped
    o = o.reshape(len(lens), Hq, most, D).permute(0, 2, 1, 3)
    O = torch.zeros_like(st["O"])
    O[at[there]] = o[there].to(O.dtype)
    return O


def _plain_prefix(st):
    c = st["case"]
    B, N, Hq, D = st["q"].shape
    Hkv, P, S, most = c["Hkv"], c["P"], c["shared"], st["most"]
    i = torch.arange(most, device=DEV)
    page = torch.where(i[None] < S, st["prefix"][(i.clamp(max=S - 1) // P)].long()[None],
                       st["table"][:, i // P].long()).clamp(min=0)  # [B, most]
    q = st["q"].float().permute(0, 2, 1, 3).reshape(B, Hkv, (Hq // Hkv) * N, D)
    k = torch.cat([st["Kp"][page, :, (i % P)[None]].permute(0, 2, 1, 3), st["Kt"]], 2).float()
    v = torch.cat([st["Vp"][page, :, (i % P)[None]].permute(0, 2, 1, 3), st["Vt"]], 2).float()
    visible = torch.cat([(i[None] < st["L"][:, None])[:, None].expand(B, N, most), st["mask"][None].expand(B, N, N)], 2)
    o = _softmax_products(q, k, v, visible[:, None, None].expand(B, 1, Hq // Hkv, N, most + N).reshape(B, 1, -1, most + N))
    return o.reshape(B, Hq, N, D).permute(0, 2, 1, 3).to(torch.bfloat16)


def _plain_store(st):
    P, lens = st["case"]["P"], st["lens"]
    table, refs = st["table"], st["refs"]
    width = table.shape[1]
    want = (torch.arange(width, device=DEV)[None] < ((st["rows"] + P - 1) // P)[:, None]) & (table < 0)
    free = (refs == 0).nonzero().flatten()
    order = want.flatten().cumsum(0).reshape(want.shape)             # lowest free page first, sequence by sequence
    served = (order[:, -1] <= free.numel()) | (want.sum(1) == 0)
    want &= served[:, None]
    new = free[(order[want] - 1)]
    table[want] = new.int()
    refs[new] = 1
    flags = torch.where(served, 0, 4).int()
    t = torch.arange(sum(lens), device=DEV)
    b = torch.bucketize(t, st["cu"][1:].long(), right=True)
    r = t - st["cu"][b]
    page = table[b, r // P].long()
    st["Kp"][page, :, r % P] = st["k"][:sum(lens)]
    st["Vp"][page, :, r % P] = st["v"][:sum(lens)]
    return {"Kp": st["Kp"], "Vp": st["Vp"], "table": table, "refs": refs, "flags": flags}


def _plain_fork(st):
    P, n = st["case"]["P"], st["src"].numel()
    table, refs, L = st["table"], st["refs"], st["L"]
    src, dst = st["src"].long(), st["dst"].long()
    width, pool = table.shape[1], refs.numel()
    length = L[src]
    part = length % P
    new = (refs == 0).nonzero().flatten()[(part > 0).cumsum(0) - 1]  # used only where a page is partly filled
    col = torch.arange(width, device=DEV)[None]
    full = (length // P)[:, None]
    rows = torch.where(col < full, table[src], torch.where((col == full) & (part > 0)[:, None], new[:, None].int(), -1))
    refs += torch.bincount(rows[rows >= 0].long(), minlength=pool).int()
    last = table[src, (length // P).clamp(max=width - 1).long()].long()
    table[dst], L[dst] = rows, length
    j = torch.arange(P, device=DEV)[None]
    f, off = ((j < part[:, None]) & (part > 0)[:, None]).nonzero(as_tuple=True)
    for pool_ in (st["Kp"], st["Vp"]):
        pool_[:, new[f], :, off] = pool_[:, last[f], :, off]
    return {"Kp": st["Kp"], "Vp": st["Vp"], "table": table, "refs": refs, "L": L, "flags": torch.zeros_like(st["flags"])}


def _plain_compact(st):
    table, refs, L = st["table"], st["refs"], st["L"]
    pool = refs.numel()
    gone = table[st["done"].long()]
    refs -= torch.bincount(gone[gone >= 0].long(), minlength=pool).int()
    table[st["done"].long()] = -1
    L[st["done"].long()] = 0
    live = refs > 0
    n_live = live.sum()
    i = torch.arange(pool, device=DEV)
    high, low = (live & (i >= n_live)).nonzero().flatten(), (~live & (i < n_live)).nonzero().flatten()
    page_map = torch.where(live, i, -1).int()
    page_map[high] = low.int()
    for pool_ in (st["Kp"], st["Vp"]):
        pool_[:, low] = pool_[:, high]
    table.copy_(torch.where(table >= 0, page_map[table.clamp(min=0).long()], table))
    refs[low], refs[high] = refs[high], 0
    return {"Kp": st["Kp"], "Vp": st["Vp"], "table": table, "refs": refs, "L": L, "page_map": page_map,
            "n_live": n_live.int().reshape(1)}


# ------------------------------------------------------------------------------------- the library's calls
def _plan(st):
    """The configuration and workspace that a program keeps between calls."""
    from medusa_speculative_decoding_heads_gb300 import binding as mb
    c, op = st["case"], st["case"]["op"]
    B = {"prompt": lambda: len(st["lens"]), "prefix": lambda: st["q"].shape[0], "store": lambda: len(st["lens"])}.get(
        op, lambda: st["table"].shape[0])()
    branching = _ints(BRANCH[c["tree"]]) if c.get("tree", 1) > 1 else [1]
    cap = max(st["lens"] + [8]) if op == "prompt" else st["table"].shape[1] * c["P"]
    cfg = mb.make_cfg(B=B, d=64, V=64, branching=branching, Hq=c.get("Hq", c["Hkv"]), Hkv=c["Hkv"], D=c.get("D", 128),
                      L_cap=cap, dtype=mb.F32 if c.get("dtype") == "f32" else mb.BF16, mode=mb.GREEDY,
                      tree_nodes=([-1], [0]) if len(branching) == 1 and c.get("tree", 1) == 1 else None)
    size = {"prompt": lambda: 0, "prefix": lambda: mb.prefix_workspace_size(cfg, c["shared"])}.get(
        op, lambda: mb.pages_workspace_size(cfg, st["pool"]))()
    st["mb"], st["cfg"], st["ws"] = mb, cfg, torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)


def _library(st):
    if "cfg" not in st:
        _plan(st)
    mb, cfg, ws, c, op = st["mb"], st["cfg"], st["ws"], st["case"], st["case"]["op"]
    if op == "prompt":
        q, k, v = st["q"], st["k"], st["v"]
        mb.prompt_attention(cfg, q, k, v, q.shape[0], q.stride(0), k.stride(0), v.stride(0), st["cu"], st["O"])
        return st["O"]
    if op == "prefix":
        mb.tree_attention_prefix(cfg, st["q"], st["Kp"], st["Vp"], st["pool"], c["P"], st["prefix"], c["shared"], st["table"],
                                 st["Kt"], st["Vt"], st["L"], st["bits"], st["O"], ws)
        return st["O"]
    Kp, Vp, table, refs = st["Kp"], st["Vp"], st["table"], st["refs"]
    out = {"Kp": Kp, "Vp": Vp, "table": table, "refs": refs}
    if op == "store":
        k, v = st["k"], st["v"]
        mb.pages_reserve(cfg, st["pool"], c["P"], st["rows"], table, refs, st["flags"], ws)
        mb.kv_store_paged(cfg, k, v, k.shape[0], k.stride(0), v.stride(0), st["cu"], None, Kp, Vp, st["pool"], c["P"], table)
        return {**out, "flags": st["flags"]}
    if op == "fork":
        mb.pages_fork(cfg, Kp, Vp, st["pool"], c["P"], c["layers"], Kp.stride(0), c["forks"], st["src"], st["dst"], table,
                      st["L"], refs, st["flags"], ws)
        return {**out, "L": st["L"], "flags": st["flags"]}
    mb.pages_free(cfg, st["pool"], c["P"], st["done"].numel(), st["done"], table, st["L"], refs)
    mb.pages_compact(cfg, Kp, Vp, st["pool"], c["P"], c["layers"], Kp.stride(0), table, refs, st["page_map"], st["n_live"], ws)
    return {**out, "L": st["L"], "page_map": st["page_map"], "n_live": st["n_live"]}


def run(state):
    _restore(state)
    if own:
        return _library(state)
    return {"prompt": _plain_prompt, "prefix": _plain_prefix, "store": _plain_store, "fork": _plain_fork,
            "compact": _plain_compact}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ work
def work(case):
    op, elt = case["op"], 4 if case.get("dtype") == "f32" else 2
    if op == "prompt":
        lens, Hq, Hkv, D = _ints(case["lens"]), case["Hq"], case["Hkv"], case["D"]
        return {"bytes": sum(lens) * (2 * Hq + 2 * Hkv) * D * elt + 4 * (len(lens) + 1),
                "flops": sum(4 * D * Hq * n * (n + 1) // 2 for n in lens)}
    if op == "prefix":
        Hq, Hkv, N, S, rest = case["Hq"], case["Hkv"], case["tree"], case["shared"], _ints(case["own"])
        pairs = int(_ancestors(_ints(BRANCH[N])).sum())
        return {"bytes": (S + sum(rest)) * Hkv * 128 * 4 + len(rest) * N * (2 * Hq + 2 * Hkv) * 128 * 2,
                "flops": sum(4 * 128 * Hq * (N * (S + n) + pairs) for n in rest)}
    P, row = case["P"], case["Hkv"] * case["D"] * elt
    if op == "store":
        lens = _ints(case["lens"])
        return {"bytes": 4 * sum(lens) * row + 4 * (case["used"] + 2 * sum(-(-n // P) for n in lens)), "flops": 0}
    if op == "fork":
        lens = _ints(case["sources"])
        part = [lens[i % len(lens)] % P for i in range(case["forks"])]
        return {"bytes": 2 * case["layers"] * row * (sum(part) + sum(n % P for n in lens[:case["forks"]]))
                + 8 * sum(-(-lens[i % len(lens)] // P) for i in range(case["forks"])), "flops": 0}
    pages = [-(-n // P) for n in _ints(case["lens"])]
    left = sum(n for b, n in enumerate(pages) if b % case["every"])
    # pages lie at random in the pool: a live one is past the live count with probability 1 - left / pool
    return {"bytes": 4 * case["layers"] * row * P * left * (1 - left / case["pool"]) + 8 * case["pool"] + 4 * sum(pages),
            "flops": 0}


# ----------------------------------------------------------------------------------------------- exact
def _exact_rows(q, k, v, visible):
    """One head: rows [R, D] against keys [n, D] in 64 bits, `visible` [R, n]; a block of rows at a time."""
    out = torch.empty_like(q)
    for r in range(0, q.shape[0], 4096):
        s = torch.einsum("rd,nd->rn", q[r:r + 4096], k) / math.sqrt(q.shape[1])
        s = torch.where(visible(r, min(q.shape[0], r + 4096)), s, -math.inf)
        p = torch.exp(s - s.max(1, keepdim=True).values)
        out[r:r + 4096] = torch.einsum("rn,nd->rd", p / p.sum(1, keepdim=True), v)
    return out


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "prompt":
        O = torch.zeros(st["O"].shape, dtype=torch.float64, device=DEV)
        G = case["Hq"] // case["Hkv"]
        cu = st["cu"].tolist()
        for a, e in zip(cu[:-1], cu[1:]):
            n = torch.arange(e - a, device=DEV)
            for h in range(case["Hq"] if e > a else 0):
                q, k, v = (x[a:e, y].double() for x, y in ((st["q"], h), (st["k"], h // G), (st["v"], h // G)))
                O[a:e, h] = _exact_rows(q, k, v, lambda r0, r1: n[None] <= n[r0:r1, None])
        return O
    if op == "prefix":
        B, N, Hq, D = st["q"].shape
        G, P, S = Hq // case["Hkv"], case["P"], case["shared"]
        O = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
        table, prefix = st["table"].tolist(), st["prefix"].tolist()
        for b, L in enumerate(st["L"].tolist()):
            pages = [prefix[x // P] if x < S else table[b][x // P] for x in range(0, L, 128)]
            k = torch.cat([st["Kp"][p, :, x % P:x % P + min(128, L - x)] for p, x in zip(pages, range(0, L, 128))] + [st["Kt"][b]], 1)
            v = torch.cat([st["Vp"][p, :, x % P:x % P + min(128, L - x)] for p, x in zip(pages, range(0, L, 128))] + [st["Vt"][b]], 1)
            see = torch.cat([torch.ones((N, L), dtype=torch.bool, device=DEV), st["mask"]], 1)
            for h in range(Hq):
                O[b, :, h] = _exact_rows(st["q"][b, :, h].double(), k[h // G].double(), v[h // G].double(),
                                         lambda r0, r1: see[r0:r1])
        return O
    P = case["P"]
    Kp, Vp = st["Kp"], st["Vp"]
    if op == "store":
        refs, table = st["refs0"].tolist(), st["table0"].tolist()
        free, cu = [p for p, n in enumerate(refs) if n == 0], st["cu"].tolist()
        for b, n in enumerate(_ints(case["lens"])):
            for i in range(-(-n // P)):
                page, rows = free.pop(0), min(P, n - i * P)
                a = cu[b] + i * P
                Kp[page, :, :rows] = st["k"][a:a + rows].transpose(0, 1)
                Vp[page, :, :rows] = st["v"][a:a + rows].transpose(0, 1)
                table[b][i], refs[page] = page, 1
        return {"Kp": Kp, "Vp": Vp, "table": _i32(table), "refs": _i32(refs), "flags": st["flags"]}
    table, refs, L = st["table0"].tolist(), st["refs0"].tolist(), st["L0"].tolist()
    if op == "fork":
        for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
            L[d] = L[s]
            for i in range(L[s] // P):
                table[d][i] = table[s][i]
                refs[table[s][i]] += 1
            if L[s] % P:
                new, old = refs.index(0), table[s][L[s] // P]
                table[d][L[s] // P], refs[new] = new, 1
                Kp[:, new, :, :L[s] % P] = Kp[:, old, :, :L[s] % P]
                Vp[:, new, :, :L[s] % P] = Vp[:, old, :, :L[s] % P]
        return {"Kp": Kp, "Vp": Vp, "table": _i32(table), "refs": _i32(refs), "L": _i32(L), "flags": st["flags"]}
    for b in st["done"].tolist():
        for p in table[b]:
            if p >= 0:
                refs[p] -= 1
        table[b], L[b] = [-1] * len(table[b]), 0
    n_live = sum(n > 0 for n in refs)
    page_map = [p if n > 0 else -1 for p, n in enumerate(refs)]
    holes = [p for p in range(n_live) if refs[p] == 0]
    for p in range(n_live, len(refs)):
        if refs[p] > 0:
            hole = holes.pop(0)
            page_map[p], refs[hole], refs[p] = hole, refs[p], 0
            Kp[:, hole], Vp[:, hole] = Kp[:, p], Vp[:, p]
    table = [[page_map[p] if p >= 0 else p for p in row] for row in table]
    return {"Kp": Kp, "Vp": Vp, "table": _i32(table), "refs": _i32(refs), "L": _i32(L), "page_map": _i32(page_map),
            "n_live": _i32([n_live])}
