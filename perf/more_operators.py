"""Cases of the norm and rotation of queries and keys, and of attention over a paged cache, with their plain forms.

Each case is one pass through an operator of the serving path: norms of queries and keys, each head by
itself, with the rotation by position; attention of a chunk of new tokens (or of single tokens) over
the pages of a cache; and the same with a sliding window and a few first rows that stay visible.
``run`` computes a case in elementary torch operations, or with ``own`` through the library's binding.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BRANCH = {7: "2,2", 22: "3,2,2", 65: "4,3,2,1", 111: "5,3,2,1,1"}   # nodes -> top-s per head
HEADS = [(32, 32), (32, 8), (40, 40), (8, 4), (16, 2), (12, 4), (28, 4), (20, 4), (6, 1), (16, 1)]
MOST_PAIRS = 2048 * (14336 + 1024.5) * 32 * 128   # (row, key) pairs times head dims of the largest attention case
MOST_KEYS = 3 << 26                               # keys times head dims of a case's pages


def _ints(text):
    return [int(x) for x in str(text).split(",") if x != ""]


def _text(values):
    return ",".join(str(int(v)) for v in values)


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi + 1))))))


def _ragged(rng, count, lo, hi):
    return [_log(rng, lo, hi) for _ in range(count)]


# ---------------------------------------------------------------------------------------------- cases
def listed():
    r = random.Random(51)
    return [
        # one user's next token, its query and key heads out of one fused projection: what counts is latency
        dict(name="rotate, 1 token", op="rotate", dtype="bf16", Hq=32, Hkv=8, D=128, T=1, N=0, rot=128, pairs=0, norm=3, fused=1,
             far=16384),
        # the trees of a batch on their way to tree attention, keys into their staged layout
        dict(name="rotate, 32 trees", op="rotate", dtype="bf16", Hq=32, Hkv=8, D=128, T=32 * 65, N=65, rot=128, pairs=0, norm=3,
             fused=1, far=16384),
        # a long prefill of a model with a key head for each query head
        dict(name="rotate, 8191 tokens", op="rotate", dtype="bf16", Hq=40, Hkv=40, D=128, T=8191, N=0, rot=128, pairs=0, norm=3,
             fused=1, far=8192),
        # the small float32 shape, half of each head rotated by neighbouring pairs, positions of a very long context
        dict(name="rotate, float32", op="rotate", dtype="f32", Hq=8, Hkv=4, D=64, T=3331, N=0, rot=32, pairs=1, norm=1, fused=0,
             far=1000000),
        # one token for each of a batch of conversations, a key head for each query head
        dict(name="chunk, 24 single tokens", op="chunk", dtype="bf16", Hq=40, Hkv=40, D=128, rows=_text([1] * 24),
             start=_text(_ragged(r, 23, 300, 4000) + [0]), P=128, pad=0, fused=1),
        # the same for the batch of the grouped-head workload, thousands of rows each
        dict(name="chunk, 32 tokens, grouped", op="chunk", dtype="bf16", Hq=32, Hkv=8, D=128, rows=_text([1] * 32),
             start=_text([r.randrange(4096, 16384) for _ in range(32)]), P=128, pad=0, fused=1),
        # the last part of a 16384-token prompt that is taken in chunks of 2048
        dict(name="chunk, 2048 after 14336", op="chunk", dtype="bf16", Hq=32, Hkv=8, D=128, rows="2048", start="14336", P=128,
             pad=0, fused=1),
        # a serving step that mixes parts of prompts with conversations, in a padded bucket
        dict(name="chunk, mixed step", op="chunk", dtype="bf16", Hq=32, Hkv=8, D=128,
             rows=_text([1] * 9 + [700, 0] + [1] * 6 + [37, 513, 1]),
             start=_text(_ragged(r, 9, 100, 8000) + [0, 900] + _ragged(r, 6, 100, 8000) + [2049, 1536, 127]), P=256, pad=45, fused=1),
        # the small float32 shape: parts of prompts and single tokens
        dict(name="chunk, float32", op="chunk", dtype="f32", Hq=8, Hkv=4, D=64, rows="129,1,700,1,0", start="600,1500,0,33,20", P=128,
             pad=0, fused=0),
        # single tokens whose layer sees the last 4096 rows and the first four
        dict(name="window, 32 single tokens", op="window", dtype="bf16", Hq=32, Hkv=8, D=128, rows=_text([1] * 32),
             start=_text(_ragged(r, 30, 100, 16000) + [4095, 4101]), P=128, pad=0, fused=1, window=4096, sinks=4),
        # a long prompt in one piece whose layer sees the last 1024 rows and the first four
        dict(name="window, 8192 tokens", op="window", dtype="bf16", Hq=32, Hkv=32, D=128, rows="8192", start="0", P=128, pad=0,
             fused=1, window=1024, sinks=4),
        # head dim 64, odd sizes: a window that ends inside a page, more first rows than a tile
        dict(name="window, odd sizes", op="window", dtype="bf16", Hq=12, Hkv=4, D=64, rows="333,1,65,0,1", start="1000,2999,0,77,150",
             P=128, pad=3, fused=0, window=201, sinks=131),
    ]


def draw(rng):
    op = rng.choice(["rotate", "chunk", "chunk", "window"])
    Hq, Hkv = rng.choice(HEADS)
    D = rng.choice([64, 128, 128])
    if op == "rotate":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        N = rng.choice([0, 0, 0] + sorted(BRANCH))
        T = N * rng.choice([1, 2, 3, 5, 8, 16, 32]) if N else _log(rng, 1, 4000 if dtype == "f32" else 8000)
        return dict(op=op, dtype=dtype, Hq=Hq, Hkv=Hkv, D=D, T=T, N=N, rot=rng.choice([D, D, D // 2, 8 * rng.randrange(0, D // 8 + 1)]),
                    pairs=rng.choice([0, 0, 1]), norm=rng.choice([3, 3, 2, 1, 0]), fused=rng.choice([0, 1]),
                    far=rng.choice([500, 16384, 131072, 1000000]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    P = rng.choice([128, 256])
    B = rng.choice([1, 1, 2, 3, 6, 11, 24, 40])
    most = MOST_PAIRS if dtype == "bf16" else MOST_PAIRS / 40   # (the largest float32 case is far smaller)
    rows, start = [], []
    for b in range(B):
        n = rng.choice([1, 1, 1, _log(rng, 1, 3000 if B < 4 else 700)])
        s = rng.choice([0, _log(rng, 1, 12000), _log(rng, 1, 3000)])
        while n * (s + n / 2) * Hq * D > most / B or (s + n) * Hkv * D > MOST_KEYS / B:
            n, s = max(1, n // 2), s // 2
        rows.append(n)
        start.append(s)
    if B > 2:
        rows[rng.randrange(B)] = 0
    case = dict(op=op, dtype=dtype, Hq=Hq, Hkv=Hkv, D=D, rows=_text(rows), start=_text(start), P=P, pad=rng.choice([0, 0, 1, 60]),
                fused=rng.choice([0, 1]))
    if op == "window":
        case.update(window=_log(rng, 1, 5000), sinks=rng.choice([0, 1, 4, 4, 64, 128, 200]))
    return case


# --------------------------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _normal(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(scale).to(dtype) if math.prod(shape) < 1 << 28 \
        else torch.randn(shape, generator=gen, device=DEV, dtype=dtype)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _offsets(rows):
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    return cu


def _width(case):
    """Block-table entries of a sequence: the longest one's pages, and one to spare."""
    return max(-(-(s + n) // case["P"]) for s, n in zip(_ints(case["start"]), _ints(case["rows"]))) + 1


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)
    Hq, Hkv, D, dt = case["Hq"], case["Hkv"], case["D"], _dtype(case)
    st = {"case": dict(case)}
    if case["op"] == "rotate":
        T, N, R = case["T"], case["N"], case["rot"]
        if case["fused"]:   # one projection's output: a row holds its q, k and v heads
            qkv = _normal(gen, (T, Hq + 2 * Hkv, D), dt, 1.5)
            q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        else:
            q, k = _normal(gen, (T, Hq, D), dt, 1.5), _normal(gen, (T, Hkv, D), dt, 1.5)
        # the trained weights of such norms are near one; a model without them has none
        qw, kw = ((1.0 + 0.2 * torch.randn(D, generator=gen, device=DEV)).to(dt) for _ in range(2))
        first = rng.randrange(max(1, case["far"] - T))
        pos = torch.arange(T, dtype=torch.int32, device=DEV) + first
        if N:   # trees: a length for each sequence, and a node's depth
            depth = torch.sort(torch.randint(0, 4, (T // N, N), generator=gen, device=DEV), 1).values
            pos = (torch.randint(0, case["far"], (T // N, 1), generator=gen, device=DEV) + depth).int().flatten()
        inv_freq = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / max(R, 1))).float()
        ko = (T // N, Hkv, N, D) if N else (T, Hkv, D)
        st.update(q=q, k=k, qw=qw if case["norm"] & 1 else None, kw=kw if case["norm"] & 2 else None, eps=1e-6, pos=pos.contiguous(),
                  inv_freq=inv_freq, qo=torch.zeros((T, Hq, D), dtype=dt, device=DEV), ko=torch.zeros(ko, dtype=dt, device=DEV))
        return st
    rows, start, P = _ints(case["rows"]), _ints(case["start"]), case["P"]
    B, T, width = len(rows), sum(rows) + case["pad"], _width(case)
    held = [-(-(s + n) // P) for s, n in zip(start, rows)]
    pool = sum(held) + 3
    ids = list(range(pool))
    rng.shuffle(ids)
    table, at = [[-1] * width for _ in range(B)], 0
    for b, n in enumerate(held):
        table[b][:n] = ids[at:at + n]
        at += n
    if case["fused"]:
        q = _normal(gen, (T, Hq + 2 * Hkv, D), dt, 2.0)[:, :Hq]
    else:
        q = _normal(gen, (T, Hq, D), dt, 2.0)
    st.update(rows=rows, first=start, q=q, cu=_i32(_offsets(rows)), start=_i32(start), table=_i32(table), pool=pool,
              Kp=_normal(gen, (pool, Hkv, P, D), dt), Vp=_normal(gen, (pool, Hkv, P, D), dt),
              O=torch.zeros((T, Hq, D), dtype=dt, device=DEV))
    return st


# ----------------------------------------------------------------------------------------- plain forms
def _plain_rotate(st):
    c = st["case"]
    R, half = c["rot"], c["rot"] // 2
    angle = st["pos"].double()[:, None] * st["inv_freq"].double()[None]   # in 64 bits: positions go far
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def one(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + st["eps"]) * w.float()
        r = y[..., :R]
        if c["pairs"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, y[..., R:]], -1).to(x.dtype)

    q, k = one(st["q"], st["qw"]), one(st["k"], st["kw"])
    if c["N"]:
        k = k.view(-1, c["N"], c["Hkv"], c["D"]).transpose(1, 2).contiguous()
    return q, k


def _plain_attention(st):
    c = st["case"]
    Hq, Hkv, D, P = c["Hq"], c["Hkv"], c["D"], c["P"]
    O, at = torch.zeros_like(st["O"]), 0
    for b, (n, s) in enumerate(zip(st["rows"], st["first"])):
        if n == 0:
            continue
        p = torch.arange(s, s + n, device=DEV)[:, None]
        j = torch.arange(s + n, device=DEV)
        if c["op"] == "window":   # what no row sees is not fetched
            j = j[(j < c["sinks"]) | (j > s - c["window"])]
        page = st["table"][b].long()[j // P]
        k = st["Kp"][page, :, j % P].float().permute(1, 2, 0)                          # [Hkv, D, keys]
        v = st["Vp"][page, :, j % P].float().transpose(0, 1)                           # [Hkv, keys, D]
        q = st["q"][at:at + n].float().transpose(0, 1).reshape(Hkv, (Hq // Hkv) * n, D) * (1.0 / math.sqrt(D))
        visible = j[None] <= p
        if c["op"] == "window":
            visible &= (j[None] > p - c["window"]) | (j[None] < c["sinks"])
        w = (q @ k).view(Hkv, Hq // Hkv, n, -1)
        w.masked_fill_(~visible, float("-inf"))
        w -= w.amax(-1, keepdim=True)
        w.exp_()
        o = (w.view(Hkv, (Hq // Hkv) * n, -1) @ v).view(Hkv, Hq // Hkv, n, D) / w.sum(-1, keepdim=True)
        O[at:at + n] = o.reshape(Hq, n, D).transpose(0, 1).to(O.dtype)
        at += n
    return O


# ------------------------------------------------------------------------------------- the library's calls
def _plan(st):
    """The configuration and workspace that a program keeps between calls."""
    from medusa_speculative_decoding_heads_gb300 import binding as mb
    c, N = st["case"], st["case"].get("N", 0)
    B = len(st["rows"]) if "rows" in st else c["T"] // N if N else 1
    cap = _width(c) * c["P"] if "rows" in st else max(c["far"], 128)
    branching = _ints(BRANCH[N]) if N else [1]
    cfg = mb.make_cfg(B=B, d=64, V=64, branching=branching, Hq=c["Hq"], Hkv=c["Hkv"], D=c["D"], L_cap=cap,
                      dtype=mb.F32 if c["dtype"] == "f32" else mb.BF16, mode=mb.GREEDY, tree_nodes=None if N else ([-1], [0]))
    size = mb.chunk_workspace_size(cfg, st["q"].shape[0]) if "rows" in st else 0
    st["mb"], st["cfg"], st["ws"] = mb, cfg, torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)


def _library(st):
    if "cfg" not in st:
        _plan(st)
    mb, cfg, c, q = st["mb"], st["cfg"], st["case"], st["q"]
    if c["op"] == "rotate":
        k, qo, ko = st["k"], st["qo"], st["ko"]
        mb.qk_norm_rotate(cfg, q, k, c["T"], q.stride(0), k.stride(0), st["qw"], st["kw"], st["eps"], st["inv_freq"], c["rot"],
                          mb.ROTATE_PAIRS if c["pairs"] else mb.ROTATE_HALVES, st["pos"], qo, ko, qo.stride(0),
                          0 if c["N"] else ko.stride(0))   # (0: the staged layout of the trees)
        return qo, ko
    args = (cfg, q, q.shape[0], q.stride(0), st["cu"], st["start"], st["Kp"], st["Vp"], st["pool"], c["P"], st["table"])
    if c["op"] == "window":
        mb.window_attention_paged(*args, c["window"], c["sinks"], st["O"], st["ws"])
    else:
        mb.chunk_attention_paged(*args, st["O"], st["ws"])
    return st["O"]


def run(state):
    if own:
        return _library(state)
    return _plain_rotate(state) if state["case"]["op"] == "rotate" else _plain_attention(state)


# ------------------------------------------------------------------------------------------------ work
def _pairs(n, s, window, sinks):
    """(row, key) pairs that rows s .. s + n - 1 see, and the keys that any of them sees."""
    if window is None:
        return n * s + n * (n + 1) // 2, s + n
    pairs = sum(min(p + 1, window + min(sinks, max(0, p + 1 - window))) for p in range(s, s + n))
    low = max(0, s - window + 1)
    return pairs, s + n - low + min(sinks, low)


def work(case):
    elt, Hq, Hkv, D = 4 if case["dtype"] == "f32" else 2, case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "rotate":
        heads = case["T"] * (Hq + Hkv)
        return {"bytes": 2 * heads * D * elt + 4 * case["T"] + 2 * case["rot"] + 2 * D * elt,
                "flops": heads * (5 * D * (case["norm"] != 0) + 3 * case["rot"])}
    seen = [_pairs(n, s, case.get("window"), case.get("sinks", 0)) for n, s in zip(_ints(case["rows"]), _ints(case["start"])) if n]
    return {"bytes": 2 * sum(_ints(case["rows"])) * Hq * D * elt + 2 * sum(k for _, k in seen) * Hkv * D * elt
            + 4 * sum(-(-k // case["P"]) for _, k in seen), "flops": 4 * D * Hq * sum(p for p, _ in seen)}


# ----------------------------------------------------------------------------------------------- exact
def _exact_rotate(case, st):
    def turn(x, w):
        out = x.double()
        if w is not None:
            size = torch.linalg.vector_norm(out, dim=-1, keepdim=True)
            out = out / torch.sqrt(size ** 2 / case["D"] + st["eps"]) * w.double()
        out = out.clone()
        for i in range(case["rot"] // 2):
            u, v = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + case["rot"] // 2)
            z = torch.polar(torch.ones_like(st["pos"], dtype=torch.float64), st["pos"].double() * float(st["inv_freq"][i]))
            z = torch.complex(out[..., u], out[..., v]) * z[:, None]
            out[..., u], out[..., v] = z.real, z.imag
        return out

    q, k = turn(st["q"], st["qw"]), turn(st["k"], st["kw"])
    if case["N"]:
        k = torch.stack([x.transpose(0, 1) for x in k.split(case["N"])])
    return q, k


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_rotate(case, st)
    O = torch.zeros(st["O"].shape, dtype=torch.float64, device=DEV)
    G, P, cu, table = case["Hq"] // case["Hkv"], case["P"], st["cu"].tolist(), st["table"].tolist()
    for b, s in enumerate(_ints(case["start"])):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        pages = table[b][:-(-(s + n) // P)]
        key = torch.arange(s + n, device=DEV)
        for h in range(case["Hkv"]):
            K, V = (torch.cat([pool[page, h] for page in pages])[:s + n].double() for pool in (st["Kp"], st["Vp"]))
            for g in range(G):
                for r in range(0, n, 2048):
                    e = min(n, r + 2048)
                    row = torch.arange(s + r, s + e, device=DEV)[:, None]
                    hidden = key > row
                    if case["op"] == "window":
                        hidden |= (key >= case["sinks"]) & (row - key >= case["window"])
                    logit = torch.einsum("rd,nd->rn", st["q"][cu[b] + r:cu[b] + e, h * G + g].double(), K) / math.sqrt(case["D"])
                    O[cu[b] + r:cu[b] + e, h * G + g] = torch.softmax(torch.where(hidden, -math.inf, logit), 1) @ V
    return O

