"""Pages of a cache: reserve, store, fork, free and compact, bit for bit against one-page-at-a-time lists."""
import ctypes
import random

import pytest
import torch

from medusa_speculative_decoding_heads_gb300 import _build, binding as mb
from oracle import serving_oracle as SO

from _helpers import gpu_ready
from _serving import cfg_for, i32, offsets

BF16, F32 = torch.bfloat16, torch.float32


class Cache:
    """Device tables and pools beside the oracle's, both driven by the same operations."""

    def __init__(self, B, width, num, dev, P=128, Hkv=2, D=64, dtype=BF16, layers=2, seed=0):
        gen = torch.Generator(device=dev).manual_seed(seed)
        self.B, self.num, self.P, self.layers, self.dev = B, num, P, layers, dev
        self.cfg = cfg_for(B, Hkv, Hkv, D, dtype, width * P)
        rnd = lambda: torch.randn((layers, num, Hkv, P, D), generator=gen, device=dev).to(dtype)
        self.Kp, self.Vp = rnd(), rnd()
        self.o = SO.Pages([[-1] * width for _ in range(B)], [0] * num, [0] * B, P, (self.Kp, self.Vp))
        self.table, self.refs, self.L = i32(self.o.table, dev), i32(self.o.refs, dev), i32(self.o.L, dev)
        self.ws = torch.full((mb.pages_workspace_size(self.cfg, num),), 255, dtype=torch.uint8, device=dev)
        self.rng = random.Random(seed)

    def set(self, table=None, refs=None, L=None):
        if table is not None:
            self.o.table = [list(r) for r in table]
        if refs is not None:
            self.o.refs = list(refs)
        if L is not None:
            self.o.L = list(L)
        self.table, self.refs, self.L = i32(self.o.table, self.dev), i32(self.o.refs, self.dev), i32(self.o.L, self.dev)

    def same(self, what=""):
        assert self.table.tolist() == self.o.table, what
        assert self.refs.tolist() == self.o.refs, what
        assert self.L.tolist() == self.o.L, what
        assert torch.equal(self.Kp, self.o.pools[0]) and torch.equal(self.Vp, self.o.pools[1]), what

    def reserve(self, rows):
        flags = torch.full((self.B,), 99, dtype=torch.int32, device=self.dev)
        mb.pages_reserve(self.cfg, self.num, self.P, i32(rows, self.dev), self.table, self.refs, flags, self.ws)
        assert flags.tolist() == self.o.reserve(rows)
        self.same(f"reserve {rows}")

    def fork(self, src, dst):
        flags = torch.full((max(len(src), 1),), 99, dtype=torch.int32, device=self.dev)
        mb.pages_fork(self.cfg, self.Kp, self.Vp, self.num, self.P, self.layers, self.Kp.stride(0), len(src),
                      i32(src, self.dev), i32(dst, self.dev), self.table, self.L, self.refs, flags, self.ws)
        assert flags.tolist()[:len(src)] == self.o.fork(src, dst), (src, dst)
        self.same(f"fork {src} -> {dst}")

    def free(self, seqs):
        mb.pages_free(self.cfg, self.num, self.P, len(seqs), i32(seqs, self.dev), self.table, self.L, self.refs)
        self.o.free(seqs)
        self.same(f"free {seqs}")

    def compact(self):
        page_map, n_live = i32([99] * self.num, self.dev), i32([99], self.dev)
        mb.pages_compact(self.cfg, self.Kp, self.Vp, self.num, self.P, self.layers, self.Kp.stride(0), self.table, self.refs,
                         page_map, n_live, self.ws)
        want_map, want_live = self.o.compact()
        assert page_map.tolist() == want_map and n_live.tolist() == [want_live]
        self.same("compact")

    def lengths(self, L):
        """The caller's own part: lengths after rows were stored."""
        self.o.L = list(L)
        self.L.copy_(i32(L, self.dev))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,P,Hkv", [(BF16, 128, 128, 2), (BF16, 64, 256, 3), (F32, 64, 128, 1), (F32, 128, 256, 2)])
def test_a_life_of_a_cache(dtype, D, P, Hkv):
    """Sequences come, fork, leave and are compacted, at random; every state equals the oracle's."""
    c = Cache(9, 5, 40, gpu_ready(), P=P, Hkv=Hkv, D=D, dtype=dtype, layers=3, seed=D + P)
    r = c.rng
    for step in range(25):
        empty = [b for b in range(c.B) if c.o.L[b] == 0 and all(p < 0 for p in c.o.table[b])]
        held = [b for b in range(c.B) if c.o.L[b] > 0]
        what = r.choice(["reserve", "fork", "free", "compact"])
        if what == "reserve":
            rows = [min(5 * P, c.o.L[b] + r.choice([0, 1, P, 2 * P - 1])) if r.random() < 0.6 else 0 for b in range(c.B)]
            c.reserve(rows)
            # each sequence now fills what it holds, up to what it asked for
            room = [next((i for i, p in enumerate(row) if p < 0), len(row)) * P for row in c.o.table]
            c.lengths([max(c.o.L[b], min(rows[b], room[b])) for b in range(c.B)])
        elif what == "fork" and held and empty:
            n = r.randrange(1, len(empty) + 1)
            c.fork([r.choice(held) for _ in range(n)], r.sample(empty, n))
        elif what == "free" and held:
            c.free([r.choice(held) for _ in range(r.randrange(1, 4))])
        else:
            c.compact()


@pytest.mark.gpu
def test_fork_lengths():
    """Zero rows, one row, a full page, one more, a full table."""
    c = Cache(12, 3, 20, gpu_ready(), seed=1)
    c.reserve([0, 1, 128, 129, 384, 0, 0, 0, 0, 0, 0, 0])
    c.lengths([0, 1, 128, 129, 384] + [0] * 7)
    c.fork([0, 1, 2, 3, 4, 3], [5, 6, 7, 8, 9, 11])
    c.fork([8], [10])            # a fork of a fork
    c.free([3, 8, 8, 1])
    c.compact()


@pytest.mark.gpu
def test_fork_refusals_on_the_device():
    """Each bad fork is refused for itself; the good ones beside it go through."""
    c = Cache(10, 3, 12, gpu_ready(), seed=2)
    c.reserve([200, 130, 0, 0, 0, 0, 0, 0, 0, 50])
    c.lengths([200, 130, 0, 0, 0, 0, 0, 0, 0, 50])
    c.fork([0, 0, -1, 10, 0, 0, 1, 2, 0, 0], [2, 3, 4, 5, -1, 10, 6, 7, 6, 1])
    c.fork([0, 1, 0], [4, 5, 4])
    c.fork([3], [3])
    c.fork([], [])
    c.lengths([200, 130, 0, 200, 0, 130, 0, 0, 0, 50])
    c.o.L[9] = 500               # longer than the table
    c.L.copy_(i32(c.o.L, c.dev))
    c.fork([9, 0], [4, 7])
    c.o.table[1][0] = 12         # a page past the pool
    c.table.copy_(i32(c.o.table, c.dev))
    c.fork([1, 0], [6, 8])


@pytest.mark.gpu
def test_out_of_pages():
    """Forks and reservations are served in order until the free pages end."""
    c = Cache(8, 4, 7, gpu_ready(), seed=3)
    c.reserve([100, 256, 0, 0, 0, 0, 0, 0])
    c.lengths([100, 256, 0, 0, 0, 0, 0, 0])
    c.fork([0, 1, 0, 0, 0, 0], [2, 3, 4, 5, 6, 7])     # four free pages: the fifth fork with a part page fails
    c.free([5])
    c.reserve([512, 300, 100, 0, -1, 513, 0, 0])
    c.reserve([100, 300, 100, 0, 0, 0, 0, 0])
    c.compact()
    c.free([0, 1, 2, 3, 4, 5, 6, 7])
    c.compact()
    assert c.o.refs == [0] * 7


@pytest.mark.gpu
def test_many_sequences():
    """More sequences, forks and free pages than the planning kernels' lists in shared memory hold."""
    c = Cache(2600, 2, 5000, gpu_ready(), Hkv=1, D=64, layers=1, seed=6)
    rows = [(37 * b) % 257 if b < 1100 else 0 for b in range(2600)]
    c.reserve(rows)
    c.lengths(rows)
    dst = list(range(1100, 2600))
    c.fork([(7 * i) % 1100 for i in range(1500)], dst)
    c.reserve([256] * 2600)                # more than there are: in order, until the free pages end
    c.free(list(range(0, 2600, 2)) + [4, 4])
    c.compact()
    c.reserve([200] * 2600)


@pytest.mark.gpu
def test_compact_many_pages():
    """More pages than one step of the scan takes, and no page in use or every page in use."""
    dev = gpu_ready()
    num, P = 20011, 128
    c = Cache(3, 8000, num, dev, P=P, Hkv=1, D=64, layers=1, seed=4)
    ids = list(range(num))
    c.rng.shuffle(ids)
    lens = [7000, 1, 4001]
    table, at, refs = [], 0, [0] * num
    for n in lens:
        table.append(ids[at:at + n] + [-1] * (8000 - n))
        for p in ids[at:at + n]:
            refs[p] = 1
        at += n
    table[1][1:3], table[1][3] = table[0][:2], num + 7      # shared pages; an id past the pool stays
    refs[table[0][0]], refs[table[0][1]] = 2, 2
    table[2][4001] = next(p for p in range(num) if refs[p] == 0)   # held without a reference: becomes -1
    c.set(table, refs, [7000 * P, 3 * P, 4001 * P])
    c.compact()
    c.compact()                                             # already compact: nothing moves
    c.reserve([7000 * P, 0, 8000 * P])
    c.set([[-1] * 8000 for _ in range(3)], [0] * num, [0] * 3)
    c.compact()
    full = Cache(1, 9, 9, dev, seed=5)
    full.reserve([9 * 128])
    full.compact()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,Hkv", [(BF16, 128, 2), (BF16, 64, 1), (F32, 64, 3), (F32, 128, 8)])
@pytest.mark.parametrize("start", [None, [0, 5, 120, 0, 250]])
def test_store(dtype, D, Hkv, start):
    """Packed rows land where their tables say; strided sources, empty sequences, rows past the table."""
    dev = gpu_ready()
    lens = [130, 1, 0, 300, 140]
    c = Cache(5, 3, 20, dev, D=D, Hkv=Hkv, dtype=dtype, layers=1, seed=6)
    c.reserve([384] * 5)
    cu = offsets(lens, 4)
    T = cu[-1] + 9
    kv = torch.randn((T, 2, Hkv, D), device=dev).to(dtype)
    k, v = kv[:, 0], kv[:, 1]
    mb.kv_store_paged(c.cfg, k, v, T, k.stride(0), v.stride(0), i32(cu, dev), None if start is None else i32(start, dev),
                      c.Kp, c.Vp, c.num, c.P, c.table)
    c.o.store(k, v, cu, start)
    c.same("store")


@pytest.mark.gpu
def test_pages_past_32_bit_offsets():
    """Pools of more than 2^31 elements a layer: a store, a fork and a compaction at their far end."""
    dev = gpu_ready()
    num = 16500
    c = Cache(3, 4, 4, dev, Hkv=8, D=128, layers=1, seed=12)
    c.num, c.o.refs = num, [1] * (num - 6) + [0] * 6     # all but the last pages belong to others
    c.Kp, c.Vp = (torch.zeros((1, num, 8, 128, 128), dtype=BF16, device=dev) for _ in range(2))
    assert c.Kp.numel() > 2 ** 31
    c.o.pools = [c.Kp.clone(), c.Vp.clone()]
    c.set()
    c.ws = torch.empty(mb.pages_workspace_size(c.cfg, num), dtype=torch.uint8, device=dev)
    c.reserve([300, 0, 0])
    k, v = (torch.randn((300, 8, 128), device=dev).to(BF16) for _ in range(2))
    mb.kv_store_paged(c.cfg, k, v, 300, 1024, 1024, i32([0, 300, 300, 300], dev), None, c.Kp, c.Vp, num, c.P, c.table)
    c.o.store(k, v, [0, 300, 300, 300], None)
    c.lengths([300, 0, 0])
    c.same("store")
    c.fork([0], [2])
    c.o.refs[5] = c.o.refs[16000] = 0
    c.set()
    c.compact()


@pytest.mark.gpu
def test_store_skips_what_it_may_not_write():
    """Negative and far starts, pages outside the pool, offsets past T or decreasing: nothing else changes."""
    dev = gpu_ready()
    c = Cache(5, 2, 10, dev, layers=1, seed=7)
    c.reserve([256, 256, 256, 256, 0])
    c.o.table[2] = [10, -7]
    c.set(table=c.o.table)
    k, v = (torch.randn((90, 2, 64), device=dev).to(BF16) for _ in range(2))
    for cu, start in (([0, 10, 40, 50, 60, 90], [250, -5, 0, 2 ** 31 - 3, 0]), ([0, 10, 40, 50, 60, 95], None),
                      ([-3, 10, 40, 50, 60, 90], None)):
        mb.kv_store_paged(c.cfg, k, v, 90, 128, 128, i32(cu, dev), None if start is None else i32(start, dev), c.Kp, c.Vp,
                          c.num, c.P, c.table)
        c.o.store(k, v, cu, start)
        c.same(f"store {cu} {start}")


@pytest.mark.gpu
def test_captured_turnover():
    """Free, reserve, fork and compact captured in one graph; replays act on the tables as they then are."""
    dev = gpu_ready()
    c = Cache(6, 4, 30, dev, seed=8)
    rows, src, dst, gone = i32([300, 200, 0, 0, 0, 0], dev), i32([0, 1], dev), i32([2, 3], dev), i32([2, 3, 4], dev)
    flags, f2 = torch.zeros(6, dtype=torch.int32, device=dev), torch.zeros(2, dtype=torch.int32, device=dev)
    page_map, n_live = i32([0] * 30, dev), i32([0], dev)
    stride = c.Kp.stride(0)

    def turn():
        mb.pages_free(c.cfg, c.num, c.P, 3, gone, c.table, c.L, c.refs)
        mb.pages_reserve(c.cfg, c.num, c.P, rows, c.table, c.refs, flags, c.ws)
        mb.pages_fork(c.cfg, c.Kp, c.Vp, c.num, c.P, c.layers, stride, 2, src, dst, c.table, c.L, c.refs, f2, c.ws)
        mb.pages_compact(c.cfg, c.Kp, c.Vp, c.num, c.P, c.layers, stride, c.table, c.refs, page_map, n_live, c.ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        turn()
    c.lengths([300, 200, 0, 0, 0, 0])
    for want in ([300, 200, 0, 0, 0, 0], [384, 10, 0, 500, 0, 0]):
        rows.copy_(i32(want, dev))
        c.lengths([300, 200] + c.o.L[2:])
        g.replay()
        c.o.free([2, 3, 4])
        c.o.reserve(want)
        c.o.fork([0, 1], [2, 3])
        c.o.compact()
        c.same(f"replayed {want}")


# ----------------------------------------------------------------------------- refusals (no GPU)
def fake(**off):
    return lambda name: ctypes.c_void_p(off.get(name, 4096)) if off.get(name, 4096) else None


def call(which, num=9, P=128, layers=2, elems=None, n=1, L_cap=512, dtype=BF16, T=4, stride=128, **off):
    _build.build()
    lib, cfg, p = mb.load(), cfg_for(3, 2, 2, 64, dtype, L_cap), fake(**off)
    elems = num * 2 * P * 64 if elems is None else elems
    c = ctypes.byref(cfg)
    if which == "reserve":
        return lib.medusa_pages_reserve(c, num, P, p("rows"), p("table"), p("refs"), p("flags"), p("ws"), None)
    if which == "fork":
        return lib.medusa_pages_fork(c, p("Kp"), p("Vp"), num, P, layers, elems, n, p("src"), p("dst"), p("table"), p("L"),
                                     p("refs"), p("flags"), p("ws"), None)
    if which == "free":
        return lib.medusa_pages_free(c, num, P, n, p("seqs"), p("table"), p("L"), p("refs"), None)
    if which == "compact":
        return lib.medusa_pages_compact(c, p("Kp"), p("Vp"), num, P, layers, elems, p("table"), p("refs"), p("map"),
                                        p("live"), p("ws"), None)
    return lib.medusa_kv_store_paged(c, p("K"), p("V"), T, stride, stride, p("cu"), None, p("Kp"), p("Vp"), num, P,
                                     p("table"), None)


NEEDS = {"reserve": ["rows", "table", "refs", "flags", "ws"],
         "fork": ["Kp", "Vp", "src", "dst", "table", "L", "refs", "flags", "ws"],
         "free": ["seqs", "table", "L", "refs"], "compact": ["Kp", "Vp", "table", "refs", "map", "live", "ws"],
         "store": ["K", "V", "cu", "Kp", "Vp", "table"]}


@pytest.mark.parametrize("which", sorted(NEEDS))
def test_refusals(which):
    for name in NEEDS[which]:
        assert call(which, **{name: 0}) == -1, name
    for name in {"Kp", "Vp", "K", "V", "ws"} & set(NEEDS[which]):
        assert call(which, **{name: 4104}) == -1, name
    assert call(which, num=0) == -1
    assert call(which, P=64) == -2 and call(which, P=192) == -2 and call(which, P=384) == -2


def test_more_refusals():
    for which in ("fork", "compact"):
        assert call(which, layers=0) == -1
        assert call(which, elems=9 * 2 * 128 * 64 - 8) == -1       # layers would overlap
        assert call(which, elems=9 * 2 * 128 * 64 + 4) == -1       # not whole 16-byte words
    assert call("fork", n=-1) == -1 and call("fork", n=4) == -1 and call("free", n=-1) == -1
    assert call("fork", n=0, src=0, dst=0) == 0 and call("free", n=0, seqs=0) == 0
    assert call("store", T=-1) == -1 and call("store", T=0, K=0, V=0, cu=0) == 0
    assert call("store", stride=127) == -1 and call("store", stride=132) == -1
    size = ctypes.c_size_t()
    cfg = cfg_for(3, 2, 2, 64, BF16)
    assert mb.raw_call("medusa_pages_workspace_size", ctypes.byref(cfg), 9, ctypes.byref(size)) == 0 and size.value > 0
    assert mb.raw_call("medusa_pages_workspace_size", ctypes.byref(cfg), 0, ctypes.byref(size)) == -1
    assert mb.raw_call("medusa_pages_workspace_size", ctypes.byref(cfg), 9, None) == -1


# ----------------------------------------------------------------------------- the lists themselves (no GPU)
def test_lists_keep_their_invariants():
    """Reference counts equal the table entries that name a page, whatever the order of operations."""
    rng = random.Random(5)
    for _ in range(30):
        o = SO.Pages([[-1] * 6 for _ in range(7)], [0] * 25, [0] * 7, 4, (torch.randn(1, 25, 1, 4, 2),))
        for _ in range(40):
            b = rng.randrange(7)
            kind = rng.randrange(4)
            if kind == 0:
                rows = [0] * 7
                rows[b] = rng.randrange(25)
                if o.reserve(rows)[b] == 0:
                    o.L[b] = max(o.L[b], rows[b])
            elif kind == 1:
                o.fork([b, b], [(b + 1) % 7, (b + 2) % 7])
            elif kind == 2:
                o.free([b, b])
            else:
                before = [[o.pools[0][0, p].clone() if p >= 0 else None for p in row] for row in o.table]
                _, live = o.compact()
                assert all(p < live for row in o.table for p in row)
                for row, old in zip(o.table, before):
                    for p, data in zip(row, old):
                        assert data is None or torch.equal(o.pools[0][0, p], data)
            for page in range(25):
                assert o.refs[page] == sum(row.count(page) for row in o.table)
