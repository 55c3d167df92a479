"""medusa_pages_fork with thousands of forks: what is refused, and what checking them costs."""
import random

import pytest
import torch

from medusa_speculative_decoding_heads_gb300 import binding as mb

from _helpers import gpu_ready
from _serving import cfg_for, i32
from test_pages import Cache


@pytest.mark.gpu
@pytest.mark.parametrize("B", [60, 1024, 1025, 3000])
def test_refusals_among_many_forks(B):
    """Destinations named twice, that are sources, that hold pages; indices out of range on both sides."""
    c = Cache(B, 2, 2 * B, gpu_ready(), Hkv=1, D=64, layers=1, seed=B)
    held = B // 3
    rows = [1 + (37 * b) % 256 if b < held else 0 for b in range(B)]
    c.reserve(rows)
    c.lengths(rows)
    r = random.Random(B)
    for _ in range(2):
        src = [r.randrange(held) for _ in range(B)]
        dst = r.sample(range(held, B), B - held) + [r.randrange(B) for _ in range(held)]
        r.shuffle(dst)
        for i in r.sample(range(B), B // 10):
            src[i] = r.choice([-1, B, 2 ** 31 - 1, -2 ** 31, dst[r.randrange(B)]])
        for i in r.sample(range(B), B // 10):
            dst[i] = r.choice([-1, B, 2 ** 31 - 1, -2 ** 31, src[i], r.randrange(B)])
        c.fork(src, dst)
        c.free(r.sample(range(held, B), (B - held) // 2))


@pytest.mark.gpu
def test_time_goes_with_the_forks():
    """Eight times as many forks take about eight times as long (16 at most): a fork's check does not read all others."""
    dev = gpu_ready()

    def us(B):
        cfg, num = cfg_for(B, 1, 1, 64, torch.bfloat16, 512), 2 * B
        sources = B // 64
        table = torch.full((B, 4), -1, dtype=torch.int32, device=dev)
        table[:sources, :2] = torch.arange(2 * sources, dtype=torch.int32, device=dev).view(sources, 2)
        refs, L = torch.zeros(num, dtype=torch.int32, device=dev), torch.zeros(B, dtype=torch.int32, device=dev)
        refs[:2 * sources], L[:sources] = 1, 130
        n = B - sources
        src, dst = i32([i % sources for i in range(n)], dev), i32(list(range(sources, B)), dev)
        Kp = torch.zeros((num, 1, 128, 64), dtype=torch.bfloat16, device=dev)
        flags, ws = i32([9] * n, dev), torch.empty(mb.pages_workspace_size(cfg, num), dtype=torch.uint8, device=dev)
        a, e = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        best = float("inf")
        for _ in range(6):
            t, r, l = table.clone(), refs.clone(), L.clone()
            torch.cuda.synchronize()
            a.record()
            mb.pages_fork(cfg, Kp, Kp, num, 128, 1, Kp.numel(), n, src, dst, t, l, r, flags, ws)
            e.record()
            torch.cuda.synchronize()
            best = min(best, 1000 * a.elapsed_time(e))
        assert not bool(flags.any())
        return best

    few, many = us(2048), us(16384)
    assert many < 16 * few, (few, many)
