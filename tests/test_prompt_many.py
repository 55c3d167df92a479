"""medusa_prompt_attention on batches of more than 32 prompts: which unit is whose, and what finding that costs."""
import random

import pytest
import torch

from _helpers import gpu_ready
from _serving import cfg_for, i32
from test_prompt_attention import call, check, make
from medusa_speculative_decoding_heads_gb300 import binding as mb

BF16, F32 = torch.bfloat16, torch.float32


def patterns(B):
    r = random.Random(B)
    few = [r.randrange(3) for _ in range(B)]
    yield "random, zeros among them", [r.choice([0, 1, r.randrange(60), r.randrange(500)]) for _ in range(B)]
    yield "longer and longer", [1 + 3 * b % 700 for b in range(B)]
    yield "shorter and shorter", [1 + 3 * (B - b) % 700 for b in range(B)]
    yield "a long one first", [2100] + few[1:]
    yield "a long one last", few[1:] + [2100]
    yield "all of one tile", [64] * B
    yield "empty but for two", [0] * (B - 2) + [130, 1]
    yield "empty", [0] * B


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,Hq,Hkv", [(BF16, 128, 3, 3), (BF16, 64, 4, 1), (F32, 64, 4, 2), (F32, 128, 3, 1)])
@pytest.mark.parametrize("B", [33, 64, 65, 333])
def test_patterns(B, dtype, D, Hq, Hkv):
    dev = gpu_ready()
    for name, lens in patterns(B):
        q, k, v, cu = make(lens, Hq, Hkv, D, dtype, dev, seed=B, pad=3, first=2)
        check(q, k, v, cu, call(q, k, v, cu), name)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_time_goes_with_the_prompts(dtype, D):
    """Eight times as many short prompts take about eight times as long (12 at most): planning a unit does not
    read the whole batch."""
    dev = gpu_ready()

    def us(B):
        r = random.Random(1)
        lens = [r.randrange(1, 60) for _ in range(B)]
        q, k, v, cu = make(lens, 8, 4, D, dtype, dev, seed=1)
        cfg, cu, O = cfg_for(B, 8, 4, D, dtype), i32(cu, dev), torch.empty_like(q)
        run = lambda: mb.prompt_attention(cfg, q, k, v, q.shape[0], q.stride(0), k.stride(0), v.stride(0), cu, O)
        a, e = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        best = float("inf")
        for _ in range(5):
            a.record()
            for _ in range(20):
                run()
            e.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(e))
        return best * 50

    few, many = us(512), us(4096)
    assert many < 12 * few, (few, many)
