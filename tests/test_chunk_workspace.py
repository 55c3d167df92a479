"""The workspace of attention of new tokens: what it has to hold, and calls that find another call's results in it."""
import pytest
import torch

from medusa_speculative_decoding_heads_gb300 import _build, binding as mb

from _helpers import gpu_ready
from _serving import cfg_for
from test_chunk_attention import BF16, F32, KINDS, Case


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (4, 1, 128), (28, 4, 128), (96, 1, 64), (40, 40, 128)])
def test_more_rows_never_need_less(Hq, Hkv, D, dtype):
    _build.build()
    cfg = cfg_for(3, Hq, Hkv, D, dtype)
    sizes = [mb.chunk_workspace_size(cfg, T) for T in list(range(0, 300)) + [511, 512, 4096, 1 << 20]]
    assert sizes[0] == 0 and sizes[1] > 0 and sizes == sorted(sizes) and all(n % 256 == 0 for n in sizes)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (3, 3)])
def test_calls_of_many_shapes_share_one_workspace(Hq, Hkv, dtype, D):
    """Larger calls' cuts and partial results lie where smaller calls have theirs; bytes past a call's own size stay."""
    dev = gpu_ready()
    shapes = [([700, 1, 1, 300], [2000, 900, 0, 5]), ([1], [3000]), ([1, 1, 1], [100, 4000, 7]), ([2], [0]), ([90, 90], [700, 0]),
              ([0, 5, 0], [3, 1300, 4]), ([1] * 40, [50 * b for b in range(40)])]
    cases = [Case(rows, start, Hq, Hkv, D, dtype, dev, seed=i, window=(None, 300)[i % 2], sinks=4 if i % 2 else 0)
             for i, (rows, start) in enumerate(shapes)]
    want = [c.call() for c in cases]
    sizes = [mb.chunk_workspace_size(c.cfg, c.T) for c in cases]
    space = torch.full((max(sizes) + 4096,), 0xA5, dtype=torch.uint8, device=dev)
    for order in (range(len(cases)), reversed(range(len(cases))), (0, 1, 0, 6, 0, 2, 4, 3)):
        for i in order:
            space[sizes[i]:] = 0xA5
            O = cases[i].call(ws=space)
            assert torch.equal(O, want[i]), shapes[i]
            assert bool((space[sizes[i]:] == 0xA5).all()), "bytes past the workspace were written"
    for c, w in zip(cases, want):
        c.check(w)
