"""medusa_tree_attention_prefix in caches with room for far more rows than the sequences have."""
import pytest
import torch

from _helpers import gpu_ready
from test_prefix_attention import Case


def capped(L, L_cap, branching, Hq, Hkv, dev, shared=256, seed=1):
    """The same batch whatever L_cap: rows, tree and pages are drawn before the capacity matters."""
    c = Case(L, shared, 128, Hq, Hkv, branching, dev, seed=seed, L_cap=L_cap)
    gen = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device=dev).to(torch.bfloat16)
    c.Q, c.Kt, c.Vt = rnd(*c.Q.shape) * 2, rnd(*c.Kt.shape), rnd(*c.Vt.shape)
    for b, n in enumerate(L):
        for i in range(0, n, 128):
            page = c.prefix[i // 128] if i < shared else c.table[b][i // 128]
            c.Kp[page], c.Vp[page] = rnd(Hkv, 128, 128), rnd(Hkv, 128, 128)
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("branching", [(1,), (4, 3, 2, 1)], ids=str)
def test_results_do_not_depend_on_the_capacity(branching):
    """A sequence's rows are divided by what it has: as long as as many ranges are planned, the bits are the same."""
    dev = gpu_ready()
    outs = []
    for L_cap in (8192, 16384, 65536):
        c = capped([3300], L_cap, branching, 32, 8, dev)
        outs.append(c.call())
        c.check(outs[-1], f"capacity {L_cap}")
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.gpu
@pytest.mark.parametrize("branching,Hq,Hkv", [((1,), 8, 2), ((1,), 8, 8), ((4, 3, 2, 1), 8, 2), ((2, 2), 12, 4)])
def test_lengths_far_below_the_capacity(branching, Hq, Hkv):
    """Lengths around each border of the ranges: nothing, one key, one range, a few, the whole cache."""
    dev = gpu_ready()
    N = {(1,): 1, (4, 3, 2, 1): 65, (2, 2): 7}[branching]
    L = [0, 1, 100, 256, 257, 383, 384, 385, 512, 513, 767, 768, 769, 3000, 8192 - N]
    c = Case(L, 256, 128, Hq, Hkv, branching, dev, seed=2, poison=True, L_cap=8192)
    c.check(c.call())
    c = Case(L[1:6] + [8192 - N + 1], 256, 128, Hq, Hkv, branching, dev, seed=3, L_cap=8192)
    O = c.call()
    assert bool((O[5] == 0).all())
    c.check(O)
