"""medusa_tree_attention_prefix: what a row does not see does not reach it."""
import pytest
import torch

from medusa_speculative_decoding_heads_gb300 import binding as mb

from _helpers import gpu_ready
from _serving import cfg_for
from test_prefix_attention import Case


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,B", [(8, 2, 3), (8, 8, 24), (16, 8, 24)])
@pytest.mark.parametrize("shared", [0, 256])
def test_bits_past_the_last_node(shared, Hq, Hkv, B):
    """Mask bits from N on name no key: single tokens (on both kernels), 7 and 65 nodes."""
    dev = gpu_ready()
    for branching in ((1,), (2, 2), (4, 3, 2, 1)):
        c = Case([shared + 17 * b for b in range(B)], shared, 128, Hq, Hkv, branching, dev, seed=B, L_cap=1024)
        word = torch.arange(128, device=dev).view(2, 64) >= c.N
        extra = [sum(1 << j for j in range(64) if word[w, j]) for w in (0, 1)]
        c.bits |= torch.tensor([x - (1 << 64) if x >> 63 else x for x in extra], dtype=torch.int64, device=dev)
        c.check(c.call(), f"{c.N} nodes")


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,B", [(8, 2, 5), (8, 8, 24), (16, 8, 24), (32, 8, 24)])
@pytest.mark.parametrize("branching", [(1,), (2, 2), (4, 3, 2, 1)], ids=str)
@pytest.mark.parametrize("most", [0, 1, 100, 128, 300, 511])
def test_shared_rows_that_no_sequence_has(most, branching, Hq, Hkv, B):
    """Every length below the shared rows (but for sequences that do not count): the rest of the prefix's
    pages holds no numbers, as memory that nothing was stored in yet."""
    dev = gpu_ready()
    L = [most - (37 * b) % (most + 1) for b in range(B)]
    L[1], L[3] = -1, 1025
    c = Case(L, 512, 128, Hq, Hkv, branching, dev, seed=most, L_cap=1024)
    for i in range(most, 512):
        page = c.prefix[i // 128]
        c.Kp[page, :, i % 128], c.Vp[page, :, i % 128] = float("nan"), float("inf") if i % 2 else float("nan")
    O = c.call()
    assert bool((O[1] == 0).all()) and bool((O[3] == 0).all())
    c.check(O)


@pytest.mark.gpu
@pytest.mark.parametrize("shared", [0, 256])
@pytest.mark.parametrize("Hq,Hkv,B", [(8, 2, 4), (8, 8, 24)])
def test_nodes_that_hold_no_numbers(shared, Hq, Hkv, B):
    """A node's key reaches the rows that see it and no others; its value stays within its sequence."""
    dev = gpu_ready()
    c = Case([shared + 40 * b for b in range(B)], shared, 128, Hq, Hkv, (2, 2), dev, seed=B + shared, L_cap=shared + 1024)
    O0 = c.call()
    c.check(O0)
    Kt, Vt = c.Kt.clone(), c.Vt.clone()
    c.Kt[0, :, 2], c.Kt[1, :, 4] = float("nan"), float("inf")
    c.Vt[2, :, 2] = float("nan")
    O = c.call()
    c.Kt, c.Vt = Kt, Vt
    for b, node in ((0, 2), (1, 4)):
        sees = c.mask[:, node].to(dev)
        assert torch.equal(O[b, ~sees], O0[b, ~sees])
        assert not bool(torch.isfinite(O[b, sees]).all(-1).any())
    assert bool(O[2, c.mask[:, 2].to(dev)].isnan().all())
    for b in range(3, B):
        assert torch.equal(O[b], O0[b])


@pytest.mark.gpu
@pytest.mark.parametrize("shared", [0, 256])
def test_a_child_that_holds_no_numbers(shared):
    """Single tokens' kernel with two nodes: the root does not see its child, neither key nor value."""
    dev = gpu_ready()
    c = Case([shared + 21 * b for b in range(20)], shared, 128, 8, 8, (1,), dev, seed=shared + 2, L_cap=shared + 512)
    c.N, c.mask = 2, torch.tensor([[True, False], [True, True]])
    c.bits = torch.tensor([[1, 0], [3, 0]], dtype=torch.int64, device=dev)
    gen = torch.Generator(device=dev).manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=gen, device=dev).to(torch.bfloat16)
    c.Q, c.Kt, c.Vt = rnd(20, 2, 8, 128) * 2, rnd(20, 8, 2, 128), rnd(20, 8, 2, 128)
    c.cfg = cfg_for(20, 8, 8, 128, torch.bfloat16, shared + 512, (1,), tree_nodes=([-1, 0], [0, 0]))
    c.ws = torch.full((max(mb.prefix_workspace_size(c.cfg, shared), 256),), 255, dtype=torch.uint8, device=dev)
    O0 = c.call()
    c.check(O0)
    c.Kt[3, :, 1], c.Vt[4, :, 1] = float("nan"), float("nan")
    O = c.call()
    assert torch.equal(O[:, 0], O0[:, 0])
    assert bool(O[3:5, 1].isnan().all()) and torch.equal(O[5:], O0[5:]) and torch.equal(O[:3], O0[:3])


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,B,branching", [(8, 2, 3, (2, 2)), (8, 2, 3, (1,)), (8, 8, 24, (1,)), (16, 8, 24, (1,))])
def test_rows_whose_scores_are_all_minus_infinity(Hq, Hkv, B, branching):
    """A sequence whose every key scores -inf gets zeros, the others are unharmed (both kernels)."""
    dev = gpu_ready()
    c = Case([300 + 5 * b for b in range(B)], 0, 128, Hq, Hkv, branching, dev, seed=B, L_cap=1024)
    c.Q[..., 0] = c.Q[..., 0].abs() + 0.5
    O0 = c.call()
    c.check(O0)
    for page in c.table[1]:
        if page >= 0:
            c.Kp[page, ..., 0] = float("-inf")
    c.Kt[1, ..., 0] = float("-inf")
    O = c.call()
    assert bool((O[1] == 0).all())
    assert torch.equal(O[0], O0[0]) and torch.equal(O[2:], O0[2:])
