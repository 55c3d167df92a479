"""medusa_tree_attention_prefix: what a row does not see does not reach it."""
import pytest
import torch

from _helpers import gpu_ready
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
