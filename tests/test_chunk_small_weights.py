"""Float32 attention of new tokens where what is far below the maximum still counts, across the cuts of the work.

A weight of 2^-130 beside a value of 2e34 is an ordinary product in float32 (weights below 2^-126 lose bits, not
all of them). The kernel keeps such weights within a part of the keys; the parts' merge has to keep them, too.

Within a part weights are relative to the part's own maximum: its sums are those of the values themselves where that
is small, and 4000 rows of 2e34 (8e37) stay below float32's 3.4e38. (Rows of 1e37 do not: such a part overflows in
any order of the keys that meets their maximum before a larger one, so the sum of |V| is bounded in the call's contract.)
"""
import math

import pytest
import torch

from oracle import serving_oracle as SO

from _helpers import gpu_ready
from _serving import assert_within, tolerance
from test_chunk_attention import F32, Case


def loud(c, depth, dev):
    """Row 0 of each sequence scores 0 and holds small values; every other key scores 2^-depth of it and holds large ones."""
    gen = torch.Generator(device=dev).manual_seed(5)
    c.q.zero_()
    c.q[..., 0] = 4.0
    c.Kp.zero_()
    c.Kp[..., 0] = -depth * math.log(2.0) * math.sqrt(c.D) / 4.0
    c.Vp.copy_(2e34 * (0.5 + 0.5 * torch.rand(c.Vp.shape, generator=gen, device=dev)))
    for row in c.table:
        if 0 <= row[0] < c.num:
            c.Kp[row[0], :, 0], c.Vp[row[0], :, 0] = 0.0, 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,start", [([1], [4000]), ([100], [3000]), ([1, 70, 1], [2500, 900, 0])], ids=str)
@pytest.mark.parametrize("depth", [120.0, 130.0])
def test_weights_below_the_normal_range_count(depth, rows, start, D):
    dev = gpu_ready()
    c = Case(rows, start, 4, 2, D, F32, dev, seed=1)
    loud(c, depth, dev)
    O = c.call()
    ref, A, S, owned = SO.chunk_attention(c.q, c.Kp, c.Vp, c.P, c.table, c.cu, c.start, c.L_cap)
    assert float(ref[owned].max()) > 1.0 + 1e-2   # beside row 0's 1.0, from the small weights
    # A weight of 2^-130 lies on a grid of 2^-149: half a step of it, 2^-20 of the weight, for its exponential and
    # for at most two products with a change of the maximum, and 2 units of the last place (2^-18) that an
    # exponential may be off there: 2^-17 covers the sum.
    tol = tolerance(F32, ref, A, S, c.L_cap) + A * 2.0 ** -17
    assert_within(O[owned], ref[owned], tol[owned], f"2^-{depth:.0f} beside 2e34")
