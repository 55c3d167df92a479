"""medusa_prompt_attention where visible scores are infinite: what the formula gives, in every type."""
import pytest
import torch

from oracle import serving_oracle as SO
from medusa_speculative_decoding_heads_gb300 import binding as mb

from _helpers import gpu_ready
from _serving import assert_within, tolerance
from test_prompt_attention import call, make

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("dead", [1, 70, 128, 200])
def test_rows_whose_scores_are_all_minus_infinity(dead, dtype, D):
    """The first `dead` keys of each prompt score -inf: rows that see only those are 0 / 0, no number; the
    others are as if those keys were not there."""
    dev = gpu_ready()
    lens = [dead, 300, dead + 1]
    q, k, v, cu = make(lens, 4, 2, D, dtype, dev, seed=dead)
    q[..., 0] = q[..., 0].abs() + 0.5
    clean = k.clone()
    for a, e in zip(cu[:-1], cu[1:]):
        k[a:min(a + dead, e), :, 0] = float("-inf")
    O = call(q, k, v, cu)
    for a, e in zip(cu[:-1], cu[1:]):
        n = min(dead, e - a)
        assert bool(O[a:a + n].isnan().all()), "rows without a finite score"
        if e - a > n:
            i = torch.arange(e - a, device=dev)
            see = (i[None] <= i[n:, None]) & (i[None] >= n)
            ref, A, S = SO.attend(q[a + n:e], clean[a:e], v[a:e], see)
            assert_within(O[a + n:e], ref, tolerance(dtype, ref, A, S, e - a), "rows behind them")
    assert mb.poll_errors() == (0, 0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64), (F32, 128)])
def test_a_score_of_infinity(dtype, D):
    """inf - inf: no number for the rows that see the key, the rows before it untouched."""
    dev = gpu_ready()
    q, k, v, cu = make([260], 4, 2, D, dtype, dev, seed=2)
    q[..., 0] = q[..., 0].abs() + 0.5
    clean = k.clone()
    k[150, :, 0] = float("inf")
    O = call(q, k, v, cu)
    ref, A, S = SO.prompt_attention(q, clean, v, cu)
    assert_within(O[:150], ref[:150], tolerance(dtype, ref, A, S, 260)[:150], "rows before the key")
    assert bool(O[150:].isnan().all())
    assert mb.poll_errors() == (0, 0, 0)
