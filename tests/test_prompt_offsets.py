"""Offsets of packed prompts that decrease somewhere: prompts ahead of that are computed, none behind it."""
import pytest
import torch

from oracle import serving_oracle as SO
from medusa_speculative_decoding_heads_gb300 import binding as mb

from _helpers import gpu_ready
from _serving import assert_within, i32, tolerance
from test_pages import Cache
from test_prompt_attention import call, make

BF16, F32 = torch.bfloat16, torch.float32

CUTS = [[0, 3000, 10, 3000], [0, 0, 700, 3000, 2999, 3000, 0, 3000], [0, 3000] * 9, [5, 4, 3000],
        list(range(0, 2000, 50)) + [2500, 60, 3000], list(range(0, 3000, 20)) + [0] + list(range(0, 3000, 40)) + [2999]]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("cu", CUTS, ids=lambda c: f"{len(c)}-{c[1]}")
def test_prompts_ahead_of_a_decrease(cu, dtype, D):
    dev = gpu_ready()
    q, k, v, _ = make([3000], 4, 2, D, dtype, dev, seed=len(cu))
    O = call(q, k, v, cu)
    good = next(i for i in range(1, len(cu)) if cu[i] < cu[i - 1])
    ref, A, S = SO.prompt_attention(q, k, v, cu[:good])
    owned = slice(cu[0], cu[good - 1])
    assert_within(O[owned], ref[owned], tolerance(dtype, ref, A, S, 3000)[owned], "ahead of the decrease")
    O[owned] = 7.0
    assert bool((O == 7.0).all())
    assert mb.poll_errors() == (0, 0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[0, 100, 10, 200], [0, 200, 5, 200, 0, 200], [7, 3, 200],
                                list(range(0, 200, 2)) + [0] + list(range(0, 200, 3)) + [200]], ids=lambda c: f"{len(c)}-{c[1]}")
def test_store_stays_in_the_tables_pages(cu):
    """Which rows are stored is not defined then, but each goes to a place of a sequence that has it."""
    dev = gpu_ready()
    B = len(cu) - 1
    c = Cache(B, 2, 2 * B + 3, dev, layers=1, seed=B)
    c.reserve([256] * B)
    k, v = (torch.randn((200, 2, 64), device=dev).to(BF16) for _ in range(2))
    Kp, Vp = c.Kp.clone(), c.Vp.clone()
    mb.kv_store_paged(c.cfg, k, v, 200, 128, 128, i32(cu, dev), None, c.Kp, c.Vp, c.num, c.P, c.table)
    c.o.store(k, v, cu, None)   # every sequence's rows
    for got, was, all_ in ((c.Kp, Kp, c.o.pools[0]), (c.Vp, Vp, c.o.pools[1])):
        assert bool(((got == was) | (got == all_)).all())


def test_oracle_stops_at_a_decrease():
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((60, h, 64), generator=gen) for h in (6, 2, 2))
    O, _, _ = SO.prompt_attention(q, k, v, [0, 20, 10, 60])
    ahead, _, _ = SO.prompt_attention(q, k, v, [0, 20])
    assert torch.equal(O, ahead) and bool((O[20:] == 0).all())
