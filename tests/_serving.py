"""Shared pieces of the prompt, prefix and page tests: configurations, inputs and derived tolerances."""
from __future__ import annotations

import numpy as np
import torch

from medusa_speculative_decoding_heads_gb300 import binding as mb, configs
from oracle import medusa_oracle as O

I32 = torch.int32


def cfg_for(B, Hq, Hkv, D, dtype, L_cap=1024, branching=(1,), tree_nodes="root"):
    """A configuration around the attention shape; the default tree is a lone root (single tokens)."""
    if tree_nodes == "root":
        tree_nodes = ([-1], [0]) if tuple(branching) == (1,) else None
    return mb.make_cfg(B=B, d=64, V=64, branching=branching, Hq=Hq, Hkv=Hkv, D=D, L_cap=L_cap,
                       dtype=mb.F32 if dtype == torch.float32 else mb.BF16, mode=configs.GREEDY, tree_nodes=tree_nodes)


def tolerance(dtype, O_ref, A, S, keys):
    """Largest error of each output value, from the arithmetic.

    Scores are float32 dot products of D exact products: off by at most D 2^-24 times the sum of
    |q_d k_d| (S holds it, scaled); scaling, the maximum and the exponential add a few units of
    2^-24 of the score and of the weight (64 covers 2-unit exponentials and the scaled arguments).
    A weight's relative error is at most twice that (numerator and sum), the sums over `keys` keys
    add 2 keys 2^-24. All of it multiplies A, the weights applied to |v|. In bf16 the weights are
    rounded before the product with v (half a step: 2^-8 of each) and so is the result (2^-8)."""
    D = O_ref.shape[-1]
    f32 = 2.0 ** -24 * (2.0 * (D + 8.0) * S.unsqueeze(-1) + 2.0 * keys + 64.0)
    if dtype == torch.float32:
        return A * f32 + 1e-30
    return A * (2.0 ** -8 + 2.0 * f32) + O_ref.abs() * 2.0 ** -8 + 1e-30


def assert_within(got, ref, tol, what):
    got = got.double()
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite values"
    over = (got - ref).abs() / tol
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.2f} times the bound at {np.unravel_index(int(over.argmax()), over.shape)}"


def ancestor_bits(branching, dev):
    """(mask [N][N] bool, bits [N][2] int64) of the Cartesian tree; branching (1,) is the lone root here."""
    if tuple(branching) == (1,):
        mask = np.ones((1, 1), dtype=bool)
    else:
        mask = O.ancestor_mask(O.tree_layout(branching)["parent"]).astype(bool)
    bits = O.mask_bits(mask.astype(np.uint8))
    return torch.from_numpy(mask), torch.from_numpy(np.ascontiguousarray(bits).astype(np.uint64).view(np.int64)).to(dev)


def i32(values, dev):
    return torch.tensor(values, dtype=I32, device=dev)


def offsets(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu
