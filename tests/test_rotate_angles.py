"""Angles of medusa_qk_norm_rotate, each held to what its own arithmetic may be off by.

The position times the frequency is reduced here in whole numbers (a frequency is a float32, so the product is
exact; 2 pi has 256 bits), so that the reference's sine and cosine are right to float64 whatever the position.
"""
import math
from functools import lru_cache

import pytest
import torch

from oracle import serving_oracle as SO

from _helpers import gpu_ready
from _serving import assert_within, i32
from test_rotate import BF16, F32, KINDS, call, freqs, make

BITS = 256


@lru_cache(None)
def two_pi():
    """2 pi 2^BITS by Machin's formula, pi / 4 = 4 arctan(1 / 5) - arctan(1 / 239), in whole numbers."""
    def arctan_of_one_over(x):
        power, total, n, sign = (1 << (BITS + 32)) // x, 0, 1, 1
        while power:
            total += sign * (power // n)
            power //= x * x
            n, sign = n + 2, -sign
        return total

    return (8 * (4 * arctan_of_one_over(5) - arctan_of_one_over(239))) >> 32


def remainder(pos, f):
    """pos f modulo 2 pi, from the exact product."""
    num, den = float(f).as_integer_ratio()
    return ((int(pos) * num << BITS) // den % two_pi()) / (1 << BITS)


def angles(pos, f):
    return torch.tensor([[remainder(p, x) for x in f.double().tolist()] for p in pos.tolist()], dtype=torch.float64, device=pos.device)


def may_be_off(pos, f):
    """Largest error of an angle, of its sine and of its cosine, for each row and pair.

    A turn's fraction for one position is cut off at 2^-64 and its constant at 2^-64 of itself; times the position,
    its first 32 bits are taken: 2 pi (2^-32 + |pos| 2^-64 (1 + |f| / 2 pi)). What is left of a quarter turn, |a| <= pi / 4,
    is rounded to float32, multiplied with a rounded constant and rounded again, 3 of 2^-24 of it: 2.4 of 2^-24. The
    series ends 2e-9 from sine and cosine and is off by at most 1.3 of 2^-24 in its roundings (half a unit of the
    last step, and what a^2 and the second-last step are off by). 4 of 2^-24 cover the three."""
    far = pos.double().abs()[:, None] * 2.0 ** -64 * (1.0 + f.double().abs()[None] / (2 * math.pi))
    return 2 * math.pi * (2.0 ** -32 + far) + 2.0 ** -22


def turned(y, a, rot, pairs):
    """(result, |y_u| + |y_v| of each pair) of heads y [T][H][D] turned by the angles a [T][rot / 2]."""
    out, M = y.clone(), y.abs()
    cos, sin = torch.cos(a)[:, None], torch.sin(a)[:, None]
    u, v = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
    out[..., u], out[..., v] = y[..., u] * cos - y[..., v] * sin, y[..., v] * cos + y[..., u] * sin
    both = M[..., u] + M[..., v]
    M[..., u], M[..., v] = both, both.clone()
    return out, M


def bound(y, out, M, off, rot, pairs, dtype, normed):
    """The norm as in test_rotate; turning adds two products and a sum, 3 of 2^-24; one rounding to the type at the end."""
    D = y.shape[-1]
    e = torch.full_like(M, (D / 2 + 8) * 2.0 ** -24 if normed else 0.0)
    u, v = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
    for s in (u, v):
        e[..., s] += off[:, None] + 3 * 2.0 ** -24
    half = {BF16: 2.0 ** -8, F32: 2.0 ** -24}[dtype]
    return M * e * (1 + half) + out.abs() * half + 1e-37


def check(q, k, qw, kw, eps, f, rot, pairs, pos, qo, ko, what):
    a, off = angles(pos, f), may_be_off(pos, f)
    for x, w, got, name in ((q, qw, qo, "queries"), (k, kw, ko, "keys")):
        y, _ = SO.norm_rotate(x, w, eps, f, 0, pairs, pos)
        out, M = turned(y, a, rot, pairs)
        assert_within(got, out, bound(y, out, M, off, rot, pairs, x.dtype, w is not None), f"{what} {name}")


FAR = [0, 1, -1, 2, 3, 100, 131071, 1000003, 2 ** 24 + 1, 77777777, -77777777, 2 ** 31 - 1, -2 ** 31]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("normed", [False, True])
def test_near_and_far_positions_by_themselves(normed, pairs, dtype, D):
    dev = gpu_ready()
    q, k, qw, kw, _ = make(len(FAR), 4, 2, D, dtype, dev, seed=3)
    qw, kw = (qw, kw) if normed else (None, None)
    pos = i32(FAR, dev)
    for f in (freqs(D, dev), torch.linspace(0.0, 7.0, D // 2, device=dev), -freqs(D, dev, 500.0),
              torch.logspace(-30, 3, D // 2, device=dev)):
        check(q, k, qw, kw, 1e-6, f, D, pairs, pos, *call(q, k, qw, kw, 1e-6, f, D, pairs, pos), f"frequencies {float(f[0])} ..")


@pytest.mark.gpu
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("rot", [8, 40, 64])
def test_every_position_of_a_context(rot, pairs):
    """(1, 0) turns into (cos, sin): float32, without a norm, positions one after another and around 2^20."""
    dev = gpu_ready()
    pos = torch.cat([torch.arange(0, 700), torch.arange(2 ** 20 - 100, 2 ** 20 + 100)]).int().to(dev)
    q = torch.zeros((pos.numel(), 1, 64), device=dev)
    u = slice(0, rot, 2) if pairs else slice(0, rot // 2)
    q[:, :, u] = 1.0
    f = freqs(rot, dev)
    check(q, q, None, None, 0.0, f, rot, pairs, pos, *call(q, q.clone(), None, None, 0.0, f, rot, pairs, pos), f"{rot} dims")


# ----------------------------------------------------------------------------------- the reference (no GPU)
def test_two_pi_and_remainders():
    assert two_pi() / (1 << BITS) == 2 * math.pi
    # 2 pi to 50 decimals, as tables have it
    assert str(two_pi() * 10 ** 50 >> BITS) == "6283185307179586476925286766559005768394338798750211"[:51]
    for p, f in ((1, 1.0), (-1, 0.5), (7, 0.25), (1000, 0.001)):
        f = float(torch.tensor(f))
        assert abs(math.remainder(remainder(p, f) - p * f, 2 * math.pi)) < 1e-12


def test_products_in_fewer_bits_are_outside():
    """What the bound is there to find: angles from a float32 product (any far position), and from a float64 one."""
    f = torch.linspace(0.0, 7.0, 64)
    for p, dtype in ((131071, torch.float32), (2 ** 31 - 1, torch.float32), (2 ** 31 - 1, torch.float64)):
        pos = torch.tensor([p], dtype=torch.int64)
        # (a remainder in float64 as good as that product's: only the product's own rounding shows)
        product = (pos.to(dtype)[:, None] * f.to(dtype)[None]).double()
        a = torch.tensor([[remainder_of(float(x)) for x in product[0]]], dtype=torch.float64)
        off = (torch.cos(a) - torch.cos(angles(pos, f))).abs().maximum((torch.sin(a) - torch.sin(angles(pos, f))).abs())
        assert float((off / may_be_off(pos, f)).max()) > 1.0


def remainder_of(x):
    num, den = x.as_integer_ratio()
    return ((num << BITS) // den % two_pi()) / (1 << BITS)
