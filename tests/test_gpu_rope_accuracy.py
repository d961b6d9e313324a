"""How near the rotation's cosines and sines are, on the GPU.

A pair (u, v) that turns by an angle a with tan a = u / v gives u cos a - v sin
a = 0: what is left of it is what the kernel's arithmetic is off by, and the
rounding to bf16 (2^-8 of the little that is left) hides none of it.  With L
the pair's length, cosine and sine each off by 2^-23 move it by at most 2^-23
(|u| + |v|) <= 2^-22.5 L; u cos a and v sin a, each at most L / 2 there, round by
2^-25 L; together less than 2^-22 L.  The angle is taken from position times
frequency to 60 digits."""

import math
from decimal import Decimal, localcontext

import pytest
import torch

import block_sparse_masked_build_gb300 as bsm

pytestmark = pytest.mark.gpu

TURN = Decimal("6.28318530717958647692528676655900576839433879875021164194988"
               "91846156328125724179972560696506842341359")
POSITIONS = (1, -1, 7, -300, 4999, 100003, -(2 ** 24) - 1, 2 ** 29 + 5,
             2 ** 31 - 1, -(2 ** 31))


def _reduced(freq, position):
    """freq * position without its whole turns, in [0, 2 pi)."""
    with localcontext() as c:
        c.prec = 100
        return float((Decimal(freq) * position) % TURN)


def _pairs(n, position, g):
    """n pairs (u, v) in bf16 and frequencies that turn them onto u' = 0; every
    second one is at or near the largest frequency."""
    u, v = (torch.randn(n, generator=g).bfloat16() for _ in range(2))
    freq = []
    for i in range(n):
        f = 63.0 if i % 2 else 60.0 * 2.0 ** (-14 * float(
            torch.rand(1, generator=g)))
        want = math.atan2(float(u[i]), float(v[i])) + math.pi * (i // 2 % 2)
        off = (want - _reduced(f, position)) % (2 * math.pi)
        if off > math.pi:
            off -= 2 * math.pi
        f += off / position
        freq.append(f if abs(f) <= 64 else f - math.copysign(
            2 * math.pi / abs(position), f))
    return u, v, freq


@pytest.mark.parametrize("position", POSITIONS)
@pytest.mark.parametrize("dim,D,inter", [(128, 128, False), (64, 64, True),
                                         (64, 128, False)])
def test_cancelling_pairs(position, dim, D, inter):
    g = torch.Generator().manual_seed(abs(position) % 1000 + dim)
    half = dim // 2
    a, b = ((slice(0, dim, 2), slice(1, dim, 2)) if inter else
            (slice(0, half), slice(half, dim)))
    at = torch.full((1, 1), position, dtype=torch.int32, device="cuda")
    for _ in range(4):
        u, v, freq = _pairs(half, position, g)
        x = torch.zeros(1, 1, 1, D, dtype=torch.bfloat16)
        x[..., a], x[..., b] = u, v
        # the same pairs turned back by the opposite frequencies
        gone, _ = bsm.norm_rope(x.cuda(), positions=at, rope=bsm.Rope(
            dim, inv_freq=freq, interleaved=inter))
        back = bsm.norm_rope_bwd(x.cuda(), positions=at, rope=bsm.Rope(
            dim, inv_freq=[-f for f in freq], interleaved=inter))[0]
        angle = torch.tensor([_reduced(f, position) for f in freq],
                             dtype=torch.float64)
        c, s = torch.cos(angle), torch.sin(angle)
        u, v = u.double(), v.double()
        size = torch.hypot(u, v)
        for got in (gone, back):
            got = got.double().cpu()[0, 0, 0]
            for y, want in ((got[a], u * c - v * s), (got[b], v * c + u * s)):
                tol = 2.0 ** -8 * want.abs() * (1 + 2.0 ** -8) \
                    + 2.0 ** -22 * size
                assert bool(((y - want).abs() <= tol).all()), (
                    float(((y - want).abs() / size).max()))
