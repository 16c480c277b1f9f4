"""Angles of kvx_cache_append_rotated at positions up to the ends of 32 bits, with frequencies and angles in 50 decimal digits. Each pair
lies across the axis that it is turned to, so that its first element comes out near zero, where f16 shows 2^-22 of the pair's size
and thereby the angle's own error."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest

from test_rotate_gpu import Case, dev, f64, kvx, torch

pytestmark = pytest.mark.gpu
getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def angles(positions, dim, base, factor):
    """(angles in radians, less whole turns, and what a frequency's 64 bits leave of each, in turns): [position][pair]."""
    logs = [-Decimal(base).ln() * 2 * i / dim for i in range(dim // 2)]
    turns = [x.exp() / Decimal(factor) / (2 * PI) for x in logs]
    a = np.array([[float((Decimal(int(p)) * t) % 1) for t in turns] for p in positions]) * (2 * math.pi)
    # the exponent's rounding 2^-53 of it, the power's a unit in the last place, the division by the factor half of one
    share = np.array([abs(float(x)) * 2.0 ** -53 + 2.0 ** -52 + 2.0 ** -53 for x in logs])
    return a, np.abs(positions.astype(np.float64))[:, None] * np.array([float(t) for t in turns]) * share


def spread(centre, n, rng):
    return np.clip(centre + rng.integers(-5000, 5001, n), -2 ** 31, 2 ** 31 - 1)


@pytest.mark.parametrize("dim,base,factor", [(64, 10000, 1), (128, 500000, 1), (128, 10000, 4)])
@pytest.mark.parametrize("pairs", [0, 1])
@pytest.mark.parametrize("far", ["2^24", "2^29", "2^31"])
def test_angles(far, pairs, dim, base, factor):
    rng = np.random.default_rng(dim + pairs)
    ends = {"2^24": [0, 1, 2 ** 24 - 1, 2 ** 24, -2 ** 24], "2^29": [2 ** 29 - 1, -2 ** 29 + 1], "2^31": [2 ** 29, 2 ** 31 - 1, -2 ** 31]}[far]
    pos = np.concatenate([ends] + [spread(e, 6, rng) for e in ends]).astype(np.int64)
    if far == "2^29":
        pos = np.clip(pos, -2 ** 29 + 1, 2 ** 29 - 1)
    angle, rounding = angles(pos, dim, base, factor)
    n, half = len(pos), dim // 2
    a, b = np.sin(angle), np.cos(angle)
    x = np.zeros((n, dim))
    ia, ib = (np.arange(0, dim, 2), np.arange(1, dim, 2)) if pairs else (np.arange(half), np.arange(half) + half)
    x[:, ia], x[:, ib] = a, b
    c = Case("f16", dim=dim, q_heads=2, heads=1, tokens=n, q_norm=False, k_norm=False)
    c.rotation = dict(dim=dim, layout=pairs, base=float(base), **(dict(scaling=1, factor=float(factor)) if factor > 1 else {}))
    c.pos, c.slots = pos.astype(np.int32), rng.permutation(c.geom.n_blocks * 16)[:n].astype(np.int64)
    c.x[:, :3 * dim] = dev(np.tile(x, (1, 3))).half()
    out = f64(c.run()).reshape(n, 2, dim)
    keys = f64(c.bufs[2].view(torch.float16).view(-1, dim)[dev(c.slots)])
    a, b = f64(c.x[:, :dim])[:, ia], f64(c.x[:, :dim])[:, ib]
    # documented: 2^-25 of a turn below position 2^29, 2^-23 beyond. Then a sine's function 2^-23 (two units in the last place) and
    # magnitude 2^-24, two products and a sum of 32 bits 2^-24 each
    turn = np.where(np.abs(pos) < 2 ** 29, 2.0 ** -25, 2.0 ** -23)[:, None] + rounding
    err = (np.abs(a) + np.abs(b)) * (2 * math.pi * turn + 2.0 ** -23 + 4 * 2.0 ** -24)
    cos, sin = np.cos(angle), np.sin(angle)
    for want, at in ((a * cos - b * sin, ia), (b * cos + a * sin, ib)):
        bound = err + 2.0 ** -11 * (np.abs(want) + err) + 2.0 ** -25
        for got in (out[:, 0, at], out[:, 1, at], keys[:, at]):
            off = np.abs(got - want) / bound
            assert (off <= 1).all(), off.max()


def test_the_reference_of_angles():
    """One angle by hand, and what 32 bits would make of it."""
    a, _ = angles(np.array([2 ** 31 - 1]), 64, 10000, 1)
    assert abs(a[0, 0] - math.fmod(2.0 ** 31 - 1, 2 * math.pi)) < 2.0 ** 28.4 * 2.5e-16   # fmod is exact, of 2 pi in 64 bits
