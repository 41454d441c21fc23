"""The rotary table against frequencies of 60 decimal digits (CPU only).

mla_rope_init computes with mantissas of 64 bits: a power to within an ulp or so, and for the scaled forms a handful of
operations, each off by half a unit of 2^-63 relative. 8 x 2^-64 of the entry (at most 2^61.4: 1.3 units) and half a
unit of rounding stay below two units of 2^-64 turns."""
import ctypes
import random
from decimal import ROUND_CEILING, ROUND_FLOOR, Decimal, getcontext

import pytest

import sparse_head_latent_b200 as mla
from sparse_head_latent_b200 import build as cuda_build

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module", autouse=True)
def lib():
    cuda_build.build()
    return mla.load_library()


def _turns(base, scaling, factor=1.0, original_len=4096.0, fast=32.0, slow=1.0):
    """Turns per position of the 32 pairs, exact."""
    base, factor = Decimal(base), Decimal(factor)
    lo = hi = Decimal(0)
    if scaling == mla.MLA_ROPE_YARN:
        at = lambda b: 64 * (Decimal(original_len) / (2 * PI * Decimal(b))).ln() / (2 * base.ln())  # noqa: E731
        lo = max(at(fast).to_integral_value(ROUND_FLOOR), Decimal(0))
        hi = min(at(slow).to_integral_value(ROUND_CEILING), Decimal(63))
    out = []
    for i in range(32):
        f = (base.ln() * (Decimal(-2 * i) / 64)).exp()
        if scaling == mla.MLA_ROPE_LINEAR:
            f /= factor
        elif scaling == mla.MLA_ROPE_YARN:
            r = min(Decimal(1), max(Decimal(0), (i - lo) / max(hi - lo, Decimal("0.001"))))
            f = f * (1 - r) + f / factor * r
        out.append(f / (2 * PI))
    return out


SETTINGS = [(10000.0, 0, 1.0, 4096.0), (1.5, 0, 1.0, 4096.0), (1e6, 0, 1.0, 4096.0), (50000.0, 0, 1.0, 4096.0),
            (10000.0, 1, 4.0, 4096.0), (10000.0, 1, 3.7, 4096.0), (10000.0, 2, 40.0, 4096.0), (50000.0, 2, 32.0, 4096.0),
            (10000.0, 2, 1.0, 4096.0), (10000.0, 2, 8.0, 3.0)]


@pytest.mark.parametrize("base,scaling,factor,original", SETTINGS)
def test_entries_are_right_to_two_units(base, scaling, factor, original):
    t = mla.make_rope(base=base, scaling=scaling, factor=factor, original_len=original)
    for got, want in zip(t.turns, _turns(base, scaling, factor, original)):
        assert abs(got - want * 2 ** 64) <= 2


@pytest.mark.parametrize("base,scaling,factor,original", SETTINGS)
def test_the_angle_is_exact_at_every_position(base, scaling, factor, original):
    # what the kernels make of it: the leading 32 bits of position * entry mod 2^64, as half turns in 24 bits
    t = mla.make_rope(base=base, scaling=scaling, factor=factor, original_len=original)
    rng = random.Random(1)
    at = [0, 1, -1, 4096, 10 ** 6, 2 ** 31 - 1, -2 ** 31] + [rng.randrange(-2 ** 31, 2 ** 31) for _ in range(40)]
    for turns, want in zip(t.turns, _turns(base, scaling, factor, original)):
        for s in at:
            half = ctypes.c_int32(((s * turns) % 2 ** 64) >> 32).value
            half = ctypes.c_float(half).value / 2 ** 31  # the nearest float
            exact = (s * want) % 1 * 2  # half turns
            off = abs(Decimal(half) - exact) % 2
            assert min(off, 2 - off) <= Decimal(2) ** -24
