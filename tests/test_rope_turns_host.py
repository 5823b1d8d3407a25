"""The rotation's turns per position, against sixty digits (no GPU)."""
import ctypes
import random
from decimal import Decimal, getcontext

import pytest

import context_blockwise_attention_step_gb300 as ra
from context_blockwise_attention_step_gb300 import _abi

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.fixture(scope="module", autouse=True)
def _setup():
    ra.build()
    getcontext().prec = 78


def units(x, pos=1):
    """x * pos / 2pi, in units of 2^-64 of a turn."""
    return Decimal(x) * pos / (2 * PI) * 2 ** 64


def apart(a, b):
    """Modulo whole turns, either way."""
    d = abs(a - b) % 2 ** 64
    return min(d, 2 ** 64 - d)


@pytest.mark.parametrize("values", [
    [10000.0 ** (-i / 64) for i in range(64)], [500000.0 ** (-i / 32) for i in range(32)],
    [-(1000000.0 ** (-i / 64)) for i in range(64)], [0.0, -0.0, 1e-300, -1e-18, 1e-18, 6.283185307179586, -6.283185307179586],
    [1e6, -1e6, 3.5e9, 2.0 ** 40, -(2.0 ** 40)],
    [random.Random(5).uniform(-7, 7) for _ in range(64)],
], ids=["1e4", "5e5", "-1e6", "edges", "large", "random"])
def test_turns_are_exact_to_a_unit(values):
    r = _abi.RaRope()
    n = len(values)
    assert _abi.lib().ra_rope_init(ctypes.byref(r), 2 * n, 0, (ctypes.c_double * n)(*values)) == _abi.RA_OK
    for got, x in zip(r.turns, values):
        assert apart(Decimal(got), units(x)) <= 1, f"{x}: {got} is off by {apart(Decimal(got), units(x))} units"
        # and so the angle of the last position there is, to less than 2^-32 of a turn
        pos = 2 ** 31 - 1
        assert apart(Decimal(got) * pos, units(x, pos)) <= 2 ** 32
