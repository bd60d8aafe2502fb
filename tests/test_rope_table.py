"""The rotation's table against its formulas in 60 decimal digits: every number is the nearest one, and the
farthest position turns as exactly as the table promises."""
from decimal import Decimal, getcontext

import pytest

import gated_pooling_gb300 as gp

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.fixture(autouse=True)
def digits():
    was = getcontext().prec
    getcontext().prec = 60
    yield
    getcontext().prec = was


def frequencies(rot, base=10000.0, scaling=0, factor=1.0, original_length=4096.0, beta_fast=32.0, beta_slow=1.0):
    log = Decimal(base).ln()
    f = [(-log * 2 * i / rot).exp() for i in range(rot // 2)]
    if scaling == 1:
        return [v / Decimal(factor) for v in f]
    if scaling == 2:
        def at(beta):
            return rot * (Decimal(original_length) / (2 * PI * Decimal(beta))).ln() / (2 * log)
        lo = min(max(at(beta_fast).__floor__(), 0), rot - 1)
        hi = min(max(at(beta_slow).__ceil__(), 0), rot - 1)
        out = []
        for i, v in enumerate(f):
            m = min(max(Decimal(i - lo) / max(Decimal(hi - lo), Decimal(0.001)), Decimal(0)), Decimal(1))
            out.append(v / Decimal(factor) * m + v * (1 - m))
        return out
    return f


CASES = [dict(), dict(base=500000.0), dict(base=1.0001), dict(base=3.7e300), dict(base=1e6, scaling=1, factor=4.0),
         dict(scaling=1, factor=7.3), dict(scaling=2, factor=16.0), dict(scaling=2, factor=40.0, original_length=8192.0,
                                                                         beta_fast=16.0, beta_slow=2.0),
         dict(scaling=2, factor=2.0, original_length=8.0), dict(base=150000.0, scaling=2, factor=32.0)]


@pytest.mark.parametrize("rot", [2, 30, 64, 128, 130, 1024])
@pytest.mark.parametrize("args", CASES)
def test_every_turn_is_the_nearest_number(rot, args):
    turns, _ = gp.csa_rope_table(rot, **args)
    want = [int((f / (2 * PI) * 2 ** 64).to_integral_value()) for f in frequencies(rot, **args)]
    assert [t % (1 << 64) for t in turns.tolist()] == want


@pytest.mark.parametrize("pos", [1, 4097, (1 << 31) - 1])
def test_far_positions_turn_as_exactly(pos):
    """Half a unit of 2^-64 of a turn, as often as the position says."""
    turns, _ = gp.csa_rope_table(128)
    for t, f in zip(turns.tolist(), frequencies(128)):
        off = (Decimal(pos * (t % (1 << 64))) / 2 ** 64 - pos * f / (2 * PI)) % 1
        assert min(off, 1 - off) <= Decimal(pos) / 2 ** 65
