"""Angles at the ends of the accepted range: every int32 position, frequencies up to 2^16 radians.

Tolerance: that of test_gpu_rotary.py without its part that grows with the distance.  An angle is off by 2^-32 of a turn (2^-29.3
radians) where the fraction is cut, by 2^-33 from the 64-bit frequency 2^31 times, and by fp32's rounding of an
eighth of a turn (2^-25.3); sine and cosine by a few units of fp32's last place, the two products by 2^-23 of |a| + |b|: below
2^-21 of it together; then half a step of fp32.
"""
from fractions import Fraction

import pytest
import torch

import rotary_ref as ref
from linear_attention_recurrence_kda_gb300 import binding as B
from test_gpu_rotary import DEV, data

pytestmark = pytest.mark.gpu


def arctan_of_one_over(n, bits):
    """Its series, in integers."""
    term = total = (1 << bits) // n
    k, sign = 1, -1
    while term:
        term //= n * n
        k += 2
        total += sign * (term // k)
        sign = -sign
    return total


def angle(position, freq):
    """position * freq radians, reduced to within half a turn with 300 bits."""
    bits = 300
    turn = Fraction(8 * (4 * arctan_of_one_over(5, bits) - arctan_of_one_over(239, bits)), 1 << bits)
    x = Fraction(freq) * position / turn
    return float((x - round(x)) * turn)


def test_the_reference():
    import math
    for p, f in ((1, 1.0), (-3, 0.25), (710, 1.0), (2 ** 31 - 1, 1.0)):
        assert abs(math.sin(angle(p, f)) - math.sin(p * f)) < 1e-15


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("adjacent", [False, True])
def test_every_position_and_frequency(adjacent, inverse):
    freqs = (65536.0, -65536.0, 60000.123, 31415.9265, 12345.678901, 1000.0 / 3, 100.0, -7.0, 6.283185307179586, 3.0, 1.0, 0.1,
             1e-3, 1e-6, 3.3e-10, 0.0)
    r = B.make_rotary(32, freqs=freqs, adjacent=adjacent)
    positions = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 1999999973, -1234567891, 2 ** 30, 104729, -1, 0]
    x = data(len(positions), 3, 64, torch.float32, 5)
    got = B.kda_rotary(r, x, positions=torch.tensor([positions], dtype=torch.int32, device=DEV), inverse=inverse)[0].double().cpu()
    t = torch.tensor([[angle(p, f) for f in freqs] for p in positions], dtype=torch.float64)[:, None] * (-1 if inverse else 1)
    xd = x.double().cpu()
    a, b = ref.split(xd, r)
    want = xd.clone()
    wa, wb = ref.split(want, r)
    wa.copy_(a * t.cos() - b * t.sin())
    wb.copy_(b * t.cos() + a * t.sin())
    tol = 2.0 ** -21 * ref.size(x, r) + 2.0 ** -24 * want.abs()
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), [(tuple(i), float((got - want)[tuple(i)])) for i in bad.nonzero()[:6].tolist()]


def test_the_same_on_the_way_into_the_cache():
    """Queries turned by the append take the same angles."""
    freqs = (60000.123,) * 4 + (12345.678901,) * 4
    r = B.make_rotary(16, freqs=freqs)
    positions = torch.tensor([[2 ** 31 - 1, -2 ** 31, 1999999973]], dtype=torch.int32, device=DEV)
    q, k, v = data(3, 4, 32, torch.float32, 6), data(3, 2, 32, torch.float32, 7), data(3, 2, 32, torch.float32, 8)
    cache = B.kda_cache_alloc(1, 16, 2, 32)
    table, lengths = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.tensor([3], dtype=torch.int32, device=DEV)
    got = B.kda_rotary_append(r, k, v, cache, table, lengths, q=q, positions=positions)
    assert torch.equal(got, B.kda_rotary(r, q, positions=positions)[0])
    turned = B.kda_rotary(r, k=k, positions=positions)[1]
    # half a step of e4m3 (2^-4 of a value, or 2^-10 in units of the scale), and both calls' fp32 roundings
    unit = cache.k_scale[0].double().cpu()[None, :, None]
    back = cache.k[0, :, :3].double().cpu().transpose(0, 1) * unit
    want = turned.double().cpu()
    assert bool(((back - want).abs() <= torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * unit) + 2.0 ** -20 * want.abs().max()).all())
