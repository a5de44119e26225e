"""How exact the rotation's angles are: far positions under frequencies that are
not small, against exact arithmetic (tests/paged_ref.py states the tolerance)."""
import math
from fractions import Fraction

import pytest
import torch

from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import RopeGeometry
from tests.test_rope_angles_host import TWO_PI

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def angle(p, f):
    """p * f modulo a turn in radians, within (-pi, pi], rounded once."""
    x = (p * Fraction(f)) % TWO_PI
    return float(x - TWO_PI if 2 * x > TWO_PI else x)


@pytest.mark.parametrize("back", [False, True])
def test_far_positions_under_any_frequency(back):
    freq = [700.25, -1e-4, 2.0 ** 20, -(2.0 ** 20 - 2.0 ** -30), 1.0, -1e-15, 123456.789, 0.0]
    geom = RopeGeometry("TND", 1, 48, 2, 16, inv_freq=freq, dtype="fp32")
    g = torch.Generator().manual_seed(3)
    q = torch.randn(48, 2, 16, generator=g)
    pos = torch.randint(-2 ** 31, 2 ** 31, (1, 48), generator=g, dtype=torch.int64)
    pos[0, :4] = torch.tensor([2 ** 31 - 1, -2 ** 31, 1, 0])
    call = swa.rope_backward if back else swa.rope
    y, _ = call(geom, q.to(DEV), None, pos.to(torch.int32).to(DEV))
    t = torch.tensor([[angle(int(p), f) for f in freq] for p in pos[0]], dtype=torch.float64)[:, None]
    if back:
        t = -t
    a, b = q.double()[..., :8], q.double()[..., 8:]
    ref = torch.cat((a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()), dim=-1)
    bound = ((a.abs() + b.abs()) * 2.0 ** -21).repeat(1, 1, 2)
    bound += 2.0 ** -24 * (ref.abs() + bound)
    assert ((y.cpu().double() - ref).abs() <= bound).all()
    assert math.isfinite(y.sum().item())


@pytest.mark.parametrize("interleaved", [False, True])
def test_sines_and_cosines_near_their_zeros(interleaved):
    """(1, 0) turned by t is (cos t, sin t): each within a few units of its own
    last place, also where it is small and the angle is not.  The angle is
    rounded to fp32 as the distance r from the nearest quarter turn (2^-24 of
    it); sine and cosine of it are within 2 ulp (2^-22), r's own error moves the
    small one by 2^-24 of itself and the other by r 2^-24 tan r <= 2^-24, and the
    product with 1 and sum with 0 are exact: 2^-22 + 2^-24 < 2^-21.  Below 2^-60
    turns the fraction's own rounding counts (|p| 2^-65 turns, tested above)."""
    freq = [math.pi * (0.5 - 2.0 ** -k) for k in range(6, 22)] + [math.pi * (1 - 2.0 ** -k) for k in range(6, 22)] + \
        [1.0, 0.7, 3.14159, 1.5707963, 2.0 ** -20, 2.0 ** -30, 6.2831853, 4.712389] + [0.1 * k for k in range(24)]
    half = len(freq)
    geom = RopeGeometry("TND", 1, 16, 1, 2 * half, inv_freq=freq, dtype="fp32", interleaved=interleaved)
    pos = torch.tensor([[0, 1, -1, 2, 3, 4, 5, -7, 11, 100, 1001, -4096, 65537, 10 ** 6, 10 ** 8, 2 ** 31 - 1]])
    q = torch.zeros(16, 1, 2 * half)
    if interleaved:
        q[..., ::2] = 1
    else:
        q[..., :half] = 1
    y, _ = swa.rope(geom, q.to(DEV), None, pos.to(torch.int32).to(DEV))
    y = y[:, 0].cpu().double()
    c, s = (y[:, ::2], y[:, 1::2]) if interleaved else (y[:, :half], y[:, half:])
    t = torch.tensor([[angle(int(p), f) for f in freq] for p in pos[0]], dtype=torch.float64)
    slack = pos.abs().double().T * 2.0 ** -65 * 2 * math.pi + 2.0 ** -52  # the fraction's rounding; the reference's
    for got, ref in ((c, t.cos()), (s, t.sin())):
        assert ((got - ref).abs() <= 2.0 ** -21 * ref.abs() + slack).all()
