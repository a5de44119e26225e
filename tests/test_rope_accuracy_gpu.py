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
