"""Rotary frequencies and angles against 60 decimal digits."""
import math
from decimal import Decimal, getcontext

import pytest
import torch

from test_rope_gpu import K, table_of

pytestmark = pytest.mark.gpu

getcontext().prec = 60
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
UNIT = 1 << 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def turns_of(rot, theta, factor=1.0, alpha=1.0, beta=4.0, context=8192.0):
    """Turns per position of every pair."""
    for i in range(rot // 2):
        u = (Decimal(-2 * i) / rot * Decimal(theta).ln()).exp() / TWO_PI
        if factor > 1:
            t = u * Decimal(context)
            if t >= Decimal(beta):
                g = Decimal(1)
            elif t <= Decimal(alpha) or math.isinf(beta):
                g = Decimal(0)
            else:
                g = (t - Decimal(alpha)) / (Decimal(beta) - Decimal(alpha))
            u *= g + (1 - g) / Decimal(factor)
        yield u


@pytest.mark.parametrize("rot,theta", [(64, 10000.0), (128, 500000.0), (2, 1.0), (256, 1e7), (50, 1.5), (128, 1.7e308)])
@pytest.mark.parametrize("kw", [dict(), dict(factor=8.0), dict(factor=40.0, alpha=0.0, beta=32.0, context=4096.0),
                                dict(factor=1.1, alpha=0.3, beta=math.inf), dict(factor=3.3, alpha=math.inf, beta=math.inf),
                                dict(factor=1e6, alpha=0.1, beta=0.7, context=1e5), dict(factor=2.0, alpha=2.0, beta=2.0)])
def test_every_frequency_is_the_nearest_unit(rot, theta, kw):
    """The kernel's error of 2^-80 is 2^-16 of a unit at most: 0.51 for the nearest."""
    for got, u in zip(table_of(rot, theta, **kw).tolist(), turns_of(rot, theta, **kw)):
        assert abs(got % UNIT - u * UNIT) <= Decimal("0.51"), (got, u * UNIT)


@pytest.mark.parametrize("far", [1, 1 << 15, 1 << 31])
def test_cosines_and_sines_of_every_angle(far):
    """Unit vectors turned.  The angle's fraction of half a turn is at most 1/4, rounded by 2^-27: pi 2^-27 = 0.4 2^-24
    of the outputs; sincospif is within one step below 1, 2^-24; the table's half unit is 2^-34 turns at 2^31."""
    rot = 128
    pos = torch.randint(-far, far, (1500,), generator=torch.Generator().manual_seed(far)).int()
    x = torch.zeros((1500, 1, rot), device="cuda")
    x[..., :rot // 2] = 1
    y = torch.empty_like(x)
    K().kvc_rope(table_of(rot), pos.cuda(), None, x, None, y, rot)
    turns = list(turns_of(rot, 10000.0))
    angle = torch.tensor([[float(p * u % 1) * 2 * math.pi for u in turns] for p in pos.tolist()], dtype=torch.float64)
    want = torch.cat((torch.cos(angle), torch.sin(angle)), -1)
    assert (y[:, 0].double().cpu() - want).abs().max().item() <= 1.4 * 2.0 ** -24 + 2 * math.pi * 2.0 ** -34
