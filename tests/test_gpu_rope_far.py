"""How far an angle is off at far positions, against decimal arithmetic of 80 digits."""

import math
from decimal import Decimal, getcontext

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import decode_attention_13_b200 as gtq  # noqa: E402

pytestmark = pytest.mark.gpu

PI = Decimal("3.1415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170680")


def angle(pos, theta, i, r):
    """pos theta^(-2i/r) less whole turns, rounded to fp64 at the end (off by 2^-53 of at most pi)."""
    getcontext().prec = 80
    a = Decimal(pos) * Decimal(theta) ** (Decimal(-2 * i) / Decimal(r))
    turns = a / (2 * PI)
    return float((turns - turns.to_integral_value()) * 2 * PI)


@pytest.mark.parametrize("pos", [0, 1, 131071, 2 ** 27 + 1, 2 ** 31 - 1, 2 ** 36 + 5, 2 ** 44 + 3, 2 ** 50 + 1])
@pytest.mark.parametrize("theta", [10000, 500000])
def test_the_angles_bound(pos, theta):
    r = 128
    cfg = gtq.make_rope(r, float(theta), dtype=gtq.DTYPE_FP32)
    x = torch.zeros((1, 1, 1, r), device="cuda")
    x[..., :r // 2] = 1.0       # y: the cosines, then the sines
    y = torch.empty_like(x)
    gtq.gtq_rope(cfg, x, y, pos0=pos)
    got = y[0, 0, 0].double().cpu().numpy()
    a = np.array([angle(pos, theta, i, r) for i in range(r // 2)])
    f = np.array([theta ** (-2.0 * i / r) for i in range(r // 2)])
    # the angle's own bound; sincospif is within 2 ulp of a value of at most 1 (2^-23), the magnitude 1 and the product by 1
    # change nothing, and the sum with 0 neither
    bound = 2.0 ** -23 + pos * f * 2.0 ** -50 + 2.0 ** -23
    err = np.maximum(np.abs(got[:r // 2] - np.cos(a)), np.abs(got[r // 2:] - np.sin(a)))
    assert np.all(err <= bound), (err / bound).max()
    assert math.isfinite(got.sum())
