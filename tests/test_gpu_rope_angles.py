"""qkmla_rope's angles at far positions, against frequencies of 50 digits.

Tolerance.  A frequency is formed in 64 bits, to 2^-48 of itself: an angle of N turns is off by N 2^-48 of a turn, and by 2^-26 of one where
its fraction becomes fp32; sine, cosine, products and sums add 5 x 6e-8 of the pair's length."""
import decimal
import math

import pytest
import torch

from test_gpu_rope_apply import Q  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

decimal.getcontext().prec = 50
PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582")
POSITIONS = [0, 1, -1, 4095, 2 ** 24, 2 ** 24 + 1, 2 ** 27 + 3, -987654321, 2 ** 31 - 1, -2 ** 31]


def turns(f):
    """The positions' angles in turns, as [-1/2, 1/2] and as they are."""
    part, whole = [], []
    for p in POSITIONS:
        n = [decimal.Decimal(p) * x / (2 * PI) for x in f]
        part.append([float(x - x.to_integral_value()) for x in n])
        whole.append([abs(float(x)) for x in n])
    return torch.tensor(part, dtype=torch.float64), torch.tensor(whole, dtype=torch.float64)


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("theta", [1.001, 1e4, 5e5, 1e8])
@pytest.mark.parametrize("d", [2, 64, 98, 256])
def test_far_positions(Q, d, theta, given):  # noqa: F811
    theta = float(torch.tensor(theta, dtype=torch.float32))
    ln = decimal.Decimal(theta).ln()
    f = [(-ln * (2 * i) / d).exp() for i in range(d // 2)]
    scaling = None
    if given:                                                  # any size and sign, as 64-bit numbers
        radians = [float(x) * 100 * (-1) ** i for i, x in enumerate(f)]
        f, scaling = [decimal.Decimal(x) for x in radians], Q.given_frequencies(radians)
    part, whole = turns(f)
    x = torch.randn((len(POSITIONS), 3, d), generator=torch.Generator().manual_seed(d))
    got = Q.rope(x.cuda(), torch.tensor(POSITIONS, dtype=torch.int64).to(torch.int32).cuda(), theta=theta, layout="half", scaling=scaling)
    z = torch.polar(torch.ones_like(part), 2 * math.pi * part)[:, None]
    a, b = x[..., :d // 2].double(), x[..., d // 2:].double()
    want = torch.complex(a, b) * z
    have = torch.complex(*(t.double().cpu() for t in (got[..., :d // 2], got[..., d // 2:])))
    bound = 2 * math.pi * (whole * 2.0 ** -48 + 2.0 ** -26) + 5 * 6e-8
    err = (have - want).abs() / torch.complex(a, b).abs()
    print(float((err / bound[:, None]).max()))
    assert (err <= bound[:, None]).all()
