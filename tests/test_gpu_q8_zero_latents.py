"""8-bit decode where the first tokens that a work item sees have an all-zero latent (scale 0).

Such a token has a weight in the softmax and none in the output, so a row's unit of the output's weights has to
come from a later tile.  Tolerances are those of test_gpu_q8_window: fp32's 1e-5 on the CUDA cores, 5e-3 of the
norm on the tensor cores.
"""
import numpy as np
import pytest

import q8_window_ref as R
from q8_inputs import replace_latents
from test_gpu_q8_window import Q, check  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [dict(), dict(H=32, G=2), dict(H=64, G=8), dict(H=16, G=1, d_c=512, d_r=64), dict(H=64, G=8, d_c=512, d_r=64),
          dict(H=128, G=8, d_c=512, d_r=64), dict(H=32, G=4, d_c=128, d_r=64)]
# (length, window, sinks, splits, tokens that are zero)
ZERO = [
    (300, 0, 0, 0, range(64)),                       # the whole first tile
    (300, 0, 0, 0, range(130)),                      # two tiles and a little
    (64, 0, 0, 0, range(63)),                        # all but the newest token
    (1000, 70, 1, 0, [0]),                           # a zero sink: the first tile's only token
    (1000, 425, 0, 0, [575]),                        # a window that starts on a tile's last token
    (1024, 0, 0, 2, range(512, 576)),                # the second item begins with a zero tile
    (1024, 0, 0, 2, range(512, 1024)),               # an item of zeros beside one that is not
    (200, 0, 0, 0, range(200)),                      # nothing but zeros: o = 0, lse finite
]


@pytest.mark.parametrize("simt", [True, False])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("k", range(len(ZERO)))
def test_zero_latents_first(Q, k, shape, simt):  # noqa: F811
    n, window, sinks, splits, zero = ZERO[k]
    c = R.Case([n, 90], window=window, sinks=sinks, **SHAPES[shape])
    lat = np.random.Generator(np.random.PCG64(k)).standard_normal((n, c.d_c)).astype(np.float32)
    lat[list(zero)] = 0
    replace_latents(c, 0, lat)
    dev = check(Q, c, simt=simt, num_splits=splits)
    if len(zero) == n:
        assert (dev.o[0] == 0).all()


def test_zero_latents_first_several_queries(Q):  # noqa: F811
    """Row blocks that span query tokens; a moving unit in rows whose first tiles differ."""
    c = R.Case([700, 260], s_q=3, H=32, G=4, window=150, sinks=66)
    g = np.random.Generator(np.random.PCG64(1))
    for b, n in enumerate(c.lens):
        lat = (g.standard_normal((n, c.d_c)) * np.exp2(g.uniform(-20, 0, (n, 1)))).astype(np.float32)
        lat[:66] = 0
        lat[n - 153:n - 100] = 0
        replace_latents(c, b, lat)
    check(Q, c, simt=False)
