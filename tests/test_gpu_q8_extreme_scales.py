"""8-bit decode of latents near the ends of fp32's range, alone and beside ordinary ones.

A latent's magnitude cancels in its logits (alpha^k) and stays in its output, so every case has a result in fp32.
Tolerance: the tensor-core kernels' 5e-3 of a row's norm, with outputs measured in units of the largest latent;
fp32's 1e-5 on the CUDA cores.
"""
import numpy as np
import pytest

import q8_window_ref as R
from q8_inputs import replace_latents, seen_slots
from test_gpu_q8_window import Device, Q  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [dict(), dict(H=32, G=2), dict(H=64, G=8, d_c=512, d_r=64), dict(H=16, G=1, d_c=512, d_r=64)]
# binades of the first tokens' latents (as many as given) and of the others'
RANGES = [(0, 0, 114), (0, 0, -114), (100, 114, -114), (100, -114, 114), (10, -100, 0), (10, 100, 0), (300, -120, -100),
          (300, 0, -118)]


@pytest.mark.parametrize("simt", [True, False])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("k", range(len(RANGES)))
def test_extreme_scales(Q, k, shape, simt):  # noqa: F811
    first, low, high = RANGES[k]
    n = 700
    c = R.Case([n, 90], outlier=1.0, **SHAPES[shape])
    g = np.random.Generator(np.random.PCG64(k))
    size = np.where(np.arange(n) < first, np.ldexp(1.0, low), np.ldexp(1.0, high))
    lat = (g.standard_normal((n, c.d_c)) * size[:, None]).astype(np.float32)
    seen, slot = seen_slots(c, 0)
    c.ak[slot] = (1 / size[seen])[:, None]
    replace_latents(c, 0, lat)
    dev = Device(Q, c, force_simt=simt, num_splits=1 if k % 2 else 0)
    o, lse = dev.run(Q)
    unit = np.abs(c.o[0]).max()
    off = np.linalg.norm((o[0] - c.o[0]) / unit) / np.linalg.norm(c.o[0] / unit)
    print(f"{off:.2e}")
    assert off <= (1e-5 if simt else 5e-3)
    assert np.abs(lse[0] - c.lse[0]).max() <= 1e-3
