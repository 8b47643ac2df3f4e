"""How far windowed and 8-bit outputs are from the 64-bit result, beside what they have to be.

Two measures.  (1) A window that covers every token adds nothing to the error of the call without one: the
windowed kernels hold the RoPE query in more bits, the rest is the same.  (2) In bf16 roundings of the exact
output: the output's own rounding counts 1, the weights' rounding to 2^-8 of each, which moves a sum of latents
by the same share of its norm, 1 more, and the RoPE query, of which the CTA-pair kernel holds a half in one part,
less than 2 more; squares add up, so a call is within 2.
"""
import numpy as np
import pytest
import torch

import q8_window_ref as R
from test_gpu_q8_window import Device, Q  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [dict(), dict(H=128, G=8, d_c=512, d_r=64), dict(H=64, G=8, d_c=512, d_r=64)]


@pytest.mark.parametrize("shape", SHAPES)
def test_covering_window_is_no_less_exact(Q, shape):  # noqa: F811
    off, off_windowed = 0.0, 0.0
    for seed in range(4):
        c = R.Case([700, 130, 64], cache="bf16", s_q=2, seed=seed, **shape)
        off += np.sum((Device(Q, c, num_splits=1).run(Q)[0] - c.o) ** 2)
        c.window = 700
        off_windowed += np.sum((Device(Q, c, num_splits=1).run(Q)[0] - c.o) ** 2)
    print(f"error with a covering window / without: {np.sqrt(off_windowed / off):.3f}")
    assert off_windowed <= off


@pytest.mark.parametrize("cache", ["q8", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("seed", range(8))
def test_error_in_roundings_of_the_output(Q, shape, cache, seed):  # noqa: F811
    g = np.random.Generator(np.random.PCG64(seed))
    lens = [int(n) for n in np.exp(g.uniform(np.log(64), np.log(3000), 3))]
    window = int(np.exp(g.uniform(np.log(16), np.log(2000))))   # (one token is its own latent: no rounding to compare with)
    c = R.Case(lens, cache=cache, window=window, sinks=int(g.choice([0, 1, 4, 70])), s_q=int(g.choice([1, 2, 3])),
               seed=seed, **shape)
    o, _ = Device(Q, c, o_dtype=torch.bfloat16).run(Q)
    rounding = np.linalg.norm(R.bf16(c.o).astype(np.float64) - c.o)
    ratio = np.linalg.norm(o - c.o) / rounding
    print(f"window {window} over {lens}: {ratio:.2f} roundings")
    assert ratio <= 2
