"""8-bit decode where one token outweighs each of very many others by 2^5 .. 2^20 and they outweigh it together.

The tensor-core kernel holds the output's weights in 8-bit parts.  What such a part leaves of a small weight
must not be lost in one direction: the softmax's denominator counts those weights in full.

Tolerance: the method's rule, 5e-3 of a row's norm.  A weight is off by 2^-8 of itself or, unbiased, by one
step of at most 2^-13 in units where the row's largest is at least 2 (4, 8, 64 behind 2048, 8192, 16384 tokens).
Rounded in proportion a step leaves at most 2^-14, over all fractions 2^-13 / sqrt(6), so N of them sqrt(N) 2^-14.3
|x| of at least 2 (4, 8, 64) x 448: with |x| = 64 sqrt(512) 3.2e-3 at N = 2000, 3.2e-3 at 8000, 2.3e-3 at 16000
and 2.7e-3 for 262144 tokens, of which 8192 lie in the coarser unit; with a mean of one deviation |x| is sqrt(2)
times that where the background does not carry the norm itself.
Every row has its own ratio.
"""
import math

import pytest
import torch

from test_gpu_q8_window import Q  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [(16, 4, 256, 32), (32, 4, 256, 32), (64, 8, 256, 64), (64, 8, 512, 64), (16, 1, 512, 64), (128, 8, 128, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("N,splits", [(2000, 1), (8000, 1), (16000, 1), (262144, 1), (262144, 0)])
@pytest.mark.parametrize("mean,at,scale", [(1.0, 0, 1.0), (1.0, 0.5, 32.0), (0.0, 0, 1.0)])
def test_heavy_token_over_background(Q, shape, N, splits, mean, at, scale):  # noqa: F811
    H, G, d_c, d_r = shape
    d, page = "cuda", 64
    gen = torch.Generator(device=d).manual_seed(N + H + d_c)
    slots = -(-N // page) * page
    kv = torch.zeros((slots, d_c + 2 * d_r), dtype=torch.uint8, device=d)
    kv_scale = torch.ones(slots, device=d)
    codes = ((torch.randn((N, d_c), generator=gen, device=d) + mean) * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
    heavy = int(at * N)
    codes[heavy] = 0
    codes[heavy, 0] = 448                                   # its latent lies in one column
    kv[:N, :d_c] = codes.view(torch.uint8)
    kv_scale[heavy] = scale
    # logits by the RoPE part alone: a row's heavy token stands 2^5 .. 2^20 above the others
    soft = 0.1
    binades = torch.linspace(5, 20, H, device=d)
    qr = torch.zeros((1, 1, H, d_r), device=d)
    qr[0, 0, :, 0] = (binades * math.log(2) / soft / 8).bfloat16().float()
    qr[0, 0, :, 1] = 1.0
    kr = torch.zeros((N, d_r), dtype=torch.bfloat16, device=d)
    kr[:, 1] = 0.5 * torch.randn(N, generator=gen, device=d)        # 5 % of spread
    kr[heavy] = 0
    kr[heavy, 0] = 8
    kv[:N, d_c:] = kr.view(torch.uint8)
    qt = torch.zeros((1, 1, H, d_c), dtype=torch.bfloat16, device=d)
    o = torch.empty((1, 1, H, d_c), device=d)
    lse = torch.empty((1, 1, H), device=d)
    call = Q.prepare_decode(qt, None, qr, None, kv, None, torch.tensor([N], dtype=torch.int32, device=d), None, page,
                            slots // page, G, soft, 1e-6, o, lse, plain=True, kv_scale=kv_scale, num_splits=splits)
    assert call.kernel_name == "tcgen05"
    call()
    assert Q.get_device_status() == 0
    logit = soft * (qr[0, 0].double() @ kr.double().t())
    p = torch.softmax(logit, dim=1) * kv_scale[:N].double()
    ref = p @ codes.double()
    off = (o[0, 0].double() - ref).norm(dim=1) / ref.norm(dim=1)
    print(f"largest row error {off.max():.2e} at 2^{binades[off.argmax()]:.1f}")
    assert off.max() <= 5e-3
    assert (lse[0, 0].double() - torch.logsumexp(logit, dim=1)).abs().max() <= 1e-3
