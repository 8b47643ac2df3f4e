"""qkmla_rope on the GPU against rotation by complex numbers in 64 bits.

Tolerance.  fp32: the angle is exact to 2^-25 of a half turn (9.4e-8 rad), sine and cosine to 2 units of 2^-24, the two
products and their sum round to 2^-24 each: a pair's error is below (9.4e-8 + 5 x 6e-8) of its length, 4e-7.  bf16 inputs
are exact; the result is rounded once, 2^-8 of the element, plus the same 4e-7 of the pair."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from qk_normed_latent_gb300 import build as B
    B.build()
    import qk_normed_latent_gb300 as Q
    return Q


def frequencies(d, theta, kind, factor=1.0, original=0, fast=32.0, slow=1.0):
    f = theta ** (-2 * np.arange(d // 2) / d)
    if kind == "linear":
        return f / factor
    if kind == "yarn":
        c = lambda turns: d * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        low, high = max(math.floor(c(fast)), 0), min(math.ceil(c(slow)), d - 1)
        ramp = np.clip((np.arange(d // 2) - low) / max(high - low, 0.001), 0, 1)
        return f / factor * ramp + f * (1 - ramp)
    return f


def exact(x, pos, f, layout, inverse=False, gain=1.0):
    turns = pos.double()[:, None] * torch.from_numpy(f / (2 * math.pi))
    turns = turns - turns.round()
    z = torch.polar(torch.ones_like(turns), (-1 if inverse else 1) * 2 * math.pi * turns) * gain
    while z.dim() < x.dim():
        z = z[:, None]
    x = x.double()
    if layout == "interleaved":
        return torch.view_as_real(torch.complex(x[..., 0::2], x[..., 1::2]) * z).flatten(-2)
    h = x.shape[-1] // 2
    y = torch.complex(x[..., :h], x[..., h:]) * z
    return torch.cat([y.real, y.imag], dim=-1)


def check(got, ref, x, layout):
    got, x = got.double().cpu(), x.double().cpu()
    d = x.shape[-1]
    pairs = x.reshape(*x.shape[:-1], d // 2, 2) if layout == "interleaved" else torch.stack([x[..., :d // 2], x[..., d // 2:]], -1)
    size = pairs.square().sum(-1).sqrt() * max(1.0, float(ref.norm() / x.norm()) if x.norm() > 0 else 1.0)
    size = size.repeat_interleave(2, -1) if layout == "interleaved" else torch.cat([size, size], -1)
    return (got - ref).abs(), size


def hold(err, ref, size, dtype):
    bound = 4e-7 * size + (ref.abs() * 2.0 ** -8 * (1 + 1e-6) if dtype == torch.bfloat16 else 0) + 1e-30
    assert (err <= bound).all(), float((err / bound).max())


SIZES = [(1, 1, 2), (3, 5, 6), (16, 16, 32), (7, 128, 64), (200, 1, 64), (33, 3, 256), (1000, 2, 20), (5, 1500, 16)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("inverse", [False, True])
def test_sizes(Q, size, layout, dtype, inverse):
    rows, heads, d = size
    g = torch.Generator().manual_seed(rows + d)
    x = torch.randn((rows, heads, d), generator=g).to(dtype)
    pos = torch.randint(0, 100000, (rows,), generator=g, dtype=torch.int32)
    out = torch.full_like(x, float("nan"), device="cuda")
    Q.rope(x.cuda(), pos.cuda(), out, layout=layout, inverse=inverse)
    assert Q.get_device_status() == 0
    ref = exact(x, pos, frequencies(d, 10000.0, "plain"), layout, inverse)
    err, sz = check(out, ref, x, layout)
    hold(err, ref, sz, dtype)


@pytest.mark.parametrize("kind,factor,original,theta", [("linear", 8.0, 0, 10000.0), ("yarn", 40.0, 4096, 10000.0), ("yarn", 4.0, 32768, 1e6),
                                                        ("yarn", 2.0, 5, 10000.0)])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_scaling(Q, kind, factor, original, theta, layout):
    x = torch.randn((50, 2, 64), generator=torch.Generator().manual_seed(1))
    pos = torch.arange(50, dtype=torch.int32) * 31337
    s = Q.linear_scaling(factor) if kind == "linear" else Q.yarn_scaling(factor, original)
    out = torch.empty_like(x, device="cuda")
    Q.rope(x.cuda(), pos.cuda(), out, theta=theta, layout=layout, scaling=s, attention_factor=1.25)
    ref = exact(x, pos, frequencies(64, theta, kind, factor, original), layout, gain=1.25)
    err, sz = check(out, ref, x, layout)
    hold(err, ref, sz * 1.25, torch.float32)


def test_positions_of_every_size(Q):
    """int32's ends, negative and far positions: the angle stays exact."""
    pos = torch.tensor([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 123456789, -987654321], dtype=torch.int32)
    x = torch.randn((8, 1, 128), generator=torch.Generator().manual_seed(2))
    out = torch.empty_like(x, device="cuda")
    Q.rope(x.cuda(), pos.cuda(), out)
    ref = exact(x, pos, frequencies(128, 10000.0, "plain"), "interleaved")
    err, sz = check(out, ref, x, "interleaved")
    # frequencies have 53 bits: 2^31 turns / 2 pi x 2^-53 are 2.4e-7 rad more on either side
    assert (err <= 1e-6 * sz).all()


def test_given_frequencies(Q):
    f = [0.0, 0.5, 3.0, -2.0]
    x = torch.randn((9, 3, 8), generator=torch.Generator().manual_seed(3))
    pos = torch.arange(9, dtype=torch.int32) * 1000
    out = torch.empty_like(x, device="cuda")
    Q.rope(x.cuda(), pos.cuda(), out, scaling=Q.given_frequencies(f))
    ref = exact(x, pos, np.array(f), "interleaved")
    err, sz = check(out, ref, x, "interleaved")
    hold(err, ref, sz, torch.float32)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("before", [128, 5])
def test_part_of_the_head_in_place(Q, layout, dtype, before):
    """The last 64 of a head's values, aligned and not; the others stay bit for bit."""
    x = torch.randn((20, 6, before + 64), generator=torch.Generator().manual_seed(4)).to(dtype)
    pos = torch.arange(20, dtype=torch.int32) * 7
    d = x.cuda()
    Q.rope(d[..., before:], pos.cuda(), layout=layout)
    assert Q.get_device_status() == 0
    assert torch.equal(d[..., :before].cpu(), x[..., :before])
    ref = exact(x[..., before:], pos, frequencies(64, 10000.0, "plain"), layout)
    err, sz = check(d[..., before:], ref, x[..., before:], layout)
    hold(err, ref, sz, dtype)


def test_strides(Q):
    """Heads outermost, rows every second one, an output with gaps."""
    x = torch.randn((4, 60, 32), generator=torch.Generator().manual_seed(5))
    pos = torch.arange(30, dtype=torch.int32)
    out = torch.full((30, 4, 48), 9.0, device="cuda")
    Q.rope(x.cuda().transpose(0, 1)[::2], pos.cuda(), out[..., 16:])
    assert (out[..., :16] == 9).all()
    src = x.transpose(0, 1)[::2]
    ref = exact(src, pos, frequencies(32, 10000.0, "plain"), "interleaved")
    err, sz = check(out[..., 16:], ref, src, "interleaved")
    hold(err, ref, sz, torch.float32)


def test_there_and_back(Q):
    x = torch.randn((100, 64), generator=torch.Generator().manual_seed(6)).cuda()
    pos = torch.randint(0, 2 ** 30, (100,), dtype=torch.int32).cuda()
    s = Q.yarn_scaling(8.0, 4096)
    y = Q.rope(x.clone(), pos, layout="half", scaling=s)
    Q.rope(y, pos, layout="half", scaling=s, inverse=True)
    assert (y - x).abs().max() <= 8e-7 * x.abs().max() * 2


def test_gradient_is_the_inverse(Q):
    """The backward pass of y = rope(x) is rope(dy, inverse), against the formula's gradient and differences."""
    x = torch.randn((6, 2, 16), generator=torch.Generator().manual_seed(7), dtype=torch.float64)
    dy = torch.randn((6, 2, 16), generator=torch.Generator().manual_seed(8), dtype=torch.float64)
    pos = torch.arange(6, dtype=torch.int32) * 1001
    f = frequencies(16, 10000.0, "plain")
    leaf = x.clone().requires_grad_()
    exact(leaf, pos, f, "half").backward(dy)
    got = Q.rope(dy.float().cuda(), pos.cuda(), layout="half", inverse=True).double().cpu()
    assert (got - leaf.grad).abs().max() <= 1e-6 * dy.abs().max() * 2
    e = torch.zeros_like(x)
    e[3, 1, 5] = 1.0
    diff = ((exact(x + e, pos, f, "half") - exact(x - e, pos, f, "half")) / 2 * dy).sum()
    assert abs(float(got[3, 1, 5] - diff)) <= 2e-6 * float(dy.abs().max())


def test_no_rows(Q):
    Q.rope(torch.empty((0, 2, 8), device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"))


def test_matches_the_fused_rotation(Q):
    """qkmla_append_rope stores what qkmla_rope, then qkmla_append do."""
    N, G, d_c, d_h, d_r = 40, 4, 128, 64, 32
    g = torch.Generator().manual_seed(9)
    c, r = torch.randn((N, d_c), generator=g).cuda(), torch.randn((N, d_r), generator=g).cuda()
    wk = torch.randn((G, d_c, d_h), generator=g).cuda()
    pos = (torch.arange(N, dtype=torch.int32) * 997).cuda()
    slots = torch.arange(N).cuda()
    kv = [torch.zeros((64, d_c + d_r), device="cuda") for _ in range(2)]
    ak = [torch.zeros((64, G), device="cuda") for _ in range(2)]
    Q.append_rope(c, r, pos, 10000.0, wk, None, slots, kv[0], ak[0], 1e-6)
    Q.append(c, Q.rope(r.clone(), pos), wk, None, slots, kv[1], ak[1], 1e-6)
    assert Q.get_device_status() == 0
    assert (kv[0] - kv[1]).abs().max() <= 1e-6 * kv[0].abs().max()
