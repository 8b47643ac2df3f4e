"""Rows read back from a cache and appended to a bf16 one: the same rows there, and decode over them gives the same.

Tolerance.  Latents are bf16 or 8-bit numbers: the bf16 cache holds them bit for bit, and alpha^k is formed from the same numbers by
the same call (two kernels: 1e-5).  A RoPE key, normalised and rounded once, is normalised and rounded again: its root mean square is
off by at most 2^-8, and each element rounded by 2^-8, 2^-7 (1 + 2^-8) together.  In decode (fp32 throughout) the RoPE part of a logit, of
root mean square sqrt(32 / 96), is then off by at most 2^-8 of itself for the common factor and 2^-8 / sqrt 3 for the roundings,
in quadrature 2.6e-3, a softmax weight and the output by sqrt 2 times that, 3.7e-3."""
import pytest
import torch

from test_gpu_q8_window import Q  # noqa: F401

pytestmark = pytest.mark.gpu

H, G, D_C, D_H, D_R, PAGE, EPS = 16, 4, 256, 64, 32, 16, 1e-6
LENS = (700, 33, 250)


def rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def decode(Q, x, kv, ak, scale, table, lens):  # noqa: F811
    o, lse = torch.empty((len(LENS), 1, H, D_C), device="cuda"), torch.empty((len(LENS), 1, H), device="cuda")
    Q.decode(*x, None, kv, ak, lens, table, PAGE, table.shape[1], G, (D_H + D_R) ** -0.5, EPS, o, lse, force_simt=True, kv_scale=scale)
    assert Q.get_device_status() == 0
    return o, lse


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cache", ["bf16", "q8"])
def test_decodes_alike(Q, cache, out):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(21)
    n = sum(LENS)
    wk = rand(g, G, D_C, D_H) / D_C ** 0.5
    pages = [-(-k // PAGE) for k in LENS]
    total = sum(pages)
    table = torch.full((3, max(pages)), -1, dtype=torch.int32, device="cuda")
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = perm[at:at + k]
        at += k
    slots = torch.cat([table[b].long()[torch.arange(k, device="cuda") // PAGE] * PAGE + torch.arange(k, device="cuda") % PAGE
                       for b, k in enumerate(LENS)])
    lens = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 700, 733, n], dtype=torch.int32, device="cuda")
    c, r = rand(g, n, D_C), rand(g, n, D_R)
    q8 = cache == "q8"
    kv = torch.zeros((total * PAGE, D_C + (2 if q8 else 1) * D_R), dtype=torch.uint8 if q8 else torch.bfloat16, device="cuda")
    scale = torch.zeros(total * PAGE, device="cuda") if q8 else None
    ak = torch.zeros((total * PAGE, G), device="cuda")
    if q8:
        Q.append_q8(c, r, wk, None, slots, kv, scale, ak, EPS)
    else:
        Q.append(c, r, wk, None, slots, kv, ak, EPS)
    # out of that cache and into a bf16 one of its own
    back = [torch.empty((n, w), dtype=out, device="cuda") for w in (D_C, D_R)]
    Q.read_cache(kv, ak, start, table, PAGE, table.shape[1], *back, kv_scale=scale)
    c2, r2 = (t.float() for t in back)
    kv2 = torch.zeros((total * PAGE, D_C + D_R), dtype=torch.bfloat16, device="cuda")
    ak2 = torch.zeros((total * PAGE, G), device="cuda")
    Q.append(c2, r2, wk, None, slots, kv2, ak2, EPS)
    assert Q.get_device_status() == 0
    # what was read is what the rows hold
    if q8:
        held = kv[slots, :D_C].view(torch.float8_e4m3fn).float() * scale[slots][:, None]
        keys = kv[slots, D_C:].contiguous().view(torch.bfloat16).float()
    else:
        held, keys = kv[slots, :D_C].float(), kv[slots, D_C:].float()
    assert torch.equal(c2, held) and torch.equal(r2, keys)
    assert torch.equal(kv2[slots, :D_C].float(), held)
    assert ((kv2[slots, D_C:].float() - keys).abs() <= 2.0 ** -7 * (1 + 2.0 ** -8) * keys.abs()).all()
    assert ((ak2 - ak)[slots].abs() <= 1e-5 * ak[slots]).all()
    # the same queries over both
    x = (rand(g, 3, 1, H, D_C).bfloat16(), rand(g, 3, 1, H).abs() * 0.1, rand(g, 3, 1, H, D_R))
    o, lse = decode(Q, x, kv, ak, scale, table, lens)
    o2, lse2 = decode(Q, x, kv2, ak2, None, table, lens)
    assert torch.linalg.norm(o - o2) <= 3.7e-3 * torch.linalg.norm(o)
    assert (lse - lse2).abs().max() <= 5 * 2.6e-3
