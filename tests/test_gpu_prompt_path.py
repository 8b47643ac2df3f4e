"""A prompt's way through the library: project_query, rope, append, prefill in chunks, decode, read_cache and back into
another cache."""
import numpy as np
import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu

H, G, D_C, D_H, D_R, D_V, PAGE, EPS = 16, 4, 256, 64, 32, 64, 16, 1e-6
SCALE = 1 / np.sqrt(D_H + D_R)


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from qk_normed_latent_gb300 import build as B
    B.build()
    import qk_normed_latent_gb300 as Q
    return Q


def rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


class Prompt:
    """One layer's weights, a prompt's inputs, and an empty cache."""

    def __init__(self, n, q8):
        g = torch.Generator(device="cuda").manual_seed(11)
        self.n, self.q8 = n, q8
        self.wq = (rand(g, H, D_H + D_R, 256) / 16).bfloat16()
        self.wk, self.wv = rand(g, G, D_C, D_H) / 16, (rand(g, G, D_C, D_V) / 16).bfloat16()
        self.gq, self.gk, self.grq = 1 + 0.1 * rand(g, D_H), 1 + 0.1 * rand(g, D_H), 1 + 0.1 * rand(g, D_R)
        self.x, self.c, self.r = rand(g, n, 256).bfloat16(), rand(g, n, D_C), rand(g, n, D_R)
        self.pages = (n + PAGE - 1) // PAGE
        self.table = torch.randperm(self.pages, generator=g, device="cuda").to(torch.int32)[None].contiguous()
        slots = self.pages * PAGE
        self.kv = torch.zeros((slots, D_C + (2 if q8 else 1) * D_R), dtype=torch.uint8 if q8 else torch.bfloat16, device="cuda")
        self.kv_scale = torch.zeros(slots, device="cuda") if q8 else None
        self.ak = torch.zeros((slots, G), device="cuda")

    def slots(self, a, b):
        t = torch.arange(a, b, device="cuda")
        return self.table[0].long()[t // PAGE] * PAGE + t % PAGE

    def queries(self, Q, a, b, scaling):
        """Rows a .. b - 1: projected without a rotation (position 0), then turned by their scaled positions."""
        q, qr = torch.empty((b - a, H, D_H), device="cuda"), torch.empty((b - a, H, D_R), device="cuda")
        pos = torch.arange(a, b, dtype=torch.int32, device="cuda")
        Q.project_query(self.x[a:b].contiguous(), self.wq, torch.zeros_like(pos), 10000.0, q, qr)
        Q.rope(qr, pos, scaling=scaling)
        return q, qr

    def append(self, Q, a, b, scaling):
        pos = torch.arange(a, b, dtype=torch.int32, device="cuda")
        r = Q.rope(self.r[a:b].clone(), pos, scaling=scaling)
        if self.q8:
            Q.append_q8(self.c[a:b].contiguous(), r, self.wk, None, self.slots(a, b), self.kv, self.kv_scale, self.ak, EPS)
        else:
            Q.append(self.c[a:b].contiguous(), r, self.wk, None, self.slots(a, b), self.kv, self.ak, EPS)

    def prefill(self, Q, weights, a, b, scaling, o):
        q, qr = self.queries(Q, a, b, scaling)
        Q.prefill(q, qr, self.gq, self.gk, self.grq, weights, self.kv, self.ak, torch.tensor([0, b - a], dtype=torch.int32, device="cuda"),
                  torch.tensor([b], dtype=torch.int32, device="cuda"), self.table, PAGE, self.pages, b, SCALE, EPS, o[a:b],
                  kv_scale=self.kv_scale)


@pytest.mark.parametrize("q8", [False, True])
def test_prompt_in_chunks_then_decode(Q, q8):
    """Chunks one after the other give what the whole prompt does, and a decode step what the last query did."""
    n, cuts = 700, [0, 1, 130, 500, 700]
    s = Q.yarn_scaling(8.0, 256)
    p = Prompt(n, q8)
    weights = Q.prefill_weights(p.wk, p.wv)
    chunked = torch.full((n, H, D_V), float("nan"), device="cuda")
    for a, b in zip(cuts, cuts[1:]):
        p.append(Q, a, b, s)
        p.prefill(Q, weights, a, b, s, chunked)
    whole = torch.full_like(chunked, float("nan"))
    p.prefill(Q, weights, 0, n, s, whole)
    assert Q.get_device_status() == 0
    # each is within 2.7e-3 of the exact result (rounding of fp16 operands), so they are within twice that of one another
    assert torch.linalg.norm(chunked - whole) <= 5.4e-3 * torch.linalg.norm(whole)
    q, qr = p.queries(Q, n - 1, n, s)
    qt, aq = torch.empty((1, H, D_C), dtype=torch.bfloat16, device="cuda"), torch.empty((1, H), device="cuda")
    Q.absorb_query(q, p.gq, p.gk, p.wk, EPS, qt, aq)
    lat, lse = torch.empty((1, 1, H, D_C), device="cuda"), torch.empty((1, 1, H), device="cuda")
    Q.decode(qt[None], aq[None], qr[None], p.grq, p.kv, p.ak, torch.tensor([n], dtype=torch.int32, device="cuda"), p.table, PAGE, p.pages,
             G, SCALE, EPS, lat, lse, kv_scale=p.kv_scale, force_simt=True)
    v = torch.empty((1, H, D_V), device="cuda")
    Q.up_project(lat.view(1, H, D_C), p.wv, v)
    assert Q.get_device_status() == 0
    # decode's bf16 (8-bit: two-part) query and weights: the method's rule, 5e-3, beside prefill's 2.7e-3
    assert torch.linalg.norm(v[0] - whole[-1]) <= 7.7e-3 * torch.linalg.norm(v)


def test_prefix_moved_to_other_positions(Q):
    """A cached prefix read back, its RoPE keys turned back and on to other positions, and appended to another cache: prefill
    over it gives what the prompt at those positions does."""
    n, shift = 200, 3000
    p = Prompt(n, False)
    weights = Q.prefill_weights(p.wk, p.wv)
    p.append(Q, 0, n, None)
    c, r = torch.empty((n, D_C), device="cuda"), torch.empty((n, D_R), device="cuda")
    Q.read_cache(p.kv, p.ak, torch.tensor([0, n], dtype=torch.int32, device="cuda"), p.table, PAGE, p.pages, c, r)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    Q.rope(r, pos, inverse=True)
    moved = Prompt(n, False)
    moved.c.copy_(c)
    Q.rope(r, pos + shift)
    Q.append(moved.c, r, moved.wk, None, moved.slots(0, n), moved.kv, moved.ak, EPS)
    # the same prompt at the shifted positions, from its inputs
    direct = Prompt(n, False)
    Q.append(direct.c, Q.rope(direct.r.clone(), pos + shift), direct.wk, None, direct.slots(0, n), direct.kv, direct.ak, EPS)
    out = []
    for x in (moved, direct):
        q, qr = torch.empty((n, H, D_H), device="cuda"), torch.empty((n, H, D_R), device="cuda")
        Q.project_query(x.x, x.wq, pos + shift, 10000.0, q, qr)
        o = torch.empty((n, H, D_V), device="cuda")
        Q.prefill(q, qr, x.gq, x.gk, x.grq, weights, x.kv, x.ak, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                  torch.tensor([n], dtype=torch.int32, device="cuda"), x.table, PAGE, x.pages, n, SCALE, EPS, o)
        out.append(o)
    assert Q.get_device_status() == 0
    # the RoPE key is rounded to bf16 twice instead of once: 2^-8 of itself more, the RoPE part of a logit by at most that times its
    # root mean square, sqrt(32 / 96), and a softmax weight by sqrt 2 times it: 3.2e-3; beside it 2.7e-3 each
    assert torch.linalg.norm(out[0] - out[1]) <= (3.2e-3 + 5.4e-3) * torch.linalg.norm(out[1])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_pipeline(Q, cache):
    """DeviceState.prefill of a step's queries: decode's result, up-projected."""
    from qk_normed_latent_gb300.pipeline import DeviceState
    w = W.small(W.WORKLOADS[4].with_(cache_dtype=cache), 3, (300, 77, 900))
    st = DeviceState(w)
    st.step()
    w_v = (torch.randn((w.G, w.d_c, 128), device="cuda") / w.d_c ** 0.5).bfloat16()
    got = st.prefill(w_v, o_dtype=torch.float32)
    want = torch.empty_like(got)
    Q.up_project(st.o.view(w.rows, w.H, w.d_c), w_v, want)
    assert Q.get_device_status() == 0
    assert torch.linalg.norm(got - want) <= 7.7e-3 * torch.linalg.norm(want)
