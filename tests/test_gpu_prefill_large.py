"""qkmla_prefill with a workspace of more than 2^32 bytes: keys and values of its last tiles lie beyond.

Tolerance as in test_gpu_prefill.py: rel-L2 2.7e-3, an lse 7e-3."""
import pytest
import torch

from test_gpu_prefill import Q  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

H, G, D_C, D_H, D_R, D_V, EPS = 8, 8, 64, 128, 64, 128, 1e-6


def exact(c, r, ak, wk, wv, q, qr, first):
    """[n, H, d_v], [n, H]: query i of one sequence sees tokens below first + i."""
    n = q.shape[0]
    q = q.double() / torch.sqrt(q.double().square().mean(-1, keepdim=True) + EPS)
    qr = qr.double() / torch.sqrt(qr.double().square().mean(-1, keepdim=True) + EPS)
    t = torch.arange(c.shape[0], device="cuda")[None, :]
    hidden = t >= first + torch.arange(n, device="cuda")[:, None]
    o, lse = [], []
    for h in range(H):
        k = (c @ wk[h].double()) * ak[:, h:h + 1].double()
        l = (q[:, h] @ k.t() + qr[:, h] @ r.t()) * (D_H + D_R) ** -0.5
        l = l.masked_fill(hidden, -torch.inf)
        lse.append(torch.logsumexp(l, dim=1))
        o.append(torch.exp(l - lse[-1][:, None]) @ (c @ wv[h].double()))
    return torch.stack(o, 1), torch.stack(lse, 1)


def test_workspace_beyond_4_gb(Q):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    lens, new, page = (1050000, 300), (2, 20), 64
    pages = -(-lens[0] // page)
    slots = 2 * pages * page                                   # contiguous: max_pages pages a sequence
    kv = rand(slots, D_C + D_R).bfloat16()
    wk, wv = rand(G, D_C, D_H) / 8, (rand(G, D_C, D_V) / 8).bfloat16()
    c = kv[:, :D_C].float()
    ak = torch.stack([torch.rsqrt((c @ w).square().mean(dim=1) + EPS) for w in wk], dim=1)
    rows = sum(new)
    q, qr = rand(rows, H, D_H), rand(rows, H, D_R)
    ones = torch.ones(D_H, device="cuda")
    o, lse = torch.empty((rows, H, D_V), device="cuda"), torch.empty((rows, H), device="cuda")
    call = Q.prepare_prefill(q, qr, ones, ones, None, Q.prefill_weights(wk, wv), kv, ak, torch.tensor([0, 2, 22], dtype=torch.int32, device="cuda"),
                             torch.tensor(lens, dtype=torch.int32, device="cuda"), None, page, pages, sum(lens), (D_H + D_R) ** -0.5, EPS, o, lse)
    assert call.args.workspace_bytes > 2 ** 32
    call()
    assert Q.get_device_status() == 0
    at = 0
    for b, (n, length) in enumerate(zip(new, lens)):
        s = slice(b * pages * page, b * pages * page + length)
        want, want_lse = exact(kv[s, :D_C].double(), kv[s, D_C:].double(), ak[s], wk, wv, q[at:at + n], qr[at:at + n], length - n + 1)
        assert torch.linalg.norm(o[at:at + n] - want) <= 2.7e-3 * torch.linalg.norm(want)
        assert (lse[at:at + n] - want_lse).abs().max() <= 7e-3
        at += n
