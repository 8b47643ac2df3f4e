"""New tokens written by qkmla_rope and qkmla_read_cache directly ahead of the append that takes them: back to back in a captured
graph, behind kernels long enough that a read ahead of its time would find the old values."""
import pytest
import torch

from test_gpu_q8_window import Q  # noqa: F401

pytestmark = pytest.mark.gpu

G, D_C, D_H, D_R, EPS, FAR = 4, 256, 64, 32, 1e-6, 200000


def rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def caches(q8, slots):
    kv = torch.zeros((slots, D_C + (2 if q8 else 1) * D_R), dtype=torch.uint8 if q8 else torch.bfloat16, device="cuda")
    return kv, torch.zeros(slots, device="cuda") if q8 else None, torch.zeros((slots, G), device="cuda")


def append(Q, q8, c, r, wk, slots, kv, scale, ak):  # noqa: F811
    if q8:
        return Q.prepare_append_q8(c, r, wk, None, slots, kv, scale, ak, EPS)
    return Q.prepare_append(c, r, wk, None, slots, kv, ak, EPS)


def replay(calls, reset, outputs, times=10):
    """The calls one by one, each waited for, and replayed from a graph: the same bits."""
    reset()
    for call in calls:
        call()
        torch.cuda.synchronize()
    want = [t.clone() for t in outputs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for call in calls:
            call()
    for _ in range(times):
        reset()
        for t in outputs:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outputs, want))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("n", [1, 16, 200])
def test_rope_then_append(Q, n, q8):  # noqa: F811
    """The last n of many keys that one call turns."""
    g = torch.Generator(device="cuda").manual_seed(n)
    raw, c, wk = rand(g, FAR, D_R), rand(g, n, D_C), rand(g, G, D_C, D_H) / 16
    x = raw.clone()
    pos = torch.randint(1, 100000, (FAR,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.arange(n, device="cuda")
    kv, scale, ak = caches(q8, 256)
    outputs = [kv, ak] + ([scale] if q8 else [])
    calls = [Q.prepare_rope(x, pos, x), append(Q, q8, c, x[-n:], wk, slots, kv, scale, ak)]
    replay(calls, lambda: x.copy_(raw), outputs)
    assert Q.get_device_status() == 0


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("n", [1, 16, 200])
def test_read_then_append(Q, n, q8):  # noqa: F811
    """The last n of many rows that one call reads back, turned to other positions between, too."""
    g = torch.Generator(device="cuda").manual_seed(n + 1)
    wk = rand(g, G, D_C, D_H) / 16
    src = rand(g, FAR, D_C + D_R).bfloat16()
    start = torch.tensor([0, FAR], dtype=torch.int32, device="cuda")
    c, r = torch.empty((FAR, D_C), device="cuda"), torch.empty((FAR, D_R), device="cuda")
    slots = torch.arange(n, device="cuda")
    pos = torch.randint(1, 100000, (n,), generator=g, device="cuda", dtype=torch.int32)
    read = Q.prepare_read_cache(src, None, start, None, 64, FAR // 64, c, r)
    for turn in (False, True):
        kv, scale, ak = caches(q8, 256)
        outputs = [kv, ak] + ([scale] if q8 else [])
        calls = [read] + ([Q.prepare_rope(r[-n:], pos, r[-n:])] if turn else []) + [append(Q, q8, c[-n:], r[-n:], wk, slots, kv, scale, ak)]
        replay(calls, lambda: (c.zero_(), r.zero_()), outputs)
    assert Q.get_device_status() == 0


def test_two_appends_behind_two_ropes(Q):  # noqa: F811
    """The second append's keys were turned before the first append, which lets it start early."""
    g = torch.Generator(device="cuda").manual_seed(3)
    raw = [rand(g, FAR, D_R) for _ in range(2)]
    xs = [t.clone() for t in raw]
    c, wk = rand(g, 16, D_C), rand(g, G, D_C, D_H) / 16
    pos = torch.randint(1, 100000, (FAR,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.arange(16, device="cuda")
    outs = [caches(False, 64) for _ in xs]
    calls = [Q.prepare_rope(x, pos, x) for x in xs] + [append(Q, False, c, x[-16:], wk, slots, *o) for x, o in zip(xs, outs)]
    replay(calls, lambda: [x.copy_(t) for x, t in zip(xs, raw)], [o[k] for o in outs for k in (0, 2)])
    assert Q.get_device_status() == 0


@pytest.mark.parametrize("q8", [False, True])
def test_layers_in_a_row(Q, q8):  # noqa: F811
    """rope, append, prefill and read_cache of three layers, nothing waiting on the host between them."""
    H, D_V, B, N, PAGE = 16, 64, 3, 130, 16
    g = torch.Generator(device="cuda").manual_seed(9)
    pages = 40
    table = torch.randperm(B * pages, generator=g, device="cuda").to(torch.int32).view(B, pages)
    lens = torch.tensor([600, 131, 333], dtype=torch.int32, device="cuda")
    start = torch.arange(0, B * N + 1, N, dtype=torch.int32, device="cuda")
    t = torch.cat([torch.arange(int(n) - N, int(n), device="cuda") for n in lens])
    b = torch.arange(B, device="cuda").repeat_interleave(N)
    slots = table.long()[b, t // PAGE] * PAGE + t % PAGE
    pos = t.to(torch.int32)
    ones_h, ones_r = torch.ones(D_H, device="cuda"), torch.ones(D_R, device="cuda")
    calls, outputs, raws, kept = [], [], [], []               # (prepared calls hold addresses alone: what they name is kept)
    for _ in range(3):
        wk, wv = rand(g, G, D_C, D_H) / 16, (rand(g, G, D_C, D_V) / 16).bfloat16()
        kv, scale, ak = caches(q8, B * pages * PAGE)
        old = torch.arange(B * pages * PAGE, device="cuda")
        past = rand(g, len(old), D_C), rand(g, len(old), D_R)
        append(Q, q8, *past, wk, old, kv, scale, ak)()
        torch.cuda.synchronize()
        raw_k, raw_q = rand(g, B * N, D_R), rand(g, B * N, H, D_R)
        k, qr, new, q = raw_k.clone(), raw_q.clone(), rand(g, B * N, D_C), rand(g, B * N, H, D_H)
        raws += [(k, raw_k), (qr, raw_q)]
        weights, first = Q.prefill_weights(wk, wv), lens - N
        o = torch.empty((B * N, H, D_V), device="cuda")
        c, r, a = (torch.empty((B * N, n), device="cuda") for n in (D_C, D_R, G))
        calls += [Q.prepare_rope(k, pos, k), Q.prepare_rope(qr, pos, qr, layout="half"),
                  append(Q, q8, new, k, wk, slots, kv, scale, ak),
                  Q.prepare_prefill(q, qr, ones_h, ones_h, ones_r, weights, kv, ak, start, lens, table, PAGE, pages, int(lens.sum()), 0.1, EPS,
                                    o, kv_scale=scale),
                  Q.prepare_read_cache(kv, ak, start, table, PAGE, pages, c, r, a, kv_scale=scale, first=first)]
        outputs += [o, c, r, a]
        kept.append((wk, wv, kv, scale, ak, new, q, weights, first))
    replay(calls, lambda: [x.copy_(y) for x, y in raws], outputs)
    assert Q.get_device_status() == 0
