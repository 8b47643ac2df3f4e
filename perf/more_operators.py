"""Measured cases of the operators that bring a prompt through the latent cache.

Three operators, each one pass as a serving program makes it:

  prefill  attention of a chunk of new tokens over the paged latent cache: keys and
           values of the cached tokens recovered from their latents, QK-normalised
           logits, a causal (or windowed) softmax, per-head values
  rope     rotary positions in both layouts, on part of a head, scaled for long contexts
  read     rows of the paged cache read back into contiguous latents and RoPE keys

`own` False: elementary torch operations.  `own` True: the library.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
LARGE = dict(H=128, G=8, G_v=8, d_c=512, d_h=128, d_r=64, d_v=128)
SMALL = dict(H=16, G=4, G_v=4, d_c=256, d_h=64, d_r=32, d_v=64)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _prefill(name, shape, cache, B, new, ctx, page, window=0, sinks=0):
    """`new`, `ctx`: bounds of the sequences' new tokens and of their whole lengths."""
    return {"name": name, "op": "prefill", "cache": cache, "B": B, "new_lo": new[0], "new_hi": new[1], "lo": ctx[0],
            "hi": ctx[1], "page": page, "window": window, "sinks": sinks, **shape}


def _rope(name, rows, heads, d, d_r, dtype, layout, factor, original, far, inverse=False):
    """d_r of each head's d values are rotated, the last ones; positions up to `far`."""
    return {"name": name, "op": "rope", "rows": rows, "heads": heads, "d": d, "d_r": d_r, "dtype": dtype,
            "layout": layout, "factor": factor, "original": original, "far": far, "inverse": inverse}


def _read(name, cache, out, B, lo, hi, page, G, d_c, d_r):
    return {"name": name, "op": "read", "cache": cache, "out": out, "B": B, "lo": lo, "hi": hi, "page": page, "G": G,
            "d_c": d_c, "d_r": d_r}


def listed():
    return [
        # a short follow-up question in one chat of a small model: the latency of a call
        _prefill("prefill_one_short", SMALL, "bf16", 1, (17, 17), (333, 333), 64),
        # a small model's batch: chunks of every length, single decode tokens among them
        _prefill("prefill_small_batch", SMALL, "bf16", 16, (1, 512), (1024, 8192), 64),
        # four whole prompts of a large model, from an empty 8-bit cache
        _prefill("prefill_large_prompts", LARGE, "q8", 4, (4096, 4096), (4096, 4096), 64),
        # one chunk of a chunked prefill in the middle of a document
        _prefill("prefill_large_chunk", LARGE, "bf16", 1, (1024, 1024), (16000, 16000), 64),
        # a question about a very long document: few rows, a long axis
        _prefill("prefill_large_long", LARGE, "q8", 1, (256, 256), (131072, 131072), 64),
        # a continuous batch: decode tokens and short chunks over ragged contexts, small pages
        _prefill("prefill_large_mixed", LARGE, "bf16", 8, (1, 300), (300, 8192), 16),
        # chunks of two long conversations behind a window and sinks
        _prefill("prefill_large_window", LARGE, "bf16", 2, (1000, 1000), (9000, 20000), 64, 4096, 4),
        # one decode step's RoPE queries of a small model
        _rope("rope_step", 16, 16, 32, 32, "f32", "interleaved", 1.0, 4096, 8192),
        # a prompt chunk's queries of a large model: the last 64 of 192 values, long-context scaling
        _rope("rope_queries", 4096, 128, 192, 64, "bf16", "half", 40.0, 4096, 163840),
        # the keys of a cached prefix turned back, to be moved to another position
        _rope("rope_keys_back", 16001, 1, 64, 64, "f32", "interleaved", 8.0, 8192, 65536, True),
        # a long shared prefix read back from the 8-bit cache
        _read("read_prefix", "q8", "bf16", 1, 32768, 32768, 64, 8, 512, 64),
        # a ragged batch's contexts read back to full precision, small pages
        _read("read_ragged", "bf16", "f32", 16, 333, 8192, 16, 4, 256, 32),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["prefill", "prefill", "prefill", "rope", "read"])
    large = rng.random() < 0.5
    shape = dict(LARGE if large else SMALL)
    if op == "rope":
        d_r = rng.choice([32, 64, 128])
        heads = rng.choice([1, 2, 16, 128])
        case = _rope("", log(1, 500000 // heads // d_r * 64), heads, d_r + rng.choice([0, 64, 128]), d_r,
                     rng.choice(["f32", "bf16"]), rng.choice(["interleaved", "half"]), rng.choice([1.0, 4.0, 40.0]),
                     rng.choice([4096, 8192]), log(16, 1000000), rng.random() < 0.3)
    elif op == "read":
        hi = log(16, 65536)
        case = _read("", rng.choice(["q8", "bf16"]), rng.choice(["bf16", "f32"]), max(1, min(log(1, 64), 131072 // hi)),
                     max(1, hi // rng.choice([1, 2, 16])), hi, rng.choice([1, 16, 48, 64, 128]), shape["G"], shape["d_c"],
                     shape["d_r"])
    else:
        H, G, G_v = rng.choice([(128, 8, 8), (64, 8, 8), (32, 4, 4), (16, 16, 16)] if large else [(16, 4, 4), (32, 4, 2), (16, 2, 4)])
        shape.update(H=H, G=G, G_v=G_v)
        hi = log(64, 65536 if large else 131072)
        lo = max(1, hi // rng.choice([1, 2, 8]))
        # every pair of a new token and a context token, padded to the longest, at most 2^25 for 128 heads
        new = log(1, max(1, min(lo, 2 ** 25 * 128 // H // hi // 2, 8192)))
        B = max(1, min(log(1, 32), 2 ** 25 * 128 // H // (hi * new), 262144 // hi))
        window = sinks = 0
        if rng.random() < 0.25:
            window, sinks = log(1, 8192), rng.choice([0, 1, 4, rng.randrange(300)])
        case = _prefill("", shape, rng.choice(["bf16", "q8"]), B, (max(1, new // rng.choice([1, 4, 64])), new), (lo, hi),
                        rng.choice([1, 16, 48, 64, 128]), window, sinks)
    return {k: v for k, v in case.items() if k != "name"}


def _spread(case, lo, hi, salt):
    """Whole numbers, one a sequence, log-uniform in [lo, hi]: part of the case, the same for every seed."""
    g = np.random.Generator(np.random.PCG64([lo, hi, case["B"], salt]))
    n = np.exp(g.uniform(math.log(lo), math.log(hi), size=case["B"]))
    return np.clip(np.round(n), lo, hi).astype(np.int64)


def _lens(case):
    return _spread(case, case["lo"], case["hi"], 0)


def _new(case):
    return np.minimum(_spread(case, case["new_lo"], case["new_hi"], 1), _lens(case))


def _seen(case, n, length):
    """(sum over the sequence's new tokens of the tokens each attends to, tokens that any of them attends to)."""
    ends = np.arange(length - n + 1, length + 1)
    if not case["window"]:
        return int(ends.sum()), length
    first = np.maximum(ends - case["window"], 0)
    head = np.minimum(first, case["sinks"])
    return int((ends - first + head).sum()), int(length - first[0] + head[0])


def work(case):
    if case["op"] == "rope":
        rotated = case["rows"] * case["heads"] * case["d_r"]
        return {"bytes": rotated * 2 * (4 if case["dtype"] == "f32" else 2) + 4 * case["rows"], "flops": 3 * rotated}
    d_c, d_r, G = case["d_c"], case["d_r"], case["G"]
    token = d_c + 2 * d_r + 4 if case["cache"] == "q8" else 2 * (d_c + d_r)
    if case["op"] == "read":
        n = int(_lens(case).sum())
        return {"bytes": n * (token + 4 * G + (d_c + d_r) * (4 if case["out"] == "f32" else 2) + 4 * G), "flops": n * d_c}
    H, G_v, d_h, d_v = case["H"], case["G_v"], case["d_h"], case["d_v"]
    seen = [_seen(case, n, length) for n, length in zip(_new(case).tolist(), _lens(case).tolist())]
    pairs, tokens, rows = sum(p for p, _ in seen), sum(t for _, t in seen), int(_new(case).sum())
    recover = 2 * d_c * (G * d_h + G_v * d_v)
    return {"bytes": tokens * (token + 4 * G) + rows * H * (4 * (d_h + d_r) + 2 * d_v) + d_c * (4 * G * d_h + 2 * G_v * d_v),
            "flops": pairs * H * 2 * (d_h + d_r + d_v) + tokens * recover}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _quantise(c):
    """e4m3 codes (as uint8) and the power-of-two scale of each row of c [N, d_c] fp32: the
    least 2^e with max|c| <= 448 2^e."""
    mant, exp = torch.frexp(c.abs().amax(dim=1))
    exp = (exp - torch.where(mant <= 0.875, 9, 8)).clamp(-126, 120)
    codes = (c * torch.ldexp(torch.ones_like(mant), -exp)[:, None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), torch.ldexp(torch.ones_like(mant), exp)


def _cache(case, gen, s):
    """A paged cache of the case's contexts, its pages in random order."""
    d_c, d_r, G, page = case["d_c"], case["d_r"], case["G"], case["page"]
    lens = _lens(case)
    pages = -(-lens // page)
    total = int(pages.sum())
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    inside = np.arange(int(pages.max()))[None, :] < pages[:, None]
    table = torch.full(inside.shape, -1, dtype=torch.int32, device="cuda")
    table[torch.from_numpy(inside).cuda()] = perm
    slots = total * page
    q8 = case["cache"] == "q8"
    kv = torch.empty((slots, d_c + 2 * d_r), dtype=torch.uint8, device="cuda") if q8 else torch.empty(
        (slots, d_c + d_r), dtype=torch.bfloat16, device="cuda")
    scale = torch.empty(slots, device="cuda") if q8 else None
    ak = torch.empty((slots, G), device="cuda")
    grk = 1 + 0.1 * torch.randn(d_r, generator=gen, device="cuda")
    for i in range(0, slots, 131072):
        n = min(131072, slots - i)
        c = torch.randn((n, d_c), generator=gen, device="cuda")
        c *= torch.where(torch.rand(n, generator=gen, device="cuda") < 0.05, 30.0, 1.0)[:, None]
        r = torch.randn((n, d_r), generator=gen, device="cuda")
        r = (r * grk * torch.rsqrt(r.square().mean(dim=1, keepdim=True) + EPS)).bfloat16()
        if q8:
            codes, sc = _quantise(c)
            kv[i:i + n, :d_c], scale[i:i + n] = codes, sc
            kv[i:i + n, d_c:] = r.view(torch.uint8)
            c = codes.view(torch.float8_e4m3fn).float() * sc[:, None]
        else:
            kv[i:i + n, :d_c], kv[i:i + n, d_c:] = c.bfloat16(), r
            c = c.bfloat16().float()
        if "wk" in s:
            ak[i:i + n] = torch.stack([torch.rsqrt((c @ w).square().mean(dim=1) + EPS) for w in s["wk"]], dim=1)
        else:
            ak[i:i + n] = torch.rand((n, G), generator=gen, device="cuda") + 0.5
    s.update(kv=kv, scale=scale, ak=ak, table=table, lens=torch.from_numpy(lens.astype(np.int32)).cuda(),
             total=int(lens.sum()))


def _starts(n):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "rope":
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        rows, heads, d, d_r = case["rows"], case["heads"], case["d"], case["d_r"]
        s["x"] = torch.randn((rows, heads, d), generator=gen, device="cuda").to(dt)
        s["positions"] = torch.randint(0, case["far"], (rows,), generator=gen, device="cuda", dtype=torch.int32)
        s["out"] = torch.empty((rows, heads, d_r), dtype=dt, device="cuda")
        return s
    d_c, d_r, G = case["d_c"], case["d_r"], case["G"]
    if case["op"] == "read":
        _cache(case, gen, s)
        dt = torch.float32 if case["out"] == "f32" else torch.bfloat16
        n = s["total"]
        s.update(starts=_starts(_lens(case)), c=torch.empty((n, d_c), dtype=dt, device="cuda"),
                 r=torch.empty((n, d_r), dtype=dt, device="cuda"), a=torch.empty((n, G), device="cuda"))
        return s
    H, G_v, d_h, d_v = case["H"], case["G_v"], case["d_h"], case["d_v"]
    s["wk"] = torch.randn((G, d_c, d_h), generator=gen, device="cuda") / math.sqrt(d_c)
    s["wv"] = (torch.randn((G_v, d_c, d_v), generator=gen, device="cuda") / math.sqrt(d_c)).bfloat16()
    _cache(case, gen, s)
    rows = int(_new(case).sum())
    s.update(q=torch.randn((rows, H, d_h), generator=gen, device="cuda"),
             qr=torch.randn((rows, H, d_r), generator=gen, device="cuda"),
             gq=1 + 0.1 * torch.randn(d_h, generator=gen, device="cuda"),
             gk=1 + 0.1 * torch.randn(d_h, generator=gen, device="cuda"),
             grq=1 + 0.1 * torch.randn(d_r, generator=gen, device="cuda"),
             starts=_starts(_new(case)), longest=int(_new(case).max()), softmax_scale=1.0 / math.sqrt(d_h + d_r),
             o=torch.empty((rows, H, d_v), dtype=torch.bfloat16, device="cuda"))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _frequencies(case, device):
    """Radians a position of each pair, in 64 bits: theta^(-2i/d), and for a context `factor` times the
    original one the slow pairs divided by it, the fast ones kept, a ramp between (32 and 1 turns within
    the original context)."""
    d, theta = case["d_r"], 10000.0
    i = torch.arange(d // 2, dtype=torch.float64, device=device)
    f = theta ** (-2 * i / d)
    if case["factor"] == 1.0:
        return f
    low, high = (d * math.log(case["original"] / (turns * 2 * math.pi)) / (2 * math.log(theta)) for turns in (32, 1))
    low, high = max(math.floor(low), 0), min(math.ceil(high), d - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return f / case["factor"] * ramp + f * (1 - ramp)


def _plain_rope(s):
    case = s["case"]
    d = case["d_r"]
    x = s["x"][..., case["d"] - d:].float()
    angle = s["positions"].double()[:, None] * _frequencies(case, "cuda")
    if case["inverse"]:
        angle = -angle
    c, n = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if case["layout"] == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        s["out"].copy_(torch.stack([a * c - b * n, a * n + b * c], dim=-1).flatten(-2))
    else:
        a, b = x[..., :d // 2], x[..., d // 2:]
        s["out"].copy_(torch.cat([a * c - b * n, a * n + b * c], dim=-1))


def _rows(s, slot):
    """Latents and RoPE keys of cache slots, in fp32."""
    d_c = s["case"]["d_c"]
    rows = s["kv"][slot]
    if s["scale"] is None:
        return rows[..., :d_c].float(), rows[..., d_c:].float()
    c = rows[..., :d_c].view(torch.float8_e4m3fn).float() * s["scale"][slot][..., None]
    return c, rows[..., d_c:].contiguous().view(torch.bfloat16).float()


def _plain_read(s):
    page = s["case"]["page"]
    at = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(s["starts"][1:].long(), at, right=True)
    t = at - s["starts"].long()[b]
    slot = s["table"].long()[b, t // page] * page + t % page
    c, r = _rows(s, slot)
    s["c"].copy_(c)
    s["r"].copy_(r)
    s["a"].copy_(s["ak"][slot])


def _plain_prefill(s):
    case = s["case"]
    B, H, G, G_v, page = case["B"], case["H"], case["G"], case["G_v"], case["page"]
    d_h, d_r, d_v, N = case["d_h"], case["d_r"], case["d_v"], s["longest"]
    length, start = s["lens"].long(), s["starts"].long()
    n = start[1:] - start[:-1]
    t = torch.arange(case["hi"], device="cuda")[:int(s["table"].shape[1]) * page].expand(B, -1)
    there = t < length[:, None]
    t = torch.where(there, t, 0)
    slot = torch.gather(s["table"].long(), 1, t // page) * page + t % page
    c, r = _rows(s, slot)                                                     # [B, L, d]
    L = t.shape[1]
    k = torch.matmul(c[:, None], s["wk"]) * s["ak"][slot].transpose(1, 2)[..., None]      # [B, G, L, d_h]
    i = torch.arange(N, device="cuda")
    row = torch.where(i < n[:, None], start[:-1, None] + i, 0)                # [B, N], short chunks padded
    q, qr = s["q"][row], s["qr"][row]
    q = q * (s["gq"] * s["gk"]) * torch.rsqrt(q.square().mean(dim=-1, keepdim=True) + EPS)
    qr = qr * s["grq"] * torch.rsqrt(qr.square().mean(dim=-1, keepdim=True) + EPS)
    q = q.transpose(1, 2).reshape(B, G, H // G * N, d_h)
    logit = torch.matmul(q, k.transpose(2, 3)).view(B, H * N, L)
    del k
    logit += torch.matmul(qr.transpose(1, 2).reshape(B, H * N, d_r), r.transpose(1, 2))
    logit = logit.view(B, H, N, L).mul_(s["softmax_scale"])
    end = (length[:, None] - n[:, None] + i + 1)[..., None]                   # [B, N, 1]
    seen = there[:, None] & (t[:, None] < end)
    if case["window"]:
        seen &= (t[:, None] < case["sinks"]) | (t[:, None] >= end - case["window"])
    logit.masked_fill_(~seen[:, None], -math.inf)
    p = logit.sub_(logit.amax(dim=-1, keepdim=True)).exp_()
    v = torch.matmul(c[:, None], s["wv"].float())                             # [B, G_v, L, d_v]
    o = torch.matmul(p.view(B, G_v, H // G_v * N, L), v).view(B, H, N, d_v) / p.sum(dim=-1, keepdim=True)
    s["o"].copy_(o.transpose(1, 2)[i < n[:, None]])


def _call(s):
    """The library's call with its arguments marshalled, as a serving loop over fixed buffers keeps it."""
    import qk_normed_latent_gb300 as Q
    case = s["case"]
    if case["op"] == "rope":
        scaling = None if case["factor"] == 1.0 else Q.yarn_scaling(case["factor"], case["original"])
        return Q.prepare_rope(s["x"][..., case["d"] - case["d_r"]:], s["positions"], s["out"], theta=10000.0,
                              layout=case["layout"], scaling=scaling, inverse=case["inverse"])
    if case["op"] == "read":
        return Q.prepare_read_cache(s["kv"], s["ak"], s["starts"], s["table"], case["page"], s["table"].shape[1],
                                    s["c"], s["r"], s["a"], kv_scale=s["scale"])
    return Q.prepare_prefill(s["q"], s["qr"], s["gq"], s["gk"], s["grq"], Q.prefill_weights(s["wk"], s["wv"]), s["kv"],
                             s["ak"], s["starts"], s["lens"], s["table"], case["page"], s["table"].shape[1], s["total"],
                             s["softmax_scale"], EPS, s["o"], kv_scale=s["scale"], window=case["window"],
                             sinks=case["sinks"])


def run(state):
    op = state["case"]["op"]
    if own:
        if "call" not in state:
            state["call"] = _call(state)
        state["call"]()
    elif op == "rope":
        _plain_rope(state)
    elif op == "read":
        _plain_read(state)
    else:
        _plain_prefill(state)
    if op == "rope":
        return state["out"]
    if op == "read":
        return {"c": state["c"], "r": state["r"], "ak": state["a"]}
    return state["o"]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_values():
    """The 256 values of e4m3 (bias 7, no infinities, all-ones is NaN)."""
    v = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(math.nan if code & 127 == 127 else -x if code & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _sequence(s, b, length):
    """Slots of a sequence's tokens, their latents and RoPE keys in 64 bits."""
    page, d_c = s["case"]["page"], s["case"]["d_c"]
    slot = (s["table"][b].long()[:, None] * page + torch.arange(page, device="cuda")).flatten()[:length]
    rows = s["kv"][slot]
    if s["case"]["cache"] == "q8":
        c = _e4m3_values()[rows[:, :d_c].long()] * s["scale"][slot].double()[:, None]
        return slot, c, rows[:, d_c:].contiguous().view(torch.bfloat16).double()
    return slot, rows[:, :d_c].double(), rows[:, d_c:].double()


def _exact_rope(s):
    case = s["case"]
    d, rows = case["d_r"], case["rows"]
    # turned by multiplication of complex numbers, the whole turns taken off the angle first
    turns = s["positions"].double()[:, None] * (_frequencies(case, "cuda") / (2 * math.pi))
    turns -= turns.round()
    z = torch.polar(torch.ones_like(turns), (-2 if case["inverse"] else 2) * math.pi * turns)[:, None]
    x = s["x"][..., case["d"] - d:].double()
    if case["layout"] == "interleaved":
        return torch.view_as_real(torch.view_as_complex(x.reshape(rows, case["heads"], d // 2, 2).contiguous()) * z).flatten(-2)
    y = torch.complex(x[..., :d // 2], x[..., d // 2:]) * z
    return torch.cat([y.real, y.imag], dim=-1)


def exact(case, seed):
    if case["op"] == "prefill" and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    lens = _lens(case).tolist()
    if case["op"] == "read":
        got = [_sequence(s, b, n) for b, n in enumerate(lens)]
        return {"c": torch.cat([c for _, c, _ in got]), "r": torch.cat([r for _, _, r in got]),
                "ak": torch.cat([s["ak"][slot].double() for slot, _, _ in got])}
    H, G, G_v = case["H"], case["G"], case["G_v"]
    o = torch.empty((s["q"].shape[0], H, case["d_v"]), dtype=torch.float64, device="cuda")
    gam = s["gq"].double() * s["gk"].double()
    at = 0
    for b, (n, length) in enumerate(zip(_new(case).tolist(), lens)):
        slot, c, r = _sequence(s, b, length)
        end = torch.arange(length - n + 1, length + 1, device="cuda")[:, None]
        t = torch.arange(length, device="cuda")[None, :]
        hidden = t >= end
        if case["window"]:
            hidden |= (t >= case["sinks"]) & (t < end - case["window"])
        kept = {}
        for h in range(H):
            g, gv = h * G // H, h * G_v // H
            if ("k", g) not in kept:
                kept["k", g] = (c @ s["wk"][g].double()) * s["ak"][slot, g].double()[:, None]
            if ("v", gv) not in kept:
                kept["v", gv] = c @ s["wv"][gv].double()
            q, qr = s["q"][at:at + n, h].double(), s["qr"][at:at + n, h].double()
            q = q * gam / torch.sqrt(q.square().mean(dim=1, keepdim=True) + EPS)
            qr = qr * s["grq"].double() / torch.sqrt(qr.square().mean(dim=1, keepdim=True) + EPS)
            logit = torch.cat([q, qr], dim=1) @ torch.cat([kept["k", g], r], dim=1).t() * s["softmax_scale"]
            o[at:at + n, h] = torch.softmax(logit.masked_fill_(hidden, -math.inf), dim=1) @ kept["v", gv]
        at += n
    return o
