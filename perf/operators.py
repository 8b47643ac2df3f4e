"""Measured cases of the 8-bit latent cache and of sliding-window decode.

Three operators, each one pass as a decoding program makes it:

  append   qkmla_append_q8: new latents into the 8-bit cache (e4m3 codes and one
           power-of-two scale a token), their alpha^k per KV group, and the
           normalised RoPE key in bf16
  q8       decode attention over that cache, over the whole context or over a
           sliding window and a few first tokens (sinks)
  window   decode attention over the bf16 cache with a sliding window and sinks

`own` False: elementary torch operations in fp32.  `own` True: the library.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attention(name, op, B, s_q, H, G, d_c, d_h, d_r, lo, hi, page, window=0, sinks=0):
    return {"name": name, "op": op, "B": B, "s_q": s_q, "H": H, "G": G, "d_c": d_c, "d_h": d_h, "d_r": d_r,
            "lo": lo, "hi": hi, "page": page, "window": window, "sinks": sinks}


def _append(name, N, G, d_c, d_h, d_r):
    return {"name": name, "op": "append", "N": N, "G": G, "d_c": d_c, "d_h": d_h, "d_r": d_r}


def listed():
    return [
        # one short chat turn: the latency of a call
        _attention("q8_one_short", "q8", 1, 1, 16, 4, 256, 64, 32, 333, 333, 64),
        # a small model's batch of ordinary contexts
        _attention("q8_small_batch", "q8", 16, 1, 16, 4, 256, 64, 32, 1024, 8192, 64),
        # a large model's decode batch of equal contexts
        _attention("q8_large_4k", "q8", 64, 1, 128, 8, 512, 128, 64, 4096, 4096, 64),
        # a few very long contexts: split over the GPU and joined
        _attention("q8_large_256k", "q8", 4, 1, 128, 8, 512, 128, 64, 262144, 262144, 64),
        # ragged serving batch with two query tokens a sequence, small pages
        _attention("q8_large_mtp_ragged", "q8", 32, 2, 128, 8, 512, 128, 64, 512, 32768, 32),
        # the same cache, long contexts read through a window and sinks
        _attention("q8_large_window", "q8", 64, 1, 128, 8, 512, 128, 64, 4096, 32768, 64, 4096, 4),
        # bf16 cache of a small model, short window: a latency-bound call
        _attention("win_small", "window", 16, 1, 16, 4, 256, 64, 32, 1024, 8192, 64, 1000, 4),
        # bf16 cache of a large model, long contexts behind an ordinary window
        _attention("win_large", "window", 64, 1, 128, 8, 512, 128, 64, 4096, 32768, 64, 4096, 4),
        # two query tokens, ragged, window larger than some contexts, sinks of several tiles
        _attention("win_large_mtp_ragged", "window", 32, 2, 128, 8, 512, 128, 64, 512, 65536, 64, 8191, 130),
        # one decode step of a small model: one token for each of 16 sequences
        _append("append_small_step", 16, 4, 256, 64, 32),
        # one decode step of a large model: two tokens for each of 128 sequences
        _append("append_large_step", 256, 8, 512, 128, 64),
        # prompts entering the cache
        _append("append_large_prompts", 16001, 8, 512, 128, 64),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    large = rng.random() < 0.5
    d_c, d_h, d_r = (512, 128, 64) if large else (256, 64, 32)
    op = rng.choice(["q8", "q8", "window", "append"])
    if op == "append":
        return {k: v for k, v in _append("", log(1, 16000), 8 if large else 4, d_c, d_h, d_r).items() if k != "name"}
    H, G = rng.choice([(64, 8), (128, 8), (128, 8), (32, 4)] if large else [(16, 4), (16, 2), (32, 4)])
    s_q = rng.choice([1, 1, 2, 3])
    hi = log(64, 65536)
    lo = min(hi, max(s_q, log(max(1, hi // 16), hi)))
    B = max(1, min(log(1, 64), 1000000 // (hi * s_q)))
    page = rng.choice([16, 32, 64, 128] if op == "q8" else [64, 128])
    window = sinks = 0
    if op == "window" or rng.random() < 0.3:
        window, sinks = log(1, 8192), rng.choice([0, 1, 4, 64, rng.randrange(300)])
    return {k: v for k, v in _attention("", op, B, s_q, H, G, d_c, d_h, d_r, lo, hi, page, window, sinks).items()
            if k != "name"}


def _lens(case):
    """Context lengths, log-uniform in [lo, hi]: part of the case, the same for every seed."""
    g = np.random.Generator(np.random.PCG64([case["lo"], case["hi"], case["B"]]))
    lens = np.exp(g.uniform(math.log(case["lo"]), math.log(case["hi"]), size=case["B"]))
    return np.clip(np.round(lens), case["lo"], case["hi"]).astype(np.int64)


def _seen(case, length, i):
    """Tokens that query i of a sequence attends to."""
    n = length - case["s_q"] + i + 1
    if not case["window"]:
        return n
    return min(n, case["window"] + min(case["sinks"], max(0, n - case["window"])))


def work(case):
    d_c, d_r, G = case["d_c"], case["d_r"], case["G"]
    if case["op"] == "append":
        N, d_h = case["N"], case["d_h"]
        read = N * (d_c + d_r) * 4 + G * d_c * d_h * 4 + d_r * 4 + N * 8
        return {"bytes": read + N * (d_c + 2 * d_r + 4 + 4 * G), "flops": 2 * N * G * d_c * d_h}
    token = (d_c + 2 * d_r + 4 if case["op"] == "q8" else 2 * (d_c + d_r)) + 4 * G
    rows = case["s_q"] * case["H"]
    tokens = flops = 0
    for n in _lens(case).tolist():
        seen = [_seen(case, n, i) for i in range(case["s_q"])]
        tokens += min(n, seen[0] + case["s_q"] - 1) if case["window"] else n
        flops += sum(seen) * case["H"] * 2 * (2 * d_c + d_r)
    query = case["B"] * rows * (2 * d_c + 4 * d_r + 4)
    return {"bytes": tokens * token + query + case["B"] * rows * d_c * 2, "flops": flops}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _quantise(c):
    """e4m3 codes (as uint8) and the power-of-two scale of each row of c [N, d_c] fp32: the
    least 2^e with max|c| <= 448 2^e, 0 for a row of zeros."""
    mant, exp = torch.frexp(c.abs().amax(dim=1))
    exp = (exp - torch.where(mant <= 0.875, 9, 8)).clamp(-126, 120)
    scale = torch.where(mant == 0, 0.0, torch.ldexp(torch.ones_like(mant), exp))
    codes = (c * torch.where(mant == 0, 0.0, torch.ldexp(torch.ones_like(mant), -exp))[:, None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), scale


def _tokens(gen, n, d, frac, by):
    """N(0,1) rows with a share `frac` of outlier rows, scaled by `by`."""
    x = torch.randn((n, d), generator=gen, device="cuda")
    out = torch.rand(n, generator=gen, device="cuda") < frac
    return x.mul_(torch.where(out, by, 1.0)[:, None]), out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    d_c, d_h, d_r, G = case["d_c"], case["d_h"], case["d_r"], case["G"]
    wk = torch.randn((G, d_c, d_h), generator=gen, device="cuda") / math.sqrt(d_c)
    grk = 1 + 0.1 * torch.randn(d_r, generator=gen, device="cuda")
    s = {"case": case, "wk": wk, "grk": grk}
    if case["op"] == "append":
        N = case["N"]
        c, out = _tokens(gen, N, d_c, 0.05, 30.0)
        r = torch.randn((N, d_r), generator=gen, device="cuda").mul_(torch.where(out, 30.0, 1.0)[:, None])
        slots = torch.randperm(N + 64, generator=gen, device="cuda")[:N].contiguous()
        s.update(c=c, r=r, slots=slots,
                 kv=torch.zeros((N + 64, d_c + 2 * d_r), dtype=torch.uint8, device="cuda"),
                 scale=torch.zeros(N + 64, device="cuda"), ak=torch.zeros((N + 64, G), device="cuda"))
        return s
    B, s_q, H, page = case["B"], case["s_q"], case["H"], case["page"]
    lens = _lens(case)
    pages = [-(-int(n) // page) for n in lens]
    total = sum(pages)
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((B, max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    slots = total * page
    q8 = case["op"] == "q8"
    kv = torch.empty((slots, d_c + 2 * d_r), dtype=torch.uint8, device="cuda") if q8 else torch.empty(
        (slots, d_c + d_r), dtype=torch.bfloat16, device="cuda")
    scale = torch.empty(slots, device="cuda") if q8 else None
    ak = torch.empty((slots, G), device="cuda")
    for i in range(0, slots, 131072):
        n = min(131072, slots - i)
        c, _ = _tokens(gen, n, d_c, 0.05, 30.0)
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
        for g in range(G):
            ak[i:i + n, g] = torch.rsqrt((c @ wk[g]).square().mean(dim=1) + EPS)
    q = torch.randn((B, s_q, H, d_h), generator=gen, device="cuda")
    gam = (1 + 0.1 * torch.randn(d_h, generator=gen, device="cuda")) * (1 + 0.1 * torch.randn(d_h, generator=gen, device="cuda"))
    qt = torch.einsum("rgpj,gnj->rgpn", (q * gam).reshape(B * s_q, G, H // G, d_h), wk)
    s.update(qt=qt.reshape(B, s_q, H, d_c).bfloat16().contiguous(),
             aq=torch.rsqrt(q.square().mean(dim=-1) + EPS),
             qr=torch.randn((B, s_q, H, d_r), generator=gen, device="cuda"),
             grq=1 + 0.1 * torch.randn(d_r, generator=gen, device="cuda"),
             kv=kv, scale=scale, ak=ak, table=table, lens=torch.from_numpy(lens.astype(np.int32)).cuda(),
             softmax_scale=1.0 / math.sqrt(d_h + d_r),
             o=torch.empty((B, s_q, H, d_c), dtype=torch.bfloat16, device="cuda"))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plain_append(s):
    case = s["case"]
    d_c = case["d_c"]
    codes, scale = _quantise(s["c"])
    c = codes.view(torch.float8_e4m3fn).float() * scale[:, None]
    k = torch.matmul(c, s["wk"])                                   # [G, N, d_h]
    r = s["r"]
    r = r * s["grk"] * torch.rsqrt(r.square().mean(dim=1, keepdim=True) + EPS)
    s["kv"][s["slots"], :d_c] = codes
    s["kv"][s["slots"], d_c:] = r.bfloat16().view(torch.uint8)
    s["scale"][s["slots"]] = scale
    s["ak"][s["slots"]] = torch.rsqrt(k.square().mean(dim=2) + EPS).t()


def _plain_attention(s):
    case = s["case"]
    B, s_q, H, G, d_c, page = case["B"], case["s_q"], case["H"], case["G"], case["d_c"], case["page"]
    window, sinks = case["window"], case["sinks"]
    n = s["lens"].long()[:, None]                                  # [B, 1]
    if window:
        first = n - s_q + 1 - window
        recent = first + torch.arange(window + s_q - 1, device="cuda")
        t = torch.cat([torch.arange(sinks, device="cuda").expand(B, sinks), recent], dim=1)
        once = torch.cat([torch.ones((B, sinks), dtype=torch.bool, device="cuda"), recent >= sinks], dim=1)
    else:
        t = torch.arange(s["table"].shape[1] * page, device="cuda").expand(B, -1)
        once = torch.ones_like(t, dtype=torch.bool)
    there = once & (t >= 0) & (t < n)
    t = torch.where(there, t, 0)
    slot = torch.gather(s["table"].long(), 1, t // page) * page + t % page
    rows = s["kv"][slot]
    if s["scale"] is not None:
        c = rows[..., :d_c].view(torch.float8_e4m3fn).float() * s["scale"][slot][..., None]
        r = rows[..., d_c:].contiguous().view(torch.bfloat16).float()
    else:
        c, r = rows[..., :d_c].float(), rows[..., d_c:].float()
    qr = s["qr"] * s["grq"] * torch.rsqrt(s["qr"].square().mean(dim=-1, keepdim=True) + EPS)
    logit = torch.matmul(s["qt"].float().reshape(B, s_q * H, d_c), c.transpose(1, 2)).view(B, s_q, G, H // G, -1)
    logit *= s["aq"].view(B, s_q, G, H // G, 1)
    logit *= s["ak"][slot].transpose(1, 2)[:, None, :, None, :]
    logit = logit.view(B, s_q * H, -1)
    logit += torch.matmul(qr.reshape(B, s_q * H, -1), r.transpose(1, 2))
    logit *= s["softmax_scale"]
    end = n[:, :, None] - s_q + 1 + torch.arange(s_q, device="cuda")[None, :, None]   # [B, s_q, 1]
    t = t[:, None, :]
    sees = there[:, None, :] & (t < end)
    if window:
        sees &= (t < sinks) | (t >= end - window)
    logit = logit.view(B, s_q, H, -1).masked_fill_(~sees[:, :, None, :], -math.inf)
    p = logit.sub_(logit.amax(dim=-1, keepdim=True)).exp_()
    o = torch.matmul(p.view(B, s_q * H, -1), c).view(B, s_q, H, d_c) / p.sum(dim=-1, keepdim=True)
    s["o"].copy_(o)


def run(state):
    case = state["case"]
    if own:
        import qk_normed_latent_gb300 as Q
        if "call" not in state:          # arguments marshalled once, workspace kept, as a decode loop does
            if case["op"] == "append":
                state["call"] = Q.prepare_append_q8(state["c"], state["r"], state["wk"], state["grk"], state["slots"],
                                                    state["kv"], state["scale"], state["ak"], EPS)
            else:
                state["call"] = Q.prepare_decode(state["qt"], state["aq"], state["qr"], state["grq"], state["kv"],
                                                 state["ak"], state["lens"], state["table"], case["page"],
                                                 state["table"].shape[1], case["G"], state["softmax_scale"], EPS,
                                                 state["o"], None, kv_scale=state["scale"], window=case["window"],
                                                 sinks=case["sinks"])
        state["call"]()
    elif case["op"] == "append":
        _plain_append(state)
    else:
        _plain_attention(state)
    if case["op"] == "append":
        d_c = case["d_c"]
        return {"codes": state["kv"][:, :d_c].view(torch.float8_e4m3fn), "rope": state["kv"][:, d_c:].view(torch.bfloat16),
                "scale": state["scale"], "ak": state["ak"]}
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


def _exact_append(s):
    case = s["case"]
    d_c, G = case["d_c"], case["G"]
    c = s["c"].double()
    top = c.abs().amax(dim=1)
    e = torch.ceil(torch.log2(top / E4M3_MAX))
    scale = torch.where(top > 0, torch.exp2(e), 0.0)
    grid = _e4m3_values()[:127]                                    # ascending, from 0 to 448
    middle = (grid[1:] + grid[:-1]) / 2
    x = torch.where(top[:, None] > 0, c / scale[:, None], 0.0)
    at = torch.bucketize(x.abs(), middle)                          # ties to the lower, mended below
    tie = (at < 126) & (x.abs() == middle[at.clamp(max=125)]) & (at % 2 == 1)
    value = grid[at + tie.long()] * torch.sign(x)
    r = s["r"].double()
    r = r * s["grk"].double() / torch.sqrt(r.square().mean(dim=1, keepdim=True) + EPS)
    n = s["kv"].shape[0]
    codes = torch.zeros((n, d_c), dtype=torch.float64, device="cuda")
    rope = torch.zeros((n, case["d_r"]), dtype=torch.float64, device="cuda")
    scales = torch.zeros(n, dtype=torch.float64, device="cuda")
    ak = torch.zeros((n, G), dtype=torch.float64, device="cuda")
    codes[s["slots"]], rope[s["slots"]], scales[s["slots"]] = value, r, scale
    stored = value * scale[:, None]
    for g in range(G):
        k = stored @ s["wk"][g].double()
        ak[s["slots"], g] = 1.0 / torch.sqrt(k.square().mean(dim=1) + EPS)
    return {"codes": codes, "rope": rope, "scale": scales, "ak": ak}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    s_q, H, G, d_c, page = case["s_q"], case["H"], case["G"], case["d_c"], case["page"]
    value = _e4m3_values()
    qr = s["qr"].double()
    qr = qr * s["grq"].double() / torch.sqrt(qr.square().mean(dim=-1, keepdim=True) + EPS)
    group = torch.arange(H, device="cuda") // (H // G)
    o = torch.empty((case["B"], s_q, H, d_c), dtype=torch.float64, device="cuda")
    for b, length in enumerate(_lens(case).tolist()):
        table = s["table"][b].long()
        for i in range(s_q):
            n = length - s_q + i + 1
            t = torch.arange(n, device="cuda")
            if case["window"]:
                t = t[(t < case["sinks"]) | (t >= n - case["window"])]
            slot = table[t // page] * page + t % page
            rows = s["kv"][slot]
            if case["op"] == "q8":
                c = value[rows[:, :d_c].long()] * s["scale"][slot].double()[:, None]
                r = rows[:, d_c:].contiguous().view(torch.bfloat16).double()
            else:
                c, r = rows[:, :d_c].double(), rows[:, d_c:].double()
            content = (s["qt"][b, i].double() @ c.t()) * s["aq"][b, i].double()[:, None] * s["ak"][slot].double().t()[group]
            p = torch.softmax((content + qr[b, i] @ r.t()) * s["softmax_scale"], dim=1)
            o[b, i] = p @ c
    return o
