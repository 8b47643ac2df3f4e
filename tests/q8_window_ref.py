"""Plain 64-bit forms of the 8-bit cache and of windowed decode, and their test inputs.

Shared by the CPU and GPU tests; uses nothing of the library.
"""
import math

import numpy as np

EPS = 1e-6
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)])[:127]


def e4m3_encode(x):
    """Codes (uint8) of x (float64, |x| <= 448) in e4m3, round to nearest even."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7)


def e4m3_decode(code):
    code = np.asarray(code, np.uint8)
    mag = np.append(E4M3, np.nan)[code & 127]
    return np.where(code & 128, -mag, mag)


def bf16(x):
    """x rounded to bf16 (nearest even), as float32."""
    u = np.asarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def bf16_bits(x):
    return (bf16(x).view(np.uint32) >> 16).astype(np.uint16)


def quantise(c):
    """Codes and scales of latents c [N, d_c] fp32 (finite)."""
    top = np.abs(c).max(axis=1).astype(np.float64)
    e = np.array([0 if t == 0 else max(math.frexp(t)[1] - (9 if math.frexp(t)[0] <= 0.875 else 8), -126) for t in top])
    scale = np.where(top > 0, 2.0 ** e, 0.0)
    x = np.where(top[:, None] > 0, c.astype(np.float64) / np.where(scale > 0, scale, 1)[:, None], 0.0)
    return e4m3_encode(x), scale


def rope_rotate(r, pos, theta):
    d = r.shape[1]
    f = theta ** (-2.0 * np.arange(d // 2) / d)
    a = pos.astype(np.float64)[:, None] * f
    out = np.empty(r.shape, np.float64)
    out[:, 0::2] = r[:, 0::2] * np.cos(a) - r[:, 1::2] * np.sin(a)
    out[:, 1::2] = r[:, 0::2] * np.sin(a) + r[:, 1::2] * np.cos(a)
    return out


def rms_normalise(x, gamma):
    x = x.astype(np.float64)
    return x * gamma / np.sqrt((x ** 2).mean(axis=-1, keepdims=True) + EPS)


def inverse_rms(c_hat, wk):
    """alpha^k [N, G] of stored latents (float64)."""
    return np.stack([1.0 / np.sqrt(((c_hat @ w.astype(np.float64)) ** 2).mean(axis=1) + EPS) for w in wk], axis=1)


def visible(n, window, sinks):
    """Tokens a query of causal length n attends to."""
    t = np.arange(max(n, 0))
    return t if window == 0 else t[(t < sinks) | (t >= n - window)]


def attention(qt, aq, qr_hat, c_hat, kr, ak, s_q, length, window, sinks, scale, plain=False):
    """o [s_q, H, d_c], lse [s_q, H] (float64) of one sequence; c_hat, kr, ak by token."""
    H, d_c = qt.shape[1:]
    g = np.arange(H) // (H // ak.shape[1])
    o = np.zeros((s_q, H, d_c))
    lse = np.full((s_q, H), -np.inf)
    for i in range(s_q):
        t = visible(length - s_q + i + 1, window, sinks)
        if not len(t):
            continue
        l = qt[i].astype(np.float64) @ c_hat[t].T
        if not plain:
            l = l * aq[i].astype(np.float64)[:, None] * ak[t].astype(np.float64).T[g]
        l = scale * (l + qr_hat[i] @ kr[t].astype(np.float64).T)
        m = l.max(axis=1, keepdims=True)
        p = np.exp(l - m)
        z = p.sum(axis=1, keepdims=True)
        o[i] = (p / z) @ c_hat[t]
        lse[i] = (m + np.log(z))[:, 0]
    return o, lse


class Case:
    """Inputs of one decode call: a paged cache of the given type (numpy), every slot that no query
    may see holding NaN, and the 64-bit result."""

    def __init__(self, lens, s_q=1, H=16, G=4, d_c=256, d_r=32, page=64, cache="q8", window=0, sinks=0, plain=False,
                 alpha="f32", contiguous=False, seed=0, spread=1.0, max_pages=None, q_scale=1.0, outlier=30.0,
                 zero=False):
        g = np.random.Generator(np.random.PCG64([seed, len(lens), s_q, H, d_c, page, window]))
        self.lens, self.s_q, self.H, self.G, self.d_c, self.d_r = list(lens), s_q, H, G, d_c, d_r
        self.page, self.window, self.sinks, self.plain, self.cache = page, window, sinks, plain, cache
        B = len(lens)
        d_h = 64
        pages = [-(-n // page) for n in lens]
        self.max_pages = max(max(pages), 1) if max_pages is None else max_pages
        total = B * self.max_pages if contiguous else max(sum(pages), 1)
        self.slots = total * page
        wk = (g.standard_normal((G, d_c, d_h)) / math.sqrt(d_c)).astype(np.float32)
        gam = 1 + 0.1 * g.standard_normal(d_h)
        self.grq = (1 + 0.1 * g.standard_normal(d_r)).astype(np.float32)
        self.scale = 1.0 / math.sqrt(d_h + d_r)
        q = g.standard_normal((B, s_q, H, d_h)) * q_scale
        qt = np.einsum("bihj,hnj->bihn", q * gam, wk.astype(np.float64)[np.arange(H) // (H // G)])
        self.qt = (bf16(qt) if cache != "f32" else qt).astype(np.float32)
        self.aq = (1.0 / np.sqrt((q ** 2).mean(axis=-1) + EPS)).astype(np.float32)
        self.qr = g.standard_normal((B, s_q, H, d_r)).astype(np.float32)
        qr_hat = self.qr.astype(np.float64) if plain else rms_normalise(self.qr, self.grq)
        if contiguous:
            self.table = None
            table = np.arange(B * self.max_pages).reshape(B, self.max_pages)
        else:
            perm = g.permutation(total)
            table = np.full((B, self.max_pages), -1)
            at = 0
            for b, n in enumerate(pages):
                table[b, :n] = perm[at:at + n]
                at += n
            self.table = table.astype(np.int32)
        # everything starts as NaN: bytes 0xFF are NaN in e4m3, bf16 and fp32 alike
        row = {"q8": d_c + 2 * d_r, "bf16": 2 * (d_c + d_r), "f32": 4 * (d_c + d_r)}[cache]
        self.kv = np.full((self.slots, row), 0xFF, np.uint8)
        self.kv_scale = np.full(self.slots, np.nan, np.float32)
        self.ak = np.full((self.slots, G), np.nan, np.float32)
        self.o = np.zeros((B, s_q, H, d_c))
        self.lse = np.full((B, s_q, H), -np.inf)
        for b, n in enumerate(lens):
            if n == 0:
                continue
            c = g.standard_normal((n, d_c))
            c *= np.where(g.random(n) < 0.05, outlier, 1.0)[:, None] * np.exp2(g.uniform(-spread, spread, n))[:, None]
            if zero:
                c[::5] = 0
            c = c.astype(np.float32)
            kr = bf16(rms_normalise(g.standard_normal((n, d_r)), np.ones(d_r)))
            seen = np.unique(np.concatenate([visible(n - s_q + i + 1, window, sinks) for i in range(s_q)])).astype(int)
            slot = table[b, seen // page] * page + seen % page
            if cache == "q8":
                codes, sc = quantise(c)
                c_hat = e4m3_decode(codes) * sc[:, None]
                self.kv[slot] = np.concatenate([codes[seen], bf16_bits(kr[seen]).view(np.uint8)], axis=1)
                self.kv_scale[slot] = sc[seen]
            elif cache == "bf16":
                c_hat = bf16(c).astype(np.float64)
                self.kv[slot] = np.concatenate([bf16_bits(c[seen]), bf16_bits(kr[seen])], axis=1).view(np.uint8)
            else:
                c_hat = c.astype(np.float64)
                self.kv[slot] = np.concatenate([c[seen], kr[seen]], axis=1).astype(np.float32).view(np.uint8)
            ak = inverse_rms(c_hat, wk).astype(np.float32)
            if alpha == "f16":
                ak = ak.astype(np.float16).astype(np.float32)
            self.ak[slot] = ak[seen]
            self.o[b], self.lse[b] = attention(self.qt[b], self.aq[b], qr_hat[b], c_hat, kr, ak, s_q, n, window, sinks,
                                               self.scale, plain)
        if alpha == "f16":
            self.ak = self.ak.astype(np.float16)
