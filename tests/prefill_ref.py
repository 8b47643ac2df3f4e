"""Prefill over the latent cache in 64 bits, from its definition, on the CPU (numpy), and the inputs of its tests.

Nothing here uses the library.  `Case` draws a paged cache as the append calls would leave it, a step's
chunks of queries, and gives the exact output."""
import numpy as np

EPS = 1e-6


def bf16(x):
    """fp32 values rounded to bfloat16 (to nearest, ties to even), as uint16 patterns; NaN stays NaN."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC1), r)


def from_bf16(u):
    return (u.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def e4m3_values():
    v = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[code] = np.nan if code & 127 == 127 else -x if code & 128 else x
    return v


def to_e4m3(x):
    """Nearest code (ties to even) of values within +-448; NaN for what is not finite."""
    grid = e4m3_values()[:127]
    a = np.abs(x)
    at = np.searchsorted((grid[1:] + grid[:-1]) / 2, a, side="left")
    tie = (at < 126) & (a == ((grid[1:] + grid[:-1]) / 2)[np.minimum(at, 125)]) & (at % 2 == 1)
    code = (at + tie).astype(np.uint8) | np.where(np.signbit(x), 128, 0).astype(np.uint8)
    return np.where(np.isfinite(x), code, 127).astype(np.uint8)


class Case:
    """lens: tokens a sequence; new: its chunk's rows.  `change(case)` may rewrite latents c, RoPE keys r, queries
    or gains before they are stored."""

    def __init__(self, lens, new, H=8, G=4, G_v=None, d_c=128, d_h=64, d_r=32, d_v=64, cache="bf16", page=16, window=0,
                 sinks=0, alpha="f32", rope_gain=True, contiguous=False, outliers=0.05, q="f32", seed=0, spare_rows=0,
                 scale=None, change=None):
        G_v = G if G_v is None else G_v
        self.__dict__.update(lens=list(lens), new=list(new), H=H, G=G, G_v=G_v, d_c=d_c, d_h=d_h, d_r=d_r, d_v=d_v,
                             cache=cache, page=page, window=window, sinks=sinks, alpha=alpha, qtype=q)
        g = np.random.Generator(np.random.PCG64([len(lens), sum(lens), sum(new), H, d_c, seed]))
        f = lambda *s: g.standard_normal(s, dtype=np.float32)  # noqa: E731
        self.B = len(lens)
        self.scale = 1 / np.sqrt(d_h + d_r) if scale is None else scale
        self.wk = f(G, d_c, d_h) / np.float32(np.sqrt(d_c))
        self.wv = bf16(f(G_v, d_c, d_v) / np.float32(np.sqrt(d_c)))
        self.gq, self.gk = 1 + np.float32(0.1) * f(d_h), 1 + np.float32(0.1) * f(d_h)
        self.grq = 1 + np.float32(0.1) * f(d_r) if rope_gain else None
        self.rows = sum(new)
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.q, self.qr = f(self.rows + spare_rows, H, d_h), f(self.rows + spare_rows, H, d_r)
        n = sum(lens)
        self.c, self.r = f(n, d_c), f(n, d_r)
        self.c *= np.where(g.random(n) < outliers, 30, 1)[:, None].astype(np.float32)
        if change is not None:
            change(self)
        if q == "bf16":
            self.q, self.qr = (from_bf16(bf16(x)).astype(np.float32) for x in (self.q, self.qr))
        # pages: each sequence's tokens in pages of its own, in random order
        pages = [-(-k // page) for k in lens]
        self.max_pages = max(1, max(pages))
        total = self.B * self.max_pages if contiguous else sum(pages) + 2
        self.table = None
        if not contiguous:
            perm = g.permutation(total).astype(np.int32)
            self.table = np.full((self.B, self.max_pages), -1, np.int32)
            at = 0
            for b, k in enumerate(pages):
                self.table[b, :k] = perm[at:at + k]
                at += k
        self.slots = total * page
        # the cache, NaN where nothing is stored
        kv = np.full((self.slots, d_c + d_r), 0x7FC1, np.uint16)
        q8 = np.full((self.slots, d_c + 2 * d_r), 0xFF, np.uint8)
        self.kv_scale = np.full(self.slots, np.nan, np.float32)
        self.ak = np.full((self.slots, G), np.nan, np.float32)
        self.slot = []
        at = 0
        for b, k in enumerate(lens):
            t = np.arange(k)
            page_of = self.table[b, t // page] if self.table is not None else b * self.max_pages + t // page
            s = page_of.astype(np.int64) * page + t % page
            self.slot.append(s)
            kv[s, :d_c] = bf16(self.c[at:at + k])
            kv[s, d_c:] = bf16(self.r[at:at + k])
            if cache == "q8":
                with np.errstate(invalid="ignore"):
                    top = np.max(np.abs(np.where(np.isfinite(self.c[at:at + k]), self.c[at:at + k], 0)), axis=1, initial=0)
                e = np.where(top > 0, np.clip(np.ceil(np.log2(np.where(top > 0, top, 1) / 448.0)), -126, 120), 0)
                self.kv_scale[s] = np.where(top > 0, 2.0 ** e, 0)
                q8[s, :d_c] = to_e4m3(self.c[at:at + k].astype(np.float64) / 2.0 ** e[:, None])
                q8[s, d_c:] = bf16(self.r[at:at + k]).view(np.uint8)
            at += k
        self.kv = q8 if cache == "q8" else kv
        self._exact()

    def stored(self, b):
        """Latents and RoPE keys of sequence b as the cache holds them."""
        rows = self.kv[self.slot[b]]
        if self.cache == "q8":
            with np.errstate(invalid="ignore"):
                c = e4m3_values()[rows[:, :self.d_c]] * self.kv_scale[self.slot[b]].astype(np.float64)[:, None]
            return c, from_bf16(np.ascontiguousarray(rows[:, self.d_c:]).view(np.uint16))
        return from_bf16(rows[:, :self.d_c]), from_bf16(rows[:, self.d_c:])

    def seen(self, b):
        """[new, len]: whether a query sees a token."""
        n, L = self.new[b], self.lens[b]
        end = (L - n + 1 + np.arange(n))[:, None]
        t = np.arange(L)[None, :]
        see = t < end
        if self.window:
            see &= (t < self.sinks) | (t >= end - self.window)
        return see

    def _exact(self):
        H, G, G_v = self.H, self.G, self.G_v
        self.o = np.zeros((self.rows, H, self.d_v))
        self.lse = np.full((self.rows, H), -np.inf)
        with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
            for b in range(self.B):
                c, r = self.stored(b)
                k = np.einsum("tn,gnj->gtj", c, self.wk.astype(np.float64))
                ak = (1 / np.sqrt((k ** 2).mean(axis=2) + EPS)).astype(np.float32)
                ak = ak.astype(np.float16).astype(np.float32) if self.alpha == "f16" else ak
                self.ak[self.slot[b]] = ak.T
                k = k * ak.astype(np.float64)[:, :, None]
                v = np.einsum("tn,gnj->gtj", c, from_bf16(self.wv))
                q = self.q[self.start[b]:self.start[b + 1]].astype(np.float64)
                qr = self.qr[self.start[b]:self.start[b + 1]].astype(np.float64)
                q = q * (self.gq.astype(np.float64) * self.gk) / np.sqrt((q ** 2).mean(axis=2, keepdims=True) + EPS)
                qr = qr / np.sqrt((qr ** 2).mean(axis=2, keepdims=True) + EPS)
                if self.grq is not None:
                    qr = qr * self.grq
                see = self.seen(b)
                for h in range(H):
                    with np.errstate(invalid="ignore"):
                        l = (q[:, h] @ k[h * G // H].T + qr[:, h] @ r.T) * self.scale
                    l = np.where(see, l, -np.inf)
                    for i in range(self.new[b]):
                        t = see[i]
                        if not t.any():
                            continue
                        row = l[i, t]
                        top = np.max(row) if np.isfinite(row).all() else np.nan
                        p = np.exp(row - top)
                        self.lse[self.start[b] + i, h] = top + np.log(p.sum())
                        self.o[self.start[b] + i, h] = (p / p.sum()) @ v[h * G_v // H][t]
