"""Chosen latents in place of a test case's random ones.

Shared by the GPU tests of the 8-bit cache and of windowed decode; uses nothing of the library.
"""
import numpy as np

import q8_window_ref as R


def seen_slots(c, b):
    """Tokens of sequence b that some query of the step sees, and their slots."""
    n = c.lens[b]
    seen = np.unique(np.concatenate([R.visible(n - c.s_q + i + 1, c.window, c.sinks) for i in range(c.s_q)])).astype(int)
    table = np.arange(len(c.lens) * c.max_pages).reshape(len(c.lens), -1) if c.table is None else c.table
    return seen, table[b, seen // c.page].astype(np.int64) * c.page + seen % c.page


def replace_latents(c, b, lat):
    """Stores lat [lens[b], d_c] (fp32, finite) as sequence b's latents in an 8-bit cache and renews its 64-bit
    result; alpha^k and the RoPE keys stay."""
    n = c.lens[b]
    seen, slot = seen_slots(c, b)
    codes, sc = R.quantise(lat[seen])
    c.kv[slot, :c.d_c], c.kv_scale[slot] = codes, sc
    c_hat, kr, ak = np.zeros((n, c.d_c)), np.zeros((n, c.d_r)), np.zeros((n, c.G))
    c_hat[seen] = R.e4m3_decode(codes) * sc[:, None]
    kr[seen] = (c.kv[slot, c.d_c:].copy().view(np.uint16).astype(np.uint32) << 16).view(np.float32)
    ak[seen] = c.ak[slot]
    qr = c.qr[b].astype(np.float64) if c.plain else R.rms_normalise(c.qr[b], c.grq)
    c.o[b], c.lse[b] = R.attention(c.qt[b], c.aq[b], qr, c_hat, kr, ak, c.s_q, n, c.window, c.sinks, c.scale, c.plain)
