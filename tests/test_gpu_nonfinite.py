"""Values that are not finite in what a query sees show in its result, and nowhere else.

o = 0 and lse = -inf say that a query has no visible token; a NaN among the tokens it sees, or in its own row,
gives NaN in o and lse, in whichever part of a split sequence it lies.  The other rows keep their results, to
the tolerance of test_gpu_q8_window.
"""
import numpy as np
import pytest
import torch

import q8_window_ref as R
from test_gpu_q8_window import Device, Q  # noqa: F401

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
# cache, CUDA cores, shape: 8-bit at 16, 32 and 64 rows; bf16 64-row kernel and CTA pair; CUDA cores of each type
KERNELS = [
    ("q8", False, dict()), ("q8", False, dict(H=32, G=2)), ("q8", False, dict(H=128, G=8, d_c=512, d_r=64)),
    ("bf16", False, dict()), ("bf16", False, dict(H=64, G=8, d_c=512, d_r=64)),
    ("bf16", False, dict(H=128, G=8, d_c=512, d_r=64)),
    ("q8", True, dict()), ("bf16", True, dict()), ("f32", True, dict()),
]
PLACES = ["latent", "rope", "alpha", "scale", "query", "alpha_q", "rope_query"]


def poison(dev, c, place, b, token, head):
    """Puts a NaN at one place; returns the heads of sequence b that it reaches."""
    slot = int(c.table[b, token // c.page]) * c.page + token % c.page
    every = np.ones(c.H, bool)
    group = np.arange(c.H) // (c.H // c.G) == 1 % c.G
    if place == "latent":
        if c.cache == "q8":
            dev.kv[slot, 5] = 0x7F
        else:
            dev.kv[slot, 5] = NAN
        return every
    if place == "rope":
        if c.cache == "q8":
            dev.kv[slot, c.d_c + 2:c.d_c + 4] = 0xFF
        else:
            dev.kv[slot, c.d_c + 1] = NAN
        return every
    if place == "alpha":
        dev.ak[slot, 1 % c.G] = NAN
        return group
    if place == "scale":
        dev.scale[slot] = NAN
        return every
    t, at = {"query": (dev.in_[0], (b, 0, head, 3)), "alpha_q": (dev.in_[1], (b, 0, head)),
             "rope_query": (dev.in_[2], (b, 0, head, 2))}[place]
    t[at] = NAN
    return np.arange(c.H) == head


def check_rows(Q, dev, c, bad):  # noqa: F811
    """Rows of `bad` [B, s_q, H] are NaN throughout, the others right."""
    dev.call()
    assert Q.get_device_status() == 0
    o, lse = dev.o.double().cpu().numpy(), dev.lse.double().cpu().numpy()
    assert np.isnan(o[bad]).all() and np.isnan(lse[bad]).all()
    fine = ~bad
    assert np.isfinite(o[fine]).all()
    assert np.linalg.norm(o[fine] - c.o[fine]) <= 5e-3 * np.linalg.norm(c.o[fine])
    assert np.abs(lse[fine] - c.lse[fine]).max() <= 2e-2


@pytest.mark.parametrize("window", [0, 3000])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("kernel,place", [(k, x) for k in range(len(KERNELS)) for x in PLACES
                                          if x != "scale" or KERNELS[k][0] == "q8"])
def test_nan_shows(Q, kernel, place, splits, window):  # noqa: F811
    cache, simt, shape = KERNELS[kernel]
    c = R.Case([1300, 200], cache=cache, window=window, sinks=4 if window else 0, **shape)
    dev = Device(Q, c, force_simt=simt, num_splits=splits)
    assert dev.call.kernel_name == ("simt" if simt else "tcgen05")
    bad = np.zeros(c.lse.shape, bool)
    bad[0, 0] = poison(dev, c, place, 0, 700, 3)            # inside the middle part of three
    check_rows(Q, dev, c, bad)


@pytest.mark.parametrize("kernel", range(len(KERNELS)))
def test_nan_in_every_token(Q, kernel):  # noqa: F811
    """Nothing but NaN: no part has a finite value, and the row is still not an empty one."""
    cache, simt, shape = KERNELS[kernel]
    for splits in (1, 3):
        c = R.Case([1300, 200, 0], cache=cache, window=1000, sinks=4, **shape)
        dev = Device(Q, c, force_simt=simt, num_splits=splits)
        slots = (c.table[0].astype(np.int64)[:, None] * c.page + np.arange(c.page)).ravel()[:1300]
        dev.ak[torch.from_numpy(slots).cuda()] = NAN
        bad = np.zeros(c.lse.shape, bool)
        bad[0] = True
        dev.call()
        assert Q.get_device_status() == 0
        o, lse = dev.o.double().cpu().numpy(), dev.lse.double().cpu().numpy()
        assert np.isnan(o[bad]).all() and np.isnan(lse[bad]).all()
        assert (o[2] == 0).all() and np.isneginf(lse[2]).all()      # the empty sequence is one
        assert np.linalg.norm(o[1] - c.o[1]) <= 5e-3 * np.linalg.norm(c.o[1])


@pytest.mark.parametrize("value", [INF, -INF])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("kernel", range(len(KERNELS)))
def test_infinite_query(Q, kernel, splits, value):  # noqa: F811
    """An infinite element of a query's row: its logits are infinities of both signs, the row is NaN."""
    cache, simt, shape = KERNELS[kernel]
    c = R.Case([1300, 200], cache=cache, window=3000, sinks=4, **shape)
    dev = Device(Q, c, force_simt=simt, num_splits=splits)
    dev.in_[0][0, 0, 5, 7] = value
    bad = np.zeros(c.lse.shape, bool)
    bad[0, 0, 5] = True
    check_rows(Q, dev, c, bad)


@pytest.mark.parametrize("kernel", range(len(KERNELS)))
@pytest.mark.parametrize("where,window", [("newest", 2000), ("newest", 0), ("oldest", 300)])
def test_nan_of_another_query(Q, kernel, where, window):  # noqa: F811
    """A NaN that only one query of the step sees -- the newest token, or the oldest of the first query's window --
    leaves the other queries' rows alone, also where a CTA holds several queries."""
    cache, simt, shape = KERNELS[kernel]
    for s_q, lens in ((2, [1300, 65]), (4, [1090, 64])):
        c = R.Case(lens, cache=cache, window=window, sinks=4 if window else 0, s_q=s_q, **shape)
        dev = Device(Q, c, force_simt=simt)
        n = lens[0]
        poison(dev, c, "latent", 0, n - 1 if where == "newest" else n - s_q + 1 - window, 0)
        bad = np.zeros(c.lse.shape, bool)
        bad[0, s_q - 1 if where == "newest" else 0] = True
        check_rows(Q, dev, c, bad)
