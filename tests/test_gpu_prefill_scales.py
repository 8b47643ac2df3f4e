"""Tokens whose latents are much larger than a row's own: hidden from it, or visible with a weight that leaves them nothing.

Tolerance.  test_gpu_prefill.py's: rel-L2 2.7e-3 with fp16 operands, 6.2e-3 where a tile's values and weights are bf16, an lse off
by up to 7e-3.  Norms are taken over the rows in question alone, since rows that see a large token would hide the others.  Where the
RoPE queries are ones, they are 1 after their normalisation (1 - 5e-7, fp16 1) and the RoPE keys here are bf16 and fp16 numbers: that
part of a logit, however large, adds no error."""
import numpy as np
import pytest
import torch

import prefill_ref as R
from test_gpu_prefill import Device, Q, compare  # noqa: F401 (Q: the fixture)

pytestmark = pytest.mark.gpu

NARROW, WIDE = 2.7e-3, 6.2e-3


def close(c, o, lse, rows, tol):
    a, b = o[rows], c.o[rows]
    rel = np.linalg.norm(a - b) / np.linalg.norm(b)
    dl = np.abs(lse[rows] - c.lse[rows]).max()
    print(f"rel-L2 {rel:.2e} lse {dl:.2e}")
    assert np.isfinite(a).all() and rel <= tol and dl <= 7e-3


@pytest.mark.parametrize("cache", ["bf16", "q8"])
@pytest.mark.parametrize("by", [2.0 ** 12, 2.0 ** 24, 2.0 ** 30, 2.0 ** 40, 2.0 ** 90])
def test_large_token_hidden_from_later_rows(Q, by, cache):  # noqa: F811
    """A token of the window's first tile that the first two rows see and the others do not."""
    def change(case):
        case.c[6] *= np.float32(by)
    c = R.Case(lens=[1024], new=[20], window=1000, outliers=0, cache=cache, change=change)       # row i sees tokens from 5 + i on
    o, lse = Device(Q, c).run(Q)
    close(c, o, lse, slice(2, 20), WIDE)
    close(c, o, lse, slice(0, 2), WIDE)


@pytest.mark.parametrize("octaves", [20, 30, 160])
@pytest.mark.parametrize("by", [2.0 ** 11, 2.0 ** 30])
@pytest.mark.parametrize("at", [5, 700])
def test_large_token_with_a_low_logit(Q, at, by, octaves):  # noqa: F811
    """Visible, and so far below the others that it adds nothing, as much as they, or more."""
    def change(case):
        case.qr[:] = 1
        case.r[:] = 0
        case.r[at] = -np.round(octaves * np.log(2) * 16) / 16 / 16        # 32 of them at scale 1 / 2: octaves ln 2
        case.c[at] *= np.float32(by)
        case.q *= np.float32(0.1)
    c = R.Case(lens=[1024], new=[20], rope_gain=False, outliers=0, scale=0.5, change=change)
    o, lse = Device(Q, c).run(Q)
    close(c, o, lse, slice(0, 20), WIDE)


@pytest.mark.parametrize("cache", ["bf16", "q8"])
def test_small_weights_beside_a_hidden_large_token(Q, cache):  # noqa: F811
    """A heavy token, many weights 2^-19 of its own that add up to a tenth of it, and, in the heavy one's tile, a token 2^11 times
    as large that most rows do not see."""
    n, heavy = 60000, 100
    def change(case):
        case.qr[:] = 1
        case.r[:] = 0
        case.r[heavy] = np.round(19 * np.log(2) * 16) / 16 / 16
        case.c += np.float32(2)                                # values with a mean: small weights count by their sum
        case.c[6] *= np.float32(2.0 ** 11)
    c = R.Case(lens=[n], new=[20], H=4, G=2, window=n - 24, rope_gain=False, outliers=0, scale=0.5, cache=cache, change=change)
    o, lse = Device(Q, c).run(Q)
    close(c, o, lse, slice(2, 20), NARROW)


@pytest.mark.parametrize("new", [1, 40])
def test_sizes_that_grow_and_fall(Q, new):  # noqa: F811
    """Every tile another size, within a tile sizes up to 2^14 apart."""
    def change(case):
        g = np.random.default_rng(3)
        n = case.c.shape[0]
        case.c *= (2.0 ** np.repeat(g.integers(-12, 13, -(-n // 128)), 128)[:n] * 2.0 ** g.integers(0, 15, n))[:, None].astype(np.float32)
    c = R.Case(lens=[4000], new=[new], outliers=0, change=change)
    compare(c, *Device(Q, c).run(Q), wide=True)


@pytest.mark.parametrize("by", [2.0 ** -20, 2.0 ** -30, 2.0 ** -38])
@pytest.mark.parametrize("zeros", [slice(0, 128), slice(256, 384), slice(130, 200)])
def test_zero_latents_beside_small_ones(Q, zeros, by):  # noqa: F811
    """A tile of zeros has no size that the others could be measured by."""
    def change(case):
        case.c *= np.float32(by)
        case.c[zeros] = 0
    c = R.Case(lens=[600], new=[50], outliers=0, change=change)
    o, lse = Device(Q, c).run(Q)
    close(c, o, lse, slice(0, 50), NARROW)


@pytest.mark.parametrize("cache", ["bf16", "q8"])
@pytest.mark.parametrize("value", [2.0 ** 30, 2.0 ** 100, float("nan")])
@pytest.mark.parametrize("sinks", [0, 2])
def test_token_that_no_row_sees_changes_nothing(Q, sinks, value, cache):  # noqa: F811
    """Not a bit of any row, where a tile holds visible tokens beside it."""
    def run(change):
        c = R.Case(lens=[1024, 300], new=[20, 7], window=1000, sinks=sinks, cache=cache, change=change)
        return c, Device(Q, c).run(Q)

    def change(case):
        case.c[3:5] *= np.float32(value)                       # the first row sees tokens from 5 on, and the sinks
    c, (o, lse) = run(None)
    compare(c, o, lse)
    _, (o2, lse2) = run(change)
    assert (o == o2).all() and (lse == lse2).all()


def test_page_that_no_row_sees(Q):  # noqa: F811
    """Pages in front of the windows may be given back: their entries are not looked up."""
    c = R.Case(lens=[1024], new=[20], window=950, page=16)                    # the first row sees tokens from 55 on
    dev = Device(Q, c)
    want = dev.run(Q)
    dev.table[0, :3] = torch.tensor([-1, 2 ** 31 - 1, -7], dtype=torch.int32)
    got = dev.run(Q)
    assert all((a == b).all() for a, b in zip(got, want))
