"""The 8-bit latent cache (qkmla_append_q8, qkmla_decode_ext) and windowed decode on the GPU, against
plain 64-bit forms.

Tolerances.  CUDA-core kernel: fp32 throughout, the fp32 rule of this method (rel-L2 and element-wise
1e-5).  Tensor-core kernels: the weights of the output product are rounded -- 8-bit cache: to the sum of
two 8-bit values, off by at most 2^-4 x 2^-4 = 2^-8 of the weight; bf16 cache: to bf16, 2^-8 -- so |o - ref|
<= 2^-8 sum_t p_t |c_t|, and rel-L2 stays within the method's rule for a bf16 cache, 5e-3, max-abs 2e-2 of
the output's scale.  lse (fp32) of the 8-bit cache has no rounded weight in it: RoPE queries as two bf16
parts leave 2^-16 of a logit part of at most d_r max|gamma| scale < 8, far below 1e-3.
"""
import math

import numpy as np
import pytest
import torch

import q8_window_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from qk_normed_latent_gb300 import build as B
    B.build()
    import qk_normed_latent_gb300 as Q
    return Q


class Device:
    """A Case's tensors on the GPU and its prepared call."""

    def __init__(self, Q, c, o_dtype=torch.float32, **kw):
        d = "cuda"
        dt = torch.float32 if c.cache == "f32" else torch.bfloat16
        self.c = c
        self.kv = torch.from_numpy(c.kv).to(d)
        if c.cache != "q8":
            self.kv = self.kv.view(dt)
        self.scale = torch.from_numpy(c.kv_scale).to(d) if c.cache == "q8" else None
        self.ak = torch.from_numpy(c.ak).to(d)
        self.o = torch.full((len(c.lens), c.s_q, c.H, c.d_c), float("nan"), dtype=o_dtype, device=d)
        self.lse = torch.full((len(c.lens), c.s_q, c.H), float("nan"), device=d)
        self.lens = torch.tensor(c.lens, dtype=torch.int32, device=d)
        self.table = None if c.table is None else torch.from_numpy(c.table).to(d)
        self.in_ = [torch.from_numpy(c.qt).to(d).to(dt), torch.from_numpy(c.aq).to(d), torch.from_numpy(c.qr).to(d),
                    torch.from_numpy(c.grq).to(d)]
        self.call = Q.prepare_decode(*self.in_, self.kv, self.ak, self.lens, self.table, c.page, c.max_pages, c.G,
                                     c.scale, R.EPS, self.o, self.lse, plain=c.plain, kv_scale=self.scale,
                                     window=c.window, sinks=c.sinks, **kw)

    def run(self, Q):
        self.call()
        assert Q.get_device_status() == 0
        return self.o.double().cpu().numpy(), self.lse.double().cpu().numpy()


def check(Q, c, simt, o_dtype=torch.float32, **kw):
    dev = Device(Q, c, o_dtype=o_dtype, force_simt=simt, **kw)
    if not simt:
        assert dev.call.kernel_name == "tcgen05"
    o, lse = dev.run(Q)
    assert np.isfinite(o).all()
    empty = np.isneginf(c.lse)
    assert (np.isneginf(lse) == empty).all()
    assert (o[empty] == 0).all()
    if empty.all():
        return dev
    d, ref = np.abs(o - c.o), np.linalg.norm(c.o)
    dl = np.abs(lse[~empty] - c.lse[~empty])
    rel, big = np.linalg.norm(o - c.o) / ref, max(1.0, np.abs(c.o).max())
    print(f"rel-L2 {rel:.2e} max {d.max():.2e} (scale {big:.2e}) lse {dl.max():.2e}")
    if simt and o_dtype == torch.float32:
        assert rel <= 1e-5 and (d <= 1e-5 * np.maximum(big, np.abs(c.o))).all()
        assert (dl <= 1e-5 * np.maximum(1, np.abs(c.lse[~empty]))).all()
    else:
        assert rel <= 5e-3 and d.max() <= 2e-2 * big
        assert dl.max() <= (1e-3 if c.cache == "q8" or simt else 2e-2)
    return dev


SIMT = [
    dict(lens=[0, 1, 2, 31, 33, 200]),
    dict(lens=[5, 64, 65], s_q=3, H=8, G=8, d_c=128, d_r=64, page=16),
    dict(lens=[1, 2, 100], s_q=3),                                          # lengths below s_q: empty rows
    dict(lens=[300, 77], window=1),
    dict(lens=[300, 77, 10], window=50, sinks=4, s_q=2),
    dict(lens=[300, 77, 10], window=33, sinks=70, H=32, G=2, page=24),
    dict(lens=[130], d_c=100, d_r=20, H=6, G=3, page=7, window=30, sinks=3),
    dict(lens=[257, 20], window=100, sinks=4, alpha="f16"),
    dict(lens=[257, 20], window=100, sinks=4, plain=True, outlier=1.0),
    dict(lens=[300, 40], contiguous=True, window=64, sinks=1),
]


@pytest.mark.parametrize("cache", ["q8", "bf16", "f32"])
@pytest.mark.parametrize("k", range(len(SIMT)))
def test_simt(Q, k, cache):
    kw = dict(SIMT[k])
    if cache != "q8" and not kw.get("window"):
        kw["window"], kw["sinks"] = 2 ** 31 - 1, 5                          # a window over everything
    check(Q, R.Case(cache=cache, **kw), simt=True)


@pytest.mark.parametrize("cache", ["q8", "bf16"])
@pytest.mark.parametrize("H", [16, 128])
def test_repeats_and_streams(Q, cache, H):
    """The same bits on every call, in order after work on the caller's stream, and from a captured graph."""
    c = R.Case([900, 333, 0, 64], cache=cache, window=300, sinks=5, s_q=2, H=H, G=4 if H == 16 else 8,
               d_c=256 if H == 16 else 512, d_r=32 if H == 16 else 64)
    dev = Device(Q, c)
    first = [x.copy() for x in dev.run(Q)]
    side = torch.cuda.Stream()
    qt = dev.in_[0].clone()
    for _ in range(5):
        dev.in_[0].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200000)
            dev.in_[0].copy_(qt)
            dev.call(side)
        side.synchronize()
        assert (dev.o.double().cpu().numpy() == first[0]).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dev.call()
    dev.o.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert (dev.o.double().cpu().numpy() == first[0]).all() and (dev.lse.double().cpu().numpy() == first[1]).all()


@pytest.mark.parametrize("splits", [1, 3, 7])
def test_simt_splits(Q, splits):
    check(Q, R.Case([200, 0, 1, 90], window=60, sinks=5, s_q=2), simt=True, num_splits=splits)


TC = [
    dict(lens=[1]),
    dict(lens=[0, 1, 2, 63, 64, 65, 127, 128, 129, 200, 400]),
    dict(lens=[1000], num_splits=1),
    dict(lens=[1000, 333], s_q=2, page=16),
    dict(lens=[5, 64, 165], s_q=3, H=32, G=4, page=32),
    dict(lens=[1, 2, 100], s_q=3),                                          # lengths below s_q: empty rows
    dict(lens=[1, 2, 300], s_q=4, H=48, G=3, page=128),
    dict(lens=[700, 77], window=1, page=64),
    dict(lens=[700, 77, 10], window=50, sinks=4, s_q=2, page=16),
    dict(lens=[1500, 177, 10], window=333, sinks=270, H=32, G=2, page=256),
    dict(lens=[1500, 900], window=256, sinks=128, H=64, G=8, d_c=512, d_r=64, s_q=3, page=32),
    dict(lens=[640, 100], H=128, G=8, d_c=512, d_r=64),
    dict(lens=[640, 100], H=16, G=1, d_c=512, d_r=64, contiguous=True),
    dict(lens=[300, 257], H=16, G=8, d_c=128, d_r=64, page=16),
    dict(lens=[300, 257], H=32, G=8, d_c=128, d_r=32, page=16, s_q=2),
    dict(lens=[300, 257], H=32, G=4, d_c=256, d_r=64, page=16, s_q=2),
    dict(lens=[257, 20], alpha="f16"),
    dict(lens=[257, 20], H=128, G=8, d_c=512, d_r=64, alpha="f16", window=100, sinks=3),
    dict(lens=[257, 20], plain=True, outlier=1.0),
    dict(lens=[2000, 900], num_splits=3),
    dict(lens=[900, 300], spread=20.0),                                     # scales over 40 binades
    dict(lens=[900, 300], spread=1.0, outlier=1e6),
    dict(lens=[900, 300], zero=True),                                       # all-zero latents: scale 0
    dict(lens=[1500], q_scale=1e-3, H=32, G=4),
    dict(lens=[3000] * 5, d_c=512, d_r=64, H=128, G=8, s_q=2),
    dict(lens=[(37 * k) % 300 for k in range(140)], window=100, sinks=5),   # planned by the scheduler kernel
]


WINDOW = [
    dict(lens=[1], window=5),
    dict(lens=[0, 1, 2, 63, 64, 65, 127, 128, 129, 300, 700], window=100, sinks=4),
    dict(lens=[1000, 333], window=1, s_q=2),
    dict(lens=[1000, 333, 70], window=64, sinks=64, s_q=3),
    dict(lens=[1, 2, 100, 400], window=70, sinks=3, s_q=4),                  # lengths below s_q
    dict(lens=[1500, 900], window=513, sinks=130, num_splits=3),
    dict(lens=[1500, 900], window=513, sinks=130, s_q=2, alpha="f16"),
    dict(lens=[700, 100], window=200, sinks=7, plain=True, outlier=1.0),
    dict(lens=[700, 100], window=200, sinks=7, contiguous=True),
    dict(lens=[400, 100], window=2 ** 31 - 1, sinks=2 ** 31 - 1),
    dict(lens=[(37 * k) % 300 for k in range(140)], window=100, sinks=5),    # planned by the scheduler kernel
]
SHAPES = [dict(), dict(H=32, G=2), dict(H=128, G=8, d_c=512, d_r=64), dict(H=64, G=8, d_c=512, d_r=64, page=128),
          dict(H=16, G=1, d_c=512, d_r=64)]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("k", range(len(WINDOW)))
def test_window_tensor_core(Q, k, shape):
    kw = dict(WINDOW[k])
    splits = kw.pop("num_splits", 0)
    if len(kw["lens"]) > 20 and SHAPES[shape].get("d_c") == 512:
        kw["lens"] = kw["lens"][:130]
    check(Q, R.Case(cache="bf16", **kw, **SHAPES[shape]), simt=False, num_splits=splits)


@pytest.mark.parametrize("H", [16, 128])
def test_window_over_everything_is_decode(Q, H):
    """A window that covers every token gives the values of the call without one.  The windowed call carries (part
    of) the RoPE query in two parts: both are within the method's rule, 5e-3 of the result's norm, and a logit's
    change is at most 2^-8 sum_j |q^r_j k^r_j| <= 2^-8 d_r max|gamma| scale < 2^-8 x 64 x 1.5 x 0.11."""
    c = R.Case([700, 130, 64], cache="bf16", H=H, G=4 if H == 16 else 8, d_c=256 if H == 16 else 512,
               d_r=32 if H == 16 else 64, s_q=2)
    a, la = Device(Q, c).run(Q)
    c.window = 700
    b, lb = Device(Q, c).run(Q)
    assert np.linalg.norm(a - b) <= 5e-3 * np.linalg.norm(a) and np.abs(la - lb).max() <= 2.0 ** -8 * 64 * 1.5 * 0.11


@pytest.mark.parametrize("k", range(len(TC)))
def test_q8_tensor_core(Q, k):
    kw = dict(TC[k])
    splits = kw.pop("num_splits", 0)
    check(Q, R.Case(**kw), simt=False, num_splits=splits)


@pytest.mark.parametrize("cache", ["q8", "bf16"])
def test_launches(Q, cache):
    """One kernel where no sequence can be split, a combine kernel where one can, a scheduler beyond 128 sequences."""
    for kw, launches in ((dict(lens=[512, 3], window=600), 1), (dict(lens=[513, 3], window=600), 2),
                         (dict(lens=[3000], window=300, sinks=60), 1), (dict(lens=[3000], window=2000), 2),
                         (dict(lens=[5] * 129, window=9), 2)):
        dev = check(Q, R.Case(cache=cache, **kw), simt=False)
        assert dev.call.launch_count == launches, kw


def test_q8_tensor_core_bf16_output(Q):
    check(Q, R.Case([600, 70], s_q=2), simt=False, o_dtype=torch.bfloat16)


def test_q8_rising_logits(Q):
    """Keys whose logits rise along the sequence move the running maximum in every tile."""
    c = R.Case([1500], plain=True, outlier=1.0, seed=3)
    g = np.random.Generator(np.random.PCG64(5))
    direction = c.qt[0, 0, 0] / np.linalg.norm(c.qt[0, 0, 0])
    lat = (0.1 * g.standard_normal((1500, c.d_c)) + np.linspace(-40, 40, 1500)[:, None] * direction).astype(np.float32)
    codes, sc = R.quantise(lat)
    t = np.arange(1500)
    slot = c.table[0, t // c.page] * c.page + t % c.page
    c.kv[slot, :c.d_c], c.kv_scale[slot] = codes, sc
    kr = (c.kv[slot, c.d_c:].copy().view(np.uint16).astype(np.uint32) << 16).view(np.float32)
    o, lse = R.attention(c.qt[0], c.aq[0], c.qr[0].astype(np.float64), R.e4m3_decode(codes) * sc[:, None], kr,
                         np.ones((1500, c.G)), 1, 1500, 0, 0, c.scale, True)
    c.o, c.lse = o[None], lse[None]
    for splits in (1, 0):
        check(Q, c, simt=False, num_splits=splits)


@pytest.mark.parametrize("binades", [8, 11, 14])
@pytest.mark.parametrize("shape", [dict(), dict(H=32, G=2), dict(H=64, G=8, d_c=512, d_r=64)])
def test_q8_heavy_token_over_flat_background(Q, shape, binades):
    """One token outweighs each of 20000 others by 2^binades, and together they outweigh it or nearly: what
    the 8-bit weights keep of small ones.  A contribution p_t s_t is off by 2^-8 of itself (2^-11 more from
    its rounding to fp16, 2^-12 for the logit) and by 2^-15 of the row's largest."""
    T = 20000
    c = R.Case([T], plain=True, outlier=1.0, seed=9, **shape)
    g = np.random.Generator(np.random.PCG64(binades))
    base = c.qt[0, 0, 0]
    c.qt[:] = R.bf16(base * (1 + 0.01 * g.standard_normal(c.qt.shape)))
    lat = (0.3 * g.standard_normal((T, c.d_c))).astype(np.float32)
    lat[0] += base * (binades * math.log(2) / (c.scale * np.linalg.norm(base) ** 2))
    codes, sc = R.quantise(lat)
    t = np.arange(T)
    slot = c.table[0, t // c.page] * c.page + t % c.page
    c.kv[slot, :c.d_c], c.kv_scale[slot] = codes, sc
    kr = (c.kv[slot, c.d_c:].copy().view(np.uint16).astype(np.uint32) << 16).view(np.float32) * np.float32(0.1)
    c.kv[slot, c.d_c:] = R.bf16_bits(kr).view(np.uint8)
    kr = R.bf16(kr)
    x = R.e4m3_decode(codes)
    o, lse = R.attention(c.qt[0], c.aq[0], c.qr[0].astype(np.float64), x * sc[:, None], kr, np.ones((T, c.G)), 1, T, 0, 0,
                         c.scale, True)
    logit = c.scale * (c.qt[0, 0].astype(np.float64) @ (x * sc[:, None]).T + c.qr[0, 0].astype(np.float64) @ kr.T)
    a = np.exp(logit - lse[0][:, None]) * sc                                  # contributions, [H, T]
    off = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12) * a + 2.0 ** -15 * a.max(axis=1, keepdims=True)
    got, got_lse = Device(Q, c).run(Q)
    assert (np.abs(got[0, 0] - o[0]) <= off @ np.abs(x) + 1e-6).all()
    assert np.abs(got_lse[0] - lse).max() <= 1e-3
    print("share of the heavy token", np.exp(logit[0, 0] - lse[0, 0]), "of the bound used",
          (np.abs(got[0, 0] - o[0]) / (off @ np.abs(x))).max(), "rel-L2", np.linalg.norm(got[0] - o) / np.linalg.norm(o))


@pytest.mark.parametrize("kw", [
    dict(H=128, G=8, d_c=128, d_r=64, s_q=8, outlier=3.0),
    dict(H=64, G=8, d_c=256, d_r=32, s_q=16, outlier=3.0, window=3000, sinks=70),
    dict(H=64, G=8, d_c=256, d_r=32, s_q=16, cache="bf16", window=100000, sinks=3),
    dict(H=128, G=8, d_c=512, d_r=64, s_q=8, cache="bf16", window=2900, sinks=130),
])
def test_ragged_batch_of_more_than_a_wave(Q, kw):
    """A plan of chunks and remainders: sequences of several chunks, of exactly one or two, of a chunk and a few
    tokens, shorter ones, empty ones.  16 row blocks put an even share near 30 tiles."""
    share = 64 * 30
    lens = [4 * share + 700, 3 * share, 2 * share + 65, share + 1100, share + 64, share, 900, 513, 512, 64, 1, 0, 0, 333, 2000, 250]
    check(Q, R.Case(lens, **kw), simt=False)


APPEND = [
    dict(N=1), dict(N=16), dict(N=33), dict(N=257, G=8, d_c=512, d_h=128, d_r=64), dict(N=5, G=3, d_c=100, d_h=36, d_r=20),
    dict(N=40, rope=True), dict(N=300, G=8, d_c=512, d_h=128, d_r=64, rope=True), dict(N=20, alpha="f16"),
    dict(N=20, plain=True), dict(N=1000, G=8, d_c=512, d_h=128, d_r=64), dict(N=130, G=2, d_c=128, d_h=64, d_r=0),
    dict(N=700, G=4, d_c=256, d_h=64, d_r=32, rope=True),
]


@pytest.mark.parametrize("k", range(len(APPEND)))
def test_append_q8(Q, k):
    """Codes and scales are exact; alpha^k is an fp32 sum of d_c products (2e-5 relative is over 300 roundings of
    2^-24), RoPE keys are bf16 (2^-8) of an fp32 value."""
    a = dict(N=16, G=4, d_c=256, d_h=64, d_r=32, rope=False, alpha="f32", plain=False)
    a.update(APPEND[k])
    N, G, d_c, d_h, d_r = a["N"], a["G"], a["d_c"], a["d_h"], a["d_r"]
    g = np.random.Generator(np.random.PCG64(k))
    c = (g.standard_normal((N, d_c)) * np.exp2(g.uniform(-4, 4, N))[:, None]).astype(np.float32)
    c[0, 0] = 448.0 * np.abs(c[0]).max()                       # one dominant value: the rest near the bottom of e4m3
    if N > 4:
        c[1] = 0
        c[2] = np.float32(1e-39)                               # below fp32's normal range
        c[3, :] = np.float32(2.0) ** -9 * (np.arange(d_c) + 0.5)  # ties
        c[4] *= np.float32(2.0 ** 60)
    r = g.standard_normal((N, d_r)).astype(np.float32)
    wk = (g.standard_normal((G, d_c, d_h)) / np.sqrt(d_c)).astype(np.float32)
    grk = (1 + 0.1 * g.standard_normal(d_r)).astype(np.float32)
    pos = g.integers(0, 200000, N).astype(np.int32)
    total = N + 9
    slots = g.permutation(total)[:N].astype(np.int64)
    skipped = g.random(N) < 0.1
    slots[skipped] = -1
    d = "cuda"
    kv = torch.full((total, d_c + 2 * d_r), 0xA5, dtype=torch.uint8, device=d)
    sc = torch.full((total,), -7.0, device=d)
    ak = torch.full((total, G), -7.0, device=d, dtype=torch.float16 if a["alpha"] == "f16" else torch.float32)
    t = lambda x: torch.from_numpy(x).to(d)  # noqa: E731
    Q.append_q8(t(c), t(r), t(wk), t(grk) if d_r else None, t(slots), kv, sc, ak, R.EPS,
                positions=t(pos) if a["rope"] else None, rope_theta=10000.0, plain=a["plain"])
    assert Q.get_device_status() == 0
    kv, sc, ak = kv.cpu().numpy(), sc.cpu().numpy().astype(np.float64), ak.double().cpu().numpy()
    codes, scale = R.quantise(c)
    live = ~skipped
    at = slots[live]
    untouched = np.setdiff1d(np.arange(total), at)
    assert (kv[untouched] == 0xA5).all() and (sc[untouched] == -7).all() and (ak[untouched] == -7).all()
    assert (sc[at] == scale[live]).all()
    got, want = kv[at, :d_c], codes[live]
    assert ((got == want) | ((got & 127 == 0) & (want & 127 == 0))).all()
    rr = R.rope_rotate(r, pos, 10000.0) if a["rope"] else r.astype(np.float64)
    ref = (rr if a["plain"] else R.rms_normalise(rr, grk)) if d_r else rr
    if d_r:
        bits = kv[at, d_c:].copy().view(np.uint16).astype(np.uint32) << 16
        np.testing.assert_allclose(bits.view(np.float32), ref[live], rtol=2.0 ** -8 + 1e-5, atol=1e-5)
    c_hat = R.e4m3_decode(codes) * scale[:, None]
    want = np.ones((N, G)) if a["plain"] else R.inverse_rms(c_hat, wk)
    if a["alpha"] == "f16":                                    # subnormal halves step by 2^-24
        np.testing.assert_allclose(ak[at], want[live], rtol=2.0 ** -11 + 2e-5, atol=2.0 ** -25)
    else:
        # a key this large squares past fp32: alpha^k is then 0 against 1e-18
        np.testing.assert_allclose(ak[at], want[live], rtol=2e-5, atol=1e-15)


def test_append_q8_not_finite(Q):
    """A value that is not finite is stored as NaN and shows; its neighbours keep codes of their own scale."""
    d = "cuda"
    c = torch.ones((3, 128), device=d)
    c[0, 5], c[1, 7] = float("nan"), float("inf")
    kv = torch.zeros((3, 128), dtype=torch.uint8, device=d)
    sc, ak = torch.zeros(3, device=d), torch.zeros((3, 1), device=d)
    Q.append_q8(c, torch.zeros((3, 0), device=d), torch.ones((1, 128, 64), device=d), None,
                torch.arange(3, device=d), kv, sc, ak, R.EPS)
    assert Q.get_device_status() == 0
    x = kv.view(torch.float8_e4m3fn).float() * sc[:, None]
    assert torch.isnan(x[0, 5]) and torch.isnan(x[1, 7])
    assert torch.isnan(ak[0]).all() and torch.isnan(ak[1]).all()
    assert (x[2] == 1).all() and (x[0, :5] == 1).all()


def test_append_q8_slot_out_of_range(Q):
    d = "cuda"
    kv = torch.zeros((4, 320), dtype=torch.uint8, device=d)
    sc, ak = torch.zeros(4, device=d), torch.zeros((4, 4), device=d)
    Q.append_q8(torch.ones((2, 256), device=d), torch.ones((2, 32), device=d), torch.ones((4, 256, 64), device=d), None,
                torch.tensor([4, 1], device=d), kv, sc, ak, R.EPS)
    assert Q.get_device_status() == Q.ERR_DEVICE_BOUNDS
    assert (sc.cpu() != 0).tolist() == [False, True, False, False]


@pytest.mark.parametrize("cache", ["q8", "bf16"])
@pytest.mark.parametrize("simt", [True, False])
def test_bad_page_and_length(Q, cache, simt):
    """A page id or a length out of range is reported; the other sequence keeps its result."""
    for bad_page in (True, False):
        c = R.Case([100, 70], cache=cache, window=0 if cache == "q8" else 500)
        dev = Device(Q, c, force_simt=simt)
        if bad_page:
            dev.table[0, 0] = 1 << 30
        else:
            dev.lens[0] = c.max_pages * c.page + 1
        dev.call()
        assert Q.get_device_status() == Q.ERR_DEVICE_BOUNDS
        assert np.linalg.norm(dev.o[1].double().cpu().numpy() - c.o[1]) <= 5e-3 * np.linalg.norm(c.o[1])


@pytest.mark.parametrize("cache,window,sinks", [("e4m3", 0, 0), ("e4m3", 300, 4), ("bf16", 300, 4)])
def test_pipeline_step(Q, cache, window, sinks):
    """The whole path -- absorb, append of the step's tokens, decode -- on the 8-bit cache and through a window,
    against the 64-bit form over what the cache then holds; the appended latents against their quantised inputs."""
    import workloads as W
    from qk_normed_latent_gb300.pipeline import DeviceState
    w = W.small(W.WORKLOADS[1].with_(cache_dtype=cache), 3, (700, 130, 64))
    st = DeviceState(w, window=window, sinks=sinks, keep_host=True)
    st.step()
    assert Q.get_device_status() == 0
    kv, ak = st.kv.cpu(), st.ak.double().cpu().numpy()
    qt, aq = st.q_tilde.double().cpu().numpy(), st.alpha_q.double().cpu().numpy()
    qr = R.rms_normalise(st.q_rope.cpu().numpy(), st.grq.cpu().numpy().astype(np.float64))
    for b, n in enumerate(int(x) for x in st.lens):
        slot = W.slots_of(st.table_np, st.page_size, b, np.arange(n))
        if cache == "e4m3":
            codes, scale = kv[slot, :w.d_c].numpy(), st.kv_scale.cpu().numpy()[slot].astype(np.float64)
            want, want_scale = R.quantise(st.host_seqs[b][0])
            assert (scale == want_scale).all() and ((codes == want) | ((codes & 127 == 0) & (want & 127 == 0))).all()
            c_hat = R.e4m3_decode(codes) * scale[:, None]
            kr = kv[slot, w.d_c:].contiguous().view(torch.bfloat16).double().numpy()
        else:
            c_hat, kr = kv[slot, :w.d_c].double().numpy(), kv[slot, w.d_c:].double().numpy()
        o, lse = R.attention(qt[b], aq[b], qr[b], c_hat, kr, ak[slot], w.s_q, n, window, sinks, w.scale)
        got = st.o[b].double().cpu().numpy()
        assert np.linalg.norm(got - o) <= 5e-3 * np.linalg.norm(o)
        assert np.abs(st.lse[b].double().cpu().numpy() - lse).max() <= 2e-2
