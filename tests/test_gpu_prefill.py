"""qkmla_prefill on the GPU against its definition in 64 bits.

Tolerance.  Operands are fp16, off by at most u = 2^-11 of themselves.  A logit's error is that of q and k
(independent, u each) and of W^K within k: with q^, k of root mean square about 1 and scale 1 / sqrt(d) its root
mean square is at most u (sqrt 2 + 1) 1.2 = 2.9 u (1.2: the gains and the spread of |q_j k_j|), and a softmax
weight's sqrt 2 times that (its own logit and the sum's); weight and value are rounded once more, u each.  Together
rel-L2 <= (4.1 + sqrt 2) u = 5.5 u = 2.7e-3 for fp32 outputs; a bf16 output adds 2^-8 in quadrature, 4.7e-3.  Where
a tile's values and weights are bf16 they are off by 2^-8 each: sqrt 2 x 2^-8 in quadrature, 6.2e-3 (bf16 output 7.3e-3).
A single element is held to 6 such errors of the output's own size (its root mean square, or |o| where larger); an
lse, with the logit error 2.9 u, to 5 of them, 7e-3."""
import numpy as np
import pytest
import torch

import prefill_ref as R

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
    """A Case's tensors on the GPU and its prepared call; outputs start as NaN."""

    def __init__(self, Q, c, o=torch.float32, total=None, lse=True):
        d = "cuda"
        self.c = c
        qt = torch.bfloat16 if c.qtype == "bf16" else torch.float32
        up = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(d)  # noqa: E731
        self.weights = Q.prefill_weights(up(c.wk), up(c.wv.view(np.int16)).view(torch.bfloat16))
        self.q, self.qr = up(c.q).to(qt), up(c.qr).to(qt)
        self.gains = [up(c.gq), up(c.gk), up(c.grq)]
        self.kv = up(c.kv) if c.cache == "q8" else up(c.kv.view(np.int16)).view(torch.bfloat16)
        self.kv_scale = up(c.kv_scale) if c.cache == "q8" else None
        self.ak = up(c.ak.astype(np.float16) if c.alpha == "f16" else c.ak)
        self.start, self.lens = up(c.start), up(np.array(c.lens, np.int32))
        self.table = up(c.table)
        rows = c.q.shape[0]
        self.o = torch.full((rows, c.H, c.d_v), float("nan"), dtype=o, device=d)
        self.lse = torch.full((rows, c.H), float("nan"), device=d) if lse else None
        self.args = (self.q, self.qr, *self.gains, self.weights, self.kv, self.ak, self.start, self.lens, self.table, c.page,
                     c.max_pages, sum(c.lens) if total is None else total, c.scale, R.EPS, self.o, self.lse)
        self.kw = dict(kv_scale=self.kv_scale, window=c.window, sinks=c.sinks)
        self.call = Q.prepare_prefill(*self.args, **self.kw)

    def run(self, Q):
        self.call()
        assert Q.get_device_status() == 0
        return self.o.double().cpu().numpy(), self.lse.double().cpu().numpy()


def compare(c, o, lse, o_dtype=torch.float32, wide=False):
    """`wide`: tiles whose values are bf16."""
    n = c.rows
    o, lse = o[:n], lse[:n]
    bad = np.isnan(c.lse)
    assert (np.isnan(lse) == bad).all()
    assert np.isnan(o[bad]).all() and np.isfinite(o[~bad]).all()
    empty = np.isneginf(c.lse)
    assert (np.isneginf(lse) == empty).all()
    assert (o[empty] == 0).all()
    there = ~bad & ~empty
    if not there.any():
        return
    a, b = o[there], c.o[there]
    tol = 6.2e-3 if wide else 2.7e-3
    if o_dtype == torch.bfloat16:
        tol = 7.3e-3 if wide else 4.7e-3
    rel = np.linalg.norm(a - b) / np.linalg.norm(b)
    rms = np.sqrt((b ** 2).mean(axis=-1, keepdims=True))
    big = (np.abs(a - b) / np.maximum(rms, np.abs(b))).max()
    dl = np.abs(lse[there] - c.lse[there]).max()
    print(f"rel-L2 {rel:.2e} largest {big:.2e} lse {dl:.2e}")
    assert rel <= tol and big <= 6 * tol and dl <= 7e-3


def check(Q, o=torch.float32, wide=False, **kw):
    c = R.Case(**kw)
    dev = Device(Q, c, o=o)
    compare(c, *dev.run(Q), o, wide)
    return dev


SHAPES = [
    dict(H=8, G=4, d_c=128, d_h=64, d_r=32, d_v=64),
    dict(H=16, G=4, d_c=256, d_h=64, d_r=32, d_v=64),
    dict(H=32, G=2, d_c=512, d_h=128, d_r=64, d_v=128),
    dict(H=8, G=8, d_c=64, d_h=128, d_r=32, d_v=64),          # a head a unit, one block of latents
    dict(H=8, G=2, G_v=8, d_c=192, d_h=64, d_r=64, d_v=128),  # a value matrix a head
    dict(H=8, G=4, G_v=1, d_c=320, d_h=128, d_r=64, d_v=64),  # an odd number of column blocks
    dict(H=128, G=1, d_c=128, d_h=64, d_r=32, d_v=128),       # two tokens a tile
]
LENGTHS = [
    dict(lens=[1], new=[1]),
    dict(lens=[5], new=[5]),
    dict(lens=[300], new=[17]),
    dict(lens=[128, 129, 127], new=[128, 1, 64], page=7),
    dict(lens=[0, 40, 3, 0, 260, 200], new=[0, 2, 3, 0, 1, 77], page=1),
    dict(lens=[700, 90], new=[33, 90], page=48, cache="q8"),
]


@pytest.mark.parametrize("k", range(len(LENGTHS)))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_shapes(Q, shape, k):
    check(Q, **SHAPES[shape], **LENGTHS[k])


@pytest.mark.parametrize("cache", ["bf16", "q8"])
@pytest.mark.parametrize("o", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("q", ["f32", "bf16"])
@pytest.mark.parametrize("alpha", ["f32", "f16"])
def test_types(Q, cache, o, q, alpha):
    check(Q, o=o, lens=[333, 64], new=[40, 64], cache=cache, q=q, alpha=alpha, rope_gain=q == "f32", contiguous=alpha == "f16")


WINDOWS = [(1, 0), (50, 4), (128, 0), (130, 200), (1000, 3), (2 ** 31 - 1, 7), (300, 128)]


@pytest.mark.parametrize("w", WINDOWS)
def test_window(Q, w):
    check(Q, lens=[900, 260, 77, 1500], new=[100, 260, 1, 513], window=w[0], sinks=w[1])


def test_long_axis_is_cut(Q):
    """Few rows over a long context: many CTAs share a query tile."""
    check(Q, lens=[40000], new=[3], H=4, G=2)
    check(Q, lens=[9000, 12, 20000], new=[1, 12, 30], H=16, G=4, d_c=64, cache="q8")


def test_query_without_a_token(Q):
    """Chunks longer than their sequences: the first queries see nothing."""
    check(Q, lens=[3, 0, 130], new=[10, 4, 300])


def test_rows_behind_the_last_sequence_stay(Q):
    c = R.Case(lens=[50, 60], new=[7, 9], spare_rows=5)
    dev = Device(Q, c, total=4000)
    dev.o.fill_(7)
    dev.lse.fill_(7)
    o, lse = dev.run(Q)
    compare(c, o, lse)
    assert (o[c.rows:] == 7).all() and (lse[c.rows:] == 7).all()


def test_strided_queries(Q):
    """Content and RoPE part of one [rows, H, d_h + d_r] array."""
    c = R.Case(lens=[300, 20], new=[30, 20])
    dev = Device(Q, c)
    both = torch.cat([dev.q, dev.qr], dim=2)
    Q.prefill(both[..., :c.d_h], both[..., c.d_h:], *dev.args[2:], **dev.kw)
    assert Q.get_device_status() == 0
    compare(c, dev.o.double().cpu().numpy(), dev.lse.double().cpu().numpy())


@pytest.mark.parametrize("cache", ["bf16", "q8"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_not_finite_token(Q, cache, value):
    """A token whose latent is not finite: NaN in the rows that see it, and in no other."""
    def change(case):
        case.c[250 - 20, 3] = value                            # a token of the chunk
        case.c[250 + 5, 0] = value                             # of the next sequence's past
    c = R.Case(lens=[250, 90], new=[40, 10], cache=cache, window=60, sinks=2, change=change)
    assert np.isnan(c.lse).any() and not np.isnan(c.lse).all()
    dev = Device(Q, c)
    compare(c, *dev.run(Q))


def test_not_finite_rope_key_and_query(Q):
    def change(case):
        case.r[190, 1] = float("nan")
        case.q[25, 3, 7] = float("nan")
        case.qr[26, 2, 0] = float("inf")
    c = R.Case(lens=[200], new=[30], change=change)
    assert np.isnan(c.lse).any() and not np.isnan(c.lse).all()
    compare(c, *Device(Q, c).run(Q))


@pytest.mark.parametrize("by", [2.0 ** -30, 2.0 ** 20, 2.0 ** 60, 2.0 ** -60])
def test_scale_of_latents(Q, by):
    """Latents of any size: their keys are normalised, their values scale.  Beyond 2^+-40 tiles hold bf16."""
    def change(case):
        case.c *= np.float32(by)
    check(Q, wide=not 2.0 ** -38 < by < 2.0 ** 30, lens=[300], new=[50], change=change)


def test_scales_far_apart(Q):
    """Tokens 2^24 and 2^80 apart, in one tile and in different ones."""
    def change(case):
        case.c[::7] *= np.float32(2.0 ** 24)
        case.c[300:420] *= np.float32(2.0 ** -80)
    check(Q, wide=True, lens=[600], new=[60], change=change)


def test_zero_latents_and_queries(Q):
    def change(case):
        case.c[:128] = 0
        case.c[140] = 0
        case.q[3] = 0
        case.qr[4] = 0
    check(Q, lens=[300], new=[50], change=change)


def test_one_heavy_token_over_many(Q):
    """A sharp softmax: one token takes most of the weight, the others' small weights still add up."""
    def change(case):
        case.qr[:] = 0
        case.qr[:, :, 0] = 1
        case.r[:] *= np.float32(0.05)
        case.r[1234] = 0
        case.r[1234, 0] = 5.0
    check(Q, lens=[5000], new=[20], H=4, G=2, scale=0.5, change=change)


@pytest.mark.parametrize("gain", [1e-4, 300.0])
def test_gains(Q, gain):
    """Large and small gains: queries carry their own power of two.  (With 300 and this scale the logits stay as they are.)"""
    def change(case):
        case.gq[:] *= np.float32(gain)
        case.grq[:] *= np.float32(gain)
    check(Q, lens=[300], new=[40], scale=1 / (gain * 10), change=change)


def test_same_bits_and_graph(Q):
    """The same bits on every call and from a captured graph, whose inputs may change under it."""
    c = R.Case(lens=[2000, 700], new=[90, 1], H=16, G=4)
    dev = Device(Q, c)
    first, _ = dev.run(Q)
    for _ in range(3):
        again, _ = dev.run(Q)
        assert (again == first).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dev.call()
    dev.lens.copy_(torch.tensor([1500, 300], dtype=torch.int32))
    dev.o.fill_(float("nan"))
    g.replay()
    assert Q.get_device_status() == 0
    got = dev.o.clone()
    dev.call()
    torch.cuda.synchronize()
    assert torch.equal(got, dev.o) and torch.isfinite(got).all() and not torch.equal(got.double().cpu(), torch.from_numpy(first))


def test_streams(Q):
    """Two calls on streams of their own, each with its workspace."""
    cases = [R.Case(lens=[800], new=[60], seed=s) for s in (1, 2)]
    devs = [Device(Q, c) for c in cases]
    streams = [torch.cuda.Stream() for _ in devs]
    torch.cuda.synchronize()
    for _ in range(3):
        for d, s in zip(devs, streams):
            d.call(s)
    assert Q.get_device_status() == 0
    for c, d in zip(cases, devs):
        compare(c, d.o.double().cpu().numpy(), d.lse.double().cpu().numpy())


def test_same_as_the_decode_path(Q):
    """prefill = absorb_query, decode_ext and up_project over the same cache."""
    c = R.Case(lens=[700, 333], new=[4, 4], H=16, G=4, d_c=256)
    dev = Device(Q, c)
    o, lse = dev.run(Q)
    wk = torch.from_numpy(c.wk).cuda()
    wv = torch.from_numpy(c.wv.view(np.int16)).cuda().view(torch.bfloat16)
    qt = torch.empty((c.rows, c.H, c.d_c), dtype=torch.bfloat16, device="cuda")
    aq = torch.empty((c.rows, c.H), device="cuda")
    Q.absorb_query(dev.q, dev.gains[0], dev.gains[1], wk, R.EPS, qt, aq)
    lat = torch.empty((2, 4, c.H, c.d_c), device="cuda")
    lse2 = torch.empty((2, 4, c.H), device="cuda")
    Q.decode(qt.view(2, 4, c.H, c.d_c), aq.view(2, 4, c.H), dev.qr.view(2, 4, c.H, c.d_r), dev.gains[2], dev.kv, dev.ak, dev.lens,
             dev.table, c.page, c.max_pages, c.G, c.scale, R.EPS, lat, lse2, window=2 ** 31 - 1, force_simt=True)
    out = torch.empty((8, c.H, c.d_v), device="cuda")
    Q.up_project(lat.view(8, c.H, c.d_c), wv, out)
    a, b = o, out.double().cpu().numpy()
    assert np.linalg.norm(a - b) <= (2.7e-3 + 5e-3) * np.linalg.norm(b)         # plus the bf16 query's rule
    assert np.abs(lse - lse2.view(8, -1).double().cpu().numpy()).max() <= 2e-2 + 7e-3


def test_many_sequences(Q):
    """More sequences than a warp looks at at once, among them idle slots (no rows, no tokens)."""
    lens = [(37 * i) % 211 for i in range(150)]
    new = [min(n, (13 * i) % 7) for i, n in enumerate(lens)]
    check(Q, lens=lens, new=new, H=4, G=2, d_c=64, page=16)


@pytest.mark.parametrize("window", [0, 100])
def test_more_tiles_than_ctas(Q, window):
    """Shares of the expansion that cut a tile, and long query lists."""
    check(Q, lens=[30000, 9000], new=[70, 5], H=4, G=4, d_c=512, d_h=128, d_r=64, d_v=128, window=window, sinks=5 if window else 0)


def test_no_rows_at_all(Q):
    """A padded step none of whose slots has a chunk: nothing is written."""
    c = R.Case(lens=[40, 0, 9], new=[0, 0, 0], spare_rows=6)
    dev = Device(Q, c)
    dev.o.fill_(3)
    dev.lse.fill_(3)
    o, lse = dev.run(Q)
    assert (o == 3).all() and (lse == 3).all()


def bounds(Q, change, keep=None):
    """The call reports what is out of range; a sequence of the step that it does not touch is right."""
    c = R.Case(lens=[200, 150, 90], new=[20, 30, 9])
    dev = Device(Q, c)
    change(dev)
    dev.call()
    assert Q.get_device_status() == Q.ERR_DEVICE_BOUNDS
    if keep is not None:
        rows = slice(int(c.start[keep]), int(c.start[keep + 1]))
        a, b = dev.o[rows].double().cpu().numpy(), c.o[rows]
        assert np.linalg.norm(a - b) <= 2.7e-3 * np.linalg.norm(b)
    # and the device is as before
    compare(c, *Device(Q, c).run(Q))


@pytest.mark.parametrize("page", [-1, 10 ** 6])
def test_bad_page(Q, page):
    bounds(Q, lambda d: d.table[1].__setitem__(2, page), keep=0)


@pytest.mark.parametrize("length", [-1, 2 ** 31 - 1, 209])
def test_bad_length(Q, length):
    bounds(Q, lambda d: d.lens.__setitem__(1, length), keep=0)


def test_total_tokens_too_small(Q):
    c = R.Case(lens=[2000, 150], new=[20, 30])
    dev = Device(Q, c, total=300)
    dev.call()
    assert Q.get_device_status() == Q.ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("start", [[0, 30, 20, 59], [0, 20, 50, 60], [3, 20, 50, 59], [0, -5, 50, 59]])
def test_chunk_starts_out_of_order(Q, start):
    bounds(Q, lambda d: d.start.copy_(torch.tensor(start, dtype=torch.int32)))


def test_workspace(Q):
    """A caller's workspace is used if it is large enough; too small a one is replaced, and refused by the C call."""
    import ctypes
    c = R.Case(lens=[100], new=[10])
    dev = Device(Q, c)
    need = Q.lib().qkmla_prefill_workspace_size(ctypes.byref(dev.call.args))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    call = Q.prepare_prefill(*dev.args, **dev.kw, workspace=ws)
    assert call.workspace is ws
    call()
    assert Q.get_device_status() == 0
    compare(c, dev.o.double().cpu().numpy(), dev.lse.double().cpu().numpy())
    call.args.workspace_bytes = need - 1
    assert Q.lib().qkmla_prefill(ctypes.byref(call.args), None) == Q.ERR_WORKSPACE


def test_results_do_not_depend_on_what_the_workspace_held(Q):
    c = R.Case(lens=[700, 40], new=[60, 3], window=200, sinks=3)
    dev = Device(Q, c)
    first = dev.run(Q)[0]
    dev.call.workspace.fill_(0xFF)
    again = dev.run(Q)[0]
    assert (first == again).all()


@pytest.mark.parametrize("cache", ["bf16", "q8"])
def test_pages_beyond_4_gb(Q, cache):
    """A cache of more than 2^32 bytes whose pages in use lie at its end."""
    c = R.Case(lens=[300, 40], new=[20, 3], H=8, G=2, d_c=512, d_h=128, d_r=64, d_v=128, page=16, cache=cache)
    dev = Device(Q, c)
    slots, width = dev.kv.shape
    far = (2 ** 32 // (width * dev.kv.element_size()) + slots) // 16 * 16 + 16
    grown = []
    for t in (dev.kv, dev.ak, dev.kv_scale):
        if t is not None:
            g = torch.empty((far, *t.shape[1:]), dtype=t.dtype, device="cuda")
            g[far - slots:] = t
            t = g
        grown.append(t)
    table = torch.where(dev.table >= 0, dev.table + (far - slots) // 16, dev.table)
    args = list(dev.args)
    args[6], args[7], args[10] = grown[0], grown[1], table
    Q.prefill(*args, **{**dev.kw, "kv_scale": grown[2]})
    assert Q.get_device_status() == 0
    compare(c, dev.o.double().cpu().numpy(), dev.lse.double().cpu().numpy())
    rows = torch.tensor([0, 300, 340], dtype=torch.int32, device="cuda")
    outs = []
    for kv, ak, scale, t in ((dev.kv, dev.ak, dev.kv_scale, dev.table), (*grown, table)):
        x = [torch.zeros((340, n), device="cuda") for n in (512, 64, 2)]
        Q.read_cache(kv, ak, rows, t, 16, c.max_pages, *x, scale)
        outs.append(x)
    assert Q.get_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_a_page_in_two_places_and_two_sequences(Q):
    """A prefix shared by two sequences, and a page that lies twice in one of them."""
    c = R.Case(lens=[64, 64], new=[1, 1], page=16, rope_gain=False)
    dev = Device(Q, c)
    dev.table[1, :2] = dev.table[0, :2]                     # the same first 32 tokens
    dev.table[1, 2] = dev.table[0, 0]                       # and the first 16 once more
    dev.run(Q)
    a, lse = dev.o[1].clone(), dev.lse[1].clone()
    # the same sequence with copies of those pages
    copy = Device(Q, c)
    at = lambda t, j: slice(int(t[j]) * 16, int(t[j]) * 16 + 16)  # noqa: E731
    spare = torch.cat([copy.kv, copy.kv.new_zeros(48, copy.kv.shape[1])]), torch.cat([copy.ak, copy.ak.new_zeros(48, copy.ak.shape[1])])
    first = copy.kv.shape[0] // 16
    for k, j in enumerate((0, 1, 0)):
        for t in spare:
            t[(first + k) * 16:(first + k + 1) * 16] = t[at(copy.table[0], j)]
        copy.table[1, k] = first + k
    args = list(copy.args)
    args[6], args[7] = spare
    Q.prefill(*args, **copy.kw)
    assert Q.get_device_status() == 0
    assert torch.equal(a, copy.o[1]) and torch.equal(lse, copy.lse[1])


def test_two_calls_at_once(Q):
    """Two prepared calls, each with its workspace, on two streams: as each alone, many times."""
    cs = [R.Case(lens=[900], new=[130], seed=1), R.Case(lens=[400, 700], new=[60, 9], seed=2)]
    devs = [Device(Q, c) for c in cs]
    alone = [d.run(Q)[0] for d in devs]
    streams = [torch.cuda.Stream() for _ in devs]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, s in zip(devs, streams):
            d.call(s)
    torch.cuda.synchronize()
    assert Q.get_device_status() == 0
    assert all((d.o.double().cpu().numpy() == a).all() for d, a in zip(devs, alone))


@pytest.mark.parametrize("H,G,G_v", [(512, 512, 512), (4, 1, 4), (128, 2, 1)])
def test_head_extremes(Q, H, G, G_v):
    check(Q, lens=[150], new=[5], H=H, G=G, G_v=G_v, d_c=64)


def test_many_empty_chunks_and_one_row(Q):
    """4096 sequences, most of them idle."""
    lens = [3 if i % 500 == 7 else 0 for i in range(4096)]
    check(Q, lens=lens, new=[1 if n else 0 for n in lens], d_c=64)


@pytest.mark.parametrize("cache", ["bf16", "q8"])
def test_contiguous_cache(Q, cache):
    check(Q, lens=[130, 1, 77], new=[40, 1, 20], contiguous=True, cache=cache)


def test_graph_replayed_over_another_step(Q):
    """A captured call takes lengths, chunks, pages and inputs as they are when it is replayed."""
    a, b = R.Case(lens=[100, 60], new=[10, 20]), R.Case(lens=[60, 100], new=[25, 5], window=0, seed=5)
    dev, other = Device(Q, a), Device(Q, b)
    dev.run(Q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dev.call()
    for name in ("q", "qr", "kv", "ak", "start", "lens", "table"):
        getattr(dev, name).copy_(getattr(other, name))
    for x, y in zip(dev.gains, other.gains):
        x.copy_(y)
    dev.weights.packed.copy_(other.weights.packed)
    dev.o.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert Q.get_device_status() == 0
    compare(b, dev.o.double().cpu().numpy(), dev.lse.double().cpu().numpy())
