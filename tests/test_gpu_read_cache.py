"""qkmla_read_cache on the GPU: the stored rows themselves, every conversion exact or rounded to nearest even, so
equal to the plain gather bit for bit."""
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


def cache(case, f32=False):
    kv = torch.from_numpy(case.kv) if case.cache == "q8" else torch.from_numpy(case.kv.view(np.int16)).view(torch.bfloat16)
    if f32:
        kv = kv.float() * 1.0000001                             # values that bf16 does not hold
    scale = torch.from_numpy(case.kv_scale).cuda() if case.cache == "q8" else None
    ak = torch.from_numpy(case.ak.astype(np.float16) if case.alpha == "f16" else case.ak).cuda()
    return kv.cuda(), scale, ak


def read(Q, case, out, firsts=None, counts=None, f32=False, spare=0):
    kv, scale, ak = cache(case, f32)
    counts = case.lens if counts is None else counts
    n = sum(counts)
    start = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    c = torch.full((n + spare, case.d_c), 5.0, dtype=out, device="cuda")
    r = torch.full((n + spare, case.d_r), 5.0, dtype=out, device="cuda")
    a = torch.full((n + spare, case.G), 5.0, device="cuda")
    first = None if firsts is None else torch.tensor(firsts, dtype=torch.int32, device="cuda")
    table = None if case.table is None else torch.from_numpy(case.table).cuda()
    Q.read_cache(kv, ak, start, table, case.page, case.max_pages, c, r, a, scale, first)
    assert Q.get_device_status() == 0
    want_c, want_r, want_a = [], [], []
    for b, k in enumerate(counts):
        f = 0 if firsts is None else firsts[b]
        s = torch.from_numpy(case.slot[b][f:f + k]).cuda()
        rows = kv[s]
        if case.cache == "q8":
            want_c.append(rows[:, :case.d_c].contiguous().view(torch.float8_e4m3fn).float() * scale[s][:, None])
            want_r.append(rows[:, case.d_c:].contiguous().view(torch.bfloat16).float())
        else:
            want_c.append(rows[:, :case.d_c].float())
            want_r.append(rows[:, case.d_c:].float())
        want_a.append(ak[s].float())
    same = lambda x, y: torch.equal(x.nan_to_num(777), y.nan_to_num(777))  # noqa: E731
    assert same(c[:n], torch.cat(want_c).to(out)) and same(r[:n], torch.cat(want_r).to(out)) and same(a[:n], torch.cat(want_a))
    assert (c[n:] == 5).all() and (r[n:] == 5).all() and (a[n:] == 5).all()


KINDS = [dict(cache="bf16"), dict(cache="q8"), dict(cache="q8", alpha="f16", contiguous=True), dict(cache="bf16", d_c=512, d_h=128, d_r=64, G=8)]


@pytest.mark.parametrize("k", range(len(KINDS)))
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("page", [1, 7, 64])
def test_types(Q, k, out, page):
    case = R.Case(lens=[0, 1, 130, 0, 77, 3, 0], new=[0] * 7, page=page, **KINDS[k])
    read(Q, case, out, spare=9)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_fp32_cache(Q, out):
    read(Q, R.Case(lens=[40, 3], new=[0, 0]), out, f32=True)


@pytest.mark.parametrize("cache_", ["bf16", "q8"])
def test_part_of_a_sequence(Q, cache_):
    case = R.Case(lens=[100, 50, 300], new=[0] * 3, cache=cache_)
    read(Q, case, torch.float32, firsts=[10, 50, 299], counts=[33, 0, 1])


@pytest.mark.parametrize("d_c,d_r", [(10, 6), (12, 4), (24, 8), (100, 20)])
@pytest.mark.parametrize("cache_", ["bf16", "q8"])
def test_odd_widths(Q, d_c, d_r, cache_):
    read(Q, R.Case(lens=[50, 21], new=[0, 0], d_c=d_c, d_r=d_r, cache=cache_), torch.bfloat16)


def test_many_sequences(Q):
    lens = [i % 5 for i in range(1000)]
    read(Q, R.Case(lens=lens, new=[0] * 1000, page=2, d_c=64, d_r=32, G=2), torch.float32)


def test_not_finite(Q):
    def change(case):
        case.c[3, 5] = float("nan")
        case.c[4, 6] = float("inf")
    for kind in ("bf16", "q8"):
        read(Q, R.Case(lens=[20], new=[0], cache=kind, change=change), torch.float32)


def test_bad_page_and_token(Q):
    """A page id or a token out of range: the status says so, its rows stay, the others are read."""
    case = R.Case(lens=[40, 40], new=[0, 0], page=16)
    kv, scale, ak = cache(case)
    table = torch.from_numpy(case.table).cuda()
    table[0, 1] = 10 ** 6
    start = torch.tensor([0, 40, 90], dtype=torch.int32, device="cuda")      # 50 tokens of a 48-token table row
    c, r = torch.full((90, case.d_c), 5.0, device="cuda"), torch.full((90, case.d_r), 5.0, device="cuda")
    Q.read_cache(kv, None, start, table, 16, case.max_pages, c, r)
    assert Q.get_device_status() == Q.ERR_DEVICE_BOUNDS
    want = kv[torch.from_numpy(case.slot[0]).cuda()][:, :case.d_c].float()
    assert torch.equal(c[:16], want[:16]) and torch.equal(c[32:40], want[32:]) and (c[16:32] == 5).all() and (c[88:] == 5).all()


def test_moved_to_another_cache(Q):
    """What append_q8 stored, read back in fp32 and appended to a bf16 cache, decodes alike."""
    case = R.Case(lens=[60], new=[0], cache="q8")
    kv, scale, ak = cache(case)
    start = torch.tensor([0, 60], dtype=torch.int32, device="cuda")
    c, r = torch.empty((60, case.d_c), device="cuda"), torch.empty((60, case.d_r), device="cuda")
    Q.read_cache(kv, ak, start, torch.from_numpy(case.table).cuda(), case.page, case.max_pages, c, r, None, scale)
    kv2, ak2 = torch.zeros((64, case.d_c + case.d_r), device="cuda"), torch.zeros((64, case.G), device="cuda")
    Q.append(c, r, torch.from_numpy(case.wk).cuda(), None, torch.arange(60).cuda(), kv2, ak2, R.EPS)
    assert Q.get_device_status() == 0
    s = torch.from_numpy(case.slot[0]).cuda()
    assert (ak2[:60] - ak[s]).abs().max() <= 1e-5 * ak[s].abs().max()


@pytest.mark.parametrize("off", [1, 2, 4, 8])
def test_alignment_of_the_outputs(Q, off):
    """Outputs `off` elements into their buffers: bases of every alignment that the call takes."""
    case = R.Case(lens=[70], new=[0])
    kv, _, ak = cache(case)
    start = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    table = torch.from_numpy(case.table).cuda()
    for out in (torch.float32, torch.bfloat16):
        got = []
        for o in (0, off):
            c, r = (torch.full((70 * d + 16,), 5.0, dtype=out, device="cuda") for d in (case.d_c, case.d_r))
            Q.read_cache(kv, ak, start, table, case.page, case.max_pages, c[o:o + 70 * case.d_c].view(70, -1), r[o:o + 70 * case.d_r].view(70, -1))
            assert (c[:o] == 5).all() and (c[o + 70 * case.d_c:] == 5).all() and (r[:o] == 5).all() and (r[o + 70 * case.d_r:] == 5).all()
            got.append((c[o:o + 70 * case.d_c], r[o:o + 70 * case.d_r]))
        assert Q.get_device_status() == 0
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
