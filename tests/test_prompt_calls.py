"""qkmla_rope, qkmla_read_cache and qkmla_prefill without a GPU: argument blocks as the compiler lays them out, and
refusals before anything is launched."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

import qk_normed_latent_gb300 as Q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 4096                     # an aligned address that nothing reads
F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def lib():
    from qk_normed_latent_gb300 import build as B
    B.build()
    return Q.lib()


@pytest.mark.parametrize("name,mirror", [("qkmla_rope_args", Q.RopeArgs), ("qkmla_read_cache_args", Q.ReadCacheArgs),
                                         ("qkmla_prefill_args", Q.PrefillArgs)])
def test_layout_matches_c(name, mirror):
    fields = [f for f, _ in mirror._fields_]
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"qkmla.h\"\nint main(void){\n"
    src += f'printf("%zu\\n", sizeof({name}));\n' + "".join(f'printf("%zu\\n", offsetof({name}, {f}));\n' for f in fields)
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write(src + "return 0;}\n")
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        vals = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert vals[0] == ctypes.sizeof(mirror)
    assert vals[1:] == [getattr(mirror, f).offset for f in fields]


def block(cls, base, kw):
    a = cls()
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


ROPE = dict(x=P, out=P, positions=P, x_row_stride=64, x_head_stride=64, out_row_stride=64, out_head_stride=64, rows=4, heads=1,
            d_r=64, theta=1e4, factor=1.0, original_context=4096, beta_fast=32.0, beta_slow=1.0)


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), Q.ERR_INVALID), (dict(out=None), Q.ERR_INVALID), (dict(positions=0), Q.ERR_INVALID), (dict(rows=-1), Q.ERR_INVALID),
    (dict(heads=0), Q.ERR_INVALID), (dict(d_r=0), Q.ERR_INVALID), (dict(d_r=63), Q.ERR_INVALID), (dict(layout=2), Q.ERR_INVALID),
    (dict(scaling=4), Q.ERR_INVALID), (dict(scaling=-1), Q.ERR_INVALID), (dict(theta=1.0), Q.ERR_INVALID),
    (dict(theta=float("inf")), Q.ERR_INVALID), (dict(theta=float("nan")), Q.ERR_INVALID), (dict(scaling=1, factor=0.0), Q.ERR_INVALID),
    (dict(scaling=2, original_context=0), Q.ERR_INVALID), (dict(scaling=2, beta_slow=0.0), Q.ERR_INVALID),
    (dict(scaling=2, beta_fast=0.5), Q.ERR_INVALID), (dict(scaling=3), Q.ERR_INVALID), (dict(attention_factor=-1.0), Q.ERR_INVALID),
    (dict(x=P + 2), Q.ERR_INVALID), (dict(dtype=2), Q.ERR_UNSUPPORTED), (dict(d_r=258), Q.ERR_UNSUPPORTED), (dict(rows=0), Q.OK),
    (dict(rows=0, x=0), Q.OK),
])
def test_rope_refuses(lib, kw, code):
    assert lib.qkmla_rope(ctypes.byref(block(Q.RopeArgs, ROPE, kw)), None) == code


def test_rope_refuses_frequencies(lib):
    for f in ([1.0, float("nan")], [float("inf"), 0.0]):
        a = block(Q.RopeArgs, ROPE, dict(d_r=4, scaling=3))
        values = (ctypes.c_double * 2)(*f)
        a.frequencies = ctypes.cast(values, ctypes.POINTER(ctypes.c_double))
        assert lib.qkmla_rope(ctypes.byref(a), None) == Q.ERR_INVALID
    assert lib.qkmla_rope(None, None) == Q.ERR_INVALID


READ = dict(kv_cache=P, ak_cache=P, out_start=P, page_table=P, num_slots=128, page_size=16, max_pages=4, B=2, rows=10, G=4, d_c=128,
            d_r=32, cache_dtype=Q.BF16, out_dtype=Q.F32, c=P, r=P, ak=P)


@pytest.mark.parametrize("kw,code", [
    (dict(kv_cache=0), Q.ERR_INVALID), (dict(out_start=0), Q.ERR_INVALID), (dict(c=0), Q.ERR_INVALID), (dict(r=0), Q.ERR_INVALID),
    (dict(ak_cache=0), Q.ERR_INVALID), (dict(rows=-1), Q.ERR_INVALID), (dict(B=0), Q.ERR_INVALID), (dict(d_c=0), Q.ERR_INVALID),
    (dict(page_size=0), Q.ERR_INVALID), (dict(num_slots=100), Q.ERR_INVALID), (dict(max_pages=2 ** 28), Q.ERR_INVALID),
    (dict(kv_scale=P), Q.ERR_INVALID), (dict(cache_dtype=Q.E4M3), Q.ERR_INVALID), (dict(cache_dtype=Q.E4M3, kv_scale=P, d_c=127), Q.ERR_INVALID),
    (dict(cache_dtype=5), Q.ERR_UNSUPPORTED), (dict(out_dtype=Q.E4M3), Q.ERR_UNSUPPORTED), (dict(kv_cache=P + 1), Q.ERR_INVALID),
    (dict(c=P + 2), Q.ERR_INVALID), (dict(first=P + 2), Q.ERR_INVALID), (dict(rows=0), Q.OK), (dict(rows=0, c=0), Q.OK),
])
def test_read_cache_refuses(lib, kw, code):
    assert lib.qkmla_read_cache(ctypes.byref(block(Q.ReadCacheArgs, READ, kw)), None) == code


PRE = dict(q=P, q_rope=P, q_row_stride=1024, q_head_stride=64, qr_row_stride=512, qr_head_stride=32, gamma_q=P, gamma_k=P, weights=P,
           kv_cache=P, ak_cache=P, chunk_start=P, seq_lens=P, page_table=P, num_slots=128, total_tokens=100, page_size=16, max_pages=4, B=2,
           rows=10, H=16, G=4, G_v=4, d_c=256, d_h=64, d_r=32, d_v=64, cache_dtype=Q.BF16, q_dtype=Q.F32, o_dtype=Q.BF16,
           softmax_scale=0.1, eps=1e-6, workspace=P, workspace_bytes=1 << 40, o=P)


@pytest.mark.parametrize("kw,code", [
    *[({name: 0}, Q.ERR_INVALID) for name in ("q", "q_rope", "gamma_q", "gamma_k", "weights", "kv_cache", "ak_cache", "chunk_start",
                                              "seq_lens", "o", "B", "H", "G", "G_v", "d_c", "d_h", "d_r", "d_v", "page_size",
                                              "max_pages", "num_slots", "softmax_scale")],
    (dict(rows=-1), Q.ERR_INVALID), (dict(H=15), Q.ERR_INVALID), (dict(G_v=3), Q.ERR_INVALID), (dict(num_slots=100), Q.ERR_INVALID),
    (dict(total_tokens=-1), Q.ERR_INVALID), (dict(window=-1), Q.ERR_INVALID), (dict(sinks=-1), Q.ERR_INVALID),
    (dict(sinks=4), Q.ERR_INVALID), (dict(eps=-1.0), Q.ERR_INVALID), (dict(kv_scale=P), Q.ERR_INVALID),
    (dict(cache_dtype=Q.E4M3), Q.ERR_INVALID), (dict(q_row_stride=1022), Q.ERR_INVALID), (dict(qr_head_stride=33), Q.ERR_INVALID),
    (dict(q=P + 8), Q.ERR_INVALID), (dict(o=P + 16), Q.ERR_INVALID), (dict(kv_cache=P + 8), Q.ERR_INVALID),
    (dict(seq_lens=P + 2), Q.ERR_INVALID), (dict(workspace=P + 128), Q.ERR_INVALID), (dict(workspace=0), Q.ERR_WORKSPACE),
    (dict(flags=Q.FLAG_PLAIN_MLA), Q.ERR_UNSUPPORTED), (dict(cache_dtype=Q.F32), Q.ERR_UNSUPPORTED), (dict(q_dtype=Q.E4M3), Q.ERR_UNSUPPORTED),
    (dict(o_dtype=Q.E4M3), Q.ERR_UNSUPPORTED), (dict(d_h=96), Q.ERR_UNSUPPORTED), (dict(d_v=192), Q.ERR_UNSUPPORTED),
    (dict(d_r=16), Q.ERR_UNSUPPORTED), (dict(d_c=96), Q.ERR_UNSUPPORTED), (dict(d_c=576), Q.ERR_UNSUPPORTED),
    (dict(H=24, G=8, G_v=8), Q.ERR_UNSUPPORTED), (dict(H=48, G=16, G_v=6), Q.ERR_UNSUPPORTED), (dict(H=256, G=1, G_v=1), Q.ERR_UNSUPPORTED),
    (dict(B=4097), Q.ERR_UNSUPPORTED), (dict(rows=0), Q.OK), (dict(rows=0, q=0, workspace=0), Q.OK),
])
def test_prefill_refuses(lib, kw, code):
    assert lib.qkmla_prefill(ctypes.byref(block(Q.PrefillArgs, PRE, kw)), None) == code


def test_prefill_weights_refuse(lib):
    size, pack = lib.qkmla_prefill_weights_size, lib.qkmla_prefill_pack_weights
    assert size(4, 4, 256, 64, 64) > 4 * 256 * 128 * 2
    for bad in ((0, 4, 256, 64, 64), (4, 4, 96, 64, 64), (4, 4, 576, 64, 64), (4, 4, 256, 96, 64), (4, 4, 256, 64, 256), (4, 600, 256, 64, 64)):
        assert size(*bad) == 0
    assert pack(P, P, 4, 4, 256, 64, 64, None, None) == Q.ERR_INVALID
    assert pack(None, P, 4, 4, 256, 64, 64, P, None) == Q.ERR_INVALID
    assert pack(P, P, 4, 4, 256, 64, 64, P + 8, None) == Q.ERR_INVALID
    assert pack(P, P, 4, 4, 256, 64, 96, P, None) == Q.ERR_UNSUPPORTED


# ---- the Python front end ----
def zeros(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype)


W = Q.PrefillWeights(zeros(16, dtype=U8), 4, 4, 256, 64, 64)


def prefill(**kw):
    a = dict(q=zeros(9, 16, 64), q_rope=zeros(9, 16, 32), gamma_q=zeros(64), gamma_k=zeros(64), gamma_rope_q=zeros(32), weights=W,
             kv_cache=zeros(64, 288, dtype=BF16), ak_cache=zeros(64, 4), chunk_start=zeros(3, dtype=I32), seq_lens=zeros(2, dtype=I32),
             page_table=zeros(2, 3, dtype=I32), page_size=16, max_pages=3, total_tokens=60, softmax_scale=0.1, eps=1e-6,
             o=zeros(9, 16, 64, dtype=BF16))
    a.update(kw)
    return Q.prepare_prefill(**a)


@pytest.mark.parametrize("name,t", [
    ("q", zeros(9, 16, 32)), ("q", zeros(9, 16, 64, dtype=torch.float16)), ("q_rope", zeros(9, 16, 32, dtype=BF16)),
    ("q_rope", zeros(8, 16, 32)), ("gamma_q", zeros(32)), ("gamma_k", zeros(64, dtype=BF16)), ("gamma_rope_q", zeros(64)),
    ("kv_cache", zeros(64, 256, dtype=BF16)), ("kv_cache", zeros(64, 288)), ("ak_cache", zeros(64, 8)),
    ("chunk_start", zeros(2, dtype=I32)), ("chunk_start", zeros(3, dtype=torch.int64)), ("seq_lens", zeros(2)),
    ("page_table", zeros(2, 4, dtype=I32)), ("o", zeros(9, 16, 128)), ("lse", zeros(9, 15)), ("kv_scale", zeros(64)),
])
def test_prefill_front_end(lib, name, t):
    with pytest.raises(ValueError, match=name):
        prefill(**{name: t})


def test_front_end_of_rope_and_read_cache(lib):
    x, pos = zeros(5, 2, 16), zeros(5, dtype=I32)
    for kw, match in ((dict(out=zeros(5, 2, 8)), "x and out"), (dict(out=zeros(5, 2, 16, dtype=BF16)), "x and out"),
                      (dict(positions=zeros(4, dtype=I32)), "positions"), (dict(positions=zeros(5)), "positions"),
                      (dict(layout="pairs"), "layout"), (dict(scaling=Q.given_frequencies([1.0])), "frequencies"),
                      (dict(x=x.transpose(1, 2), out=x.transpose(1, 2)), "last dimension"), ({}, "CUDA device"),
                      (dict(attention_factor=0.0), "attention_factor|CUDA device")):
        with pytest.raises(ValueError, match=match):
            Q.prepare_rope(**{**dict(x=x, positions=pos, out=x), **kw})
    read = dict(kv_cache=zeros(64, 288, dtype=BF16), ak_cache=zeros(64, 4), out_start=zeros(3, dtype=I32), page_table=zeros(2, 3, dtype=I32),
                page_size=16, max_pages=3, c=zeros(9, 256), r=zeros(9, 32), ak=zeros(9, 4))
    for kw, match in ((dict(kv_cache=zeros(64, 288, dtype=U8)), "8-bit"), (dict(kv_scale=zeros(64)), "kv_scale"), (dict(r=zeros(9, 32, dtype=BF16)), "r is"),
                      (dict(r=zeros(8, 32)), "r is"), (dict(ak=zeros(8, 4)), "ak is"), (dict(first=zeros(3, dtype=I32)), "first"),
                      (dict(page_table=zeros(3, 3, dtype=I32)), "page_table"), (dict(c=zeros(9, 128)), "kv_cache"), ({}, "CUDA device")):
        with pytest.raises(ValueError, match=match):
            Q.prepare_read_cache(**{**read, **kw})
    with pytest.raises(ValueError, match="CUDA device"):
        prefill()
    with pytest.raises(Q.QkmlaError):
        Q.prefill_weights(zeros(4, 256, 96), zeros(4, 256, 64, dtype=BF16))
