"""Host side of the 8-bit cache and of windowed decode: refusals before any launch, the argument
block's layout, and the test oracle itself."""
import ctypes
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

import q8_window_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def Q():
    from qk_normed_latent_gb300 import build as B
    B.build()
    import qk_normed_latent_gb300 as Q
    return Q


def test_ext_args_layout_matches_c(Q):
    fields = [f for f, _ in Q.DecodeExtArgs._fields_]
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"qkmla.h\"\nint main(void){\n"
    src += 'printf("%zu\\n", sizeof(qkmla_decode_ext_args));\n'
    src += "".join(f'printf("%zu\\n", offsetof(qkmla_decode_ext_args, {f}));\n' for f in fields) + "return 0;}\n"
    with tempfile.TemporaryDirectory() as d:
        open(os.path.join(d, "t.c"), "w").write(src)
        exe = os.path.join(d, "t")
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), os.path.join(d, "t.c"), "-o", exe], check=True)
        vals = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert vals == [ctypes.sizeof(Q.DecodeExtArgs)] + [getattr(Q.DecodeExtArgs, f).offset for f in fields]


def args(Q, **kw):
    """A valid argument block with addresses that are never read: validation comes first."""
    a = Q.DecodeArgs()
    for f in ("q_tilde", "alpha_q", "q_rope", "kv_cache", "ak_cache", "seq_lens", "page_table", "o"):
        setattr(a, f, 4096)
    a.num_slots, a.page_size, a.max_pages = 640, 64, 10
    a.B, a.s_q, a.H, a.G, a.d_c, a.d_r = 2, 1, 16, 4, 256, 32
    a.cache_dtype, a.o_dtype, a.softmax_scale, a.eps = Q.E4M3, Q.BF16, 0.1, 1e-6
    x = Q.DecodeExtArgs(4096, 0, 0)
    for k, v in kw.items():
        setattr(x if k in ("kv_scale", "window", "sinks") else a, k, v)
    return a, x


@pytest.mark.parametrize("kw,code", [
    (dict(window=-1), "INVALID"), (dict(window=5, sinks=-1), "INVALID"), (dict(sinks=4), "INVALID"),
    (dict(kv_scale=None), "INVALID"), (dict(cache_dtype=1), "INVALID"), (dict(cache_dtype=0), "INVALID"),
    (dict(kv_scale=4098), "INVALID"), (dict(d_c=255), "INVALID"), (dict(H=15), "INVALID"), (dict(B=0), "INVALID"),
    (dict(q_tilde=None), "INVALID"), (dict(q_tilde=4097), "INVALID"), (dict(num_slots=100), "INVALID"),
    (dict(softmax_scale=0.0), "INVALID"), (dict(d_c=514), "UNSUPPORTED"), (dict(H=12), "UNSUPPORTED"),
    (dict(o_dtype=2), "UNSUPPORTED"), (dict(cache_dtype=3, kv_scale=None), "UNSUPPORTED"),
])
def test_decode_ext_refuses(Q, kw, code):
    a, x = args(Q, **kw)
    lib = Q.lib()
    assert lib.qkmla_decode_ext(ctypes.byref(a), ctypes.byref(x), None) == getattr(Q, "ERR_" + code)
    assert lib.qkmla_decode_ext_workspace_size(ctypes.byref(a), ctypes.byref(x)) == 0
    assert lib.qkmla_decode_ext_kernel_name(ctypes.byref(a), ctypes.byref(x)) == b"invalid"
    assert lib.qkmla_decode_ext_launch_count(ctypes.byref(a), ctypes.byref(x)) == 0


def test_null_blocks(Q):
    a, x = args(Q)
    lib = Q.lib()
    assert lib.qkmla_decode_ext(None, ctypes.byref(x), None) == Q.ERR_INVALID
    assert lib.qkmla_decode_ext(ctypes.byref(a), None, None) == Q.ERR_INVALID


def test_e4m3_is_no_type_of_the_other_calls(Q):
    a, _ = args(Q)
    f = ctypes.c_void_p(4096)
    lib = Q.lib()
    assert lib.qkmla_decode(ctypes.byref(a), None) == Q.ERR_UNSUPPORTED
    assert lib.qkmla_append(f, f, f, None, f, 1, 4, 256, 64, 32, 1e-6, 0, f, Q.E4M3, f, 64, None) == Q.ERR_UNSUPPORTED


def test_append_q8_refuses(Q):
    f, lib = ctypes.c_void_p(4096), Q.lib()

    def call(c=f, r=f, pos=None, theta=0.0, wk=f, slots=f, N=4, G=4, d_c=256, d_h=64, d_r=32, eps=1e-6, kv=f, sc=f, ak=f,
             num=64):
        return lib.qkmla_append_q8(c, r, pos, theta, wk, None, slots, N, G, d_c, d_h, d_r, eps, 0, kv, sc, ak, num, None)

    for kw in (dict(c=None), dict(r=None), dict(wk=None), dict(slots=None), dict(kv=None), dict(sc=None), dict(ak=None),
               dict(N=-1), dict(G=0), dict(d_c=0), dict(d_c=255), dict(d_h=257), dict(eps=-1.0), dict(num=0),
               dict(pos=f, theta=1.0), dict(pos=f, theta=1e4, d_r=31), dict(kv=ctypes.c_void_p(4097)),
               dict(sc=ctypes.c_void_p(4098))):
        assert call(**kw) == Q.ERR_INVALID, kw
    assert call(d_c=514) == Q.ERR_UNSUPPORTED
    assert call(d_r=66) == Q.ERR_UNSUPPORTED
    assert call(N=0, c=None) == Q.OK


def test_front_end_refuses(Q):
    kv, sc = torch.zeros((64, 320), dtype=torch.uint8), torch.zeros(64)
    with pytest.raises(ValueError, match="8-bit cache"):
        Q._check_q8_cache(kv, sc, 256, 16)
    with pytest.raises(ValueError, match="kv_scale"):
        Q._check_q8_cache(kv, None, 256, 32)
    with pytest.raises(ValueError, match="kv_scale"):
        Q._check_q8_cache(kv, sc[:63], 256, 32)
    Q._check_q8_cache(kv, sc, 256, 32)


def test_oracle_e4m3_against_torch():
    x = np.concatenate([R.E4M3, (R.E4M3[1:] + R.E4M3[:-1]) / 2, np.linspace(0, 448, 4001)])
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn)          # exact in fp64 -> one rounding
    np.testing.assert_array_equal(R.e4m3_decode(R.e4m3_encode(x)), want.double().numpy())
    codes = np.arange(256, dtype=np.uint8)
    np.testing.assert_array_equal(R.e4m3_decode(codes), torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy())


def test_oracle_scale_is_the_least():
    c = np.array([[448.0], [448.1], [1.0], [0.0], [1e-38], [7 / 8]], np.float32)
    _, s = R.quantise(c)
    assert s.tolist() == [1.0, 2.0, 2.0 ** -8, 0.0, 2.0 ** -126, 2.0 ** -9]


def test_oracle_window():
    assert R.visible(10, 0, 0).tolist() == list(range(10))
    assert R.visible(10, 3, 2).tolist() == [0, 1, 7, 8, 9]
    assert R.visible(4, 3, 2).tolist() == [0, 1, 2, 3]
    assert R.visible(0, 3, 2).tolist() == [] and R.visible(-2, 3, 2).tolist() == []
