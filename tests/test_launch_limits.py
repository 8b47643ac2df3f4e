"""Sizes beyond a launch's limits are refused on the host."""
import ctypes

from test_q8_window import Q, args  # noqa: F401


def test_launch_limits_are_refused(Q):  # noqa: F811
    """More rows than an int counts, and more groups than a grid takes."""
    lib, f = Q.lib(), ctypes.c_void_p(4096)
    a, x = args(Q, B=1 << 20, s_q=1 << 7, H=16)
    assert lib.qkmla_decode_ext(ctypes.byref(a), ctypes.byref(x), None) == Q.ERR_INVALID
    assert lib.qkmla_append_q8(f, f, None, 0.0, f, None, f, 4, 65536, 256, 64, 32, 1e-6, 0, f, f, f, 64, None) == Q.ERR_INVALID


def test_token_counts_beyond_int_are_refused(Q):  # noqa: F811
    """max_pages x page_size wrapped to a negative length, behind which every sequence looked too long."""
    lib = Q.lib()
    for pages in (1 << 25, (1 << 25) - 1):
        a, x = args(Q, max_pages=pages)
        assert lib.qkmla_decode_ext(ctypes.byref(a), ctypes.byref(x), None) == Q.ERR_INVALID
        a, x = args(Q, max_pages=pages, cache_dtype=Q.BF16)
        assert lib.qkmla_decode(ctypes.byref(a), None) == Q.ERR_INVALID


def test_window_beyond_int_means_every_token(Q):  # noqa: F811
    """ctypes cuts a Python int to 32 bits: 2^32 + 5 was a window of 5."""
    for n, want in ((0, 0), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 63, 2 ** 31 - 1),
                    (-1, -1), (-2 ** 32, -1)):
        assert Q.DecodeExtArgs(None, Q._c_int(n), 0).window == want
