"""qkmla_rope refuses outputs whose rows or heads share elements, before anything is launched: a broadcast tensor in place."""
import ctypes

import pytest

import qk_normed_latent_gb300 as Q

P = 4096                     # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    from qk_normed_latent_gb300 import build as B
    B.build()
    return Q.lib()


@pytest.mark.parametrize("rows,heads,row_stride,head_stride", [
    (4, 1, 0, 64), (1, 4, 64, 0), (4, 4, 0, 64), (4, 4, 256, 0), (4, 1, 63, 64), (4, 2, 256, 32), (4, 1, -32, 64), (2, 2, -2 ** 40, 2),
])
@pytest.mark.parametrize("in_place", [True, False])
def test_shared_outputs(lib, rows, heads, row_stride, head_stride, in_place):
    a = Q.RopeArgs(x=P, out=P if in_place else 1 << 40, positions=P, x_row_stride=row_stride, x_head_stride=head_stride,
                   out_row_stride=row_stride, out_head_stride=head_stride, rows=rows, heads=heads, d_r=64, theta=1e4)
    assert lib.qkmla_rope(ctypes.byref(a), None) == Q.ERR_INVALID


def test_strides_that_are_not_used(lib):
    """One row or one head has no stride; no row at all is no call."""
    a = Q.RopeArgs(x=P, out=P, positions=P, rows=0, heads=1, d_r=64, theta=1e4)
    assert lib.qkmla_rope(ctypes.byref(a), None) == Q.OK
    a = Q.RopeArgs(x=P, out=P, positions=P, rows=1, heads=1, d_r=64, theta=1e4, dtype=2)
    assert lib.qkmla_rope(ctypes.byref(a), None) == Q.ERR_UNSUPPORTED       # refused for its type, not for its strides
