"""Query tiles without a token among others: chunks longer than their sequences give a CTA many pieces of work in a row
that have nothing to convert or to multiply, and then pieces that have."""
import numpy as np
import pytest
import torch

import prefill_ref as R
from test_gpu_prefill import Device, Q, compare  # noqa: F401 (Q: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,new", [
    ([3, 200], [2500, 60]),                                   # two tokens a tile: 8 pieces a CTA without a token
    ([0, 200, 2, 150, 1, 90], [1300, 60, 1300, 50, 700, 90]),
    ([1], [4000]),
])
def test_many_pieces_without_tiles(Q, lens, new):  # noqa: F811
    c = R.Case(lens=lens, new=new, H=128, G=1, d_c=128, d_h=64, d_r=32, d_v=128)
    dev = Device(Q, c)
    o, lse = dev.run(Q)
    compare(c, o, lse)
    for _ in range(20):
        dev.o.fill_(float("nan"))
        again, _ = dev.run(Q)
        assert (again == o).all()


def test_many_pieces_without_tiles_in_a_graph(Q):  # noqa: F811
    """The same call replayed over steps with and without tokens."""
    c = R.Case(lens=[150, 180], new=[900, 180], H=128, G=1, d_c=128, d_h=64, d_r=32, d_v=128)
    dev = Device(Q, c)
    want, _ = dev.run(Q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dev.call()
    lens = dev.lens.clone()
    for step in range(6):
        dev.lens.copy_(lens if step % 2 else torch.zeros_like(lens))
        dev.o.fill_(float("nan"))
        g.replay()
        assert Q.get_device_status() == 0
        got = dev.o.double().cpu().numpy()
        assert (got == (want if step % 2 else np.zeros_like(want))).all()
