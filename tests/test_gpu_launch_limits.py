"""Split counts whose items are more than a grid's y takes."""
import pytest

import q8_window_ref as R
from test_gpu_q8_window import Device, Q, check  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache,window", [("q8", 0), ("q8", 9), ("bf16", 9), ("bf16", 0)])
def test_more_items_than_a_grid_takes(Q, cache, window):  # noqa: F811
    """300 sequences x 256 splits: the CUDA-core kernel, whose splits are the grid's y."""
    lens = [1 + k % 40 for k in range(300)]
    c = R.Case(lens, cache=cache, window=window)
    dev = Device(Q, c, num_splits=256)
    assert dev.call.kernel_name == "simt"
    o, _ = dev.run(Q)
    assert abs(o - c.o).max() <= 1e-5 * max(1.0, abs(c.o).max())
    check(Q, c, simt=False, num_splits=218)                                       # 65400 items
