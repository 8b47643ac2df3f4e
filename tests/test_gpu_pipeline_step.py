"""The whole step over the 8-bit cache and through a window, in the one line that users are shown."""
import pytest
import torch

from test_gpu_q8_window import Q  # noqa: F401

pytestmark = pytest.mark.gpu


def test_documented_step_runs(Q):  # noqa: F811
    import workloads as W
    from qk_normed_latent_gb300 import pipeline
    workload = W.small(W.WORKLOADS[1], 2, (700, 130))
    state = pipeline.DeviceState(workload.with_(cache_dtype="e4m3"), window=4096, sinks=4)
    state.step()
    assert state.q8 and (state.window, state.sinks) == (4096, 4)
    assert Q.get_device_status() == 0 and bool(torch.isfinite(state.o.float()).all())
