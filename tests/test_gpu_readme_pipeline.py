"""The whole step as the README writes it."""
import os
import re

import pytest
import torch

from test_gpu_q8_window import Q  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_step_runs(Q):  # noqa: F811
    import workloads as W
    from qk_normed_latent_gb300 import pipeline
    text = open(os.path.join(ROOT, "README.md")).read()
    line, = re.findall(r"`(pipeline\.DeviceState\([^`]*)`", text)
    assert 'cache_dtype="e4m3"' in line and "window=4096, sinks=4" in line
    made = []

    class State(pipeline.DeviceState):
        def step(self, *args, **kw):
            made.append(self)
            super().step(*args, **kw)

    shim = type("pipeline", (), {"DeviceState": State})
    eval(line, {"pipeline": shim, "workload": W.small(W.WORKLOADS[1], 2, (700, 130))})
    st, = made
    assert st.q8 and (st.window, st.sinks) == (4096, 4)
    assert Q.get_device_status() == 0 and bool(torch.isfinite(st.o.float()).all())
