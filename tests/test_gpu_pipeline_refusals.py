"""The pipeline passes on what the call refuses."""
import pytest

from test_gpu_q8_window import Q  # noqa: F401

pytestmark = pytest.mark.gpu


def test_sinks_without_a_window_are_refused(Q):  # noqa: F811
    """As qkmla_decode_ext refuses them; they were left out for a bf16 cache."""
    import workloads as W
    from qk_normed_latent_gb300.pipeline import DeviceState
    for dtype in ("bf16", "e4m3"):
        st = DeviceState(W.small(W.WORKLOADS[1].with_(cache_dtype=dtype), 2, (700, 130)), sinks=4)
        with pytest.raises(Q.QkmlaError):
            st.step()
