"""DeviceState.prefill: weights as they are at each call, outputs of its own, and what it refuses."""
import pytest
import torch

import workloads as W
from test_gpu_q8_window import Q  # noqa: F401

pytestmark = pytest.mark.gpu


def state(cache="bf16", **kw):
    from qk_normed_latent_gb300.pipeline import DeviceState
    st = DeviceState(W.small(W.WORKLOADS[4].with_(cache_dtype=cache), 3, (300, 77, 900)), **kw)
    st.step()
    return st


def values(w, G_v, d_v, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((G_v, w.d_c, d_v), generator=g, device="cuda") / w.d_c ** 0.5).bfloat16()


def expect(Q, st, got, w_v):
    """Decode's output, up-projected: within decode's rule, 5e-3, beside prefill's 2.7e-3."""
    want = torch.empty_like(got)
    Q.up_project(st.o.view(st.w.rows, st.w.H, st.w.d_c), w_v, want)
    assert Q.get_device_status() == 0
    assert torch.linalg.norm(got - want) <= 7.7e-3 * torch.linalg.norm(want)


def test_weights_changed_in_place(Q):  # noqa: F811
    st = state()
    w_v = values(st.w, st.w.G, 128, 1)
    expect(Q, st, st.prefill(w_v, torch.float32), w_v)
    w_v.copy_(values(st.w, st.w.G, 128, 2))
    expect(Q, st, st.prefill(w_v, torch.float32), w_v)


def test_views_of_one_storage(Q):  # noqa: F811
    st = state()
    w_v = values(st.w, st.w.G, 128, 3)
    half = w_v.view(-1)[:st.w.G // 2 * st.w.d_c * 128].view(st.w.G // 2, st.w.d_c, 128)
    slim = w_v.view(-1)[:st.w.G * st.w.d_c * 64].view(st.w.G, st.w.d_c, 64)
    for v in (w_v, half, slim):
        got = st.prefill(v, torch.float32)
        assert got.shape == (st.w.rows, st.w.H, v.shape[2])
        expect(Q, st, got, v)


def test_results_are_the_callers(Q):  # noqa: F811
    st = state()
    a, b = values(st.w, st.w.G, 128, 4), values(st.w, st.w.G, 128, 5)
    first = st.prefill(a, torch.float32)
    kept = first.clone()
    w_v = Q.prefill_weights(st.wk, a)
    assert torch.equal(st.prefill(w_v, torch.float32), kept)                 # weights laid out once, by the caller
    st.prefill(b, torch.float32)
    a.copy_(b)
    st.prefill(a, torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(first, kept)


def test_on_a_stream(Q):  # noqa: F811
    st = state()
    w_v = values(st.w, st.w.G, 128, 6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [st.prefill(w_v, torch.float32, stream=s) for _ in range(4)]
    s.synchronize()
    for o in outs:
        expect(Q, st, o, w_v)


def test_plain_attention_is_refused(Q):  # noqa: F811
    """Prefill normalises; a state without the normalisation gave that other attention."""
    st = state(plain=True)
    with pytest.raises(Q.QkmlaError) as e:
        st.prefill(values(st.w, st.w.G, 128, 7))
    assert e.value.code == Q.ERR_UNSUPPORTED
