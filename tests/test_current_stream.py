"""The current stream's handle comes from a private call of torch where it has one, else from the public form."""
import types

import qk_normed_latent_gb300 as Q


def fake(raw):
    def current_stream(device=None):
        assert device in (None, 3)
        return types.SimpleNamespace(cuda_stream=77)
    c = types.SimpleNamespace(**({"_cuda_getCurrentRawStream": raw} if raw else {}))
    return types.SimpleNamespace(_C=c, cuda=types.SimpleNamespace(current_device=lambda: 3, current_stream=current_stream))


def test_with_and_without_the_private_call(monkeypatch):
    seen = []
    monkeypatch.setattr(Q, "_torch", lambda: fake(lambda device: seen.append(device) or 55))
    assert Q._stream(None) == 55 and seen == [3]
    monkeypatch.setattr(Q, "_torch", lambda: fake(None))
    assert Q._stream(None) == 77
    assert Q._stream(12) == 12 and Q._stream(types.SimpleNamespace(cuda_stream=9)) == 9
