"""What the Python wrappers do around the library's calls, without a GPU."""
import contextlib
import types

import torch

from state_space_model_scan_gb300 import api


def test_calls_run_with_their_tensors_gpu_current(monkeypatch):
    """Whichever GPU is current, a call launches on that of its tensors: with no stream given, the library takes the
    current GPU's current stream."""
    state = {"current": 0, "seen": []}

    @contextlib.contextmanager
    def device(d):
        before, state["current"] = state["current"], d.index
        yield
        state["current"] = before
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["current"])
    monkeypatch.setattr(torch.cuda, "device", device)

    def f(x, other=None, stream=None):
        state["seen"].append(state["current"])
        return x
    on = api._on_stream(f)
    x = types.SimpleNamespace(device=torch.device("cuda", 1))
    assert on(x) is x and on(x=x) is x and on(types.SimpleNamespace(device=torch.device("cuda", 0))) is not x
    assert state["seen"] == [1, 1, 0] and state["current"] == 0
    for name in ("ssd_forward", "ssd_backward", "gated_norm_forward", "gated_norm_backward", "conv1d_forward", "conv1d_backward",
                 "complex_ssd_forward"):
        assert getattr(api, name).__wrapped__ is not None
