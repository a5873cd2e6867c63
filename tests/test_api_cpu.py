"""What the Python wrappers do around the library's calls, and when its binding is built, without a GPU."""
import contextlib
import os
import types

import torch

from state_space_model_scan_gb300 import api, build


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


def test_binding_is_built_again_for_another_torch(monkeypatch, tmp_path):
    compiled = []

    def run(cmd, **kw):
        compiled.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build, "BUILT_FOR", str(tmp_path / "_binding.txt"), raising=False)
    monkeypatch.setattr(build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(build.subprocess, "run", run)
    build.build_binding()
    build.build_binding()
    assert len(compiled) == 1 and os.path.exists(build.BINDING)
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    build.build_binding()
    build.build_binding()
    assert len(compiled) == 2
    monkeypatch.setattr(torch, "__file__", str(tmp_path / "torch" / "__init__.py"))
    build.build_binding()
    assert len(compiled) == 3
