"""Calls with nothing in them, no tokens, no heads of keys, and calls that several threads make for the first time."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import state_space_model_scan_gb300 as pkg
from state_space_model_scan_gb300 import _lib

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_call_without_tokens_leaves_a_status(dtype, packed):
    """The workspace's contents need not be initialised, and its status is that of the call."""
    z = lambda *s, t=dtype: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    S = 3 if packed else 2
    a = [z(1 if packed else 2, 0, 1, 64), z(1 if packed else 2, 0, 1, 64), z(1 if packed else 2, 0, 2, 64), z(1 if packed else 2, 0, 2, t=F32), z(1 if packed else 2, 0, 2, t=F32)]
    init = torch.randn(S, 2, 64, 64, device="cuda")
    cu = torch.zeros(S + 1, dtype=torch.int32, device="cuda") if packed else None
    ws = torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda")

    class Same:
        def get(self, n):
            assert n <= ws.numel()
            return ws
    d = pkg.gated_delta_backward(*a, a[2], initial_states=init, dfinal_states=init, cu_seqlens=cu, workspace=Same())
    assert torch.equal(d["dinitial_states"], init)
    assert _lib.query_status(ws) == _lib.SSD_OK
    # the forward through C, whose workspace Python allocates by itself
    ws.fill_(7)
    p = _lib.DeltaProblem(1 if packed else 2, 0, 2, 1, 64, 64, S if packed else 0, 0.125, _lib.SSD_BF16 if dtype == BF16 else _lib.SSD_F32)
    f, out = _lib.DeltaArgs(), torch.empty_like(init)
    for name, t in (("initial_states", init), ("final_states", out)):
        d = _lib.Tensor()
        d.ptr, d.dtype = t.data_ptr(), _lib.SSD_F32
        for i, s in enumerate(t.stride()):
            d.stride[i] = s
        setattr(f, name, d)
    if packed:
        f.cu_seqlens = cu.data_ptr()
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert _lib.load().ssd_delta_fwd(ctypes.byref(p), ctypes.byref(f), ctypes.c_void_p(ws.data_ptr()), ctypes.c_size_t(ws.numel()), st) == 0
    assert torch.equal(out, init) and _lib.query_status(ws) == _lib.SSD_OK


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [64, 40, 7])
def test_weights_of_no_key_heads_have_gradients_of_zero(dtype, dim):
    q, k = torch.randn(2, 9, 3, dim, device="cuda").to(dtype), torch.empty(2, 9, 0, dim, device="cuda", dtype=dtype)
    w = 1 + torch.rand(2, dim, device="cuda")
    dq = torch.randn_like(q)
    want = pkg.qk_norm_backward(q, None, dq, None, w[0])
    for _ in range(4):
        full = torch.full((dim,), float("nan"), device="cuda")             # what is allocated next holds NaN
        del full
        got = pkg.qk_norm_backward(q, k, dq, k, w[0], w[1])
        assert torch.equal(got["dq"], want["dq"]) and torch.equal(got["dq_weight"], want["dq_weight"])
        assert not got["dk_weight"].any() and got["dk"].shape == k.shape
    got = pkg.qk_norm_backward(q, k, dq, k, None, w[1])                    # the keys' weights alone
    assert torch.equal(got["dq"], pkg.qk_norm_backward(q, None, dq, None)["dq"]) and not got["dk_weight"].any()


FIRST = r"""
import sys, threading
import torch
import state_space_model_scan_gb300 as pkg

def one(K, back):
    r = lambda *s: torch.rand(*s, device="cuda") / 16
    x = [r(1, 2, 1, K), r(1, 2, 1, K), r(1, 2, H, 32), -r(1, 2, H), r(1, 2, H)]
    gate.wait()
    return pkg.gated_delta_backward(*x, x[2]) if back else pkg.gated_delta_forward(*x)

torch.zeros(1, device="cuda")
for H in (2, 64, 200):                         # 8, 16 or 32 values a block
    for back in (False, True):
        sizes, errors = [8, 256, 40, 200, 100, 256, 8, 256], []
        gate = threading.Barrier(len(sizes))
        def work(K):
            try:
                one(K, back)
            except Exception as e:
                errors.append(e)
        ts = [threading.Thread(target=work, args=(K,)) for K in sizes]
        [t.start() for t in ts]
        [t.join() for t in ts]
        torch.cuda.synchronize()
        if errors:
            sys.exit("refused: %r" % errors)
"""


def test_threads_that_launch_a_kernel_for_the_first_time():
    """Eight threads, each with another size of the keys, and so of the shared memory that the same kernel is launched with."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
