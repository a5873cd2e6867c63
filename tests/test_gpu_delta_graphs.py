"""The autograd node of the gated delta rule on its tensor-core path (more than 256 tokens x heads; test_gpu_delta_autograd.py's calls are
smaller and run in fp32), and the norm of queries and keys beside it: threads, streams, retained graphs, hooks, checkpoints, strided
gradients, one graph in several threads.  Bit for bit as the calls without a graph, or as one another."""
import threading

import pytest
import torch
import torch.utils.checkpoint

import state_space_model_scan_gb300 as pkg
from state_space_model_scan_gb300 import _lib

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dinitial_states")


def leaves(seed=0, L=200, H=4, V=64, K=128):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    unit = lambda t: torch.nn.functional.normalize(t, dim=-1)  # noqa: E731
    x = [unit(r(1, L, 2, K)).to(BF16), unit(r(1, L, 2, K)).to(BF16), r(1, L, H, V).to(BF16), -torch.rand(1, L, H, generator=g, device="cuda"),
         torch.rand(1, L, H, generator=g, device="cuda"), r(1, H, V, K)]
    return [t.requires_grad_() for t in x]


def qk_leaves(seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return [t.requires_grad_() for t in (r(2, 9, 3, 64).to(BF16), r(2, 9, 1, 64).to(BF16), r(64), r(64))]


OPS = {"delta": (pkg.GatedDeltaFunction, leaves), "qk": (pkg.QKNormFunction, qk_leaves)}


def same(a, b):
    return all(torch.equal(s, t) for s, t in zip(a, b))


def total(out):
    return sum(o.float().sum() for o in out)


def test_these_calls_take_the_tensor_cores():
    """What is kept says which path a call takes: states, values and matrices of a chunk and head (4 of each here) in bf16, 90 KB, or
    states and values in fp32."""
    import ctypes
    for L, H, tc in ((200, 4, True), (65, 4, True), (64, 4, False), (70, 2, False)):
        n = ctypes.c_size_t()
        p = _lib.DeltaProblem(1, L, H, 2, 64, 128, 0, 0.1, _lib.SSD_BF16)
        assert _lib.load().ssd_delta_chunk_states_size(ctypes.byref(p), ctypes.byref(n)) == 0
        chunks = -(-L // 64) * H
        assert (n.value // chunks > 65536) == tc and (tc or n.value == chunks * (64 * 128 + 64 * 64) * 4)


def test_a_graph_gives_what_the_calls_give():
    x = leaves()
    out = pkg.GatedDeltaFunction.apply(*x)
    w = [torch.randn_like(o) for o in out]
    got = torch.autograd.grad(out, x, w, retain_graph=True)
    a = [t.detach() for t in x]
    d = pkg.gated_delta_backward(*a[:5], w[0], initial_states=a[5], dfinal_states=w[1])
    assert same(got, [d[n] for n in NAMES]) and same(got, torch.autograd.grad(out, x, w))
    with pytest.raises(RuntimeError):
        torch.autograd.grad(out, x, w)
    again = torch.autograd.grad(pkg.GatedDeltaFunction.apply(*x, None, None, False), x, w)
    assert same(got, again)


def test_strided_and_expanded_gradients():
    x = leaves()
    out = pkg.GatedDeltaFunction.apply(*x)
    for w in ([torch.randn(*o.shape[:-1], 2 * o.shape[-1], device="cuda").to(o.dtype)[..., ::2] for o in out],
              [torch.randn(*o.shape[:-1], o.shape[-1] + 3, device="cuda").to(o.dtype)[..., 1:-2] for o in out],
              [torch.ones((), dtype=o.dtype, device="cuda").expand_as(o) for o in out]):
        a = torch.autograd.grad(out, x, w, retain_graph=True)
        assert same(a, torch.autograd.grad(out, x, [t.contiguous() for t in w], retain_graph=True))


@pytest.mark.parametrize("op", OPS)
def test_threads_and_streams(op):
    """Eight threads, each with its own stream, inputs and size (tensor maps are encoded by all of them at once)."""
    f, make = OPS[op]
    xs = [make(i, 130 + 30 * i) if op == "delta" else make(i) for i in range(8)]
    want = [torch.autograd.grad(total(f.apply(*x)), x) for x in xs]
    torch.cuda.synchronize()
    got, errors = [None] * len(xs), []

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(8):
                    got[i] = torch.autograd.grad(total(f.apply(*xs[i])), xs[i])
            st.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not errors
    assert all(same(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("retain", [True, False])
@pytest.mark.parametrize("op", OPS)
def test_one_graph_in_several_threads(op, retain):
    """Threads that go through the same graph at once: each has the gradients, or, where the graph is given up by the first, that or
    torch's error."""
    f, make = OPS[op]
    x = make()
    want = torch.autograd.grad(total(f.apply(*x)), x)
    for _ in range(5):
        loss, got, errors, gate = total(f.apply(*x)), [], [], threading.Barrier(4)

        def work():
            gate.wait()
            try:
                got.append(torch.autograd.grad(loss, x, retain_graph=retain))
            except RuntimeError as e:
                errors.append(e)

        ts = [threading.Thread(target=work) for _ in range(4)]
        [t.start() for t in ts]
        [t.join() for t in ts]
        torch.cuda.synchronize()
        assert all(same(g, want) for g in got) and len(got) + len(errors) == 4
        assert len(got) == 4 if retain else all("second time" in str(e) or "freed" in str(e) for e in errors)


def test_saved_tensor_hooks_and_checkpoints():
    x = leaves()
    f = pkg.GatedDeltaFunction.apply
    want = torch.autograd.grad(total(f(*x)), x)
    with torch.autograd.graph.save_on_cpu():
        out = f(*x)
    assert same(want, torch.autograd.grad(total(out), x))
    assert same(want, torch.autograd.grad(total(torch.utils.checkpoint.checkpoint(f, *x, use_reentrant=False)), x))


@pytest.mark.parametrize("op", OPS)
def test_a_captured_step_through_autograd(op):
    """Forward and backward captured into a CUDA graph and replayed on new values; meanwhile an eager graph of other leaves lives."""
    f, make = OPS[op]
    x, y = make(1), make(2)
    other = f.apply(*make(3))
    want = []
    for src in (x, y):
        out = f.apply(*src)
        want.append(([o.detach() for o in out], torch.autograd.grad(total(out), src)))
        del out
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(total(f.apply(*x)), x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f.apply(*x)
        d = torch.autograd.grad(total(out), x)
    for src, (o, g) in ((y, want[1]), (make(1), want[0])):
        with torch.no_grad():
            for s, t in zip(x, src):
                s.copy_(t)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert same([t.detach() for t in out], o) and same(d, g)
    assert all(torch.isfinite(t).all() for t in other)
