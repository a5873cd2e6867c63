"""The autograd nodes of the gated delta rule and of the norm of queries and keys: what a graph holds and when it lets go, what it
refuses, and from which thread and stream its backward runs.  Results are compared bit for bit with the calls without a graph."""
import threading

import pytest
import torch
import torch.utils.checkpoint

import state_space_model_scan_gb300 as pkg

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def delta_leaves(dtype=BF16, L=70, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    unit = lambda t: torch.nn.functional.normalize(t, dim=-1)  # noqa: E731
    t = [unit(r(1, L, 1, 64)).to(dtype), unit(r(1, L, 1, 64)).to(dtype), r(1, L, 2, 32).to(dtype), -torch.rand(1, L, 2, generator=g, device="cuda"),
         torch.rand(1, L, 2, generator=g, device="cuda"), r(1, 2, 32, 64)]
    return [x.requires_grad_() for x in t]


def qk_leaves(dtype=BF16, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return [x.requires_grad_() for x in (r(2, 9, 3, 40).to(dtype), r(2, 9, 1, 40).to(dtype), r(40), r(40))]


OPS = {"delta": (pkg.GatedDeltaFunction, delta_leaves), "qk": (pkg.QKNormFunction, qk_leaves)}


@pytest.mark.parametrize("op", OPS)
def test_a_graph_serves_once_or_is_retained(op):
    f, make = OPS[op]
    x = make()
    out = f.apply(*x)
    w = [torch.randn_like(o) for o in out]
    a = torch.autograd.grad(out, x, w, retain_graph=True)
    b = torch.autograd.grad(out, x, w)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    with pytest.raises(RuntimeError):
        torch.autograd.grad(out, x, w)
    torch.autograd.backward(f.apply(*x), w)                                 # into the leaves, twice: gradients add up
    torch.autograd.backward(f.apply(*x), w)
    assert all(torch.equal(t.grad, 2 * s) for s, t in zip(a, x))


@pytest.mark.parametrize("op", OPS)
def test_an_input_written_in_between_is_refused(op):
    f, make = OPS[op]
    x = make()
    y = [t * 1 for t in x]
    out = f.apply(*y)
    y[1].data_ptr()
    with torch.no_grad():
        y[1].mul_(2)
    with pytest.raises(RuntimeError, match="inplace|in-place|modified"):
        torch.autograd.grad(out[0].float().sum(), x[0])


@pytest.mark.parametrize("op", OPS)
def test_some_inputs_some_outputs_no_graph(op):
    f, make = OPS[op]
    x = make()
    full = torch.autograd.grad([o.float().sum() for o in f.apply(*x)], x)
    y = [t.detach() for t in x]
    y[1].requires_grad_()
    part, = torch.autograd.grad([o.float().sum() for o in f.apply(*y)], y[1])
    assert torch.equal(part, full[1])
    with torch.no_grad():
        assert not any(o.requires_grad for o in f.apply(*x))
    assert not any(o.requires_grad for o in f.apply(*[t.detach() for t in x]))
    for i in (0, 1):                                                        # one output alone: the other's gradient is zero
        out = f.apply(*x)
        w = [torch.zeros_like(o) for o in out]
        w[i] = torch.randn_like(out[i])
        a, b = torch.autograd.grad(out[i], x, w[i], allow_unused=True), torch.autograd.grad(f.apply(*x), x, w)
        assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("op", OPS)
def test_a_second_differentiation_is_refused(op):
    f, make = OPS[op]
    x = make()
    d, = torch.autograd.grad(f.apply(*x)[0].float().sum(), x[0], create_graph=True)
    assert d.requires_grad
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        torch.autograd.grad(d.float().sum(), x[0])


def test_a_gradient_that_does_not_fit_is_an_error_and_not_an_end():
    """What the backward refuses on the engine's thread reaches the caller as the same exception."""
    x = delta_leaves()
    out = pkg.GatedDeltaFunction.apply(*x)
    saved = x[3].data
    x[3].data = saved.to(torch.float64)                                     # behind autograd's back: g of a type that is refused
    try:
        with pytest.raises((ValueError, RuntimeError)):
            torch.autograd.grad(out[0].float().sum(), x[0])
    finally:
        x[3].data = saved
    assert torch.isfinite(torch.autograd.grad(pkg.GatedDeltaFunction.apply(*x)[0].float().sum(), x[0])[0]).all()


@pytest.mark.parametrize("op", OPS)
def test_strided_and_expanded_gradients(op):
    f, make = OPS[op]
    x = make()
    out = f.apply(*x)
    one = torch.ones((), device="cuda")
    w = [torch.randn(*o.shape[:-1], 2 * o.shape[-1], device="cuda").to(o.dtype)[..., ::2] for o in out]
    a = torch.autograd.grad(out, x, w, retain_graph=True)
    b = torch.autograd.grad(out, x, [t.contiguous() for t in w], retain_graph=True)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    a = torch.autograd.grad(out, x, [one.to(o.dtype).expand_as(o) for o in out], retain_graph=True)
    b = torch.autograd.grad(out, x, [torch.ones_like(o) for o in out])
    assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("op", OPS)
def test_threads_and_streams(op):
    """Four threads, each its own stream: forward and backward of their own inputs, as alone."""
    f, make = OPS[op]
    xs = [make(seed=i) for i in range(4)]
    want = [torch.autograd.grad([o.float().sum() for o in f.apply(*x)], x) for x in xs]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(5):
                    got[i] = torch.autograd.grad([o.float().sum() for o in f.apply(*xs[i])], xs[i])
            st.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not errors
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


@pytest.mark.parametrize("op", OPS)
def test_saved_tensor_hooks_and_checkpoints(op):
    f, make = OPS[op]
    x = make()
    want = torch.autograd.grad(f.apply(*x)[0].float().sum(), x[:2], allow_unused=True)
    with torch.autograd.graph.save_on_cpu():
        out = f.apply(*x)[0]
    got = torch.autograd.grad(out.float().sum(), x[:2], allow_unused=True)
    again = torch.autograd.grad(torch.utils.checkpoint.checkpoint(lambda *t: f.apply(*t)[0], *x, use_reentrant=False).float().sum(), x[:2],
                                allow_unused=True)
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, again) if a is not None)
