"""Forward-mode differentiation: no operator has it, and each says so, where a result without its tangent would be wrong in silence."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import state_space_model_scan_gb300 as pkg

pytestmark = pytest.mark.gpu


def rand(*s):
    return torch.rand(*s, device="cuda")


def delta():
    return [rand(1, 70, 1, 64) / 8, rand(1, 70, 1, 64) / 8, rand(1, 70, 2, 32), -rand(1, 70, 2), rand(1, 70, 2), rand(1, 2, 32, 64)]


def qk():
    return [rand(2, 9, 3, 40), rand(2, 9, 1, 40), rand(40), rand(40), rand(9, 8), rand(9, 8)]


def scan():
    return [rand(1, 20, 16), rand(1, 20, 16), -rand(16, 8), rand(1, 20, 1, 8), rand(1, 20, 1, 8)]


OPS = {"delta": (pkg.GatedDeltaFunction, delta), "qk": (pkg.QKNormFunction, qk), "selective": (pkg.SelectiveScanFunction, scan)}


@pytest.mark.parametrize("op,i", [("delta", i) for i in range(6)] + [("qk", i) for i in range(6)] + [("selective", 0)])
def test_a_tangent_is_refused(op, i):
    f, make = OPS[op]
    x = make()
    with fwd.dual_level():
        y = list(x)
        y[i] = fwd.make_dual(x[i], torch.ones_like(x[i]))
        with pytest.raises(NotImplementedError):
            f.apply(*y)
        with torch.no_grad(), pytest.raises(NotImplementedError):
            f.apply(*y)
        assert all(torch.isfinite(o).all() for o in f.apply(*x))           # without one it runs there as anywhere
    assert all(torch.isfinite(o).all() for o in f.apply(*x))


@pytest.mark.parametrize("op", OPS)
def test_transforms_are_refused(op):
    f, make = OPS[op]
    x = make()
    with pytest.raises((RuntimeError, NotImplementedError, ValueError)):
        torch.func.jvp(lambda t: f.apply(t, *x[1:])[0], (x[0],), (torch.ones_like(x[0]),))
    with pytest.raises((RuntimeError, NotImplementedError, ValueError)):
        torch.func.vmap(lambda t: f.apply(t, *x[1:])[0])(x[0][None].expand(3, *x[0].shape))


@pytest.mark.parametrize("op", ["delta", "qk"])
def test_a_tangent_of_an_output_gradient_is_refused(op):
    f, make = OPS[op]
    x = [t.requires_grad_() for t in make()]
    out = f.apply(*x)[0]
    w = torch.ones_like(out)
    with fwd.dual_level():
        with pytest.raises(NotImplementedError):
            torch.autograd.grad(out, x[0], fwd.make_dual(w, w), retain_graph=True)
    assert torch.isfinite(torch.autograd.grad(out, x[0], w)[0]).all()
