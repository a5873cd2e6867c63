"""The autograd nodes of the gated delta rule, on its tensor-core path (more than 256 tokens x heads), and of the norm of queries and keys,
where one graph is gone through by several threads."""
import threading

import pytest
import torch

import state_space_model_scan_gb300 as pkg

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


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
