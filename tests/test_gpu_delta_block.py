"""The gated delta rule's operators together, as a block uses them: convolution, norm and rotation of queries and keys,
the rule, the gated norm; prompts in pieces and tokens one by one against whole prompts, and gradients through all of it.

Tolerances (relative 2-norm).  Serving, as for the other blocks' example: pieces and steps recompute the same bf16
pipeline with other roundings of a few intermediate results (each 2^-9 at most in the mean, carried on by sums of random signs):
2e-2; an 8-bit snapshot is off by up to half of 1/127 of each row's largest value: 3e-2.
Gradients: one rounding to bf16 is 2^-8 / sqrt(3) = 2.3e-3 in the mean square.  A gradient of the rule is a sum of up to
four products with five roundings each; the unit queries and keys add two to every product: 2 sqrt(7) 2.3e-3 = 1.22e-2, and
the rounding of a gradient before and after the norm's backward two more: 1.26e-2.  In fp32: 2e-5 for the rule, and as
much again for what the norm makes of it: 4e-5.
Differences: both ends are h along the gradient with h = 1e-2 in the mean square, so the cubic term is 1e-4 of the slope times a
curvature of order ten at most, and fp32 outputs (2e-5 each, of random sign over their thousands) add less: 2e-3."""
import os
import sys

import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
F32, BF16 = torch.float32, torch.bfloat16


def rel(a, b):
    a, b = a.detach(), b.detach()
    return float((a.double() - b.double()).norm() / b.double().norm().clamp(min=1e-300))


@pytest.mark.parametrize("shape", [dict(), dict(nheads=6, headdim=128, ngroups=3, dstate=128), dict(nheads=3, headdim=40, ngroups=1,
                                                                                                  dstate=24)])
@pytest.mark.parametrize("lens", [(150, 37, 64), (5, 300, 2)])
def test_serving(shape, lens):
    import decode
    import delta_block
    r = decode.run(delta_block.DeltaBlock(**shape), lens=lens)
    torch.cuda.synchronize()
    assert r["pieces"] <= 2e-2 and r["steps"] <= 2e-2 and r["fork"] <= 3e-2, r


def plain(p, rate, a_bias, heads, table, cu, positions):
    """mix in float64, token by token."""
    H, P, G, N = heads
    q, k, v, a, b = p.split([G * N, G * N, H * P, H, H], -1)
    q, k, v = q.unflatten(-1, (G, N)), k.unflatten(-1, (G, N)), v.unflatten(-1, (H, P))
    g, beta = -rate * F.softplus(a + a_bias), torch.sigmoid(b)

    def norm(x):
        x = x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()
        if table is None:
            return x
        c, s = (t.double()[positions.long()][:, :, None] for t in table)
        h = c.shape[-1]
        x1, x2, rest = x[..., :h], x[..., h:2 * h], x[..., 2 * h:]
        return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s, rest], -1)

    q, k = (norm(t).repeat_interleave(H // G, 2) for t in (q, k))
    outs = []
    rows = [(0, i, j) for i, j in zip(cu, cu[1:])] if cu else [(r, 0, p.shape[1]) for r in range(p.shape[0])]
    for r, i, j in rows:
        S = p.new_zeros(H, P, N)
        for t in range(i, j):
            S = torch.exp(g[r, t])[:, None, None] * S
            u = beta[r, t][:, None] * (v[r, t] - (S @ k[r, t][..., None])[..., 0])
            S = S + u[..., None] * k[r, t][:, None]
            outs.append(N ** -0.5 * (S @ q[r, t][..., None])[..., 0])
    return torch.stack(outs).view(p.shape[0], p.shape[1], H, P)


def problem(heads, B, L, dtype, rotary, lens=None, seed=3):
    H, P, G, N = heads
    gen = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    p, w = r(B, L, 2 * G * N + H * (P + 2)).to(dtype), r(B, L, H, P).to(dtype)
    rate, a_bias = torch.exp(r(H)), r(H) - 2.0
    angle = 30.0 * torch.rand(L, rotary // 2, generator=gen, device="cuda") if rotary else None
    cu, pos = None, torch.arange(L, device="cuda").expand(B, L)
    if lens:
        cu = [0] + torch.tensor(lens).cumsum(0).tolist()
        pos = torch.cat([torch.arange(n) for n in lens])[None].cuda()
    return p, w, rate, a_bias, (angle.cos(), angle.sin()) if rotary else None, cu, pos.int().contiguous()


SHAPES = [  # (heads, headdim, groups, dstate), batch, tokens, type, rotated features, lengths
    ((4, 64, 2, 64), 2, 130, BF16, 32, None),
    ((2, 128, 1, 128), 1, 141, BF16, 0, [1, 75, 0, 65]),
    ((3, 40, 1, 24), 1, 97, F32, 24, [33, 64]),
    ((2, 72, 2, 48), 2, 70, F32, 0, None),
]


@pytest.mark.parametrize("heads,B,L,dtype,rotary,lens", SHAPES)
def test_gradients_together(heads, B, L, dtype, rotary, lens):
    from delta_block import mix
    p, w, rate, a_bias, table, cu, pos = problem(heads, B, L, dtype, rotary, lens)
    cu_dev = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    leaves = [t.detach().requires_grad_() for t in (p, rate, a_bias)]
    o = mix(*leaves, heads, table, cu_dev, pos)
    got = torch.autograd.grad((o.float() * w.float()).sum(), leaves)
    exact = [t.detach().double().requires_grad_() for t in (p, rate, a_bias)]
    oo = plain(*exact, heads, table, cu, pos)
    want = torch.autograd.grad((oo * w.double()).sum(), exact)
    H, P, G, N = heads
    tol_o, tol = (2e-5, 4e-5) if dtype == F32 else (6.1e-3, 1.26e-2)     # sqrt(7) 2.3e-3 for the outputs
    assert rel(o, oo) <= tol_o
    parts = [G * N, G * N, H * P, H, H]
    for name, a, b in zip("qkvab", got[0].split(parts, -1), want[0].split(parts, -1)):
        assert rel(a, b) <= tol, name
    for a, b in zip(got[1:], want[1:]):
        assert rel(a, b) <= tol


def test_gradient_is_the_slope():
    from delta_block import mix
    heads, B, L, dtype, rotary, lens = SHAPES[2]
    p, w, rate, a_bias, table, cu, pos = problem(heads, B, L, dtype, rotary, lens)
    cu_dev = torch.tensor(cu, dtype=torch.int32, device="cuda")
    f = lambda x: (mix(x, rate, a_bias, heads, table, cu_dev, pos).double() * w.double()).sum()  # noqa: E731
    x = p.detach().requires_grad_()
    d, = torch.autograd.grad(f(x), x)
    h = 1e-2 * d / d.square().mean().sqrt()
    with torch.no_grad():
        slope = float(f(p + h) - f(p - h)) / 2
    assert abs(slope / float((d.double() * h.double()).sum()) - 1) <= 2e-3


def test_captured_step_is_the_eager_one():
    """Forward and backward of the block's middle in one graph, replayed on new inputs: bit for bit the eager results."""
    from delta_block import mix
    heads, B, L, dtype, rotary, lens = SHAPES[0]
    p, w, rate, a_bias, table, cu, pos = problem(heads, B, L, dtype, rotary, lens)
    other = problem(heads, B, L, dtype, rotary, lens, seed=8)[0]

    def step(x):
        x = x.detach().requires_grad_()
        o = mix(x, rate, a_bias, heads, table, None, pos)
        return o.detach(), *torch.autograd.grad(o, x, w)

    eager = [step(x) for x in (p, other)]
    x = p.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(x)
    torch.cuda.current_stream().wait_stream(side)
    for src, want in zip((p, other), eager):
        x.copy_(src)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_training_runs():
    import delta_block
    losses, layer = delta_block.train(steps=2, tokens=100)
    assert all(torch.isfinite(torch.tensor(losses)))
    for name, t in layer.named_parameters():
        assert t.grad is not None and torch.isfinite(t.grad).all() and t.grad.abs().max() > 0, name
