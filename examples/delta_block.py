"""A gated delta rule block: prompts, single tokens and snapshots as a server would run them, and a training step.

The block is projections around a causal convolution and the gated delta rule, whose queries and keys are brought
to unit length per head (and, with a table, rotated by their positions) on the way:

    u -> in_proj -> [z | q k v | a | b];  q k v -> convolution -> qk_norm (l2) -> gated delta rule (g from a, beta from b)
      -> gated norm with z -> out_proj

A request keeps two things between calls, each in a pool of slots: the convolution's window and the rule's state.

    python examples/delta_block.py

runs it with random weights as decode.py does its blocks: packed prompts in pieces, a captured decode step replayed and
a fork from an 8-bit snapshot, then a few training steps.
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from state_space_model_scan_gb300.api import (GatedDeltaFunction, QKNormFunction, conv1d_prompt, conv1d_step,  # noqa: E402
                                              gated_delta_forward, gated_delta_step, gated_norm_forward, qk_norm_forward)


class DeltaBlock:
    def __init__(self, width=512, nheads=8, headdim=64, ngroups=2, dstate=64, slots=8, device="cuda", seed=0):
        gen = torch.Generator(device).manual_seed(seed)
        r = lambda *s, scale=1.0: torch.randn(*s, generator=gen, device=device) * scale  # noqa: E731
        self.H, self.P, self.G, self.N = nheads, headdim, ngroups, dstate
        self.di, self.gn = nheads * headdim, ngroups * dstate
        self.dc = self.di + 2 * self.gn
        pad = -(self.di + self.dc + 2 * nheads) % 8        # rows of a multiple of 16 bytes, so that a slice of one is aligned
        self.w_in = r(width, self.di + self.dc + 2 * nheads + pad, scale=width ** -0.5).bfloat16()
        self.w_out = r(self.di, width, scale=self.di ** -0.5).bfloat16()
        self.conv_w, self.conv_b = r(self.dc, 4, scale=0.4), r(self.dc, scale=0.1)
        self.rate, self.a_bias = torch.exp(r(nheads)), r(nheads) - 3.0
        self.norm_w = torch.ones(self.di, device=device)
        self.windows = torch.zeros(slots, 3, self.dc, dtype=torch.bfloat16, device=device)
        self.states = torch.zeros(slots, nheads, headdim, dstate, device=device)

    def _split(self, p):
        z, qkv, a, b, _ = p.split([self.di, self.dc, self.H, self.H, p.shape[-1] - self.di - self.dc - 2 * self.H], -1)
        return z.contiguous(), qkv.contiguous(), -self.rate * F.softplus(a.float() + self.a_bias), torch.sigmoid(b.float())

    def _heads(self, qkv):
        q, k, v = qkv.split([self.gn, self.gn, self.di], -1)
        return q.unflatten(-1, (self.G, self.N)), k.unflatten(-1, (self.G, self.N)), v.unflatten(-1, (self.H, self.P))

    def _out(self, o, z):
        y, _ = gated_norm_forward(o.flatten(-2), self.norm_w, self.P, z=z)
        return y @ self.w_out

    def prompt(self, u, cu, slots, fresh):
        """u [1, tokens, width]: packed prompt pieces, sequence i going on in slot slots[i] (from zeros where fresh)."""
        z, qkv, g, beta = self._split(u @ self.w_in)
        q, k, v = self._heads(conv1d_prompt(qkv, self.conv_w, self.conv_b, self.windows, cu_seqlens=cu, state_indices=slots,
                                            has_initial=~fresh))
        q, k = qk_norm_forward(q, k, mode="l2")
        init = torch.where(fresh[:, None, None, None], 0.0, self.states[slots.long()])
        o, final = gated_delta_forward(q, k, v, g, beta, initial_states=init, cu_seqlens=cu)
        self.states[slots.long()] = final
        return self._out(o, z)

    def step(self, u, slots):
        """u [requests, width]: the next token of each."""
        z, qkv, g, beta = self._split(u @ self.w_in)
        q, k, v = self._heads(conv1d_step(qkv, self.conv_w, self.conv_b, self.windows, state_indices=slots))
        q, k = (t[0] for t in qk_norm_forward(q[None], k[None], mode="l2"))
        return self._out(gated_delta_step(self.states, q, k, v, g, beta, state_indices=slots), z)


def mix(p, rate, a_bias, heads, table=None, cu_seqlens=None, positions=None):
    """The differentiable middle of the block: p [batch, tokens, 2 G N + H (P + 2)] = [q | k | v | a | b], heads = (H, P, G, N);
    table: (cos, sin) of the rotation."""
    H, P, G, N = heads
    q, k, v, a, b = p.split([G * N, G * N, H * P, H, H], -1)
    q, k, v = q.unflatten(-1, (G, N)), k.unflatten(-1, (G, N)), v.unflatten(-1, (H, P))
    cos, sin = table if table is not None else (None, None)
    q, k = QKNormFunction.apply(q, k, None, None, cos, sin, positions, "l2")
    g, beta = -rate * F.softplus(a.float() + a_bias), torch.sigmoid(b.float())
    return GatedDeltaFunction.apply(q, k, v, g, beta, None, cu_seqlens)[0]


class DeltaLayer(torch.nn.Module):
    """in_proj -> mix -> out_proj with a residual, for training."""

    def __init__(self, width=256, nheads=4, headdim=64, ngroups=2, dstate=64, rotary=32, rows=4096):
        super().__init__()
        self.heads = nheads, headdim, ngroups, dstate
        self.w_in = torch.nn.Linear(width, 2 * ngroups * dstate + nheads * (headdim + 2), bias=False)
        self.w_out = torch.nn.Linear(nheads * headdim, width, bias=False)
        self.log_rate, self.a_bias = torch.nn.Parameter(torch.zeros(nheads)), torch.nn.Parameter(torch.full((nheads,), -3.0))
        angle = torch.arange(rows)[:, None] * 10000.0 ** (-torch.arange(rotary // 2) / (rotary // 2))
        self.register_buffer("cos", angle.cos(), persistent=False)
        self.register_buffer("sin", angle.sin(), persistent=False)

    def forward(self, u, cu_seqlens=None, positions=None):
        with torch.autocast("cuda", torch.bfloat16):
            p = self.w_in(u)
            o = mix(p, torch.exp(self.log_rate), self.a_bias, self.heads, (self.cos, self.sin), cu_seqlens, positions)
            return u + self.w_out(o.flatten(-2))


def train(steps=5, batch=2, tokens=512, width=256, seed=0):
    """A few steps of AdamW towards a fixed random target; returns the losses and the layer."""
    torch.manual_seed(seed)
    layer = DeltaLayer(width).cuda()
    opt = torch.optim.AdamW(layer.parameters(), lr=1e-3)
    u, want = torch.randn(2, batch, tokens, width, device="cuda").unbind(0)
    losses = []
    for _ in range(steps):
        loss = F.mse_loss(layer(u), want)
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses, layer


if __name__ == "__main__":
    import decode
    print("DeltaBlock", {k: float("%.3g" % v) for k, v in decode.run(DeltaBlock(), time_steps=200).items()})
    print("training", [float("%.4g" % v) for v in train()[0]])
