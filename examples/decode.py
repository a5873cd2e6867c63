"""Prompts, single tokens and snapshots of two state-space blocks, as a server would run them.

Each block is projections around a causal convolution and a scan: ``HeadBlock`` with one decay rate per head
(ssd_forward / ssd_step and the gated norm), ``ChannelBlock`` with one per channel and state
(selective_scan_forward / selective_scan_step).  Its requests keep two things between calls, each in a
pool of slots: the convolution's window and the scan's state.

    python examples/decode.py

runs both with random weights: prompts of different lengths packed on one axis, a decode step captured in a CUDA
graph and replayed, and a request forked from an 8-bit snapshot; it checks that prompts fed in pieces and
token by token give what whole prompts give, and prints the time of a decode step.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from state_space_model_scan_gb300.api import (conv1d_prompt, conv1d_step, gated_norm_forward, selective_scan_forward,  # noqa: E402
                                              selective_scan_step, snapshot_load, snapshot_store, split_xbc, ssd_forward,
                                              ssd_step)


class HeadBlock:
    """One rate per head: in_proj -> [z | x B C | dt], convolution over x B C, scan, gated norm, out_proj."""

    def __init__(self, width=512, nheads=16, headdim=64, ngroups=1, dstate=128, slots=8, device="cuda", seed=0):
        g = torch.Generator(device).manual_seed(seed)
        r = lambda *s, scale=1.0: torch.randn(*s, generator=g, device=device) * scale  # noqa: E731
        self.H, self.P, self.G, self.N = nheads, headdim, ngroups, dstate
        self.di, self.dc = nheads * headdim, nheads * headdim + 2 * ngroups * dstate
        self.w_in = r(width, self.di + self.dc + nheads, scale=width ** -0.5).bfloat16()
        self.w_out = r(self.di, width, scale=self.di ** -0.5).bfloat16()
        self.conv_w, self.conv_b = r(self.dc, 4, scale=0.4), r(self.dc, scale=0.1)
        self.A, self.D, self.dt_bias = -torch.exp(r(nheads)), r(nheads), r(nheads) - 3.0
        self.norm_w = torch.ones(self.di, device=device)
        self.windows = torch.zeros(slots, 3, self.dc, dtype=torch.bfloat16, device=device)
        self.states = torch.zeros(slots, nheads, headdim, dstate, device=device)

    def prompt(self, u, cu, slots, fresh):
        """u [1, tokens, width]: packed prompt pieces, sequence i going on in slot slots[i] (from zeros where fresh)."""
        p = u @ self.w_in
        z, xbc, dt = p[..., :self.di], p[..., self.di:self.di + self.dc].contiguous(), p[..., self.di + self.dc:].float()
        xbc = conv1d_prompt(xbc, self.conv_w, self.conv_b, self.windows, cu_seqlens=cu, state_indices=slots,
                            has_initial=~fresh)
        x, B, C = split_xbc(xbc, self.H, self.P, self.G, self.N)
        init = torch.where(fresh[:, None, None, None], 0.0, self.states[slots.long()])
        y, final = ssd_forward(x, dt, self.A, B, C, D=self.D, dt_bias=self.dt_bias, initial_states=init, cu_seqlens=cu)
        self.states[slots.long()] = final
        y, _ = gated_norm_forward(y.flatten(-2), self.norm_w, self.di // self.G, z=z.contiguous())
        return y @ self.w_out

    def step(self, u, slots):
        """u [requests, width]: the next token of each."""
        p = u @ self.w_in
        xbc = conv1d_step(p[:, self.di:self.di + self.dc], self.conv_w, self.conv_b, self.windows, state_indices=slots)
        hp, gn = self.di, self.G * self.N
        x, B, C = xbc[:, :hp].unflatten(-1, (self.H, self.P)), xbc[:, hp:hp + gn].unflatten(-1, (self.G, self.N)), \
            xbc[:, hp + gn:].unflatten(-1, (self.G, self.N))
        y = ssd_step(self.states, x, p[:, self.di + self.dc:].float(), self.A, B, C, D=self.D, dt_bias=self.dt_bias,
                     state_indices=slots)
        y, _ = gated_norm_forward(y.flatten(-2), self.norm_w, self.di // self.G, z=p[:, :self.di].contiguous())
        return y @ self.w_out


class ChannelBlock:
    """One rate per channel and state: in_proj -> [x | z], convolution, x_proj -> [dt | B | C], scan, out_proj."""

    def __init__(self, width=512, channels=1024, dstate=16, rank=32, slots=8, device="cuda", seed=0):
        g = torch.Generator(device).manual_seed(seed)
        r = lambda *s, scale=1.0: torch.randn(*s, generator=g, device=device) * scale  # noqa: E731
        self.C, self.N, self.R = channels, dstate, rank
        self.w_in = r(width, 2 * channels, scale=width ** -0.5).bfloat16()
        self.w_x = r(channels, rank + 2 * dstate, scale=channels ** -0.5).bfloat16()
        self.w_dt = r(rank, channels, scale=0.5 * rank ** -0.5).bfloat16()
        self.w_out = r(channels, width, scale=channels ** -0.5).bfloat16()
        self.conv_w, self.conv_b = r(channels, 4, scale=0.4), r(channels, scale=0.1)
        self.A = -torch.arange(1, dstate + 1, device=device).float().repeat(channels, 1)
        self.D, self.dt_bias = r(channels), r(channels) - 3.0
        self.windows = torch.zeros(slots, 3, channels, dtype=torch.bfloat16, device=device)
        self.states = torch.zeros(slots, channels, dstate, device=device)

    def _dt_b_c(self, x):
        q = x @ self.w_x
        B, C = (q[..., self.R + k * self.N:self.R + (k + 1) * self.N].unsqueeze(-2) for k in (0, 1))
        return q[..., :self.R] @ self.w_dt, B, C

    def prompt(self, u, cu, slots, fresh):
        p = u @ self.w_in
        x, z = p[..., :self.C], p[..., self.C:]
        x = conv1d_prompt(x, self.conv_w, self.conv_b, self.windows, cu_seqlens=cu, state_indices=slots, has_initial=~fresh)
        dt, B, C = self._dt_b_c(x)
        init = torch.where(fresh[:, None, None], 0.0, self.states[slots.long()])
        y, final = selective_scan_forward(x, dt, self.A, B, C, D=self.D, z=z, dt_bias=self.dt_bias, initial_states=init,
                                          cu_seqlens=cu)
        self.states[slots.long()] = final
        return y @ self.w_out

    def step(self, u, slots):
        p = u @ self.w_in
        x = conv1d_step(p[:, :self.C], self.conv_w, self.conv_b, self.windows, state_indices=slots)
        dt, B, C = self._dt_b_c(x)
        y = selective_scan_step(self.states, x, dt, self.A, B, C, D=self.D, z=p[:, self.C:], dt_bias=self.dt_bias,
                                state_indices=slots)
        return y @ self.w_out


def snapshots_for(block, count):
    """Room for `count` 8-bit snapshots of a block's states, and their windows beside them."""
    st, w = block.states, block.windows
    return dict(q=torch.empty(count, *st.shape[1:], dtype=torch.int8, device=st.device),
                scale=torch.empty(count, *st.shape[1:-1], device=st.device),
                windows=torch.empty(count, *w.shape[1:], dtype=w.dtype, device=w.device))


def put_aside(block, snaps, slot, at):
    snapshot_store(block.states, snaps["q"], snaps["scale"], state_indices=slot, slots=at)
    snaps["windows"][at.long()] = block.windows[slot.long()]


def take_up(block, snaps, at, slot):
    snapshot_load(snaps["q"], snaps["scale"], block.states, slots=at, state_indices=slot)
    block.windows[slot.long()] = snaps["windows"][at.long()]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def run(block, lens=(150, 37, 64), new_tokens=12, width=512, seed=1, time_steps=0):
    """Prompts, graph-replayed steps and a fork; returns relative differences from whole prompts (and us per step)."""
    n, total = len(lens), [v + new_tokens for v in lens]
    g = torch.Generator("cuda").manual_seed(seed)
    text = [torch.randn(t, width, generator=g, device="cuda").bfloat16() for t in total]   # each request's tokens
    cu = lambda ls: _i32([0] + torch.tensor(ls).cumsum(0).tolist())  # noqa: E731
    slots, fresh, goes_on = _i32([5, 2, 0][:n]), torch.ones(n, dtype=torch.bool, device="cuda"), \
        torch.zeros(n, dtype=torch.bool, device="cuda")
    whole = block.prompt(torch.cat(text)[None], cu(total), slots, fresh)[0].split(total)
    # the same prompts in two pieces, the second going on from the first
    half = [v // 2 for v in lens]
    block.prompt(torch.cat([t[:h] for t, h in zip(text, half)])[None], cu(half), slots, fresh)
    rest = [v - h for v, h in zip(lens, half)]
    out = block.prompt(torch.cat([t[h:v] for t, h, v in zip(text, half, lens)])[None], cu(rest), slots, goes_on)[0].split(rest)
    res = {"pieces": max(rel(o, w[h:v]) for o, w, h, v in zip(out, whole, half, lens))}
    # an 8-bit snapshot of the first request after its prompt
    snaps, one = snapshots_for(block, 4), _i32([3])
    put_aside(block, snaps, slots[:1], one)
    # token by token, one captured step replayed
    u = torch.stack([t[v] for t, v in zip(text, lens)])
    keep = [t.clone() for t in (block.windows, block.states)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(u, slots)                      # libraries set themselves up outside the capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = block.step(u, slots)
    torch.cuda.current_stream().wait_stream(side)
    for t, k in zip((block.windows, block.states), keep):
        t.copy_(k)
    got = []
    for i in range(new_tokens):
        u.copy_(torch.stack([t[v + i] for t, v in zip(text, lens)]))
        graph.replay()
        got.append(y.clone())
    got = torch.stack(got, 1)
    res["steps"] = max(rel(got[k], whole[k][lens[k]:]) for k in range(n))
    # a new request that goes on from the snapshot with the same tokens
    fork = _i32([7])
    take_up(block, snaps, one, fork)
    again = torch.stack([block.step(text[0][lens[0] + i][None], fork)[0] for i in range(new_tokens)])
    res["fork"] = rel(again, got[0])
    if time_steps:
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(time_steps):
            graph.replay()
        b.record()
        torch.cuda.synchronize()
        res["us_per_step"] = a.elapsed_time(b) / time_steps * 1e3
    return res


if __name__ == "__main__":
    for cls in (HeadBlock, ChannelBlock):
        print(cls.__name__, {k: float("%.3g" % v) for k, v in run(cls(), time_steps=200).items()})
