"""Measured cases of the operators that carry a state-space block from training into serving.

Four operators, each in a plain form (elementary torch operations in 32 bits) and as a user
calls it in this package:

* the selective scan: a state-space scan whose decay rates A[channel][state] differ from channel
  to channel and from state to state, over prompts (``scan``) and as a training step with every
  gradient (``train``);
* the short causal convolution with the window that a sequence carries from call to call, over
  prompts (``conv_prompt``) and for one token per request (``conv_step``);
* the recurrence's step for one token per request on a pool of states, with one decay rate per
  head (``ssd_step``) and with one per channel and state (``scan_step``);
* 8-bit snapshots of states, written and read back (``snapshot``).

``own`` selects the package's operators; otherwise the plain forms run.
"""
import math

import torch

own = False

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # One user's prompt of two thousand tokens at a mid-sized block's width, gated, from a zero state.
        dict(name="scan_prompt", op="scan", batch=1, seqlen=2048, channels=4096, groups=1, dstate=16, dtype="bf16",
             dt_dtype="bf16", gate=True, carried=False, nseqs=0),
        # Continuous batching: prompts and prompt pieces of mixed lengths packed on one token axis,
        # each going on from the state that its last piece left.
        dict(name="scan_packed", op="scan", batch=1, seqlen=16111, channels=4096, groups=1, dstate=16, dtype="bf16",
             dt_dtype="bf16", gate=True, carried=True, nseqs=9),
        # A training step's scan, forward and backward, at an ordinary micro-batch.
        dict(name="train_2x2048", op="train", batch=2, seqlen=2048, channels=4096, groups=1, dstate=16, dtype="bf16",
             dt_dtype="bf16", gate=True, carried=False, nseqs=0),
        # The same in 32 bits at odd sizes: a channel count and a state size that fill no tile, two groups.
        dict(name="train_f32_odd", op="train", batch=3, seqlen=517, channels=998, groups=2, dstate=11, dtype="f32",
             dt_dtype="f32", gate=False, carried=True, nseqs=0),
        # Packed prompt pieces through the convolution at the benchmark block's x|B|C width.
        dict(name="conv_prompt_packed", op="conv_prompt", seqlen=8191, nseqs=6, channels=6144, width=4, dtype="bf16"),
        # One token for each of 64 running requests through the same convolution.
        dict(name="conv_step_64", op="conv_step", batch=64, channels=6144, width=4, dtype="bf16"),
        # A single user's next token at the benchmark block's heads: what one request waits for.
        dict(name="ssd_step_1", op="ssd_step", batch=1, nheads=64, headdim=64, groups=8, dstate=128, dtype="bf16",
             state_dtype="f32", gate=True),
        # A loaded server's step with the states stored in 16 bits.
        dict(name="ssd_step_256", op="ssd_step", batch=256, nheads=80, headdim=64, groups=1, dstate=128, dtype="bf16",
             state_dtype="bf16", gate=False),
        # A few requests in 32 bits at odd sizes.
        dict(name="scan_step_3", op="scan_step", batch=3, channels=1001, groups=1, dstate=13, dtype="f32",
             dt_dtype="f32", state_dtype="f32", gate=True),
        # A loaded server's step of the per-channel recurrence.
        dict(name="scan_step_192", op="scan_step", batch=192, channels=8192, groups=1, dstate=16, dtype="bf16",
             dt_dtype="bf16", state_dtype="f32", gate=True),
        # Two requests' states put aside and taken up again (a shared prefix, a preempted request).
        dict(name="snapshot_2", op="snapshot", count=2, nheads=24, headdim=33, dstate=20, state_dtype="bf16"),
        # A server swaps out 96 requests' states and swaps them in again.
        dict(name="snapshot_96", op="snapshot", count=96, nheads=64, headdim=64, dstate=128, state_dtype="f32"),
    ]


def _len(rng, lo, hi):
    """A length spread over the logarithm of [lo, hi]: odd, or an odd multiple of 64 where that fits."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.3 and n >= 64:
        return max(64, n // 128 * 128 - 64)
    return min(hi, max(lo, n | 1))


def draw(rng):
    op = rng.choice(["scan", "train", "conv_prompt", "conv_step", "ssd_step", "scan_step", "snapshot"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    gate = rng.random() < 0.6
    if op in ("scan", "train"):
        groups = rng.choice([1, 1, 1, 2])
        channels = groups * _len(rng, 33, 4095)
        most = (1 << 25) if op == "scan" else (1 << 24)          # tokens x channels
        tokens = _len(rng, 1, min(16001, most // channels))
        batch = 1
        if rng.random() < 0.5:
            batch = rng.choice([2, 3, 4])
            tokens = max(1, tokens // batch)
        nseqs = rng.choice([0, 2, 5, 11]) if batch == 1 and tokens >= 64 else 0
        return dict(op=op, batch=batch, seqlen=tokens, channels=channels, groups=groups,
                    dstate=rng.choice([16, 16, 16, 8, 13, 32]) if op == "scan" else rng.choice([16, 16, 8, 13]),
                    dtype=dtype, dt_dtype=rng.choice([dtype, "f32"]), gate=gate,
                    carried=rng.random() < 0.5, nseqs=nseqs)
    if op == "conv_prompt":
        channels = 8 * _len(rng, 5, 1001)
        tokens = _len(rng, 1, min(8191, (1 << 25) // channels))
        return dict(op=op, seqlen=tokens, nseqs=rng.choice([1, 2, 6, 40]) if tokens >= 40 else 1, channels=channels,
                    width=rng.choice([4, 4, 3, 2]), dtype=dtype)
    if op == "conv_step":
        return dict(op=op, batch=_len(rng, 1, 255), channels=8 * _len(rng, 5, 1001), width=rng.choice([4, 4, 3, 2]),
                    dtype=dtype)
    if op == "ssd_step":
        groups = rng.choice([1, 2, 8])
        nheads = groups * rng.choice([1, 3, 5, 8])
        return dict(op=op, batch=_len(rng, 1, 255), nheads=nheads, headdim=rng.choice([64, 64, 32, 24]), groups=groups,
                    dstate=rng.choice([128, 128, 64, 40]), dtype=dtype, state_dtype=rng.choice(["f32", "bf16"]),
                    gate=gate)
    if op == "scan_step":
        groups = rng.choice([1, 1, 2])
        return dict(op=op, batch=_len(rng, 1, 191), channels=groups * _len(rng, 33, 4095), groups=groups,
                    dstate=rng.choice([16, 16, 8, 13, 32]), dtype=dtype, dt_dtype=rng.choice([dtype, "f32"]),
                    state_dtype=rng.choice(["f32", "bf16"]), gate=gate)
    return dict(op=op, count=_len(rng, 1, 95), nheads=rng.choice([5, 24, 64]), headdim=rng.choice([64, 33]),
                dstate=rng.choice([128, 64, 20, 16]), state_dtype=rng.choice(["f32", "bf16"]))


# ---------------------------------------------------------------------------- inputs
def _cuts(case, seed):
    """cu_seqlens of the packed sequences: seqlen tokens cut at random places (some pieces may be tiny)."""
    r = torch.Generator().manual_seed(seed + 17)
    inner = torch.randint(0, case["seqlen"] + 1, (case["nseqs"] - 1,), generator=r).sort().values
    return torch.cat([torch.zeros(1, dtype=torch.int64), inner, torch.tensor([case["seqlen"]])]).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def steps(*shape):
        """dt_bias whose softplus is log-uniform on [1e-3, 1e-1]."""
        return torch.log(torch.expm1(torch.exp(math.log(1e-3) + uniform(*shape) * math.log(100.0))))

    s = {"case": case}
    if op in ("scan", "train"):
        Bt, L, Dm, G, N = (case[k] for k in ("batch", "seqlen", "channels", "groups", "dstate"))
        td, tt = _DTYPE[case["dtype"]], _DTYPE[case["dt_dtype"]]
        ns = case["nseqs"] or Bt
        s.update(x=normal(Bt, L, Dm, dtype=td), dt=normal(Bt, L, Dm, dtype=tt, scale=0.5),
                 A=-torch.arange(1, N + 1, device="cuda") * torch.exp(0.2 * normal(Dm, N)),
                 B=normal(Bt, L, G, N, dtype=td), C=normal(Bt, L, G, N, dtype=td), D=normal(Dm),
                 z=normal(Bt, L, Dm, dtype=td) if case["gate"] else None, dt_bias=steps(Dm),
                 init=normal(ns, Dm, N, scale=0.1) if case["carried"] else None,
                 cu=_cuts(case, seed).cuda() if case["nseqs"] else None)
        if op == "train":
            s.update(dy=normal(Bt, L, Dm, dtype=td), dfinal=normal(ns, Dm, N, scale=0.1))
        # where each token's sequence starts and ends, for the plain form
        first = torch.zeros(Bt, L, dtype=torch.bool)
        last = torch.zeros(Bt, L, dtype=torch.bool)
        if case["nseqs"]:
            cu = _cuts(case, seed).long()
            full = cu[1:] > cu[:-1]
            first[0, cu[:-1][full]] = True
            last[0, cu[1:][full] - 1] = True
            seq = torch.searchsorted(cu, torch.arange(L), right=True) - 1
            s["seq"] = seq.unsqueeze(0).cuda()
            s["empty"] = (~full).cuda()
        else:
            first[:, 0] = True
            last[:, -1] = True
            s["seq"] = torch.arange(Bt).unsqueeze(1).expand(Bt, L).contiguous().cuda()
            s["empty"] = torch.zeros(Bt, dtype=torch.bool, device="cuda")
        s["first"], s["last"] = first.cuda(), last.cuda()
        s["first_at"] = s["first"].nonzero(as_tuple=True)
        s["last_at"] = s["last"].nonzero(as_tuple=True)
    elif op in ("conv_prompt", "conv_step"):
        Cn, K, td = case["channels"], case["width"], _DTYPE[case["dtype"]]
        n = case["nseqs"] if op == "conv_prompt" else case["batch"]
        slots = n + 3                                             # the pool has free slots too
        rows = (1, case["seqlen"]) if op == "conv_prompt" else (n,)
        s.update(u=normal(*rows, Cn, dtype=td), w=normal(Cn, K, scale=0.5), bias=normal(Cn, scale=0.1),
                 window=normal(slots, K - 1, Cn, dtype=td),
                 slot=torch.randperm(slots, generator=torch.Generator().manual_seed(seed))[:n].to(torch.int32).cuda())
        if op == "conv_prompt":
            cu = _cuts(case, seed)
            s["cu"] = cu.cuda()
            s["seq"] = (torch.searchsorted(cu.long(), torch.arange(case["seqlen"]), right=True) - 1).cuda()
            s["has"] = (uniform(n) < 0.7).to(torch.uint8)         # some sequences start here
    elif op == "snapshot":
        n, H, P, N, td = case["count"], case["nheads"], case["headdim"], case["dstate"], _DTYPE[case["state_dtype"]]
        slots = n + 2
        perm = [torch.randperm(slots, generator=torch.Generator().manual_seed(seed + k))[:n].to(torch.int32).cuda()
                for k in range(3)]
        # heads of very different sizes, as decay rates of 1 to 16 leave them
        size = torch.exp(2.0 * normal(slots, H, 1, 1))
        s.update(states=(normal(slots, H, P, N) * size).to(td), back=torch.zeros(slots, H, P, N, dtype=td, device="cuda"),
                 q=torch.zeros(slots, H, P, N, dtype=torch.int8, device="cuda"),
                 scale=torch.zeros(slots, H, P, device="cuda"), src=perm[0], slot=perm[1], dst=perm[2])
    else:
        n, G, N, td, sd = case["batch"], case["groups"], case["dstate"], _DTYPE[case["dtype"]], _DTYPE[case["state_dtype"]]
        slots = n + 3
        s["slot"] = torch.randperm(slots, generator=torch.Generator().manual_seed(seed))[:n].to(torch.int32).cuda()
        s.update(B=normal(n, G, N, dtype=td), C=normal(n, G, N, dtype=td))
        if op == "ssd_step":
            H, P = case["nheads"], case["headdim"]
            s.update(x=normal(n, H, P, dtype=td), dt=normal(n, H, scale=0.5), A=-torch.exp(uniform(H) * math.log(16.0)),
                     D=normal(H), z=normal(n, H, P, dtype=td) if case["gate"] else None, dt_bias=steps(H),
                     state=normal(slots, H, P, N, dtype=sd))
        else:
            Dm = case["channels"]
            s.update(x=normal(n, Dm, dtype=td), dt=normal(n, Dm, dtype=_DTYPE[case["dt_dtype"]], scale=0.5),
                     A=-torch.arange(1, N + 1, device="cuda") * torch.exp(0.2 * normal(Dm, N)), D=normal(Dm),
                     z=normal(n, Dm, dtype=td) if case["gate"] else None, dt_bias=steps(Dm),
                     state=normal(slots, Dm, N, dtype=sd))
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    return (_OWN if own else _PLAIN)[op](s)


def _own_scan(s):
    from state_space_model_scan_gb300.api import selective_scan_forward
    y, final = selective_scan_forward(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                                      initial_states=s["init"], cu_seqlens=s["cu"])
    return {"y": y, "final": final}


def _own_train(s):
    from state_space_model_scan_gb300.api import selective_scan_backward, selective_scan_forward
    kw = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], initial_states=s["init"], cu_seqlens=s["cu"])
    y, final, kept = selective_scan_forward(s["x"], s["dt"], s["A"], s["B"], s["C"], keep_chunk_states=True, **kw)
    out = selective_scan_backward(s["x"], s["dt"], s["A"], s["B"], s["C"], s["dy"], dfinal_states=s["dfinal"],
                                  chunk_states=kept, **kw)
    out["y"], out["final"] = y, final
    return out


def _own_conv_prompt(s):
    from state_space_model_scan_gb300.api import conv1d_prompt
    out = conv1d_prompt(s["u"], s["w"], s["bias"], s["window"], cu_seqlens=s["cu"], state_indices=s["slot"],
                        has_initial=s["has"])
    return {"out": out, "window": s["window"]}


def _own_conv_step(s):
    from state_space_model_scan_gb300.api import conv1d_step
    return {"out": conv1d_step(s["u"], s["w"], s["bias"], s["window"], state_indices=s["slot"]), "window": s["window"]}


def _own_ssd_step(s):
    from state_space_model_scan_gb300.api import ssd_step
    y = ssd_step(s["state"], s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                 state_indices=s["slot"])
    return {"y": y, "state": s["state"]}


def _own_scan_step(s):
    from state_space_model_scan_gb300.api import selective_scan_step
    y = selective_scan_step(s["state"], s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
                            dt_bias=s["dt_bias"], state_indices=s["slot"])
    return {"y": y, "state": s["state"]}


def _own_snapshot(s):
    from state_space_model_scan_gb300.api import snapshot_load, snapshot_store
    snapshot_store(s["states"], s["q"], s["scale"], state_indices=s["src"], slots=s["slot"])
    snapshot_load(s["q"], s["scale"], s["back"], slots=s["slot"], state_indices=s["dst"])
    return {"back": s["back"], "scale": s["scale"]}


# ---------------------------------------------------------------------------- plain forms
def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _linear_scan(a, b):
    """h[t] = a[t] h[t-1] + b[t] along dimension 1, by doubling: after the pass with distance d every place holds
    the composition of its last 2 d steps, so log2(length) passes of whole-tensor operations do it (the loop
    runs over the distances, not over the tokens)."""
    d = 1
    while d < a.shape[1]:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _scan_states(s):
    """(a, h, dt, x, B, C): decays and states [batch, seqlen, channels, dstate] and the inputs in 32 bits."""
    Dm, G = s["A"].shape[0], s["B"].shape[2]
    x, dt = s["x"].float(), _softplus(s["dt"].float() + s["dt_bias"])
    B = s["B"].float().repeat_interleave(Dm // G, 2)
    C = s["C"].float().repeat_interleave(Dm // G, 2)
    a = torch.exp(dt.unsqueeze(-1) * s["A"])
    b = (dt * x).unsqueeze(-1) * B
    if s["init"] is not None:
        at = s["first_at"]
        b[at] += a[at] * s["init"][s["seq"][at]]
    h = _linear_scan(a * ~s["first"][..., None, None], b)
    return a, h, dt, x, B, C


def _finals(s, h):
    ns = s["cu"].numel() - 1 if s["cu"] is not None else h.shape[0]
    final = torch.zeros(ns, *h.shape[2:], device=h.device)
    if s["init"] is not None:
        final = torch.where(s["empty"][:, None, None], s["init"], final)
    at = s["last_at"]
    final[s["seq"][at]] = h[at]
    return final


def _plain_scan(s):
    _, h, _, x, _, C = _scan_states(s)
    y = (h * C).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return {"y": y.to(s["x"].dtype), "final": _finals(s, h)}


def _plain_train(s):
    a, h, dt, x, B, C = _scan_states(s)
    Bt, L, Dm, N = h.shape
    G = s["B"].shape[2]
    td = s["x"].dtype
    y = (h * C).sum(-1) + s["D"] * x
    dy = s["dy"].float()
    out = {}
    if s["z"] is not None:
        z = s["z"].float()
        sg = 1.0 / (1.0 + torch.exp(-z))
        out["dz"] = (dy * y * sg * (1.0 + z * (1.0 - sg))).to(td)
        dy, y = dy * z * sg, y * z * sg
    out["y"], out["final"] = y.to(td), _finals(s, h)
    # the gradient of the state after every token, from the end
    c = dy.unsqueeze(-1) * C
    at = s["last_at"]
    c[at] += s["dfinal"][s["seq"][at]]
    nxt = torch.cat([a[:, 1:] * ~s["first"][:, 1:, None, None], torch.zeros_like(a[:, :1])], 1)
    g = _linear_scan(nxt.flip(1), c.flip(1)).flip(1)
    prev = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1) * ~s["first"][..., None, None]
    if s["init"] is not None:
        at = s["first_at"]
        prev[at] = s["init"][s["seq"][at]]
        dinit = s["dfinal"] * s["empty"][:, None, None]
        dinit[s["seq"][at]] = (a[at] * g[at])
        out["dinitial_states"] = dinit
    q = g * a * prev
    dtx = (g * B).sum(-1)
    ddt = dtx * x + (q * s["A"]).sum(-1)
    raw = s["dt"].float() + s["dt_bias"]
    draw_ = ddt * torch.where(raw > 20.0, torch.ones_like(raw), 1.0 / (1.0 + torch.exp(-raw)))
    out["dx"] = (dtx * dt + s["D"] * dy).to(td)
    out["ddt"] = draw_.to(s["dt"].dtype)
    out["dA"] = (q * dt.unsqueeze(-1)).sum((0, 1))
    out["dB"] = (g * (dt * x).unsqueeze(-1)).view(Bt, L, G, Dm // G, N).sum(3).to(td)
    out["dC"] = (h * dy.unsqueeze(-1)).view(Bt, L, G, Dm // G, N).sum(3).to(td)
    out["dD"] = (dy * x).sum((0, 1))
    out["ddt_bias"] = draw_.sum((0, 1))
    return out


def _plain_conv_prompt(s):
    u, cu, K = s["u"][0].float(), s["cu"].long(), s["w"].shape[1]
    slot = s["slot"].long()
    hist = s["window"][slot].float() * s["has"][:, None, None]
    L, seq = u.shape[0], s["seq"]
    t = torch.arange(L, device=u.device)
    back = t.unsqueeze(1) - (K - 1) + torch.arange(K, device=u.device)            # [L, K]
    old = back - cu[seq].unsqueeze(1)                                             # below 0: in the carried window
    taps = torch.where((old >= 0).unsqueeze(-1), u[back.clamp(min=0)],
                       hist[seq.unsqueeze(1), (old + K - 1).clamp(0, K - 2)])
    pre = s["bias"] + (taps * s["w"].t()).sum(1)
    # the new windows: the last K - 1 rows of (old window, sequence)
    end = (cu[1:] - cu[:-1]).unsqueeze(1) - (K - 1) + torch.arange(K - 1, device=u.device)
    new = torch.where((end >= 0).unsqueeze(-1), u[(cu[:-1].unsqueeze(1) + end).clamp(0, L - 1)],
                      hist.gather(1, (end + K - 1).clamp(0, K - 2).unsqueeze(-1).expand(-1, -1, u.shape[1])))
    s["window"][slot] = new.to(s["window"].dtype)
    return {"out": _silu(pre).to(s["u"].dtype).unsqueeze(0), "window": s["window"]}


def _plain_conv_step(s):
    slot = s["slot"].long()
    taps = torch.cat([s["window"][slot].float(), s["u"].float().unsqueeze(1)], 1)
    pre = s["bias"] + (taps * s["w"].t()).sum(1)
    s["window"][slot] = taps[:, 1:].to(s["window"].dtype)
    return {"out": _silu(pre).to(s["u"].dtype), "window": s["window"]}


def _plain_ssd_step(s):
    slot, H, G = s["slot"].long(), s["A"].shape[0], s["B"].shape[1]
    x, dt = s["x"].float(), _softplus(s["dt"] + s["dt_bias"])
    B, C = (s[k].float().repeat_interleave(H // G, 1) for k in ("B", "C"))
    h = s["state"][slot].float() * torch.exp(dt * s["A"])[..., None, None]
    h = h + (dt.unsqueeze(-1) * x).unsqueeze(-1) * B.unsqueeze(2)
    y = (h * C.unsqueeze(2)).sum(-1) + s["D"][:, None] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["state"][slot] = h.to(s["state"].dtype)
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


def _plain_scan_step(s):
    slot, Dm, G = s["slot"].long(), s["A"].shape[0], s["B"].shape[1]
    x, dt = s["x"].float(), _softplus(s["dt"].float() + s["dt_bias"])
    B, C = (s[k].float().repeat_interleave(Dm // G, 1) for k in ("B", "C"))
    h = s["state"][slot].float() * torch.exp(dt.unsqueeze(-1) * s["A"]) + (dt * x).unsqueeze(-1) * B
    y = (h * C).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["state"][slot] = h.to(s["state"].dtype)
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


def _plain_snapshot(s):
    h = s["states"][s["src"].long()].float()
    most = h.abs().amax(-1)
    used = most >= 1e-30
    inv = torch.where(used, 127.0 / most, torch.zeros_like(most))
    s["q"][s["slot"].long()] = torch.round(h * inv.unsqueeze(-1)).to(torch.int8)
    s["scale"][s["slot"].long()] = torch.where(used, most / 127.0, torch.zeros_like(most))
    back = s["q"][s["slot"].long()].float() * s["scale"][s["slot"].long()].unsqueeze(-1)
    s["back"][s["dst"].long()] = back.to(s["back"].dtype)
    return {"back": s["back"], "scale": s["scale"]}


_PLAIN = {"scan": _plain_scan, "train": _plain_train, "conv_prompt": _plain_conv_prompt, "conv_step": _plain_conv_step,
          "ssd_step": _plain_ssd_step, "scan_step": _plain_scan_step, "snapshot": _plain_snapshot}
_OWN = {"scan": _own_scan, "train": _own_train, "conv_prompt": _own_conv_prompt, "conv_step": _own_conv_step,
        "ssd_step": _own_ssd_step, "scan_step": _own_scan_step, "snapshot": _own_snapshot}


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    es = 2 if case.get("dtype") == "bf16" else 4
    if op in ("scan", "train"):
        Bt, L, Dm, G, N = (case[k] for k in ("batch", "seqlen", "channels", "groups", "dstate"))
        et = 2 if case["dt_dtype"] == "bf16" else 4
        tok, ns, e = Bt * L, case["nseqs"] or Bt, Bt * L * Dm * N
        acts = tok * Dm * (es * (3 if case["gate"] else 2) + et) + 2 * tok * G * N * es
        states = ns * Dm * N * 4 * (2 if case["carried"] else 1)
        par = Dm * N * 4 + 2 * Dm * 4
        if op == "scan":     # exp, its argument, the input's product, two multiply-adds
            return {"bytes": acts + states + par, "flops": 7 * e}
        grads = tok * Dm * (es * (3 if case["gate"] else 2) + et) + 2 * tok * G * N * es
        return {"bytes": acts + grads + 2 * states + 2 * par, "flops": 7 * e + 18 * e}
    if op == "conv_prompt":
        n = case["seqlen"] * case["channels"]
        win = 2 * case["nseqs"] * (case["width"] - 1) * case["channels"] * es
        return {"bytes": 2 * n * es + win + case["channels"] * (case["width"] + 1) * 4, "flops": n * (2 * case["width"] + 4)}
    if op == "conv_step":
        n = case["batch"] * case["channels"]
        return {"bytes": 2 * n * es * case["width"] + case["channels"] * (case["width"] + 1) * 4,
                "flops": n * (2 * case["width"] + 4)}
    if op == "snapshot":
        rows = case["count"] * case["nheads"] * case["headdim"]
        n, sb = rows * case["dstate"], 2 if case["state_dtype"] == "bf16" else 4
        return {"bytes": 2 * (n * (sb + 1) + rows * 4), "flops": 4 * n}
    sb = 2 if case["state_dtype"] == "bf16" else 4
    rows = case["nheads"] * case["headdim"] if op == "ssd_step" else case["channels"]
    n, N = case["batch"], case["dstate"]
    acts = n * rows * es * (3 if case["gate"] else 2) + 2 * n * case["groups"] * N * es
    if op == "ssd_step":
        par, dts = 3 * case["nheads"] * 4, n * case["nheads"] * 4
    else:
        par, dts = rows * (N + 2) * 4, n * rows * (2 if case["dt_dtype"] == "bf16" else 4)
    return {"bytes": 2 * n * rows * N * sb + acts + dts + par, "flops": 6 * n * rows * N}


# ---------------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]]({k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
                               for k, v in s.items()})


def _exact_scan(s):
    """The recurrence one token at a time; for a training step, its derivative one token at a time from the end."""
    case, x, A, Dv, z = s["case"], s["x"], s["A"], s["D"], s["z"]
    Bt, L, Dm = x.shape
    G, N = s["B"].shape[2:]
    train = case["op"] == "train"
    raw = s["dt"] + s["dt_bias"]
    dt = torch.nn.functional.softplus(raw, threshold=1e9)
    grp = torch.arange(Dm, device=x.device) // (Dm // G)
    cu = s["cu"].tolist() if s["cu"] is not None else None
    spans = [(0, k, cu[k], cu[k + 1]) for k in range(len(cu) - 1)] if cu else [(None, None, 0, L)]
    zero = torch.zeros(len(spans) if cu else Bt, Dm, N, dtype=torch.float64, device=x.device)
    init = s["init"] if s["init"] is not None else zero
    final, y = init.clone(), torch.zeros_like(x)
    keep = torch.zeros(L, Bt, Dm, N, dtype=torch.float64, device=x.device) if train else None   # h before each token
    for row, k, t0, t1 in spans:          # a packed sequence, or all rows of the batch at once
        rows, sts = (slice(0, 1), slice(k, k + 1)) if cu else (slice(None), slice(None))
        h = init[sts].clone()
        for t in range(t0, t1):
            if train:
                keep[t, rows] = h
            h = torch.exp(dt[rows, t, :, None] * A) * h + (dt[rows, t] * x[rows, t]).unsqueeze(-1) * s["B"][rows, t][:, grp]
            y[rows, t] = torch.einsum("bdn,bdn->bd", h, s["C"][rows, t][:, grp])
        final[sts] = h
    y = y + Dv * x
    gate = z * torch.sigmoid(z) if z is not None else torch.ones_like(y)
    if not train:
        return {"y": y * gate, "final": final}
    out = {"y": y * gate, "final": final}
    dy = s["dy"] * gate
    if z is not None:
        sg = torch.sigmoid(z)
        out["dz"] = s["dy"] * y * (sg + z * sg * (1 - sg))
    dtx, da = torch.zeros_like(x), torch.zeros_like(x)
    dA = torch.zeros_like(A)
    dB = torch.zeros(Bt, L, G, N, dtype=torch.float64, device=x.device)
    dC = torch.zeros_like(dB)
    dinit = torch.zeros_like(init)
    for row, k, t0, t1 in spans:
        rows, sts = (slice(0, 1), slice(k, k + 1)) if cu else (slice(None), slice(None))
        g = s["dfinal"][sts].clone()
        for t in range(t1 - 1, t0 - 1, -1):
            Bv, Cv = s["B"][rows, t][:, grp], s["C"][rows, t][:, grp]
            decay = torch.exp(dt[rows, t, :, None] * A)
            u = (dt[rows, t] * x[rows, t]).unsqueeze(-1)
            before = keep[t, rows]
            g = g + dy[rows, t].unsqueeze(-1) * Cv
            dC[rows, t] = ((decay * before + u * Bv) * dy[rows, t].unsqueeze(-1)).view(-1, G, Dm // G, N).sum(2)
            dB[rows, t] = (g * u).view(-1, G, Dm // G, N).sum(2)
            dtx[rows, t] = (g * Bv).sum(-1)
            g = g * decay
            q = g * before
            da[rows, t] = (q * A).sum(-1)
            dA += (q * dt[rows, t].unsqueeze(-1)).sum(0)
        dinit[sts] = g
    if s["init"] is not None:
        out["dinitial_states"] = dinit
    ddt = (dtx * x + da) * torch.sigmoid(raw)
    out.update(dx=dtx * dt + Dv * dy, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(dy * x).sum((0, 1)), ddt_bias=ddt.sum((0, 1)))
    return out


def _exact_conv(s):
    """Each sequence's rows behind its carried window, convolved as a sum over taps of shifted rows."""
    K, window = s["w"].shape[1], s["window"].clone()
    step = s["case"]["op"] == "conv_step"
    u = s["u"] if step else s["u"][0]
    out = torch.zeros_like(u)
    cu = list(range(u.shape[0] + 1)) if step else s["cu"].tolist()
    has = [1] * (len(cu) - 1) if step else s["has"].tolist()
    for k, slot in enumerate(s["slot"].tolist()):
        n = cu[k + 1] - cu[k]
        rows = torch.cat([s["window"][slot] * has[k], u[cu[k]:cu[k + 1]]])
        pre = s["bias"].expand(n, -1).clone()
        for j in range(K):
            pre += s["w"][:, j] * rows[j:j + n]
        out[cu[k]:cu[k + 1]] = pre * torch.sigmoid(pre)
        window[slot] = rows[rows.shape[0] - (K - 1):]
    return {"out": out if step else out.unsqueeze(0), "window": window}


def _exact_step(s):
    """One step of the recurrence for each request, request by request."""
    state, y = s["state"].clone(), torch.zeros_like(s["x"])
    per_head = s["case"]["op"] == "ssd_step"
    G = s["B"].shape[1]
    for k, slot in enumerate(s["slot"].tolist()):
        h, x = state[slot], s["x"][k]
        dt = torch.nn.functional.softplus(s["dt"][k] + s["dt_bias"], threshold=1e9)
        B, C = (s[n][k].repeat_interleave(s["A"].shape[0] // G, 0) for n in ("B", "C"))
        if per_head:
            h = torch.exp(dt * s["A"])[:, None, None] * h + torch.einsum("h,hp,hn->hpn", dt, x, B)
            y[k] = torch.einsum("hpn,hn->hp", h, C) + s["D"][:, None] * x
        else:
            h = torch.exp(dt[:, None] * s["A"]) * h + (dt * x)[:, None] * B
            y[k] = torch.einsum("dn,dn->d", h, C) + s["D"] * x
        state[slot] = h
    if s["z"] is not None:
        y = y * s["z"] * torch.sigmoid(s["z"])
    return {"y": y, "state": state}


def _exact_snapshot(s):
    back, scale = s["back"].clone(), s["scale"].clone()
    for i, j, k in zip(s["src"].tolist(), s["slot"].tolist(), s["dst"].tolist()):
        most = s["states"][i].abs().amax(-1)
        scale[j] = torch.where(most < 1e-30, torch.zeros_like(most), most / 127)
        unit = torch.where(scale[j] > 0, scale[j], torch.ones_like(most)).unsqueeze(-1)
        back[k] = torch.round(s["states"][i] / unit) * scale[j].unsqueeze(-1)
    return {"back": back, "scale": scale}


_EXACT = {"scan": _exact_scan, "train": _exact_scan, "conv_prompt": _exact_conv, "conv_step": _exact_conv,
          "ssd_step": _exact_step, "scan_step": _exact_step, "snapshot": _exact_snapshot}
