"""Measured cases of the operators that carry a gated-delta block through training and serving.

Four operators, each in a plain form (elementary torch operations in 32 bits) and as a user
calls it in this package:

* the gated delta rule over prompts and packed prompt pieces (``prompt``): per value head a state
  that decays, forgets what a key held and takes up the new value,
      S <- a S,  u = beta (v - S k),  S <- S + u k^T,  o = scale S q;
* the same as a training step with every gradient (``train``);
* its step for one token per request on a pool of states (``step``);
* the norm of each head of queries and keys with the rotation by position in the same pass, for
  prompts and single tokens (``qk``) and as a training step (``qk_train``).

``own`` selects the package's operators; otherwise the plain forms run.
"""
import math

import torch

own = False

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 64


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # One user's long prompt at a mid-sized block's heads: latency counts, few heads fill the card.
        dict(name="prompt_8192", op="prompt", batch=1, seqlen=8192, key_heads=16, nheads=32, dstate=128, headdim=128,
             dtype="bf16", gate_dtype="f32", nseqs=0, carried=False, state_dtype="f32"),
        # Continuous batching: pieces of mixed lengths packed on one token axis, each going on from its state.
        dict(name="prompt_packed", op="prompt", batch=1, seqlen=16111, key_heads=16, nheads=16, dstate=128, headdim=128,
             dtype="bf16", gate_dtype="bf16", nseqs=9, carried=True, state_dtype="f32"),
        # A short prompt in 32 bits at odd sizes.
        dict(name="prompt_f32_odd", op="prompt", batch=2, seqlen=77, key_heads=2, nheads=6, dstate=48, headdim=72,
             dtype="f32", gate_dtype="f32", nseqs=0, carried=True, state_dtype="f32"),
        # A training step at an ordinary micro-batch.
        dict(name="train_2x2048", op="train", batch=2, seqlen=2048, key_heads=16, nheads=32, dstate=128, headdim=128,
             dtype="bf16", gate_dtype="bf16", nseqs=0, carried=False, state_dtype="bf16"),
        # The same in 32 bits at odd sizes, from a given state.
        dict(name="train_f32_odd", op="train", batch=3, seqlen=331, key_heads=3, nheads=3, dstate=64, headdim=96,
             dtype="f32", gate_dtype="f32", nseqs=0, carried=True, state_dtype="f32"),
        # A single user's next token: what one request waits for.
        dict(name="step_1", op="step", batch=1, key_heads=16, nheads=32, dstate=128, headdim=128, dtype="bf16",
             gate_dtype="bf16", state_dtype="f32"),
        # A loaded server's step.
        dict(name="step_192", op="step", batch=192, key_heads=16, nheads=32, dstate=128, headdim=128, dtype="bf16",
             gate_dtype="f32", state_dtype="f32"),
        # The queries and keys of a long prompt, normalised by their mean square and rotated.
        dict(name="qk_8192", op="qk", batch=1, seqlen=8192, query_heads=32, key_heads=8, dim=128, rotary=128,
             mode="rms", weighted=True, interleaved=False, dtype="bf16"),
        # One token for each of 64 requests, to unit length, without a rotation: what precedes a delta step.
        dict(name="qk_step_64", op="qk", batch=64, seqlen=1, query_heads=16, key_heads=16, dim=128, rotary=0,
             mode="l2", weighted=False, interleaved=False, dtype="bf16"),
        # A training step of the norm and rotation at an ordinary micro-batch.
        dict(name="qk_train_2x2048", op="qk_train", batch=2, seqlen=2048, query_heads=32, key_heads=8, dim=128,
             rotary=64, mode="rms", weighted=True, interleaved=False, dtype="bf16"),
        # The same in 32 bits at odd sizes, neighbouring pairs rotated.
        dict(name="qk_train_f32_odd", op="qk_train", batch=3, seqlen=211, query_heads=5, key_heads=1, dim=72,
             rotary=36, mode="rms", weighted=True, interleaved=True, dtype="f32"),
    ]


def _len(rng, lo, hi):
    """A length spread over the logarithm of [lo, hi]: odd, or an odd multiple of 64 where that fits."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.3 and n >= 64:
        return max(64, n // 128 * 128 - 64)
    return min(hi, max(lo, n | 1))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "train", "step", "qk", "qk_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("qk", "qk_train"):
        dim = rng.choice([128, 128, 64, 256, 96])
        tokens = _len(rng, 1, 8191 if op == "qk" else 4095)
        batch = rng.choice([1, 2, 3]) if tokens >= 3 else 1
        rotary = rng.choice([dim, dim // 2, 0])
        return dict(op=op, batch=batch, seqlen=max(1, tokens // batch), query_heads=rng.choice([32, 16, 8, 5]),
                    key_heads=rng.choice([8, 4, 1]), dim=dim, rotary=rotary, mode=rng.choice(["rms", "l2"]),
                    weighted=rng.random() < 0.7, interleaved=rotary > 0 and rng.random() < 0.3, dtype=dtype)
    K, V = rng.choice([(128, 128), (128, 128), (128, 128), (64, 64), (64, 128), (96, 48)])
    key_heads = rng.choice([16, 8, 4, 1, 3])
    nheads = key_heads * rng.choice([1, 2, 2, 3])
    gate = rng.choice([dtype, "f32"]) if op != "train" else dtype
    state = rng.choice(["f32", "bf16"])
    if op == "step":
        return dict(op=op, batch=_len(rng, 1, 191), key_heads=key_heads, nheads=min(nheads, 32 // key_heads * key_heads), dstate=K,
                    headdim=V, dtype=dtype, gate_dtype=gate, state_dtype=state)
    # 32 bits: a test's or a small model's size
    most = {"prompt": 1 << 18, "train": 1 << 17}[op] // (8 if dtype == "f32" else 1)   # tokens x heads
    tokens = _len(rng, 1, min(16001, most // nheads))
    batch = rng.choice([2, 3, 4]) if tokens >= 4 and rng.random() < 0.5 else 1
    nseqs = rng.choice([0, 2, 5, 11]) if batch == 1 and tokens >= 64 else 0
    return dict(op=op, batch=batch, seqlen=max(1, tokens // batch), key_heads=key_heads, nheads=nheads, dstate=K,
                headdim=V, dtype=dtype, gate_dtype=gate, nseqs=nseqs, carried=rng.random() < 0.5,
                state_dtype=dtype if op == "train" else state)


# ---------------------------------------------------------------------------- inputs
def _lengths(case, seed):
    """Lengths of the packed sequences: seqlen tokens cut at random places (some pieces may be tiny)."""
    r = torch.Generator().manual_seed(seed + 17)
    inner = torch.randint(0, case["seqlen"] + 1, (case["nseqs"] - 1,), generator=r).sort().values.tolist()
    cuts = [0] + inner + [case["seqlen"]]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    td = _DTYPE[case["dtype"]]

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"case": case}
    if op in ("qk", "qk_train"):
        B, L, Hq, Hk, D, R = (case[k] for k in ("batch", "seqlen", "query_heads", "key_heads", "dim", "rotary"))
        train = op == "qk_train"
        qkv = normal(B, L, (Hq + 2 * Hk) * D, dtype=td)              # a projection's output: queries, keys, values
        s["q"] = qkv[..., :Hq * D].unflatten(-1, (Hq, D))
        s["k"] = qkv[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
        s["wq"] = 1.0 + normal(D, scale=0.1) if case["weighted"] else None
        s["wk"] = 1.0 + normal(D, scale=0.1) if case["weighted"] else None
        s["cos"] = s["sin"] = s["positions"] = None
        if R:
            rows = 32768
            rate = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
            angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * rate
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
            first = torch.randint(0, rows - L, (B, 1), generator=g, device="cuda")
            s["positions"] = (first + torch.arange(L, device="cuda")).to(torch.int32)
        if train:
            s["q"], s["k"] = s["q"].detach().requires_grad_(), s["k"].detach().requires_grad_()
            s["wq"] = None if s["wq"] is None else s["wq"].requires_grad_()
            s["wk"] = None if s["wk"] is None else s["wk"].requires_grad_()
            s["dq"], s["dk"] = normal(B, L, Hq, D, dtype=td), normal(B, L, Hk, D, dtype=td)
        return s

    B, L = case["batch"], case.get("seqlen", 1)
    Hk, H, K, V = (case[k] for k in ("key_heads", "nheads", "dstate", "headdim"))
    tg, ts = _DTYPE[case["gate_dtype"]], _DTYPE[case["state_dtype"]]
    # what a convolution with SiLU leaves: queries and keys brought to unit length per head, values as they are
    xbc = torch.nn.functional.silu(normal(B, L, 2 * Hk * K + H * V)).to(td)
    q, k = xbc[..., :2 * Hk * K].float().unflatten(-1, (2, Hk, K)).unbind(-3)
    q = (q * torch.rsqrt(q.square().sum(-1, keepdim=True) + 1e-6)).to(td)
    k = (k * torch.rsqrt(k.square().sum(-1, keepdim=True) + 1e-6)).to(td)
    v = xbc[..., 2 * Hk * K:].unflatten(-1, (H, V))
    rate = torch.exp(torch.rand(H, generator=g, device="cuda") * math.log(16.0))
    bias = torch.log(torch.expm1(torch.exp(math.log(1e-3) + torch.rand(H, generator=g, device="cuda") * math.log(100.0))))
    decay = (-rate * torch.nn.functional.softplus(normal(B, L, H, scale=0.5) + bias)).to(tg)
    beta = torch.sigmoid(normal(B, L, H)).to(tg)
    s.update(q=q, k=k, v=v, g=decay, beta=beta, scale=K ** -0.5)
    if op == "step":
        slots = B + 3                                                  # a pool with some slots free
        s.update(q=q[:, 0], k=k[:, 0], v=v[:, 0], g=decay[:, 0], beta=beta[:, 0])
        s["state"] = normal(slots, H, V, K, dtype=ts, scale=0.1)
        s["slots"] = torch.randperm(slots, generator=g, device="cuda")[:B].to(torch.int32)
        return s
    lens = _lengths(case, seed) if case["nseqs"] else [L] * B
    S = len(lens)
    s["longest"] = max(lens)
    s["cu"] = None
    if case["nseqs"]:
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    s["init"] = normal(S, H, V, K, dtype=ts, scale=0.1) if case["carried"] else None
    if op == "train":
        for name in ("q", "k", "v", "g", "beta", "init"):
            s[name] = None if s[name] is None else s[name].detach().requires_grad_()
        s["do"] = normal(B, L, H, V, dtype=td)
        s["dfinal"] = normal(S, H, V, K, dtype=ts, scale=0.1) if case["carried"] else None
    return s


# ---------------------------------------------------------------------------- plain forms
def _pieces(t, s, chunks):
    """[batch, seqlen, heads, ...] as [sequences, heads, chunks, 64, ...] in 32 bits, with zeros past each sequence's end."""
    t = t.float()
    if s["cu"] is None:
        t = torch.nn.functional.pad(t, (0, 0) * (t.dim() - 2) + (0, chunks * _CHUNK - t.shape[1]))
    else:
        at = s["cu"][:-1, None].long() + torch.arange(chunks * _CHUNK, device=t.device)
        inside = at < s["cu"][1:, None]
        t = t[0][at.clamp(max=t.shape[1] - 1)]
        t = torch.where(inside.view(inside.shape + (1,) * (t.dim() - 2)), t, 0.0)
    return t.unflatten(1, (chunks, _CHUNK)).movedim(3, 1)


def _joined(o, s, seqlen):
    """The inverse of _pieces for the output."""
    o = o.movedim(1, 3).flatten(1, 2)
    if s["cu"] is None:
        return o[:, :seqlen]
    t = torch.arange(seqlen, device=o.device)
    seq = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    return o[seq, t - s["cu"].long()[seq]][None]


def _plain_delta(s):
    """The rule in chunks of 64 tokens: within a chunk a triangular system, from chunk to chunk the state (one pass of
    the loop for each chunk: the state that enters it is needed first)."""
    chunks = max(1, -(-s["longest"] // _CHUNK))
    per = s["v"].shape[2] // s["q"].shape[2]
    q = _pieces(s["q"], s, chunks).repeat_interleave(per, 1) * s["scale"]
    k = _pieces(s["k"], s, chunks).repeat_interleave(per, 1)
    v, g, beta = _pieces(s["v"], s, chunks), _pieces(s["g"], s, chunks), _pieces(s["beta"], s, chunks)
    G = g.double().cumsum(-1)
    low = torch.ones(_CHUNK, _CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = torch.where(low, G[..., :, None] - G[..., None, :], -math.inf).exp().float()
    since, until, whole = G.exp().float(), (G[..., -1:] - G).exp().float(), G[..., -1].exp().float()
    system = torch.where(low.tril(-1), (k @ k.mT) * decay, 0.0) * beta[..., None, :]
    eye = torch.eye(_CHUNK, device=q.device)
    solve = torch.linalg.solve_triangular(eye + system, eye.expand_as(system), upper=False, unitriangular=True)
    inner = (q @ k.mT) * decay
    S = s["init"].float() if s["init"] is not None else torch.zeros(q.shape[0], v.shape[1], v.shape[-1], q.shape[-1], device=q.device)
    out = []
    for c in range(chunks):
        u = solve[:, :, c] @ (v[:, :, c] - since[:, :, c, :, None] * (k[:, :, c] @ S.mT))
        w = beta[:, :, c, :, None] * u
        out.append(since[:, :, c, :, None] * (q[:, :, c] @ S.mT) + inner[:, :, c] @ w)
        S = whole[:, :, c, None, None] * S + (until[:, :, c, :, None] * w).mT @ k[:, :, c]
    return _joined(torch.stack(out, 2), s, s["q"].shape[1]), S


def _plain_step(s):
    at = s["slots"].long()
    per = s["v"].shape[1] // s["q"].shape[1]
    q, k = (s[n].float().repeat_interleave(per, 1) for n in ("q", "k"))
    S = s["state"][at].float() * s["g"].float().exp()[..., None, None]
    u = s["beta"].float()[..., None] * (s["v"].float() - (S @ k[..., None])[..., 0])
    S = S + u[..., None] * k[..., None, :]
    s["state"][at] = S.to(s["state"].dtype)
    return ((S @ q[..., None])[..., 0] * s["scale"]).to(s["v"].dtype)


def _plain_qk(x, w, s):
    case = s["case"]
    x = x.float()
    m = x.square().mean(-1, keepdim=True) if case["mode"] == "rms" else x.square().sum(-1, keepdim=True)
    y = x * torch.rsqrt(m + 1e-6)
    y = y if w is None else y * w
    if case["rotary"]:
        R = case["rotary"]
        cos, sin = (s[n][s["positions"].long()][:, :, None] for n in ("cos", "sin"))
        a, b = (y[..., 0:R:2], y[..., 1:R:2]) if case["interleaved"] else (y[..., :R // 2], y[..., R // 2:R])
        a, b = a * cos - b * sin, a * sin + b * cos
        r = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
        y = torch.cat([r, y[..., R:]], -1)
    return y


def _grads(outputs, grads, s, names):
    names = [n for n in names if s[n] is not None]
    return {"d" + n: t for n, t in zip(names, torch.autograd.grad(outputs, [s[n] for n in names], grads))}


# ---------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import state_space_model_scan_gb300 as pkg
    if op == "prompt":
        if own:
            o, final = pkg.gated_delta_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], initial_states=s["init"],
                                               cu_seqlens=s["cu"], state_dtype=_DTYPE[case["state_dtype"]])
        else:
            o, final = _plain_delta(s)
            o, final = o.to(s["v"].dtype), final.to(_DTYPE[case["state_dtype"]])
        return {"o": o, "final": final}
    if op == "train":
        if own:
            o, final = pkg.GatedDeltaFunction.apply(s["q"], s["k"], s["v"], s["g"], s["beta"], s["init"], s["cu"], s["scale"])
        else:
            o, final = _plain_delta(s)
            o, final = o.to(s["v"].dtype), final.to(_DTYPE[case["state_dtype"]])
        outputs, grads = ([o, final], [s["do"], s["dfinal"]]) if s["init"] is not None else ([o], [s["do"]])
        return {"o": o.detach(), **_grads(outputs, grads, s, ("q", "k", "v", "g", "beta", "init"))}
    if op == "step":
        if own:
            o = pkg.gated_delta_step(s["state"], s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], state_indices=s["slots"])
        else:
            o = _plain_step(s)
        return {"o": o, "state": s["state"]}
    if own and op == "qk":
        q, k = pkg.qk_norm_forward(s["q"], s["k"], s["wq"], s["wk"], cos=s["cos"], sin=s["sin"], positions=s["positions"],
                                   mode=case["mode"], interleaved=case["interleaved"], eps=1e-6)
    elif own:
        q, k = pkg.QKNormFunction.apply(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["positions"], case["mode"],
                                        case["interleaved"], 1e-6)
    else:
        q, k = (_plain_qk(x, w, s).to(x.dtype) for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])))
    if op == "qk":
        return {"q": q, "k": k}
    return {"q": q.detach(), "k": k.detach(), **_grads([q, k], [s["dq"], s["dk"]], s, ("q", "k", "wq", "wk"))}


# ---------------------------------------------------------------------------- work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("qk", "qk_train"):
        tokens = case["batch"] * case["seqlen"]
        vals = tokens * (case["query_heads"] + case["key_heads"]) * case["dim"]
        table = tokens * (4 + 4 * case["rotary"])                       # positions and rows of the table
        passes = 2 if case["op"] == "qk" else 5                         # read, write; and read again with dy, dx written
        return {"bytes": passes * vals * e + (1 if case["op"] == "qk" else 2) * table, "flops": (6 if case["op"] == "qk" else 20) * vals}
    Hk, H, K, V = (case[k] for k in ("key_heads", "nheads", "dstate", "headdim"))
    eg, es = (2 if case[n] == "bf16" else 4 for n in ("gate_dtype", "state_dtype"))
    tokens = case["batch"] * case.get("seqlen", 1)
    ins = tokens * (2 * Hk * K * e + H * V * e + 2 * H * eg)
    outs = tokens * H * V * e
    if case["op"] == "step":
        return {"bytes": ins + outs + 2 * case["batch"] * H * V * K * es, "flops": 8 * case["batch"] * H * V * K}
    S = case["nseqs"] or case["batch"]
    state = S * H * V * K * es
    # a token and head: the state read by key and by query and written, half of each 64 x 64 product
    flops = tokens * H * (6 * K * V + 2 * _CHUNK * (K + V))
    if case["op"] == "prompt":
        return {"bytes": ins + outs + (2 if case["carried"] else 1) * state, "flops": flops}
    back = tokens * H * (12 * K * V + _CHUNK * (4 * K + 6 * V))
    return {"bytes": 3 * ins + 2 * outs + (4 * state if case["carried"] else 0), "flops": flops + back}


# ---------------------------------------------------------------------------- in 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] in ("qk", "qk_train"):
            return _exact_qk(case, s)
        if case["op"] == "step":
            at, per = s["slots"].long(), case["nheads"] // case["key_heads"]
            state = s["state"].double()
            q, k = (s[n].double()[:, torch.arange(case["nheads"], device="cuda") // per] for n in ("q", "k"))
            old = torch.exp(s["g"].double())[:, :, None, None] * state[at]
            read = (old * k[:, :, None, :]).sum(-1)
            new = old + (s["beta"].double()[:, :, None] * (s["v"].double() - read))[..., None] * k[:, :, None, :]
            state[at] = new
            return {"o": case["dstate"] ** -0.5 * (new * q[:, :, None, :]).sum(-1), "state": state}
        return _exact_delta(case, s)


def _exact_delta(case, s):
    """One token after the other, all sequences at once; the gradients by the adjoint of that loop."""
    train = case["op"] == "train"
    H, K, V, T = case["nheads"], case["dstate"], case["headdim"], s["longest"]
    scale, per = case["dstate"] ** -0.5, H // case["key_heads"]
    cu = s["cu"].tolist() if s["cu"] is not None else None
    S = len(cu) - 1 if cu else case["batch"]
    if S * H * V * K * 8 * T > (6 << 30) * (8 if train else 100) or T > 20000:
        return None

    def rows(t):                                                          # [sequences, longest, ...], zeros past the end
        if cu is None:
            return t.double()
        r = torch.zeros(S, T, *t.shape[2:], dtype=torch.float64, device="cuda")
        for i in range(S):
            r[i, :cu[i + 1] - cu[i]] = t[0, cu[i]:cu[i + 1]].double()
        return r

    def flat(t):
        if cu is None:
            return t
        return torch.cat([t[i, :cu[i + 1] - cu[i]] for i in range(S)])[None]

    head = torch.arange(H, device="cuda") // per
    q, k = rows(s["q"])[:, :, head], rows(s["k"])[:, :, head]
    v, a, beta = rows(s["v"]), rows(s["g"]).exp(), rows(s["beta"])
    h = s["init"].double() if s["init"] is not None else torch.zeros(S, H, V, K, dtype=torch.float64, device="cuda")
    o, err, kept = torch.empty_like(v), torch.empty_like(v), []
    for t in range(T):
        if train:
            kept.append(h)
        h = a[:, t, :, None, None] * h
        err[:, t] = v[:, t] - torch.matmul(h, k[:, t, :, :, None])[..., 0]
        h = h + (beta[:, t, :, None] * err[:, t])[..., None] * k[:, t, :, None, :]
        o[:, t] = scale * torch.matmul(h, q[:, t, :, :, None])[..., 0]
    if not train:
        return {"o": flat(o), "final": h}
    do = rows(s["do"])
    dh = s["dfinal"].double() if s["dfinal"] is not None else torch.zeros_like(h)
    dq, dk, dv, da, dbeta = (torch.zeros_like(x) for x in (q, k, v, a, beta))
    for t in reversed(range(T)):
        qt, kt, dot = q[:, t], k[:, t], do[:, t]
        dh = dh + scale * dot[..., None] * qt[..., None, :]
        dq[:, t] = scale * torch.matmul(dot[..., None, :], h)[..., 0, :]
        u = beta[:, t, :, None] * err[:, t]
        du = torch.matmul(dh, kt[..., None])[..., 0]
        dbeta[:, t] = (du * err[:, t]).sum(-1)
        dv[:, t] = beta[:, t, :, None] * du
        old = kept.pop()
        faded = a[:, t, :, None, None] * old
        dk[:, t] = torch.matmul(u[..., None, :], dh)[..., 0, :] - torch.matmul(dv[:, t, :, None, :], faded)[..., 0, :]
        dfaded = dh - dv[:, t, :, :, None] * kt[..., None, :]
        da[:, t] = (dfaded * faded).sum((-1, -2))                          # times a: the gradient of log a
        dh = a[:, t, :, None, None] * dfaded
        h = old
    shared = lambda t: flat(t.unflatten(2, (case["key_heads"], per)).sum(3))  # noqa: E731
    r = {"o": flat(o), "dq": shared(dq), "dk": shared(dk), "dv": flat(dv), "dg": flat(da), "dbeta": flat(dbeta)}
    if s["init"] is not None:
        r["dinit"] = dh
    return r


def _exact_qk(case, s):
    R, D = case["rotary"], case["dim"]
    r = {}
    for n, w in (("q", s["wq"]), ("k", s["wk"])):
        x = s[n].double()
        power = x.pow(2).sum(-1, keepdim=True)
        rstd = (power / D + 1e-6 if case["mode"] == "rms" else power + 1e-6) ** -0.5
        wd = torch.ones(D, dtype=torch.float64, device="cuda") if w is None else w.double()
        y = x * rstd * wd
        if R:
            i = torch.arange(R // 2, device="cuda")
            first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + R // 2)
            at = s["positions"].long()
            c, sn = s["cos"].double()[at].unsqueeze(2), s["sin"].double()[at].unsqueeze(2)

            def turn(t, sign):
                z = t.clone()
                z[..., first] = t[..., first] * c - sign * t[..., second] * sn
                z[..., second] = sign * t[..., first] * sn + t[..., second] * c
                return z
        else:
            turn = lambda t, sign: t  # noqa: E731
        r[n] = turn(y, 1)
        if case["op"] == "qk_train":
            dy = turn(s["d" + n].double(), -1)
            if w is not None:
                r["dw" + n] = (dy * x * rstd).flatten(0, 2).sum(0)
            dn = dy * wd
            r["d" + n] = rstd * dn - x * rstd ** 3 / (D if case["mode"] == "rms" else 1) * (dn * x).sum(-1, keepdim=True)
    return r
