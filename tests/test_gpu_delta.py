"""The gated delta rule on the GPU against the float64 oracle: chunks, packed sequences, every gradient, single tokens.

Tolerances (relative 2-norm).  A rounding to bf16 is off by at most 2^-8 of the value, 2^-8 / sqrt(3) = 2.3e-3 in the mean
square.  A bf16 output of the tensor-core path goes through at most five (the state as an operand, the matrix inside
the chunk, the values, a decay's factor, the output itself): sqrt(5) x 2.3e-3 = 5.1e-3.  A gradient adds up
to four such products of either sign: twice that.  Everything in fp32, and fp32 states of either path: 64 terms and
two or three products in a row, each carried to 2^-17 at least: 2e-5."""
import numpy as np
import pytest
import torch

import state_space_model_scan_gb300 as pkg
from oracle import delta as oracle

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
OUT = {F32: 2e-5, BF16: 5.1e-3}
GRAD = {F32: 2e-5, BF16: 1.02e-2}


def np64(t):
    return t.detach().double().cpu().numpy()


def rel(a, b):
    b = np.asarray(b, np.float64)
    return float(np.linalg.norm(np64(a).reshape(b.shape) - b) / max(np.linalg.norm(b), 1e-300))


def make(B, L, G, H, V, K, dtype, gdtype=F32, nseqs=None, init=None, seed=0, train=False):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r, dtype=torch.float64)  # noqa: E731
    silu = torch.nn.functional.silu
    unit = lambda t: t / t.norm(dim=-1, keepdim=True).clamp(min=1e-6)  # noqa: E731
    S = nseqs or B
    x = dict(q=unit(silu(n(B, L, G, K))).to(dtype), k=unit(silu(n(B, L, G, K))).to(dtype), v=silu(n(B, L, H, V)).to(dtype),
             g=(-torch.linspace(0.01, 4.0, H, dtype=torch.float64) * torch.rand(B, L, H, generator=r, dtype=torch.float64)).to(gdtype),
             beta=torch.rand(B, L, H, generator=r, dtype=torch.float64).to(gdtype))
    x["init"] = (0.1 * n(S, H, V, K)).to(init) if init else None
    if train:
        x["do"], x["dfinal"] = n(B, L, H, V).to(dtype), (0.1 * n(S, H, V, K)).to(init or F32)
    return {k: None if t is None else t.cuda() for k, t in x.items()}


def want(x, scale, cu=None, back=False):
    """The oracle's o, final (and gradients) for a batch of rows, or for one packed row."""
    B = x["q"].shape[0]
    rows = []
    for b in range(B):
        a = [np64(x[n][b]) for n in ("q", "k", "v", "g", "beta")]
        init = None if x["init"] is None else np64(x["init"] if cu is not None else x["init"][b:b + 1])
        r = dict(zip(("o", "final"), oracle.forward(*a, scale, init, cu)))
        if back:
            df = np64(x["dfinal"] if cu is not None else x["dfinal"][b:b + 1])
            r.update(oracle.backward(*a, scale, np64(x["do"][b]), init, df, cu))
        rows.append(r)
    out = {n: np.stack([r[n] for r in rows]) for n in rows[0] if n not in ("final", "dinit")}
    for n in ("final", "dinit"):
        if n in rows[0]:
            out[n] = np.concatenate([r[n] for r in rows])
    return out


def packed(lens):
    return torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device="cuda")


CASES = [  # B, L, groups, heads, headdim, dstate, dtype, gates, lengths, initial states
    (1, 1, 1, 1, 128, 128, BF16, BF16, None, None),
    (2, 64, 2, 2, 128, 128, BF16, F32, None, F32),
    (1, 65, 1, 3, 128, 128, BF16, BF16, None, BF16),
    (1, 200, 2, 4, 128, 128, BF16, F32, [63, 0, 1, 136], F32),
    (2, 130, 1, 2, 64, 64, BF16, BF16, None, F32),
    (1, 150, 2, 2, 48, 96, BF16, F32, [150], None),
    (1, 129, 1, 2, 128, 72, BF16, F32, [1, 64, 64], BF16),
    (1, 70, 1, 2, 33, 57, BF16, BF16, None, F32),
    (1, 66, 1, 1, 160, 200, BF16, F32, None, F32),
    (1, 1, 1, 2, 5, 3, F32, F32, None, F32),
    (2, 77, 2, 6, 72, 48, F32, F32, None, F32),
    (1, 160, 3, 3, 96, 64, F32, F32, [64, 0, 0, 95, 1], F32),
    (1, 130, 1, 2, 256, 256, F32, F32, None, None),
    (1, 65, 1, 1, 1, 1, F32, F32, None, BF16),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(str(v) for v in c[:6]) + "-" + str(c[6])[6:])
def test_forward(case):
    B, L, G, H, V, K, dtype, gd, lens, init = case
    x = make(B, L, G, H, V, K, dtype, gd, lens and len(lens), init)
    cu = None if lens is None else packed(lens)
    o, f = pkg.gated_delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], initial_states=x["init"], cu_seqlens=cu, state_dtype=F32)
    w = want(x, K ** -0.5, None if cu is None else cu.tolist())
    assert o.dtype == dtype and rel(o, w["o"]) <= OUT[dtype]
    assert f.dtype == F32 and rel(f, w["final"]) <= OUT[F32]
    o2, f2 = pkg.gated_delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], initial_states=x["init"], cu_seqlens=cu)
    assert f2.dtype == (init or F32) and torch.equal(o, o2) and torch.equal(f2, f.to(f2.dtype))


@pytest.mark.parametrize("kept", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(str(v) for v in c[:6]) + "-" + str(c[6])[6:])
def test_backward(case, kept):
    B, L, G, H, V, K, dtype, gd, lens, init = case
    x = make(B, L, G, H, V, K, dtype, gd, lens and len(lens), init, train=True)
    cu = None if lens is None else packed(lens)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    states = None
    if kept:
        states = pkg.gated_delta_forward(*a, scale=0.3, initial_states=x["init"], cu_seqlens=cu, keep_chunk_states=True)[2]
    d = pkg.gated_delta_backward(*a, x["do"], scale=0.3, initial_states=x["init"], dfinal_states=x["dfinal"], cu_seqlens=cu, chunk_states=states)
    w = want(x, 0.3, None if cu is None else cu.tolist(), back=True)
    for n, like in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("dbeta", "beta")):
        assert d[n].dtype == x[like].dtype and d[n].shape == x[like].shape
        assert rel(d[n], w[n]) <= GRAD[dtype], n
    assert ("dinitial_states" in d) == (init is not None)
    if init is not None:
        assert d["dinitial_states"].dtype == init and rel(d["dinitial_states"], w["dinit"]) <= GRAD[dtype]


def test_long_sequences_and_memory_of_the_past():
    """2000 tokens of heads that forget slowly and quickly: what the chunks carry does not drift."""
    x = make(1, 2000, 1, 2, 128, 128, BF16)
    x["g"][..., 0] *= 0.01
    o, f = pkg.gated_delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"])
    w = want(x, 128 ** -0.5)
    for h in range(2):
        assert rel(o[:, :, h], w["o"][:, :, h]) <= OUT[BF16] and rel(f[:, h], w["final"][:, h]) <= OUT[F32]


@pytest.mark.parametrize("B,L,G,H,lens,init", [(1, 1500, 1, 1, None, F32), (1, 1301, 1, 2, [700, 3, 0, 598], BF16), (3, 700, 1, 1, None, None),
                                               (1, 900, 1, 2, [1, 899], None), (1, 640, 2, 2, None, F32)])
def test_chains_in_segments(B, L, G, H, lens, init):
    """Few heads and many chunks: the chains are cut, their segments joined; every output as of a whole one."""
    x = make(B, L, G, H, 128, 128, BF16, F32, lens and len(lens), init, train=True, seed=4)
    x["g"] *= 0.02                                                     # the past matters across segments
    cu = None if lens is None else packed(lens)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, f, kept = pkg.gated_delta_forward(*a, initial_states=x["init"], cu_seqlens=cu, state_dtype=F32, keep_chunk_states=True)
    d = pkg.gated_delta_backward(*a, x["do"], initial_states=x["init"], dfinal_states=x["dfinal"], cu_seqlens=cu, chunk_states=kept)
    w = want(x, 128 ** -0.5, None if cu is None else cu.tolist(), back=True)
    assert rel(o, w["o"]) <= OUT[BF16] and rel(f, w["final"]) <= OUT[F32]
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert rel(d[n], w[n]) <= GRAD[BF16], n
    if init is not None:
        assert rel(d["dinitial_states"], w["dinit"]) <= GRAD[BF16]
    assert torch.equal(pkg.gated_delta_forward(*a, initial_states=x["init"], cu_seqlens=cu)[0], o)
    d2 = pkg.gated_delta_backward(*a, x["do"], initial_states=x["init"], dfinal_states=x["dfinal"], cu_seqlens=cu)
    assert all(torch.equal(d[n], d2[n]) for n in d)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gates_at_their_ends(dtype):
    """Decays of 1 and of 0 (g = -inf, fp32's lowest value, -300 next to small ones), beta of 0, 1 and 2."""
    x = make(1, 150, 1, 4, 128, 128, dtype, train=True, init=F32)
    x["g"][..., 0] = 0
    x["g"][0, [0, 63, 64, 100], 1] = -float("inf")
    x["g"][0, [5, 70], 2] = torch.finfo(F32).min
    x["g"][0, ::40, 3] = -300
    x["beta"][0, 10:20] = 0
    x["beta"][0, 20:30] = 1
    x["beta"][0, 90:100] = 2
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, f = pkg.gated_delta_forward(*a, initial_states=x["init"])
    d = pkg.gated_delta_backward(*a, x["do"], initial_states=x["init"], dfinal_states=x["dfinal"])
    y = dict(x, g=x["g"].double().clamp(min=-800))     # the oracle's exponential underflows there, its product with 0 stays 0
    w = want(y, 128 ** -0.5, back=True)
    for h in range(4):
        assert rel(o[:, :, h], w["o"][:, :, h]) <= OUT[dtype] and rel(f[:, h], w["final"][:, h]) <= OUT[F32]
        for n in ("dv", "dg", "dbeta"):
            assert rel(d[n][:, :, h], w[n][:, :, h]) <= GRAD[dtype], (n, h)
    for n in ("dq", "dk"):
        assert rel(d[n], w[n]) <= GRAD[dtype], n
    assert rel(d["dinitial_states"], w["dinit"]) <= GRAD[dtype]


def test_sequences_never_meet():
    """NaN and infinities of one packed sequence stay there, forwards and backwards, at every place of the chunk's edge."""
    lens = [64, 1, 40, 90, 0, 5]
    x = make(1, 200, 1, 2, 128, 128, BF16, nseqs=6, init=F32, train=True)
    cu = packed(lens)
    a = lambda y: [y[n] for n in ("q", "k", "v", "g", "beta")]  # noqa: E731
    o, f = pkg.gated_delta_forward(*a(x), initial_states=x["init"], cu_seqlens=cu)
    d = pkg.gated_delta_backward(*a(x), x["do"], initial_states=x["init"], dfinal_states=x["dfinal"], cu_seqlens=cu)
    for s in (1, 2, 3):
        y = {n: t.clone() for n, t in x.items()}
        i = slice(int(cu[s]), int(cu[s + 1]))
        for n in ("q", "k", "v", "g", "beta", "do"):
            y[n][0, i] = float("nan") if n != "v" else float("inf")
        y["init"][s] = float("nan")
        o2, f2 = pkg.gated_delta_forward(*a(y), initial_states=y["init"], cu_seqlens=cu)
        d2 = pkg.gated_delta_backward(*a(y), y["do"], initial_states=y["init"], dfinal_states=y["dfinal"], cu_seqlens=cu)
        rest = [t for t in range(200) if not i.start <= t < i.stop]
        others = [j for j in range(6) if j != s]
        assert torch.equal(o[0, rest], o2[0, rest]) and torch.equal(f[others], f2[others])
        for n in ("dq", "dk", "dv", "dg", "dbeta"):
            assert torch.equal(d[n][0, rest], d2[n][0, rest]), n
        assert torch.equal(d["dinitial_states"][others], d2["dinitial_states"][others])
        assert not torch.isfinite(o2[0, i]).any()


def test_no_tokens():
    x = make(2, 0, 1, 2, 128, 128, BF16, init=F32, train=True)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, f = pkg.gated_delta_forward(*a, initial_states=x["init"])
    assert o.shape == (2, 0, 2, 128) and torch.equal(f, x["init"])
    assert not pkg.gated_delta_forward(*a)[1].any()
    d = pkg.gated_delta_backward(*a, x["do"], initial_states=x["init"], dfinal_states=x["dfinal"])
    assert torch.equal(d["dinitial_states"], x["dfinal"]) and d["dq"].shape == x["q"].shape


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_and_addresses(dtype):
    """Views of one projection, heads before tokens, rows that start at odd elements, one gate for all tokens: the
    same values, bit for bit."""
    x = make(2, 100, 1, 2, 128, 128, dtype, dtype, train=True)
    names = ("q", "k", "v", "g", "beta")
    a = [x[n] for n in names]
    o, f = pkg.gated_delta_forward(*a)
    d = pkg.gated_delta_backward(*a, x["do"])

    def heads_first(t):
        return t.transpose(1, 2).contiguous().transpose(1, 2)

    def odd(t):
        w = torch.full((t.shape[0], t.shape[1], t[0, 0].numel() + 3), float("nan"), dtype=t.dtype, device="cuda")
        w[..., 1:-2] = t.flatten(2)
        return w[..., 1:-2].unflatten(2, t.shape[2:])
    for way in (heads_first, odd):
        b = [way(t) for t in a]
        o2, f2 = pkg.gated_delta_forward(*b)
        d2 = pkg.gated_delta_backward(*b, way(x["do"]))
        assert torch.equal(o, o2) and torch.equal(f, f2) and all(torch.equal(d[n], d2[n]) for n in d)
    one = x["beta"][:, :1].expand(-1, 100, -1)
    o3 = pkg.gated_delta_forward(*a[:4], one)[0]
    assert torch.equal(o3, pkg.gated_delta_forward(*a[:4], one.contiguous())[0])


def test_autograd_streams_and_workspace():
    x = make(1, 190, 2, 4, 128, 128, BF16, BF16, init=F32, train=True)
    leaves = [x[n].detach().requires_grad_() for n in ("q", "k", "v", "g", "beta", "init")]
    o, f = pkg.GatedDeltaFunction.apply(*leaves)
    grads = torch.autograd.grad([o, f], leaves, [x["do"], x["dfinal"]])
    a = [t.detach() for t in leaves]
    d = pkg.gated_delta_backward(*a[:5], x["do"], initial_states=a[5], dfinal_states=x["dfinal"])
    names = ("dq", "dk", "dv", "dg", "dbeta", "dinitial_states")
    assert all(torch.equal(g, d[n]) for g, n in zip(grads, names))
    # what is kept and what is computed again are the same; an output that nothing came of
    o2, f2 = pkg.GatedDeltaFunction.apply(*leaves, None, None, False)
    assert torch.equal(o, o2)
    assert all(torch.equal(g, h) for g, h in zip(grads, torch.autograd.grad([o2, f2], leaves, [x["do"], x["dfinal"]])))
    only_f = torch.autograd.grad(pkg.GatedDeltaFunction.apply(*leaves)[1], leaves, x["dfinal"])
    d0 = pkg.gated_delta_backward(*a[:5], torch.zeros_like(x["do"]), initial_states=a[5], dfinal_states=x["dfinal"])
    assert all(torch.equal(g, d0[n]) for g, n in zip(only_f, names))
    o3 = pkg.GatedDeltaFunction.apply(*leaves)[0]
    with pytest.raises(RuntimeError):
        torch.autograd.grad(torch.autograd.grad(o3.float().sum(), leaves[0], create_graph=True)[0].float().sum(), leaves[0])
    # another stream, a workspace of the caller's
    st, ws = torch.cuda.Stream(), pkg.Workspace()
    st.wait_stream(torch.cuda.current_stream())
    d2 = pkg.gated_delta_backward(*a[:5], x["do"], initial_states=a[5], dfinal_states=x["dfinal"], workspace=ws, stream=st)
    o4, _ = pkg.gated_delta_forward(*a[:5], initial_states=a[5], stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(o4, o.detach()) and all(torch.equal(d[n], d2[n]) for n in names)


def test_training_step_in_a_graph():
    """Captured forward and backward, replayed on new values, while an eager graph of other leaves lives."""
    x = make(1, 130, 1, 2, 128, 128, BF16, BF16, train=True)
    y = make(1, 130, 1, 2, 128, 128, BF16, BF16, train=True, seed=5)
    names = ("q", "k", "v", "g", "beta")
    held = [y[n].clone().requires_grad_() for n in names]
    eager = pkg.GatedDeltaFunction.apply(*held)[0]
    a = [x[n].clone() for n in names]

    def step():
        o, f, kept = pkg.gated_delta_forward(*a, keep_chunk_states=True)
        return o, pkg.gated_delta_backward(*a, x["do"], chunk_states=kept)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, d = step()
    for src in (x, y):
        for t, n in zip(a, names):
            t.copy_(src[n])
        graph.replay()
        o2, d2 = step()
        assert torch.equal(o, o2) and all(torch.equal(d[n], d2[n]) for n in d)
    assert torch.equal(eager, o)


# ---- single tokens
@pytest.mark.parametrize("B,G,H,V,K,dtype,gd,sd", [
    (1, 16, 32, 128, 128, BF16, BF16, F32), (9, 2, 4, 128, 128, BF16, F32, BF16), (17, 1, 3, 72, 48, F32, F32, F32),
    (3, 1, 2, 64, 256, BF16, BF16, F32), (8, 1, 2, 17, 200, F32, F32, BF16), (2, 1, 1, 5, 7, BF16, F32, F32), (5, 2, 2, 33, 1, F32, F32, F32),
    (20, 1, 2, 48, 96, BF16, BF16, BF16)])
def test_step(B, G, H, V, K, dtype, gd, sd):
    x = make(B, 1, G, H, V, K, dtype, gd, init=sd)
    pool = torch.randn(B + 4, H, V, K, device="cuda").to(sd)
    slots = torch.randperm(B + 4, device="cuda")[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, B + 4                                 # padding
    old = pool.clone()
    a = [x[n][:, 0] for n in ("q", "k", "v", "g", "beta")]
    o = pkg.gated_delta_step(pool, *a, state_indices=slots)
    touched = torch.zeros(B + 4, dtype=torch.bool)
    for b in range(B):
        s = int(slots[b])
        if not 0 <= s < B + 4:
            assert not o[b].any()
            continue
        touched[s] = True
        wo, ws = oracle.step(np64(old[s]), *[np64(t[b]) for t in a], K ** -0.5)
        # fp32 sums of up to 256 terms; a bf16 output or state is rounded once, by 2^-8 at most
        assert rel(o[b], wo) <= (2e-6 if dtype == F32 else 4e-3) and rel(pool[s], ws) <= (2e-6 if sd == F32 else 4e-3)
    assert torch.equal(pool[~touched.cuda()], old[~touched.cuda()])


def test_steps_are_the_scan():
    x = make(2, 67, 1, 2, 64, 128, F32, init=F32)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, f = pkg.gated_delta_forward(*a, initial_states=x["init"])
    pool = x["init"].clone()
    got = torch.stack([pkg.gated_delta_step(pool, *[t[:, i] for t in a]) for i in range(67)], 1)
    assert rel(got, np64(o)) <= 2e-5 and rel(pool, np64(f)) <= 2e-5


def test_step_in_place_is_seen_and_strided():
    x = make(3, 2, 1, 2, 32, 64, BF16)
    big = torch.zeros(4, 3, 2, 32, 64, device="cuda")
    pool = big[:, 1]                                                   # slots lie apart
    plain = torch.zeros(4, 2, 32, 64, device="cuda")
    a = [x[n][:, 1] for n in ("q", "k", "v", "g", "beta")]
    before = pool._version
    o = pkg.gated_delta_step(pool, *a)
    assert pool._version > before
    assert torch.equal(o, pkg.gated_delta_step(plain, *[t.contiguous() for t in a])) and torch.equal(pool, plain)
    assert not big[:, [0, 2]].any()


def test_refusals():
    x = make(1, 10, 2, 4, 16, 16, F32, init=F32, train=True)
    a = {n: x[n] for n in ("q", "k", "v", "g", "beta")}
    run = pkg.gated_delta_forward
    for name, bad in (("q", x["q"][:, :9]), ("k", x["k"].to(BF16)), ("v", x["v"][0]), ("g", x["g"].double()), ("beta", x["beta"][..., :3]),
                      ("q", x["q"].transpose(2, 3)), ("k", x["k"].cpu())):
        with pytest.raises(ValueError):
            run(**{**a, name: bad})
    with pytest.raises(ValueError):
        run(**a, initial_states=x["init"][:, :2])
    with pytest.raises(ValueError):
        run(**a, cu_seqlens=torch.tensor([0, 10], device="cuda"))      # int64
    with pytest.raises(ValueError):
        run(**a, state_dtype=torch.float16)
    with pytest.raises(TypeError):
        run(**a, scale="one")
    with pytest.raises(pkg.api._lib.SSDError):                         # heads that no group divides
        run(x["q"][:, :, [0, 1, 1]], x["k"][:, :, [0, 1, 1]], x["v"], x["g"], x["beta"])
    with pytest.raises(pkg.api._lib.SSDError):
        wide = torch.zeros(1, 10, 4, 257, device="cuda")
        run(x["q"], x["k"], wide, x["g"], x["beta"])
    two = make(2, 10, 2, 4, 16, 16, F32)
    with pytest.raises(pkg.api._lib.SSDError):                         # packed rows come alone
        run(*[two[n] for n in a], cu_seqlens=packed([4, 6]))
    with pytest.raises(ValueError):
        pkg.gated_delta_backward(**a, do=x["do"], chunk_states=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        pkg.gated_delta_step(x["init"][:0], *[t[:, 0] for t in a.values()])
    with pytest.raises(ValueError):
        pkg.gated_delta_step(x["init"], *[t[:, 0] for t in a.values()], state_indices=torch.zeros(2, dtype=torch.int32, device="cuda"))
