"""Norm and rotation of queries and keys on the GPU against the float64 oracle.

Tolerances (relative 2-norm): fp32 sums of up to 512 terms and a handful of operations, 2e-6; the weights' gradients are fp32 sums
over all tokens and heads, 4e-6; a bf16 output is rounded once, by 2^-8 of its value at most, 3.9e-3."""
import numpy as np
import pytest
import torch

import state_space_model_scan_gb300 as pkg
from oracle import delta as oracle

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 2e-6, BF16: 3.91e-3}


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def rel(a, b):
    return float(np.linalg.norm(np64(a) - b) / max(np.linalg.norm(b), 1e-300))


def make(B, L, Hq, Hk, D, R, dtype, weighted=True, rows=40, seed=0):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r, dtype=torch.float64)  # noqa: E731
    qkv = n(B, L, (Hq + 2 * Hk) * D).to(dtype).cuda()
    x = dict(q=qkv[..., :Hq * D].unflatten(-1, (Hq, D)), k=qkv[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D)) if Hk else None)
    x["wq"], x["wk"] = (((1 + 0.2 * n(D)).float().cuda() if weighted and (i == 0 or Hk) else None) for i in range(2))
    x["dq"], x["dk"] = n(B, L, Hq, D).to(dtype).cuda(), n(B, L, Hk, D).to(dtype).cuda() if Hk else None
    x["cos"] = x["sin"] = x["pos"] = None
    if R:
        angle = torch.arange(rows, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
        x["cos"], x["sin"] = angle.cos().float().cuda(), angle.sin().float().cuda()
        x["pos"] = torch.randint(0, rows, (B, L), generator=r).to(torch.int32).cuda()
    return x


def run(x, **kw):
    return pkg.qk_norm_forward(x["q"], x["k"], x["wq"], x["wk"], x["cos"], x["sin"], x["pos"], **kw)


def back(x, **kw):
    return pkg.qk_norm_backward(x["q"], x["k"], x["dq"], x["dk"], x["wq"], x["wk"], x["cos"], x["sin"], x["pos"], **kw)


def check(x, dtype, **kw):
    q, k = run(x, **kw)
    d = back(x, **kw)
    for n, y in (("q", q), ("k", k)):
        if x[n] is None:
            assert y is None and "d" + n not in d
            continue
        B, L, H, D = x[n].shape
        flat = lambda t: np64(t).reshape(B * L, H, D)  # noqa: E731
        pos = np.tile(np.arange(L), B) if x["pos"] is None else np64(x["pos"]).reshape(-1).astype(int)
        a = dict(w=np64(x["w" + n]), cos=np64(x["cos"]), sin=np64(x["sin"]), positions=pos, **kw)
        assert y.dtype == dtype and rel(y.reshape(B * L, H, D), oracle.qk_forward(flat(x[n]), **a)) <= TOL[dtype]
        dx, dw = oracle.qk_backward(flat(x[n]), flat(x["d" + n]), **a)
        # dx = rstd (dn - n <dn, n>) is the difference of two terms, each right to 2e-6 of itself (in one dimension
        # they are the same but for eps / x^2 of them): what is allowed is that, and the rounding of dx
        xs = flat(x[n])
        power = (xs * xs).sum(-1) / (D if kw["mode"] == "rms" else 1) + kw["eps"]
        terms = np.linalg.norm(np.linalg.norm(flat(x["d" + n]) * (1.0 if x["w" + n] is None else np64(x["w" + n])), axis=-1) / np.sqrt(power))
        off = np.linalg.norm(np64(d["d" + n]).reshape(dx.shape) - dx)
        assert d["d" + n].dtype == dtype and off <= TOL[dtype] * np.linalg.norm(dx) + 2e-6 * terms
        if x["w" + n] is not None:
            assert rel(d["d%s_weight" % n], dw) <= 4e-6
        else:
            assert "d%s_weight" % n not in d
    return q, k, d


@pytest.mark.parametrize("mode", ["rms", "l2"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,L,Hq,Hk,D,R,dtype", [
    (1, 1, 1, 1, 128, 128, BF16), (2, 37, 32, 8, 128, 64, BF16), (1, 300, 5, 1, 64, 64, BF16), (3, 11, 6, 2, 256, 128, BF16),
    (1, 9, 3, 3, 96, 96, BF16), (1, 5, 2, 1, 512, 256, BF16), (1, 7, 3, 2, 72, 36, BF16), (2, 13, 3, 0, 128, 0, BF16),
    (2, 37, 8, 4, 128, 128, F32), (1, 21, 5, 1, 72, 36, F32), (1, 8, 2, 2, 200, 200, F32), (1, 4, 2, 1, 512, 512, F32), (1, 6, 1, 1, 7, 4, F32),
    (1, 3, 4, 5, 1, 0, F32)])
def test_against_the_oracle(B, L, Hq, Hk, D, R, dtype, mode, interleaved):
    check(make(B, L, Hq, Hk, D, R, dtype), dtype, mode=mode, interleaved=interleaved, eps=1e-5)


def test_many_tokens_without_weights_and_default_positions():
    x = make(2, 700, 9, 2, 128, 128, BF16, weighted=False, rows=700)
    x["pos"] = None
    check(x, BF16, mode="l2", interleaved=False, eps=1e-6)
    x = make(1, 1500, 8, 2, 128, 128, F32)
    check(x, F32, mode="rms", interleaved=False, eps=1e-6)


@pytest.mark.parametrize("D", [128, 72])
def test_padding(D):
    """Positions outside the table: zeros, whatever the token holds; an empty table: nothing but zeros."""
    x = make(2, 10, 5, 1, D, 64 if D == 128 else 36, BF16)
    x["pos"][0, 3], x["pos"][1, 9], x["pos"][0, 0] = -1, 40, -2 ** 31
    for n in ("q", "k", "dq", "dk"):
        x[n] = x[n].clone()
        x[n][0, 3] = float("nan")
    q, k = run(x)
    d = back(x)
    for t in (q, k, d["dq"], d["dk"]):
        assert not t[0, 3].any() and not t[1, 9].any() and not t[0, 0].any() and torch.isfinite(t).all()
    y = {n: (t if t is None or t.dim() < 3 else t.clone()) for n, t in x.items()}
    for n in ("q", "k", "dq", "dk"):
        y[n][0, 3] = 1.0
    check(y, BF16, mode="rms", interleaved=False, eps=1e-6)
    assert torch.equal(d["dq_weight"], back(y)["dq_weight"])
    x["cos"], x["sin"] = x["cos"][:0], x["sin"][:0]
    q, k = run(x)
    d = back(x)
    assert not any(t.any() for t in (q, k, *d.values()))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_and_addresses(dtype):
    """Any strides of what is read give the same values (other sums where a row starts between the pieces)."""
    x = make(2, 30, 6, 2, 128, 128, dtype)
    q, k = run(x)
    d = back(x)
    y = dict(x, **{n: x[n].transpose(1, 2).contiguous().transpose(1, 2) for n in ("q", "k", "dq", "dk")})
    q2, k2 = run(y)
    d2 = back(y)
    assert torch.equal(q, q2) and torch.equal(k, k2) and all(torch.equal(d[n], d2[n]) for n in d)

    def odd(t):
        w = torch.zeros(t.shape[0], t.shape[1], t[0, 0].numel() + 3, dtype=t.dtype, device="cuda")
        w[..., 1:-2] = t.flatten(2)
        return w[..., 1:-2].unflatten(2, t.shape[2:])
    check(dict(x, **{n: odd(x[n]) for n in ("q", "k", "dq", "dk")}), dtype, mode="rms", interleaved=False, eps=1e-6)
    z = dict(x, q=x["q"][:, :1].expand(-1, 30, -1, -1))
    assert torch.equal(run(z)[0], run(dict(z, q=z["q"].contiguous()))[0])


def test_zero_vectors_and_no_tokens():
    x = make(1, 4, 2, 1, 128, 128, BF16)
    x["q"] = torch.zeros_like(x["q"])
    q, _ = run(x)
    assert not q.any() and torch.isfinite(back(x)["dq"]).all()
    x = make(1, 0, 2, 1, 128, 128, BF16)
    q, k = run(x)
    assert q.shape == (1, 0, 2, 128) and not back(x)["dq_weight"].any()


def test_autograd_streams_and_graph():
    x = make(2, 65, 6, 2, 128, 64, BF16)
    leaves = [x[n].detach().clone().requires_grad_() for n in ("q", "k", "wq", "wk")]
    q, k = pkg.QKNormFunction.apply(*leaves, x["cos"], x["sin"], x["pos"], "rms", True, 1e-6)
    grads = torch.autograd.grad([q, k], leaves, [x["dq"], x["dk"]])
    d = back(x, interleaved=True)
    assert all(torch.equal(g, d[n]) for g, n in zip(grads, ("dq", "dk", "dq_weight", "dk_weight")))
    st, ws = torch.cuda.Stream(), pkg.Workspace()
    st.wait_stream(torch.cuda.current_stream())
    d2 = back(x, interleaved=True, workspace=ws, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(d[n], d2[n]) for n in d)
    back(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, dd = run(x), back(x)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, run(x))) and all(torch.equal(dd[n], v) for n, v in back(x).items())
    only_q = torch.autograd.grad(pkg.QKNormFunction.apply(leaves[0], None)[0].float().sum(), leaves[0])[0]
    assert torch.isfinite(only_q).all()


def test_refusals():
    x = make(1, 4, 2, 1, 16, 8, F32)
    for change in (dict(q=x["q"][0]), dict(k=x["k"].to(BF16)), dict(wq=x["wq"][:8]), dict(wk=x["wk"].double()), dict(cos=x["cos"][:5]),
                   dict(sin=None), dict(pos=x["pos"].long()), dict(pos=x["pos"][:, :3]), dict(k=None), dict(q=x["q"].transpose(2, 3)), dict(q=x["q"].cpu())):
        with pytest.raises(ValueError):
            run({**x, **change})
    with pytest.raises(ValueError):
        run(x, mode="layer")
    with pytest.raises(ValueError):
        wide = torch.zeros(40, 9, device="cuda")
        run({**x, "cos": wide, "sin": wide})
    with pytest.raises(pkg.api._lib.SSDError):
        big = torch.zeros(1, 1, 1, 513, device="cuda")
        pkg.qk_norm_forward(big, None)
    with pytest.raises(pkg.api._lib.SSDError):
        run(x, eps=-1.0)
