"""The gated delta rule, its single-token step, and the norm of queries and keys with the rotation, in float64 -- TEST
INFRASTRUCTURE ONLY.

Gated delta rule, value head h with the keys and queries of group h // (H // G) and a state S [V, K]:

    S <- exp(g) S,  u = beta (v - S k),  S <- S + u k^T,  o = scale S q

one token after the other; the backward is the exact adjoint of that loop.  Pinned by tests/test_oracle_delta.py: central
differences of every gradient, the plain linear attention that orthonormal keys give, one token at a time against the
whole, packed sequences against separate ones.
"""
import numpy as np


def _spans(L, cu):
    return [(0, L)] if cu is None else [(int(cu[k]), int(cu[k + 1])) for k in range(len(cu) - 1)]


def step(S, q, k, v, g, beta, scale):
    """One token: S [H, V, K], q, k [G, K], v [H, V], g, beta [H]; returns o [H, V], the new S."""
    rep = v.shape[0] // q.shape[0]
    q, k = np.repeat(q, rep, 0), np.repeat(k, rep, 0)
    S = np.exp(g)[:, None, None] * S
    u = beta[:, None] * (v - np.einsum("hvk,hk->hv", S, k))
    S = S + u[:, :, None] * k[:, None, :]
    return scale * np.einsum("hvk,hk->hv", S, q), S


def forward(q, k, v, g, beta, scale, init=None, cu=None):
    """One row: q, k [L, G, K], v [L, H, V], g, beta [L, H], init [S, H, V, K]; returns o [L, H, V], final [S, H, V, K]."""
    L, H, V = v.shape
    spans = _spans(L, cu)
    final = np.zeros((len(spans), H, V, q.shape[2])) if init is None else np.array(init, np.float64)
    o = np.zeros((L, H, V))
    for s, (t0, t1) in enumerate(spans):
        for t in range(t0, t1):
            o[t], final[s] = step(final[s], q[t], k[t], v[t], g[t], beta[t], scale)
    return o, final


def backward(q, k, v, g, beta, scale, do, init=None, dfinal=None, cu=None):
    """Gradients of sum(do * o) + sum(dfinal * final)."""
    L, H, V = v.shape
    G, K = q.shape[1:]
    rep = H // G
    spans = _spans(L, cu)
    d = dict(dq=np.zeros((L, H, K)), dk=np.zeros((L, H, K)), dv=np.zeros(v.shape), dg=np.zeros(g.shape), dbeta=np.zeros(g.shape),
             dinit=np.zeros((len(spans), H, V, K)))
    for s, (t0, t1) in enumerate(spans):
        S = np.zeros((H, V, K)) if init is None else np.array(init[s], np.float64)
        kept = []
        for t in range(t0, t1):
            kept.append(S)
            S = step(S, q[t], k[t], v[t], g[t], beta[t], scale)[1]
        dS = np.zeros((H, V, K)) if dfinal is None else np.array(dfinal[s], np.float64)
        for t in reversed(range(t0, t1)):
            qt, kt = np.repeat(q[t], rep, 0), np.repeat(k[t], rep, 0)
            faded = np.exp(g[t])[:, None, None] * kept[t - t0]
            err = v[t] - np.einsum("hvk,hk->hv", faded, kt)
            u = beta[t][:, None] * err
            new = faded + u[:, :, None] * kt[:, None, :]
            d["dq"][t] = scale * np.einsum("hvk,hv->hk", new, do[t])
            dS = dS + scale * do[t][:, :, None] * qt[:, None, :]
            du = np.einsum("hvk,hk->hv", dS, kt)
            d["dbeta"][t] = (du * err).sum(-1)
            derr = beta[t][:, None] * du
            d["dv"][t] = derr
            d["dk"][t] = np.einsum("hvk,hv->hk", dS, u) - np.einsum("hvk,hv->hk", faded, derr)
            dfaded = dS - derr[:, :, None] * kt[:, None, :]
            d["dg"][t] = (dfaded * faded).sum((-1, -2))
            dS = np.exp(g[t])[:, None, None] * dfaded
        d["dinit"][s] = dS
    for n in ("dq", "dk"):
        d[n] = d[n].reshape(L, G, rep, K).sum(2)
    return d


# ---- queries and keys
def _turn(x, cos, sin, interleaved, sign):
    """x [..., D], cos, sin [..., R / 2]: the rotation by the angle (sign 1) or the opposite one (-1)."""
    h = cos.shape[-1]
    y = x.copy()
    a, b = (np.arange(0, 2 * h, 2), np.arange(1, 2 * h, 2)) if interleaved else (np.arange(h), np.arange(h, 2 * h))
    y[..., a] = x[..., a] * cos - sign * x[..., b] * sin
    y[..., b] = sign * x[..., a] * sin + x[..., b] * cos
    return y


def _qk_rows(positions, cos, sin):
    """The tokens' rows of the table and which tokens are none (a position outside it)."""
    ok = (positions >= 0) & (positions < len(cos))
    at = np.where(ok, positions, 0)
    return (cos[at][:, None], sin[at][:, None], ok) if len(cos) else (np.ones((len(at), 1, cos.shape[1])), np.zeros((len(at), 1, cos.shape[1])), ok)


def qk_forward(x, w=None, cos=None, sin=None, positions=None, mode="rms", interleaved=False, eps=1e-6):
    """x [L, H, D]; w [D]; cos, sin [rows, R / 2]; positions [L]."""
    m = (x * x).mean(-1, keepdims=True) if mode == "rms" else (x * x).sum(-1, keepdims=True)
    y = x / np.sqrt(m + eps) * (1.0 if w is None else w)
    if cos is None:
        return y
    c, s, ok = _qk_rows(np.arange(len(x)) if positions is None else positions, cos, sin)
    return np.where(ok[:, None, None], _turn(y, c, s, interleaved, 1), 0.0)


def qk_backward(x, dy, w=None, cos=None, sin=None, positions=None, mode="rms", interleaved=False, eps=1e-6):
    """dx [L, H, D] and dw [D]."""
    D = x.shape[-1]
    n = D if mode == "rms" else 1
    rstd = 1 / np.sqrt((x * x).sum(-1, keepdims=True) / n + eps)
    d = np.array(dy, np.float64)
    if cos is not None:
        c, s, ok = _qk_rows(np.arange(len(x)) if positions is None else positions, cos, sin)
        d = np.where(ok[:, None, None], _turn(d, c, s, interleaved, -1), 0.0)
    dw = (d * x * rstd).sum((0, 1))
    d = d * (1.0 if w is None else w)
    return rstd * d - x * rstd ** 3 * (d * x).sum(-1, keepdims=True) / n, dw
