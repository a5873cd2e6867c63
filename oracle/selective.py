"""The selective scan, its single-token step, the convolution with a carried window and 8-bit state snapshots in
float64 -- TEST INFRASTRUCTURE ONLY.

Selective scan: per channel d (B/C group g = d // (channels // groups)) and state n,

    dt = softplus(dt_raw + dt_bias),  h <- exp(dt A[d, n]) h + dt x B[g, n],  y = (sum_n C[g, n] h + D x) silu(z)

one token after the other; the backward is the exact adjoint of that loop.  Pinned by
tests/test_oracle_selective.py: central differences of every gradient, a closed form, the per-head scan where
all channels of a head share a rate, and one token at a time against the whole sequence.
"""
import numpy as np


def softplus(v):
    return np.logaddexp(0.0, v)


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def _spans(L, cu):
    return [(0, L)] if cu is None else [(int(cu[k]), int(cu[k + 1])) for k in range(len(cu) - 1)]


def forward(x, dt, A, B, C, D=None, z=None, dt_bias=None, init=None, cu=None):
    """One row: x, dt, z [L, Dm]; B, C [L, G, N]; A [Dm, N]; init [S, Dm, N]; returns y [L, Dm], final [S, Dm, N]."""
    L, Dm = x.shape
    N = A.shape[1]
    grp = np.arange(Dm) // (Dm // B.shape[1])
    dts = softplus(dt + (0.0 if dt_bias is None else dt_bias))
    spans = _spans(L, cu)
    final = np.zeros((len(spans), Dm, N)) if init is None else np.array(init, np.float64)
    y = np.zeros((L, Dm))
    for s, (t0, t1) in enumerate(spans):
        h = final[s].copy()
        for t in range(t0, t1):
            h = np.exp(dts[t][:, None] * A) * h + (dts[t] * x[t])[:, None] * B[t][grp]
            y[t] = (h * C[t][grp]).sum(1)
        final[s] = h
    if D is not None:
        y = y + D * x
    if z is not None:
        y = y * z * sigmoid(z)
    return y, final


def backward(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, init=None, dfinal=None, cu=None):
    """Gradients of sum(dy y) + sum(dfinal final) as a dict (names of the inputs with a d before)."""
    L, Dm = x.shape
    G, N = B.shape[1:]
    grp = np.arange(Dm) // (Dm // G)
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    dts = softplus(raw)
    spans = _spans(L, cu)
    before = np.zeros((L, Dm, N))
    ysum = np.zeros((L, Dm))
    for s, (t0, t1) in enumerate(spans):
        h = np.zeros((Dm, N)) if init is None else np.array(init[s], np.float64)
        for t in range(t0, t1):
            before[t] = h
            h = np.exp(dts[t][:, None] * A) * h + (dts[t] * x[t])[:, None] * B[t][grp]
            ysum[t] = (h * C[t][grp]).sum(1)
    Dv = np.zeros(Dm) if D is None else D
    out = dict(dA=np.zeros((Dm, N)), dB=np.zeros((L, G, N)), dC=np.zeros((L, G, N)))
    if z is not None:
        sg = sigmoid(z)
        out["dz"] = dy * (ysum + Dv * x) * sg * (1.0 + z * (1.0 - sg))
        dy = dy * z * sg
    dx, ddt = np.zeros((L, Dm)), np.zeros((L, Dm))
    dinit = np.zeros((len(spans), Dm, N))
    for s, (t0, t1) in enumerate(spans):
        g = np.zeros((Dm, N)) if dfinal is None else np.array(dfinal[s], np.float64)
        for t in range(t1 - 1, t0 - 1, -1):
            Bv, Cv = B[t][grp], C[t][grp]
            a = np.exp(dts[t][:, None] * A)
            u = dts[t] * x[t]
            g = g + dy[t][:, None] * Cv
            np.add.at(out["dC"][t], grp, (a * before[t] + u[:, None] * Bv) * dy[t][:, None])
            np.add.at(out["dB"][t], grp, g * u[:, None])
            e = (g * Bv).sum(1)
            q = g * a * before[t]
            dx[t] = e * dts[t]
            ddt[t] = e * x[t] + (q * A).sum(1)
            out["dA"] += q * dts[t][:, None]
            g = g * a
        dinit[s] = g
    out["dx"] = dx + Dv * dy
    out["ddt"] = ddt * sigmoid(raw)
    out["dD"] = (dy * x).sum(0)
    out["ddt_bias"] = out["ddt"].sum(0)
    out["dinitial_states"] = dinit
    return out


def step(h, x, dt, A, B, C, D=None, z=None, dt_bias=None):
    """One token of one request.  Per channel: h [Dm, N], A [Dm, N], x, dt [Dm]; per head: h [H, P, N], A, dt [H], x
    [H, P]; B, C [G, N].  Returns the new state and y."""
    H = A.shape[0]
    grp = np.arange(H) // (H // B.shape[0])
    dts = softplus(dt + (0.0 if dt_bias is None else dt_bias))
    if A.ndim == 1:
        h = np.exp(dts * A)[:, None, None] * h + (dts[:, None] * x)[:, :, None] * B[grp][:, None, :]
        y = (h * C[grp][:, None, :]).sum(2)
        y = y if D is None else y + D[:, None] * x
    else:
        h = np.exp(dts[:, None] * A) * h + (dts * x)[:, None] * B[grp]
        y = (h * C[grp]).sum(1)
        y = y if D is None else y + D * x
    return h, (y if z is None else y * z * sigmoid(z))


def conv(u, w, bias, window, silu=True):
    """One sequence: u [n, channels] after window [K - 1, channels]; returns out and the new window."""
    K = w.shape[1]
    rows = np.concatenate([window, u])
    out = np.zeros(u.shape) + (0.0 if bias is None else bias)
    for k in range(K):
        out = out + w[:, k] * rows[k:k + u.shape[0]]
    return (out * sigmoid(out) if silu else out), rows[rows.shape[0] - (K - 1):]


def snapshot(h):
    """(q, scale) of rows [..., N] in the arithmetic the definition names, each operation rounded to fp32."""
    h = np.asarray(h, np.float32)
    with np.errstate(all="ignore"):
        m = np.abs(h).max(-1)
        ok = (m >= np.float32(1e-30)) & np.isfinite(m)
        inv = np.where(ok, (np.float32(1) / m) * np.float32(127), np.float32(0)).astype(np.float32)
        scale = np.where(ok, m / np.float32(127), np.where(np.isfinite(m), np.float32(0), np.float32("nan")))
        q = np.where(ok[..., None], np.rint(h * inv[..., None]), 0).astype(np.int8)
    return q, scale.astype(np.float32)
