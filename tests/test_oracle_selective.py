"""Pins of the float64 oracle of the selective scan, its step, the carried convolution and the snapshots (CPU)."""
import numpy as np
import pytest

from oracle import conv1d as oc
from oracle import selective as osel
from oracle import sequential


def make(L=7, Dm=6, G=2, N=3, S=1, seed=0):
    r = np.random.RandomState(seed)
    i = dict(x=r.randn(L, Dm), dt=0.5 * r.randn(L, Dm), A=-np.exp(r.randn(Dm, N)), B=r.randn(L, G, N), C=r.randn(L, G, N))
    o = dict(D=r.randn(Dm), z=r.randn(L, Dm), dt_bias=r.randn(Dm) - 1.0, init=r.randn(S, Dm, N))
    return i, o, r.randn(L, Dm), r.randn(S, Dm, N)


def test_closed_form_of_one_channel():
    """Constant inputs and one state: a geometric series."""
    n, dt, A = 9, 0.3, -1.7
    raw = np.log(np.expm1(dt))
    one = np.ones((n, 1))
    y, fin = osel.forward(2.0 * one, raw * one, np.array([[A]]), np.ones((n, 1, 1)), np.ones((n, 1, 1)))
    a = np.exp(dt * A)
    want = dt * 2.0 * (1 - a ** np.arange(1, n + 1)) / (1 - a)
    assert np.allclose(y[:, 0], want, rtol=1e-13) and np.isclose(fin[0, 0, 0], want[-1], rtol=1e-13)


def test_one_rate_per_head_is_the_per_head_scan(oracle_lib):
    H, P, G, N, L = 4, 3, 2, 5, 20
    r = np.random.RandomState(1)
    x, dt, A = r.randn(L, H, P), 0.5 * r.randn(L, H), -np.exp(r.randn(H))
    B, C, D, z, bias = r.randn(L, G, N), r.randn(L, G, N), r.randn(H), r.randn(L, H, P), r.randn(H)
    init = r.randn(1, H, P, N)
    y, fin = sequential.forward(x, dt, A, B, C, D=D, z=z, dt_bias=bias, init=init, cu=[0, L])
    rep = lambda v: np.repeat(v, P, -1)  # noqa: E731
    ys, fs = osel.forward(x.reshape(L, -1), rep(dt), np.repeat(np.repeat(A, P)[:, None], N, 1), B, C, rep(D),
                          z.reshape(L, -1), rep(bias), init.reshape(1, H * P, N))
    assert np.allclose(ys, y.reshape(L, -1), rtol=1e-11) and np.allclose(fs.reshape(fin.shape), fin, rtol=1e-11)
    h, outs = init[0], []
    for t in range(L):
        h, o = osel.step(h, x[t], dt[t], A, B[t], C[t], D, z[t], bias)
        outs.append(o)
    assert np.allclose(np.stack(outs), y, rtol=1e-11) and np.allclose(h, fin[0], rtol=1e-11)


def test_steps_are_the_scan_and_packed_is_separate():
    i, o, _, _ = make(S=3, L=9)
    cu = [0, 4, 4, 9]
    y, fin = osel.forward(**i, **o, cu=cu)
    assert np.array_equal(fin[1], o["init"][1])
    for s in range(3):
        h, t0 = o["init"][s], cu[s]
        for t in range(t0, cu[s + 1]):
            h, yt = osel.step(h, i["x"][t], i["dt"][t], i["A"], i["B"][t], i["C"][t], o["D"], o["z"][t], o["dt_bias"])
            assert np.allclose(yt, y[t], rtol=1e-12)
        assert np.allclose(h, fin[s], rtol=1e-12)


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 7]])
def test_gradients_are_central_differences(cu):
    i, o, dy, df = make(S=1 if cu is None else 3)
    g = osel.backward(**i, dy=dy, **o, dfinal=df, cu=cu)

    def loss(**k):
        y, fin = osel.forward(**{**i, **o, **k}, cu=cu)
        return (y * dy).sum() + (fin * df).sum()
    r = np.random.RandomState(2)
    for name in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "init"):
        v = (i if name in i else o)[name]
        d = r.randn(*v.shape)
        num = (loss(**{name: v + 1e-6 * d}) - loss(**{name: v - 1e-6 * d})) / 2e-6
        ana = (g["dinitial_states" if name == "init" else "d" + name] * d).sum()
        assert abs(num - ana) <= 1e-6 * max(1.0, abs(ana)), name


def test_carried_convolution_is_the_whole_ones():
    r = np.random.RandomState(3)
    u, w, b = r.randn(11, 4), r.randn(4, 4), r.randn(4)
    want, _ = oc.forward(u, w, b)
    win = np.zeros((3, 4))
    for t0, t1 in ((0, 1), (1, 3), (3, 3), (3, 10), (10, 11)):
        out, win = osel.conv(u[t0:t1], w, b, win)
        assert np.allclose(out, want[t0:t1], rtol=1e-13)
    assert np.array_equal(win, u[-3:])


def test_snapshot_rows():
    h = np.array([[0.0, 0.0, 0.0], [1.0, -2.0, 0.5], [1e-31, 0.0, -1e-32], [np.inf, 1.0, 0.0], [np.nan, 1.0, 2.0]])
    q, s = osel.snapshot(h)
    assert (q[0] == 0).all() and s[0] == 0 and (q[2] == 0).all() and s[2] == 0
    assert q[1].tolist() == [64, -127, 32] and s[1] == np.float32(2) / np.float32(127)     # 63.5 and 31.75: half to even
    assert np.isnan(s[3:]).all() and (q[3:] == 0).all()
