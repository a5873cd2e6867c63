"""The float64 oracle of the gated delta rule and of the norm and rotation of queries and keys, pinned by what does not share
its code: central differences, closed forms, torch's autograd."""
import numpy as np
import pytest

from oracle import delta as D


def make(L=9, G=2, H=4, K=5, V=3, seed=0, nseq=1):
    r = np.random.default_rng(seed)
    q, k = r.normal(size=(L, G, K)), r.normal(size=(L, G, K))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return dict(q=q, k=k, v=r.normal(size=(L, H, V)), g=-r.uniform(0, 1, (L, H)), beta=r.uniform(0, 1, (L, H)),
                init=r.normal(size=(nseq, H, V, K))), r.normal(size=(L, H, V)), r.normal(size=(nseq, H, V, K))


@pytest.mark.parametrize("cu", [None, [0, 4, 4, 9]])
def test_gradients_are_the_differences(cu):
    x, do, df = make(nseq=1 if cu is None else 3)

    def loss(**y):
        o, f = D.forward(y["q"], y["k"], y["v"], y["g"], y["beta"], 0.7, y["init"], cu)
        return (o * do).sum() + (f * df).sum()
    d = D.backward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.7, do, x["init"], df, cu)
    r = np.random.default_rng(3)
    for name in x:
        way = r.normal(size=x[name].shape)
        e = 1e-6
        want = (loss(**{**x, name: x[name] + e * way}) - loss(**{**x, name: x[name] - e * way})) / (2 * e)
        # central differences of a smooth function: e^2, and 1e-16 / e of cancellation
        assert abs((d["d" + name] * way).sum() - want) <= 1e-8 * max(1.0, abs(want)), name


def test_orthonormal_keys_make_a_table():
    """Keys of an orthonormal set, no decay, beta 1: the state holds each key's last value."""
    K, V = 4, 3
    r = np.random.default_rng(1)
    keys = np.linalg.qr(r.normal(size=(K, K)))[0]
    at = [0, 1, 2, 1, 3, 0]
    v = r.normal(size=(len(at), 1, V))
    k = keys[at][:, None]
    z = np.zeros((len(at), 1))
    o, f = D.forward(k, k, v, z, z + 1, 1.0)
    assert np.allclose(o, v, atol=1e-12)
    assert np.allclose(f[0, 0] @ keys.T, np.stack([v[5, 0], v[3, 0], v[2, 0], v[4, 0]], -1), atol=1e-12)


def test_beta_zero_is_a_fading_readout():
    x, _, _ = make()
    o, f = D.forward(x["q"], x["k"], x["v"], x["g"], 0 * x["beta"], 1.0, x["init"])
    fade = np.exp(np.cumsum(x["g"], 0))
    assert np.allclose(f[0], fade[-1][:, None, None] * x["init"][0])
    assert np.allclose(o[3], np.einsum("hvk,hk->hv", fade[3][:, None, None] * x["init"][0], np.repeat(x["q"][3], 2, 0)))


def test_packed_is_separate():
    x, do, df = make(nseq=3)
    cu = [0, 4, 4, 9]
    o, f = D.forward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.5, x["init"], cu)
    for s in range(3):
        i = slice(cu[s], cu[s + 1])
        os_, fs = D.forward(x["q"][i], x["k"][i], x["v"][i], x["g"][i], x["beta"][i], 0.5, x["init"][s:s + 1])
        assert np.array_equal(o[i], os_) and np.array_equal(f[s], fs[0])


@pytest.mark.parametrize("mode", ["rms", "l2"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_against_complex_numbers_and_differences(mode, interleaved):
    r = np.random.default_rng(2)
    L, H, Dm, R = 5, 3, 10, 6
    x, w, dy = r.normal(size=(L, H, Dm)), r.normal(size=Dm), r.normal(size=(L, H, Dm))
    angle = np.arange(20)[:, None] * np.array([1.0, 0.3, 0.01])
    pos = np.array([3, 19, 0, -1, 7])
    kw = dict(cos=np.cos(angle), sin=np.sin(angle), positions=pos, mode=mode, interleaved=interleaved, eps=1e-3)
    y = D.qk_forward(x, w, **kw)
    n = x / np.sqrt((x ** 2).sum(-1, keepdims=True) / (Dm if mode == "rms" else 1) + 1e-3) * w
    z = n[..., 0:R:2] + 1j * n[..., 1:R:2] if interleaved else n[..., :R // 2] + 1j * n[..., R // 2:R]
    z = z * np.exp(1j * angle[np.maximum(pos, 0)])[:, None]
    turned = np.stack([z.real, z.imag], -1).reshape(L, H, R) if interleaved else np.concatenate([z.real, z.imag], -1)
    want = np.concatenate([turned, n[..., R:]], -1)
    want[3] = 0
    assert np.allclose(y, want, atol=1e-12)
    dx, dw = D.qk_backward(x, dy, w, **kw)
    for name, val, got in (("x", x, dx), ("w", w, dw)):
        way = r.normal(size=val.shape)
        e = 1e-6
        f = lambda s: (D.qk_forward(x + (s * way if name == "x" else 0), w + (s * way if name == "w" else 0), **kw) * dy).sum()  # noqa: E731
        num = (f(e) - f(-e)) / (2 * e)
        assert abs((got * way).sum() - num) <= 1e-7 * max(1.0, abs(num)), name
