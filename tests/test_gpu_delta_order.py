"""The gated delta rule's tensor-core kernels where one part of a block works in memory that another part has used: states that come in,
joins of segments, tiles that leave.  What orders them is in the kernels; here the calls that need it are made often, at the sizes and
addresses that reach it, and compared bit for bit with one another, or with the oracle (tolerances of test_gpu_delta.py)."""
import pytest
import torch

import state_space_model_scan_gb300 as pkg
import test_gpu_delta as t

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("q", "k", "v", "g", "beta")


def step(x, cu=None):
    """One training step, with what the forward kept and without."""
    a = [x[n] for n in NAMES]
    o, f, kept = pkg.gated_delta_forward(*a, initial_states=x["init"], cu_seqlens=cu, state_dtype=F32, keep_chunk_states=True)
    rest = dict(initial_states=x["init"], dfinal_states=x["dfinal"], cu_seqlens=cu)
    d, d2 = pkg.gated_delta_backward(*a, x["do"], chunk_states=kept, **rest), pkg.gated_delta_backward(*a, x["do"], **rest)
    assert all(torch.equal(d[n], d2[n]) for n in d)
    return dict(o=o, f=f, **d)


def check(got, x, cu=None):
    w = t.want(x, x["q"].shape[-1] ** -0.5, None if cu is None else cu.tolist(), back=True)
    assert t.rel(got["o"], w["o"]) <= t.OUT[BF16] and t.rel(got["f"], w["final"]) <= t.OUT[F32]
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert t.rel(got[n], w[n]) <= t.GRAD[BF16], n
    if x["init"] is not None:
        assert t.rel(got["dinitial_states"], w["dinit"]) <= t.GRAD[BF16]


@pytest.mark.parametrize("init", [F32, BF16])
@pytest.mark.parametrize("V,K", [(128, 128), (128, 64), (72, 128)])
def test_states_that_come_in_are_read_before_states_are_kept(V, K, init):
    """A step from given states, to given gradients of the final ones, in a full card (160 chains): their rows pass through the memory
    from which the kept states leave.  The first state that is kept is the one that came in."""
    x = t.make(4, 70, 40, 40, V, K, BF16, F32, None, init, train=True)
    first = step(x)
    for h in (0, 17, 39):                                    # (the oracle goes token by token)
        y = {n: v[:1, :, h:h + 1] if n not in ("init", "dfinal") else v[:1, h:h + 1] for n, v in x.items()}
        check({n: v[:1, :, h:h + 1] if n not in ("f", "dinitial_states") else v[:1, h:h + 1] for n, v in first.items()}, y)
    for _ in range(30):
        again = step(x)
        assert all(torch.equal(first[n], again[n]) for n in first)


def odd_rows(x, names=("q", "k", "v", "do")):
    """The same values in rows that start at odd elements, which no tensor map describes."""
    def odd(v):
        w = torch.full((*v.shape[:2], v[0, 0].numel() + 3), float("nan"), dtype=v.dtype, device="cuda")
        w[..., 1:-2] = v.flatten(2)
        return w[..., 1:-2].unflatten(2, v.shape[2:])
    return {n: odd(v) if n in names else v for n, v in x.items()}


@pytest.mark.parametrize("B,H,L,lens,V,K", [(1, 2, 64 * 33, None, 128, 128), (1, 2, 64 * 33 - 7, None, 72, 48), (2, 2, 64 * 30 + 1, None, 64, 128),
                                            (1, 3, 2176, [1700, 0, 64, 1, 411], 128, 40), (1, 1, 64 * 40, None, 33, 57)])
def test_segments_of_smaller_heads_and_odd_rows(B, H, L, lens, V, K):
    """Chains in up to eleven segments, the last with up to nine joins before it, of states that are a part of 128 x 128."""
    x = t.make(B, L, 1, H, V, K, BF16, F32, lens and len(lens), F32, seed=3, train=True)
    x["g"] *= 0.02                                           # the past matters across segments
    cu = None if lens is None else t.packed(lens)
    first = step(x, cu)
    check(first, x, cu)
    for y in (x, odd_rows(x), odd_rows(x, ("k", "do"))):
        for _ in range(5):
            again = step(y, cu)
            assert all(torch.equal(first[n], again[n]) for n in first)


@pytest.mark.parametrize("names", [("q", "k"), ("k",), ("q", "do"), ("v",)])
def test_tiles_of_gradients_have_left_before_they_are_filled_anew(names):
    """352 chunks and groups on 152 blocks, so that each takes two or three; those of rows that no tensor map describes are filled by
    all of a block's threads, and dK's and dQ's of the chunk before leave from the same memory.  As of aligned rows, bit for bit."""
    x = t.make(1, 64 * 44, 8, 8, 64, 64, BF16, F32, None, F32, train=True)
    first = step(x)
    y = {n: v[:, :, 5:6] if n not in ("init", "dfinal") else v[:, 5:6] for n, v in x.items()}
    check({n: v[:, :, 5:6] if n not in ("f", "dinitial_states") else v[:, 5:6] for n, v in first.items()}, y)
    y = odd_rows(x, names)
    for _ in range(10):
        again = step(y)
        assert all(torch.equal(first[n], again[n]) for n in first)


@pytest.mark.parametrize("B,L,H,V,K,dtype,at", [(2, 200, 4, 128, 128, BF16, 100), (2, 200, 4, 64, 72, BF16, 64), (1, 64 * 30, 2, 128, 128, BF16, 64 * 20 + 63),
                                                (2, 140, 2, 40, 24, F32, 100), (1, 130, 2, 200, 40, BF16, 129)])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta"])
def test_a_token_that_is_not_finite_reaches_its_chunk_and_what_follows(B, L, H, V, K, dtype, at, name):
    """Tokens of earlier chunks, other heads and other rows stay as they are, bit for bit."""
    x = t.make(B, L, 2, H, V, K, dtype, F32, None, F32)
    a = [x[n] for n in NAMES]
    o, f = pkg.gated_delta_forward(*a, initial_states=x["init"])
    y = {n: v.clone() for n, v in x.items()}
    y[name][0, at, 0] = float("nan")
    o2, f2 = pkg.gated_delta_forward(*[y[n] for n in NAMES], initial_states=y["init"])
    own = H // 2 if name in ("q", "k") else 1                # heads of the first group
    assert torch.equal(o2[0, :at // 64 * 64], o[0, :at // 64 * 64])
    assert torch.equal(o2[0, :, own:], o[0, :, own:]) and torch.equal(f2[0, own:], f[0, own:])
    assert torch.equal(o2[1:], o[1:]) and torch.equal(f2[1:], f[1:])
    assert not torch.isfinite(o2[0, at, 0]).all()
    if name != "q":                                          # (a query is read and not kept)
        assert not torch.isfinite(o2[0, at:, 0]).any(-1).any() and not torch.isfinite(f2[0, 0]).all()
