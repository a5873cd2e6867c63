"""The selective scan (a decay rate per channel and state) on the GPU, forward and backward, against the float64
oracle: types, state sizes and channel counts that fill no tile, groups, chunk edges, packed sequences down
to none, strided inputs, long decays, differences, reproducibility and refusals.

Tolerances (relative 2-norm).  bf16 outputs are rounded once to 8 bits: at most 2^-9 each, 2^-8 allowed.  fp32:
a decay has a relative error near 2^-22 and a state remembers some 1 / (dt |A|) <= 100 tokens at these inputs'
typical rates, so 100 x 2^-22 = 2.4e-5; twice that is allowed."""
import numpy as np
import pytest
import torch

from oracle import selective as osel
from state_space_model_scan_gb300 import _lib
from state_space_model_scan_gb300.api import SelectiveScanFunction, selective_scan_backward, selective_scan_forward, selective_scan_step
from helpers import rel_l2

pytestmark = pytest.mark.gpu
TD = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {torch.bfloat16: 2.0 ** -8, torch.float32: 5e-5}


def make(Bt=1, L=33, Dm=33, G=1, N=16, dtype="f32", dt_dtype=None, z=True, D=True, bias=True, init=True, lens=None, seed=0,
         state_dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    if lens is not None:
        Bt, L = 1, sum(lens)
    S = Bt if lens is None else len(lens)
    td = TD[dtype]

    def n(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)
    i = dict(x=n(Bt, L, Dm).to(td), dt=(0.5 * n(Bt, L, Dm)).to(TD[dt_dtype or dtype]),
             A=(-torch.arange(1, N + 1, dtype=torch.float64) * torch.exp(0.2 * n(Dm, N))).float(),
             B=n(Bt, L, G, N).to(td), C=n(Bt, L, G, N).to(td), D=n(Dm).float() if D else None,
             z=n(Bt, L, Dm).to(td) if z else None,
             dt_bias=torch.log(torch.expm1(torch.exp(np.log(1e-3) + torch.rand(Dm, generator=g, dtype=torch.float64) * np.log(100)))).float()
             if bias else None, init=(0.3 * n(S, Dm, N)).to(state_dtype) if init else None,
             cu=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32) if lens is not None else None)
    i["dy"] = n(Bt, L, Dm).to(td)
    i["dfinal"] = n(S, Dm, N).to(state_dtype)
    return i


def dev(i):
    return {k: None if v is None else v.cuda() for k, v in i.items()}


def h(t):
    return None if t is None else t.detach().double().cpu().numpy()


def oracle(i):
    """Forward and backward over all rows, in the tensors' shapes."""
    keys = ("x", "dt", "B", "C", "z", "dy")
    o = {k: h(v) for k, v in i.items() if k != "cu"}
    cu = None if i["cu"] is None else i["cu"].numpy()
    res = {}
    for b in range(i["x"].shape[0]):
        r = {k: None if o[k] is None else o[k][b] for k in keys}
        sts = slice(None) if cu is not None else slice(b, b + 1)
        init = None if o["init"] is None else o["init"][sts]
        y, fin = osel.forward(r["x"], r["dt"], o["A"], r["B"], r["C"], o["D"], r["z"], o["dt_bias"], init, cu)
        g = osel.backward(r["x"], r["dt"], o["A"], r["B"], r["C"], r["dy"], o["D"], r["z"], o["dt_bias"], init,
                          o["dfinal"][sts], cu)
        for k, v in dict(g, y=y[None], final=fin).items():
            if k in ("dx", "ddt", "dB", "dC", "dz"):
                v = v[None]
            if k in ("dA", "dD", "ddt_bias"):
                res[k] = res.get(k, 0) + v
            else:
                res.setdefault(k, []).append(v)
    return {k: np.concatenate(v) if isinstance(v, list) else v for k, v in res.items()}


def kw(d):
    return dict(D=d["D"], z=d["z"], dt_bias=d["dt_bias"], initial_states=d["init"], cu_seqlens=d["cu"])


def gpu(i, keep=True):
    d = dev(i)
    a = (d["x"], d["dt"], d["A"], d["B"], d["C"])
    y, final, kept = selective_scan_forward(*a, keep_chunk_states=True, **kw(d))
    g = selective_scan_backward(*a, d["dy"], dfinal_states=d["dfinal"], chunk_states=kept if keep else None, **kw(d))
    torch.cuda.synchronize()
    return dict(g, y=y, final=final)


def check(i, keep=True):
    got, want = gpu(i, keep), oracle(i)
    for k, v in got.items():
        assert torch.isfinite(v).all(), k
        assert rel_l2(h(v), want[k]) <= TOL[v.dtype], (k, rel_l2(h(v), want[k]))
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 127, 129, 300])
def test_lengths(dtype, L):
    check(make(Bt=2, L=L, Dm=40, dtype=dtype, seed=L))


@pytest.mark.parametrize("N", [1, 4, 13, 16, 17, 32, 40, 64, 65, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_state_sizes(N, dtype):
    check(make(L=70, Dm=37, N=N, dtype=dtype, seed=N))


@pytest.mark.parametrize("Dm,G", [(1, 1), (31, 1), (64, 2), (66, 3), (257, 1), (600, 2)])
def test_channels_and_groups(Dm, G):
    check(make(Bt=2, L=45, Dm=Dm, G=G, seed=Dm))


@pytest.mark.parametrize("drop", ["z", "D", "bias", "init"])
def test_absent_inputs(drop):
    i = make(L=65, Dm=34, **{drop: False})
    got = check(i)
    for name, out in (("z", "dz"), ("D", "dD"), ("bias", "ddt_bias"), ("init", "dinitial_states")):
        assert (out in got) == (name != drop)


def test_wide_batches_take_the_same_values():
    """Many channels in flight (no split over time) and few (split): one batch row against itself alone."""
    i = make(Bt=24, L=200, Dm=512, dtype="bf16", seed=3)
    d = dev(i)
    y, fin = selective_scan_forward(d["x"], d["dt"], d["A"], d["B"], d["C"], **kw(d))
    one = {k: (v[5:6] if k in ("x", "dt", "B", "C", "z", "init") else v) for k, v in d.items()}
    y1, fin1 = selective_scan_forward(one["x"], one["dt"], one["A"], one["B"], one["C"], **kw(one))
    assert rel_l2(h(y[5:6]), h(y1)) <= TOL[torch.bfloat16]
    assert rel_l2(h(fin[5:6]), h(fin1)) <= TOL[torch.float32]


@pytest.mark.parametrize("dtype,dt_dtype", [("bf16", "f32"), ("bf16", "bf16")])
def test_dt_types(dtype, dt_dtype):
    got = check(make(L=90, Dm=48, dtype=dtype, dt_dtype=dt_dtype))
    assert got["ddt"].dtype == TD[dt_dtype]


@pytest.mark.parametrize("lens", [[5], [1, 1, 1], [0, 3, 0, 64, 200, 0], [33, 31, 32, 1, 95], [300, 2, 129]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_sequences(lens, dtype):
    check(make(lens=lens, Dm=35, G=1, N=16, dtype=dtype, seed=len(lens)))


@pytest.mark.parametrize("dtype,N", [("bf16", 16), ("f32", 13), ("f32", 40)])
@pytest.mark.parametrize("shape", [dict(L=1300), dict(L=2561, G=2), dict(Bt=2, L=999), dict(lens=[1, 1200, 0, 257, 900, 3]), dict(lens=[1025])])
def test_long_sequences_of_few_channels(dtype, N, shape):
    """Few channels, many tokens: the sequences are cut into segments whose ends are joined."""
    for keep in (True, False):
        check(make(Dm=6, N=N, dtype=dtype, seed=N, **shape), keep)


def test_packed_is_separate_and_poison_stays_in_its_sequence():
    i = make(lens=[40, 37, 64], Dm=33, N=16, z=True)
    clean = gpu(i)
    for k in ("x", "B", "dt", "z", "dy"):
        i[k][:, 40:77] = float("nan")
    i["init"][1] = float("inf")
    bad = gpu(i)
    for k in ("y", "dx", "ddt", "dB", "dC", "dz"):
        assert torch.equal(bad[k][:, :40], clean[k][:, :40]) and torch.equal(bad[k][:, 77:], clean[k][:, 77:]), k
    assert torch.equal(bad["final"][0], clean["final"][0]) and torch.equal(bad["final"][2], clean["final"][2])
    assert torch.isnan(bad["y"][:, 40:77]).all()


def test_no_tokens():
    i = make(Bt=2, L=0, Dm=33)
    got = gpu(i)
    assert torch.equal(got["final"].cpu(), i["init"]) and torch.equal(got["dinitial_states"].cpu(), i["dfinal"])
    assert got["dA"].abs().max() == 0 and got["dD"].abs().max() == 0 and got["ddt_bias"].abs().max() == 0
    i = make(lens=[0, 0], Dm=33, init=False)
    assert gpu(i)["final"].abs().max() == 0


def test_states_in_16_bits():
    i = make(L=70, Dm=40, state_dtype=torch.bfloat16)
    got = check(i)
    assert got["final"].dtype == got["dinitial_states"].dtype == torch.bfloat16


def test_backward_without_kept_states_is_the_same():
    for i in (make(L=150, Dm=70, dtype="bf16"), make(lens=[70, 0, 129], Dm=40)):
        a, b = gpu(i), gpu(i, keep=False)
        for k in a:
            assert torch.equal(a[k], b[k]), k


def test_runs_repeat_bit_for_bit():
    i = make(Bt=2, L=333, Dm=300, G=2, dtype="bf16")
    a, b = gpu(i), gpu(i)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_strided_views():
    """x, z side by side in one buffer, B and C in another, an odd element offset, dy a slice."""
    i = make(Bt=2, L=77, Dm=31, N=13, dtype="bf16")
    d = dev(i)
    want = gpu(i)
    xz = torch.empty(2, 77, 63, dtype=torch.bfloat16, device="cuda")
    xz[..., 1:32], xz[..., 32:] = d["x"], d["z"]
    bc = torch.empty(2, 77, 1, 27, dtype=torch.bfloat16, device="cuda")
    bc[..., :13], bc[..., 14:] = d["B"], d["C"]
    d.update(x=xz[..., 1:32], z=xz[..., 32:], B=bc[..., :13], C=bc[..., 14:])
    big = torch.zeros(2, 80, 40, dtype=torch.bfloat16, device="cuda")
    big[:, 2:79, 5:36] = d["dy"]
    a = (d["x"], d["dt"], d["A"], d["B"], d["C"])
    y, fin = selective_scan_forward(*a, **kw(d))
    g = selective_scan_backward(*a, big[:, 2:79, 5:36], dfinal_states=d["dfinal"], **kw(d))
    for k, v in dict(g, y=y, final=fin).items():
        assert torch.equal(v, want[k]), k


def test_extreme_steps():
    """Steps whose softplus is its argument, vanishing steps, and decays that underflow to zero."""
    i = make(L=64, Dm=48)
    i["dt"][:, ::3] = 30.0
    i["dt"][:, 1::3] = -40.0
    check(i)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gate_far_below_zero(dtype):
    # Every term has one sign, so that each element keeps its own relative accuracy: the type's rounding and a
    # state's, as in the tolerances above, where silu(z) is as small as e^-40 too.
    i = make(Bt=2, L=40, Dm=48, N=16, dtype=dtype, seed=23)
    for k in ("x", "B", "C", "D", "init", "dy", "dfinal"):
        i[k] = i[k].abs() + 0.125
    i["dfinal"] = torch.zeros_like(i["dfinal"])
    i["z"] = torch.linspace(-40, -2, i["z"].numel(), dtype=torch.float64).reshape(i["z"].shape).to(i["z"].dtype)
    got, want = gpu(i), oracle(i)
    for k in ("y", "dx", "dz"):
        err = np.abs(h(got[k]) - want[k]) / np.abs(want[k])
        assert err.max() < TOL[i["x"].dtype], (k, err.max())
    d = dev(i)
    state = d["init"].clone()
    y = selective_scan_step(state, d["x"][:, 0], d["dt"][:, 0], d["A"], d["B"][:, 0], d["C"][:, 0], D=d["D"], z=d["z"][:, 0],
                            dt_bias=d["dt_bias"])
    err = np.abs(h(y) - want["y"][:, 0]) / np.abs(want["y"][:, 0])
    assert err.max() < TOL[i["x"].dtype], err.max()


def test_autograd_and_another_stream():
    i = make(Bt=2, L=50, Dm=33, dtype="f32")
    d = dev(i)
    want = gpu(i)
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "init")
    v = {k: d[k].clone().requires_grad_() for k in names}
    y, fin = SelectiveScanFunction.apply(*(v[k] for k in names), None)
    ((y * d["dy"]).sum() + (fin * d["dfinal"]).sum()).backward()
    for k in names:
        assert torch.equal(v[k].grad, want["d" + {"init": "initial_states"}.get(k, k)]), k
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = (d["x"], d["dt"], d["A"], d["B"], d["C"])
    y2, fin2 = selective_scan_forward(*a, stream=s, **kw(d))
    g2 = selective_scan_backward(*a, d["dy"], dfinal_states=d["dfinal"], stream=s, **kw(d))
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y2, want["y"]) and torch.equal(fin2, want["final"]) and torch.equal(g2["dA"], want["dA"])


def test_autograd_of_one_output():
    i = make(Bt=2, L=20, Dm=32, dtype="f32", seed=29)
    d = dev(i)
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "init")
    a = (d["x"], d["dt"], d["A"], d["B"], d["C"])
    none = torch.zeros_like(d["dy"]), torch.zeros_like(d["dfinal"])
    for only_y in (True, False):
        v = {k: d[k].clone().requires_grad_() for k in names}
        y, fin = SelectiveScanFunction.apply(*(v[k] for k in names), None)
        (y.sum() if only_y else fin.sum()).backward()      # gradients that are one value, expanded
        want = selective_scan_backward(*a, torch.ones_like(d["dy"]) if only_y else none[0],
                                       dfinal_states=none[1] if only_y else torch.ones_like(d["dfinal"]), **kw(d))
        for k in names:
            assert torch.equal(v[k].grad, want["d" + {"init": "initial_states"}.get(k, k)]), k
    x = d["x"].clone().requires_grad_()
    y, _ = SelectiveScanFunction.apply(x, *a[1:], None, None, None, None, None)
    g, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


@pytest.mark.parametrize("name", ["x", "dt", "A", "B", "C", "D", "z", "dt_bias", "init"])
def test_gradients_against_differences(name):
    """The derivative along a random direction, from two forwards.  The loss sums some 4000 products with fp32 errors
    near 1e-6 of their size, the step is 2^-6 of the inputs' spread: noise / (2 step) near 1e-3 of the
    derivative's scale, curvature as much; 2% allowed."""
    i = make(L=60, Dm=33, N=16, seed=5)
    d = dev(i)
    g = gpu(i)["d" + {"init": "initial_states"}.get(name, name)].double()
    v = torch.randn(d[name].shape, generator=torch.Generator().manual_seed(1)).cuda()
    v = v * (d[name].abs() if name == "A" else 1.0)
    step = 2.0 ** -6

    def loss(sign):
        e = dict(d)
        e[name] = (d[name] + sign * step * v).contiguous()
        y, fin = selective_scan_forward(e["x"], e["dt"], e["A"], e["B"], e["C"], **kw(e))
        return float((y.double() * d["dy"].double()).sum() + (fin.double() * d["dfinal"].double()).sum())
    num = (loss(1) - loss(-1)) / (2 * step)
    ana = float((g * v.double()).sum())
    size = float((g * v.double()).norm())
    assert abs(num - ana) <= 0.02 * max(abs(ana), size), (num, ana)


def test_refusals():
    i = dev(make(L=10, Dm=32))
    a = [i["x"], i["dt"], i["A"], i["B"], i["C"]]
    for k, bad in ((1, i["dt"].double()), (1, i["dt"][:, :5]), (2, i["A"][:, :3]), (2, i["A"].t().contiguous().t()),
                   (3, i["B"].bfloat16()), (3, i["B"][0]), (4, i["C"].cpu()), (0, i["x"].half()),
                   (0, i["x"].transpose(1, 2).contiguous().transpose(1, 2))):
        b = list(a)
        b[k] = bad
        with pytest.raises(ValueError):
            selective_scan_forward(*b)
    with pytest.raises(ValueError):
        selective_scan_forward(*a, initial_states=i["init"][:, :4])
    with pytest.raises(ValueError):
        selective_scan_forward(*a, cu_seqlens=torch.tensor([0, 10], device="cuda"))       # int64
    with pytest.raises(ValueError):
        selective_scan_backward(*a, i["dy"], chunk_states=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(_lib.SSDError) as e:                                              # 33 % 2 != 0
        selective_scan_forward(i["x"], i["dt"], i["A"], i["B"].expand(1, 10, 3, 16).contiguous(),
                               i["C"].expand(1, 10, 3, 16).contiguous())
    assert e.value.code == 1
    j = dev(make(L=10, Dm=32, N=129))
    with pytest.raises(_lib.SSDError) as e:
        selective_scan_forward(j["x"], j["dt"], j["A"], j["B"], j["C"])
    assert e.value.code == 2


def test_autograd_keeps_states_for_gradients_only(monkeypatch):
    """Chunk states are kept where a backward can follow, and not where the caller would rather compute them again."""
    from state_space_model_scan_gb300 import api
    d = dev(make(Bt=2, L=50, Dm=33, dtype="f32"))
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "init")
    args = [d[k] for k in names]
    forward, kept = api.selective_scan_forward, []

    def spy(*a, keep_chunk_states=False, **k):
        kept.append(keep_chunk_states)
        return forward(*a, keep_chunk_states=keep_chunk_states, **k)
    monkeypatch.setattr(api, "selective_scan_forward", spy)
    want, _ = SelectiveScanFunction.apply(*args, None)
    assert kept.pop() is False and not want.requires_grad
    leaves = [t.clone().requires_grad_() for t in args]
    with torch.no_grad():
        y, _ = SelectiveScanFunction.apply(*leaves, None)
    assert kept.pop() is False and not y.requires_grad and torch.equal(y, want)
    grads = []
    for k in (True, False):
        y, fin = SelectiveScanFunction.apply(*leaves, keep_chunk_states=k)
        assert kept.pop() is k
        grads.append(torch.autograd.grad((y * d["dy"]).sum() + (fin * d["dfinal"]).sum(), leaves))
    for a, b in zip(*grads):
        assert torch.equal(a, b)


def whole_case(dtype, N, packed, Dm):
    """A batch with enough (sequence, channel) pairs for the form that does not split sequences over time: 16384, packed
    65536.  Packed lengths: none, one, chunk and tile edges, one long."""
    if not packed:
        return make(Bt=17 if Dm > 512 else 33, L=45, Dm=Dm, N=N, G=1, dtype=dtype, seed=N)
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 64, 0, 70, 3, 129]
    lens += [1 + k % 5 for k in range((65536 + Dm - 1) // Dm - len(lens))]
    return make(lens=lens, Dm=Dm, N=N, dtype=dtype, seed=N)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,Dm", [(16, 1000), (13, 1003), (32, 512), (29, 999), (64, 1000), (128, 1000), (128, 997)])
@pytest.mark.parametrize("packed", [False, True])
def test_sequences_that_are_not_split(dtype, N, Dm, packed):
    """Values, kept states, final states and the gradients that start from the kept states, or recompute them, in that form;
    channels that are taken in fours and channels that are not.  Checked on some of the channels (B and C alone couple
    them: all of dy's other channels are zero)."""
    i = whole_case(dtype, N, packed, Dm)
    cols = np.unique(np.concatenate([np.arange(3), np.linspace(5, Dm - 6, 9).astype(int), np.arange(Dm - 3, Dm)]))
    off = torch.ones(Dm, dtype=torch.bool)
    off[cols] = False
    i["dy"][..., off] = 0
    i["dfinal"][:, off] = 0
    got, again = gpu(i), gpu(i, keep=False)
    part = dict(i)
    for k in ("x", "dt", "z", "dy"):
        part[k] = i[k][..., cols]
    for k in ("A", "D", "dt_bias"):
        part[k] = i[k][cols]
    for k in ("init", "dfinal"):
        part[k] = i[k][:, cols]
    want = oracle(part)
    for k, v in got.items():
        assert torch.isfinite(v).all(), k
        assert torch.equal(v, again[k]), k
        w = h(v)
        if k in ("y", "dx", "ddt", "dz"):
            w = w[..., cols]
        elif k in ("dA", "dD", "ddt_bias"):
            w = w[cols]
        elif k in ("final", "dinitial_states"):
            w = w[:, cols]
        assert rel_l2(w, want[k]) <= TOL[v.dtype], (k, rel_l2(w, want[k]))


@pytest.mark.parametrize("N,G", [(32, 1), (64, 1), (128, 1), (20, 2), (64, 2), (124, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_states_in_wide_rows(N, G, dtype):
    """Channels and states that allow four elements an access, at state sizes above 16."""
    check(make(Bt=2, L=70, Dm=72, N=N, G=G, dtype=dtype, seed=N))


def some_channels(i, cols, want_keys, got):
    """got's values at these channels against the oracle's, which runs on them alone."""
    part = dict(i)
    for k in ("x", "dt", "z", "dy"):
        part[k] = None if i[k] is None else i[k][..., cols]
    for k in ("A", "D", "dt_bias"):
        part[k] = None if i[k] is None else i[k][cols]
    for k in ("init", "dfinal"):
        part[k] = None if i[k] is None else i[k][:, cols]
    want = oracle(part)
    for k in want_keys:
        v = got[k]
        w = h(v)[..., cols] if k in ("y", "dx", "ddt", "dz") else h(v)[cols] if k in ("dA", "dD", "ddt_bias") else h(v)[:, cols]
        assert torch.isfinite(v).all() and rel_l2(w, want[k]) <= TOL[v.dtype], (k, rel_l2(w, want[k]))


@pytest.mark.parametrize("opt", [dict(z=False), dict(D=False, bias=False), dict(init=False), dict(state_dtype=torch.bfloat16),
                                 dict(dt_dtype="f32"), dict(L=1), dict(L=200, Bt=9, Dm=1900)])
@pytest.mark.parametrize("G", [1, 2])
def test_options_where_sequences_are_not_split(opt, G):
    """Absent inputs, types, groups whose channels are taken in fours (and, 501 of them, are not), one token, many tiles."""
    i = make(**dict(dict(Bt=17, L=40, Dm=1002, G=G, dtype="bf16", seed=G), **opt))
    got = gpu(i)
    Dm = i["x"].shape[2]
    cols = np.concatenate([np.arange(4), np.arange(Dm // G - 2, Dm // G), np.arange(Dm - 3, Dm)]) if G == 1 else None
    keys = ["y", "final", "dx", "ddt", "dA"] + [k for k in ("dz", "dD", "ddt_bias", "dinitial_states") if k in got]
    if G == 1:
        some_channels(i, np.unique(cols), keys, got)
    else:                                             # as many channels of each group
        part = np.concatenate([g * (Dm // G) + np.r_[0:3, Dm // G - 3:Dm // G] for g in range(G)])
        some_channels(i, part, keys, got)


def test_poison_stays_in_its_sequence_where_they_are_not_split():
    i = make(lens=[17, 3, 33] + [2] * 64, Dm=1000, dtype="bf16", seed=2)
    clean = gpu(i)
    for k in ("x", "B", "dt", "z", "dy"):
        i[k][:, 20:53] = float("nan")
    i["init"][2] = float("inf")
    bad = gpu(i)
    for k in ("y", "dx", "ddt", "dB", "dC", "dz"):
        assert torch.equal(bad[k][:, :20], clean[k][:, :20]) and torch.equal(bad[k][:, 53:], clean[k][:, 53:]), k
    keep = [s for s in range(67) if s != 2]
    assert torch.equal(bad["final"][keep], clean["final"][keep]) and torch.isnan(bad["y"][:, 20:53]).all()


@pytest.mark.parametrize("shape", [dict(Bt=2, L=37), dict(lens=[1, 0, 40, 17]), dict(L=1300), dict(Bt=33, L=21, Dm=512)])
def test_rates_that_forget_everything(shape):
    """A = -inf, and fp32's lowest value: the state is the last token's term alone, and no step of another rate, sequence end
    or tile end makes a NaN of it.  (Their decays have no gradient; the oracle's rate is -1e30.)"""
    i = make(**dict(dict(Dm=6, N=16), **shape))
    i["A"][:, 3], i["A"][::2, 5] = float("-inf"), torch.finfo(torch.float32).min
    i["dt"].clamp_(min=-3.0)
    got = gpu(i)
    state = i["init"][:1].cuda()
    y = selective_scan_step(state, *(t.cuda().contiguous() for t in (i["x"][:1, 0], i["dt"][:1, 0], i["A"], i["B"][:1, 0], i["C"][:1, 0])),
                            D=i["D"].cuda(), z=i["z"][:1, 0].cuda(), dt_bias=i["dt_bias"].cuda())
    i["A"].clamp_(min=-1e30)
    want = oracle(i)
    for k, v in got.items():
        assert torch.isfinite(v).all(), k
        assert rel_l2(h(v), want[k]) <= TOL[v.dtype], (k, rel_l2(h(v), want[k]))
    assert rel_l2(h(y), want["y"][:1, 0]) <= TOL[torch.float32]
