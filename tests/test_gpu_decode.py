"""Decoding on the GPU: the single-token steps on a pool of states, the convolution with a carried window, and 8-bit
snapshots, against the float64 oracle; prompts in pieces and tokens one by one against whole prompts.

Tolerances (relative 2-norm): bf16 results are rounded once, at most 2^-9: 2^-8 allowed.  fp32 steps take a dozen
operations with errors near 2^-22 each: 4e-6 allowed; over a sequence, 5e-5 as for the scan."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import conv1d as oconv
from oracle import selective as osel
from state_space_model_scan_gb300 import _lib
from state_space_model_scan_gb300.api import (conv1d_backward, conv1d_forward, conv1d_prompt, conv1d_step, selective_scan_forward,
                                              selective_scan_step, snapshot_load, snapshot_store, ssd_forward, ssd_step)
from helpers import rel_l2

pytestmark = pytest.mark.gpu
TD = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {torch.bfloat16: 2.0 ** -8, torch.float32: 4e-6}


def h(t):
    return None if t is None else t.detach().double().cpu().numpy()


def gen(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)


def step_inputs(n, H, P, G, N, dtype="f32", state_dtype="f32", selective=False, slots=None, seed=0, dt_dtype=None):
    r = gen(seed)
    td = TD[dtype]
    xs = (n, H) if selective else (n, H, P)
    st = (H, N) if selective else (H, P, N)
    slots = n + 2 if slots is None else slots
    i = dict(x=r(*xs).to(td), dt=(0.5 * r(n, H)).to(TD[dt_dtype or ("f32" if not selective else dtype)]),
             A=-torch.exp(r(H, N) if selective else r(H)).float(), B=r(n, G, N).to(td), C=r(n, G, N).to(td), D=r(H).float(),
             z=r(*xs).to(td), dt_bias=(r(H) - 3.0).float(), state=r(slots, *st).to(TD[state_dtype]))
    i["idx"] = torch.randperm(slots, generator=torch.Generator().manual_seed(seed))[:n].to(torch.int32)
    return i


def run_step(i, selective, drop=(), d=None):
    d = {k: v.cuda() for k, v in i.items()} if d is None else d
    f = selective_scan_step if selective else ssd_step
    opt = {k: (None if k in drop else d[k]) for k in ("D", "z", "dt_bias")}
    y = f(d["state"], d["x"], d["dt"], d["A"], d["B"], d["C"], state_indices=d["idx"], **opt)
    torch.cuda.synchronize()
    return y, d["state"]


def check_step(i, selective, drop=()):
    y, state = run_step(i, selective, drop)
    want = h(i["state"])
    ys = np.zeros(i["x"].shape)
    for k, s in enumerate(i["idx"].tolist()):
        if not 0 <= s < want.shape[0]:
            continue
        opt = {q: None if q in drop else (h(i[q])[k] if q == "z" else h(i[q])) for q in ("D", "z", "dt_bias")}
        want[s], ys[k] = osel.step(want[s], h(i["x"])[k], h(i["dt"])[k], h(i["A"]), h(i["B"])[k], h(i["C"])[k],
                                   opt["D"], opt["z"], opt["dt_bias"])
    assert rel_l2(h(y), ys) <= TOL[y.dtype], rel_l2(h(y), ys)
    assert rel_l2(h(state), want) <= TOL[state.dtype], rel_l2(h(state), want)
    idle = [s for s in range(want.shape[0]) if s not in i["idx"].tolist()]
    assert torch.equal(state[idle].cpu(), i["state"][idle])
    return y, state


@pytest.mark.parametrize("dtype,state_dtype", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("n,H,P,G,N", [(1, 4, 64, 2, 128), (3, 6, 17, 3, 64), (5, 2, 64, 1, 40), (2, 3, 5, 1, 1),
                                       (2, 2, 33, 2, 256), (1, 1, 1, 1, 129), (7, 5, 24, 5, 20), (2, 4, 8, 4, 132)])
def test_ssd_step(n, H, P, G, N, dtype, state_dtype):
    check_step(step_inputs(n, H, P, G, N, dtype, state_dtype, seed=N), False)


@pytest.mark.parametrize("dtype,state_dtype", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("n,Dm,G,N", [(1, 64, 1, 16), (3, 33, 1, 13), (2, 130, 2, 16), (4, 7, 7, 8), (1, 1, 1, 1),
                                      (3, 200, 1, 128), (2, 30, 3, 256), (5, 257, 1, 32)])
def test_selective_scan_step(n, Dm, G, N, dtype, state_dtype):
    check_step(step_inputs(n, Dm, 1, G, N, dtype, state_dtype, selective=True, seed=Dm), True)


@pytest.mark.parametrize("selective", [False, True])
@pytest.mark.parametrize("drop", [("z",), ("D",), ("dt_bias",), ("z", "D", "dt_bias")])
def test_step_absent_inputs(selective, drop):
    check_step(step_inputs(2, 6, 8, 2, 16, selective=selective), selective, drop)


@pytest.mark.parametrize("selective", [False, True])
def test_step_padding_requests(selective):
    """Requests without a slot (negative, or past the pool) answer zeros and touch nothing, whatever they hold."""
    i = step_inputs(5, 4, 8, 2, 16, selective=selective, slots=6)
    i["idx"][1], i["idx"][3] = -1, 6
    i["x"][1] = float("nan")
    i["z"][3] = float("inf")
    y, _ = check_step(i, selective)
    assert y[1].abs().max() == 0 and y[3].abs().max() == 0
    i["idx"][:] = -1
    y, state = run_step(i, selective)
    assert y.abs().max() == 0 and torch.equal(state.cpu(), i["state"])


def test_step_poison_stays_in_its_request():
    i = step_inputs(3, 4, 8, 2, 16)
    clean, st = run_step(i, False)
    i["state"][i["idx"][1]] = float("nan")
    i["x"][1] = float("inf")
    bad, st2 = run_step(i, False)
    assert torch.equal(bad[[0, 2]], clean[[0, 2]]) and torch.isnan(bad[1]).all()
    assert torch.equal(st2[i["idx"][[0, 2]].long()], st[i["idx"][[0, 2]].long()])


def test_step_strided_pool_and_rows():
    """A pool that is a slice of a larger one, x/B/C as views of a conv output row, unaligned rows."""
    H, P, G, N = 4, 8, 2, 16
    i = step_inputs(3, H, P, G, N, "bf16", "f32")
    want, st = run_step(i, False)
    d = {k: v.cuda() for k, v in i.items()}
    row = torch.cat([d["x"].flatten(1), d["B"].flatten(1), d["C"].flatten(1)], 1)
    odd = torch.zeros(3, row.shape[1] + 3, dtype=row.dtype, device="cuda")
    odd[:, 1:-2] = row
    row = odd[:, 1:-2]
    hp, gn = H * P, G * N
    d["x"], d["B"], d["C"] = row[:, :hp].unflatten(1, (H, P)), row[:, hp:hp + gn].unflatten(1, (G, N)), row[:, hp + gn:].unflatten(1, (G, N))
    pool = torch.full((d["state"].shape[0], 2, H, P, N), 7.0, device="cuda")
    pool[:, 1] = d["state"]
    d["state"] = pool[:, 1]
    y, got = run_step(i, False, d=d)
    assert torch.equal(y, want) and torch.equal(got, st) and (pool[:, 0] == 7.0).all()
    # a pool whose rows start off 16 bytes takes single loads: the same values to rounding
    raw = torch.zeros(st.numel() + 1, device="cuda")
    raw[1:] = i["state"].cuda().flatten()
    d["state"] = raw[1:].view(st.shape)
    y, got = run_step(i, False, d=d)
    assert rel_l2(h(y), h(want)) <= TOL[torch.bfloat16] and rel_l2(h(got), h(st)) <= TOL[torch.float32]


def test_steps_continue_a_prompt():
    """The per-head scan's final state, then tokens one by one, against the whole prompt; and so for the selective scan."""
    H, P, G, N, L, cut = 4, 64, 2, 128, 140, 131
    r = gen(3)
    x, z = r(2, L, H, P).float().cuda(), r(2, L, H, P).float().cuda()
    B, C = r(2, L, G, N).float().cuda(), r(2, L, G, N).float().cuda()
    dt, A, D = (0.5 * r(2, L, H)).float().cuda(), -torch.exp(r(H)).float().cuda(), r(H).float().cuda()
    bias = (r(H) - 3).float().cuda()
    y, fin = ssd_forward(x, dt, A, B, C, D=D, z=z, dt_bias=bias, chunk_size=64)
    _, state = ssd_forward(x[:, :cut].contiguous(), dt[:, :cut].contiguous(), A, B[:, :cut].contiguous(),
                           C[:, :cut].contiguous(), D=D, z=z[:, :cut].contiguous(), dt_bias=bias, chunk_size=64)
    for t in range(cut, L):
        yt = ssd_step(state, x[:, t], dt[:, t], A, B[:, t], C[:, t], D=D, z=z[:, t], dt_bias=bias)
        assert rel_l2(h(yt), h(y[:, t])) <= 5e-5
    assert rel_l2(h(state), h(fin)) <= 5e-5
    Dm, N = 100, 16
    x, z, dt = (r(2, L, Dm).float().cuda() for _ in range(3))
    B, C = r(2, L, 1, N).float().cuda(), r(2, L, 1, N).float().cuda()
    A, D, bias = -torch.exp(r(Dm, N)).float().cuda(), r(Dm).float().cuda(), (r(Dm) - 3).float().cuda()
    y, fin = selective_scan_forward(x, dt, A, B, C, D=D, z=z, dt_bias=bias)
    y1, state = selective_scan_forward(x[:, :cut], dt[:, :cut], A, B[:, :cut], C[:, :cut], D=D, z=z[:, :cut], dt_bias=bias)
    assert rel_l2(h(y1), h(y[:, :cut])) <= 5e-5
    for t in range(cut, L):
        yt = selective_scan_step(state, x[:, t], dt[:, t], A, B[:, t], C[:, t], D=D, z=z[:, t], dt_bias=bias)
        assert rel_l2(h(yt), h(y[:, t])) <= 5e-5
    assert rel_l2(h(state), h(fin)) <= 5e-5


# ------------------------------------------------------------------ the convolution's carried window
def conv_inputs(Cn, K, dtype, slots, shape, seed=0, bias=True):
    r = gen(seed)
    return (r(*shape, Cn).to(TD[dtype]), (0.5 * r(Cn, K)).float(), (0.1 * r(Cn)).float() if bias else None,
            r(slots, K - 1, Cn).to(TD[dtype]))


def check_prompt(u, w, bias, win, lens=None, idx=None, has=None, silu=True):
    """lens: packed sequences of row 0, else batch rows."""
    cu = None if lens is None else np.concatenate([[0], np.cumsum(lens)])
    n = u.shape[0] if lens is None else len(lens)
    d = [None if t is None else t.cuda() for t in (u, w, bias, win)]
    out = conv1d_prompt(*d, cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"),
                        state_indices=None if idx is None else torch.tensor(idx, dtype=torch.int32, device="cuda"),
                        has_initial=None if has is None else torch.tensor(has, dtype=torch.uint8, device="cuda"), silu=silu)
    torch.cuda.synchronize()
    want, wwin = np.zeros(u.shape), h(win)
    for s in range(n):
        slot = s if idx is None else idx[s]
        real = 0 <= slot < win.shape[0]
        old = wwin[slot] if real and (has is None or has[s]) else np.zeros(win.shape[1:])
        rows = h(u[s]) if lens is None else h(u[0, cu[s]:cu[s + 1]])
        o, new = osel.conv(rows, h(w), h(bias), old, silu)
        if lens is None:
            want[s] = o
        else:
            want[0, cu[s]:cu[s + 1]] = o
        if real:
            wwin[slot] = new
    assert rel_l2(h(out), want) <= TOL[out.dtype], rel_l2(h(out), want)
    assert np.array_equal(h(d[3]), wwin)          # windows are copied, never computed
    return out, d[3]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("B,L,Cn", [(1, 1, 8), (2, 2, 264), (3, 63, 64), (1, 130, 2048 + 8)])
def test_conv_prompt_rows(dtype, K, B, L, Cn):
    check_prompt(*conv_inputs(Cn, K, dtype, B + 1, (B, L), seed=K))


@pytest.mark.parametrize("lens", [[3, 0, 1, 2, 200, 5, 64, 63, 1], [64, 64, 128], [1] * 20, [0, 0, 7], [66, 2, 60, 4]])
def test_conv_prompt_packed(lens):
    n = len(lens)
    u, w, b, win = conv_inputs(48, 4, "f32", n + 3, (1, sum(lens)), seed=n)
    idx = np.random.RandomState(n).permutation(n + 3)[:n].tolist()
    check_prompt(u, w, b, win, lens, idx, [(k * 7) % 3 != 0 for k in range(n)])


def test_conv_prompt_padding_and_options():
    lens = [5, 1, 70, 2]
    u, w, b, win = conv_inputs(40, 4, "bf16", 3, (1, 78))
    check_prompt(u, w, None, win, lens, [2, -1, 0, 3], silu=False)
    win[1] = float("nan")                          # a fresh sequence does not read its slot
    out, _ = check_prompt(u, w, b, win, lens, [2, 1, 0, -5], [1, 0, 1, 1])
    assert torch.isfinite(out).all()


def test_conv_pieces_and_tokens_make_the_whole():
    """A prompt in pieces of odd lengths, then single tokens: bit for bit the convolution of the whole."""
    u, w, b, win = (t.cuda() for t in conv_inputs(72, 4, "bf16", 2, (2, 150)))
    win.zero_()
    whole = conv1d_forward(u, w, b)
    at = 0
    for n in (1, 2, 3, 65, 64, 7):
        out = conv1d_prompt(u[:, at:at + n], w, b, win)
        assert torch.equal(out, whole[:, at:at + n]), n
        at += n
    for t in range(at, 150):
        assert rel_l2(h(conv1d_step(u[:, t].contiguous(), w, b, win)), h(whole[:, t])) <= TOL[torch.bfloat16]
    assert torch.equal(win, u[:, -3:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("n,Cn", [(1, 8), (3, 1032), (70, 64)])
def test_conv_step(dtype, K, n, Cn):
    u, w, b, win = conv_inputs(Cn, K, dtype, n + 2, (n,), seed=K + n)
    idx = np.random.RandomState(n).permutation(n + 2)[:n]
    if n > 2:
        idx[1] = -1
    d = [t.cuda() for t in (u, w, b, win)]
    out = conv1d_step(*d, state_indices=torch.tensor(idx, dtype=torch.int32, device="cuda"))
    want, wwin = np.zeros(u.shape), h(win)
    for k, s in enumerate(idx):
        o, new = osel.conv(h(u[k:k + 1]), h(w), h(b), wwin[s] if s >= 0 else np.zeros((K - 1, Cn)))
        want[k] = o[0]
        if s >= 0:
            wwin[s] = new
    assert rel_l2(h(out), want) <= TOL[out.dtype]
    assert np.array_equal(h(d[3]), wwin)


# ------------------------------------------------------------------ snapshots
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,mid,N", [(1, (1,), 1), (3, (4, 5), 16), (2, (3, 33), 20), (2, (7,), 128), (1, (5,), 129),
                                     (2, (3,), 256), (1, (9,), 516), (1, (2,), 1024)])
def test_snapshots(dtype, n, mid, N):
    """The stored values and scales bit for bit (one quotient, one product and one rounding each), and what reads back."""
    r = gen(N)
    slots = n + 2
    st = (r(slots, *mid, N) * torch.exp(2 * r(slots, *mid, 1))).to(TD[dtype])
    st[0, ..., 0, :] = 0.0
    src, snap, dst = ([(k + o) % slots for k in range(n)] for o in (0, 1, 2))
    q = torch.full((slots, *mid, N), 55, dtype=torch.int8, device="cuda")
    sc = torch.full((slots, *mid), 5.0, device="cuda")
    back = torch.full(st.shape, 3.0, dtype=st.dtype, device="cuda")
    I = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    snapshot_store(st.cuda(), q, sc, state_indices=I(src), slots=I(snap))
    snapshot_load(q, sc, back, slots=I(snap), state_indices=I(dst))
    torch.cuda.synchronize()
    wq, ws = osel.snapshot(st.float().numpy())
    for k in range(n):
        assert np.array_equal(q[snap[k]].cpu().numpy(), wq[src[k]]) and np.array_equal(sc[snap[k]].cpu().numpy(), ws[src[k]])
        val = torch.from_numpy(wq[src[k]].astype(np.float32) * ws[src[k]][..., None]).to(st.dtype)
        assert torch.equal(back[dst[k]].cpu(), val)
        err = np.abs(val.double().numpy() - h(st[src[k]]))
        lim = ws[src[k]][..., None] * (0.5 + 1e-5) + np.abs(h(st[src[k]])) * (2.0 ** -8 if dtype == "bf16" else 1e-6)
        assert (err <= lim).all()
    for s in set(range(slots)) - set(snap):
        assert (q[s] == 55).all() and (sc[s] == 5.0).all()
    for s in set(range(slots)) - set(dst):
        assert (back[s] == 3.0).all()


@pytest.mark.parametrize("N", [16, 13])
def test_snapshot_rows_that_cannot_be_kept(N):
    """A NaN or an infinity makes its row read back as NaN and no other; tiny rows become zeros."""
    st = torch.randn(1, 6, N, generator=torch.Generator().manual_seed(0)).cuda()
    st[0, 1, 3], st[0, 2, 0], st[0, 3, 5] = float("nan"), float("inf"), float("-inf")
    st[0, 4] *= 1e-32
    q, sc, back = torch.empty(1, 6, N, dtype=torch.int8, device="cuda"), torch.empty(1, 6, device="cuda"), torch.empty_like(st)
    snapshot_store(st, q, sc)
    snapshot_load(q, sc, back)
    assert torch.isnan(back[0, 1:4]).all() and (back[0, 4] == 0).all() and sc[0, 4] == 0
    assert torch.isfinite(back[0, [0, 5]]).all()
    # pairs with an index out of range are skipped
    before = back.clone()
    snapshot_load(q, sc, back, slots=torch.tensor([0, 1, -1], dtype=torch.int32, device="cuda"),
                  state_indices=torch.tensor([1, 0, 0], dtype=torch.int32, device="cuda"))
    assert torch.equal(torch.nan_to_num(back, 9.0), torch.nan_to_num(before, 9.0))


def test_graph_capture_and_streams():
    """The steps allocate nothing but their outputs: a captured decode step replays on the pool's current states."""
    i = step_inputs(2, 4, 8, 2, 16)
    d = {k: v.cuda() for k, v in i.items()}
    eager = d["state"].clone()
    for _ in range(3):
        want = ssd_step(eager, d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"], dt_bias=d["dt_bias"], state_indices=d["idx"])
    pool = d["state"].clone()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            y = ssd_step(pool, d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"], dt_bias=d["dt_bias"], state_indices=d["idx"])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(pool, eager)
    pool = d["state"].clone()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        y = ssd_step(pool, d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"], dt_bias=d["dt_bias"], state_indices=d["idx"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want) and torch.equal(pool, eager)


def test_refusals():
    i = {k: v.cuda() for k, v in step_inputs(2, 4, 8, 2, 16).items()}
    a = dict(state=i["state"], x=i["x"], dt=i["dt"], A=i["A"], B=i["B"], C=i["C"])
    for k, bad in (("dt", i["dt"].bfloat16()), ("dt", i["dt"][:, :2]), ("A", i["A"][:3]), ("B", i["B"].bfloat16()),
                   ("C", i["C"][..., :8]), ("state", i["state"][..., :8]), ("state", i["state"].half()),
                   ("state", i["state"].transpose(2, 3)), ("x", i["x"].cpu()), ("state", i["state"][:1])):
        with pytest.raises(ValueError):
            ssd_step(**dict(a, **{k: bad}))
    with pytest.raises(ValueError):
        ssd_step(**a, state_indices=i["idx"].long())
    with pytest.raises(ValueError):
        ssd_step(**a, state_indices=i["idx"][:1])
    with pytest.raises(ValueError):
        selective_scan_step(i["state"], i["x"], i["dt"], i["A"], i["B"], i["C"])
    big = {k: v.cuda() for k, v in step_inputs(1, 2, 2, 1, 257).items()}
    with pytest.raises(_lib.SSDError) as e:
        ssd_step(big["state"], big["x"], big["dt"], big["A"], big["B"], big["C"])
    assert e.value.code == 2
    u, w, b, win = (t.cuda() for t in conv_inputs(16, 4, "f32", 2, (2, 5)))
    for args in ((u, w, b, win[:, :2]), (u, w, b, win.bfloat16()), (u, w, b, win[:1]), (u, w[:8], b, win), (u[0], w, b, win)):
        with pytest.raises(ValueError):
            conv1d_prompt(*args)
    with pytest.raises(ValueError):
        conv1d_prompt(u, w, b, win, has_initial=torch.ones(2, device="cuda"))
    with pytest.raises(_lib.SSDError) as e:
        conv1d_step(u[:, 0, :12].contiguous(), w[:12].contiguous(), b[:12], torch.zeros(2, 3, 12, device="cuda"))
    assert e.value.code == 2
    st = i["state"]
    q, sc = torch.empty(st.shape, dtype=torch.int8, device="cuda"), torch.empty(st.shape[:-1], device="cuda")
    for args in ((st, q[:, :2], sc), (st, q.float(), sc), (st, q, sc[:, 0]), (st.double(), q, sc), (st, q[:1], sc[:1])):
        with pytest.raises(ValueError):
            snapshot_store(*args)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_conv_silu_far_below_zero(dtype):
    """Each element's own relative accuracy where silu is as small as e^-40.  All products of an output have one sign, so
    the sum before the activation is off by some 2^-22 of 40, 1e-5, and its silu by as much of itself; a result's rounding:
    2^-8 allowed in bf16, 5e-5 in fp32.  So for the gradients: below -2 silu' keeps its sign too."""
    Cn, K, L = 64, 4, 150
    r = gen(41)
    w = (0.5 + r(Cn, K).abs()).float()
    w = w / w.sum(1, keepdim=True)
    depth = torch.linspace(2.5, 40, Cn, dtype=torch.float64)
    u = (-depth * (1 + 0.02 * r(1, L, Cn))).to(TD[dtype])
    win = (-depth * (1 + 0.02 * r(1, K - 1, Cn))).to(TD[dtype])
    dout = (r(1, L, Cn).abs() + 0.125).to(TD[dtype])
    lim = 2.0 ** -8 if dtype == "bf16" else 5e-5

    def close(got, want, what):
        err = np.abs(h(got) - want) / np.abs(want)
        assert err.max() <= lim, (what, err.max())
    ud, wd, pool, dd = u.cuda(), w.cuda(), win.cuda(), dout.cuda()
    want, _ = osel.conv(h(u[0]), h(w), None, h(win[0]))
    close(conv1d_prompt(ud, wd, None, pool.clone())[0], want, "prompt")
    steps = [conv1d_step(ud[:, t], wd, None, pool)[0] for t in range(L)]
    close(torch.stack(steps), want, "step")
    # from zeros the first sums are smaller, of one sign all the same
    want, _ = oconv.forward(h(u[0]), h(w), None)
    close(conv1d_forward(ud, wd, None)[0], want, "forward")
    bias = -2.0 * torch.ones(Cn)
    du, dw, db = conv1d_backward(ud, wd, dd, bias.cuda())
    odu, odw, odb = oconv.backward(h(u[0]), h(w), h(dout[0]), h(bias))
    close(du[0], odu, "du")
    close(dw, odw, "dw")
    close(db, odb, "db")


def test_selective_step_past_32_bits():
    """B and C of 2^23 + 8 groups of 256 states: the last groups' elements lie past 2^31 (22 GB in all)."""
    Dm, N = (1 << 23) + 8, 256
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    state, B, C = r(1, Dm, N), r(1, Dm, N), r(1, Dm, N)
    A = torch.empty(Dm, N, device="cuda").uniform_(-2, -0.5, generator=g)
    x, dt = r(1, Dm), r(1, Dm)
    parts = (slice(0, 4), slice((1 << 23) - 4, (1 << 23) + 8))
    before = [h(state[0, p]) for p in parts]
    y = selective_scan_step(state, x, dt, A, B, C)
    for p, old in zip(parts, before):
        new, want = osel.step(old, h(x[0, p]), h(dt[0, p]), h(A[p]), h(B[0, p]), h(C[0, p]))
        assert rel_l2(h(y[0, p]), want) <= TOL[torch.bfloat16] and rel_l2(h(state[0, p]), new) <= TOL[torch.bfloat16]


def test_step_on_an_empty_pool():
    """No slots: every request is padding.  Through C a single request's rows have no stride to speak of."""
    i = {k: v.cuda() for k, v in step_inputs(1, 4, 8, 2, 16).items()}
    for stride in (0, 32, 40):
        y = torch.full((1, 32), 7.0, device="cuda")
        p = _lib.StepProblem(1, 0, 4, 8, 2, 16, 0, stride, 0, 0, 0, 0, stride, 0, 0, 0, 0)
        a = [i[k].data_ptr() for k in ("state", "idx", "x", "dt", "A", "B", "C")]
        assert _lib.load().ssd_step(ctypes.byref(p), *a, None, None, None, y.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        assert (y == 0).all()
    y = ssd_step(i["state"][:0], *(i[k] for k in ("x", "dt", "A", "B", "C")), state_indices=i["idx"])
    assert y.shape == i["x"].shape and (y == 0).all()


def in_place_calls():
    """(name, tensors that the call writes, call)"""
    i = {k: v.cuda() for k, v in step_inputs(2, 4, 8, 2, 16).items()}
    j = {k: v.cuda() for k, v in step_inputs(2, 4, 8, 2, 16, selective=True).items()}
    u, w, b, win = (t.cuda() for t in conv_inputs(16, 4, "f32", 2, (2, 5)))
    st = i["state"].clone()
    q, sc = torch.zeros(st.shape, dtype=torch.int8, device="cuda"), torch.zeros(st.shape[:-1], device="cuda")
    a = ("x", "dt", "A", "B", "C")
    return [("ssd_step", [i["state"]], lambda: ssd_step(i["state"], *(i[k] for k in a), state_indices=i["idx"])),
            ("selective_scan_step", [j["state"]], lambda: selective_scan_step(j["state"], *(j[k] for k in a), state_indices=j["idx"])),
            ("conv1d_prompt", [win], lambda: conv1d_prompt(u, w, b, win)),
            ("conv1d_step", [win], lambda: conv1d_step(u[:, 0].contiguous(), w, b, win)),
            ("snapshot_store", [q, sc], lambda: snapshot_store(st, q, sc)),
            ("snapshot_load", [st], lambda: snapshot_load(q, sc, st))]


@pytest.mark.parametrize("k", range(6))
def test_updates_in_place_are_seen_by_autograd(k):
    """What a call writes counts as changed: a graph that saved it for its backward says so."""
    name, written, call = in_place_calls()[k]
    before = [t._version for t in written]
    leaf = torch.ones((), device="cuda", requires_grad=True)
    graph = (leaf * written[-1]).sum()
    call()
    assert all(t._version > v for t, v in zip(written, before)), name
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        graph.backward()


def test_pools_made_in_inference_mode():
    for k in range(6):
        with torch.inference_mode():
            _, written, call = in_place_calls()[k]
        call()
        with torch.inference_mode():
            call()


@pytest.mark.parametrize("dtype,state_dtype", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("n,H,P,G,N", [(8, 3, 64, 1, 128), (9, 4, 33, 2, 64), (17, 2, 5, 1, 40), (33, 2, 64, 1, 16), (8, 2, 67, 2, 8),
                                       (9, 3, 64, 3, 4), (8, 2, 130, 1, 256), (10, 2, 24, 2, 132)])
def test_ssd_step_of_many_requests(n, H, P, G, N, dtype, state_dtype):
    """Eight rows in flight a thread (from eight requests on): rows that fill no block, rows of fewer lanes than rows in
    flight, padding requests."""
    i = step_inputs(n, H, P, G, N, dtype, state_dtype, seed=N + n)
    check_step(i, False)
    i["idx"][2], i["idx"][n - 1] = -1, i["state"].shape[0]
    y, _ = check_step(i, False)
    assert y[2].abs().max() == 0 and y[n - 1].abs().max() == 0
    check_step(i, False, ("z", "D"))
