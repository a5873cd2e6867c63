"""The gated delta rule where a call could go wrong: chains cut into segments or spread over more blocks against the same heads in a
full card, offsets past 32 bits, graphs that run at once, cu_seqlens that make no sense.

Tolerances (relative 2-norm).  The same chunks in segments: states in fp32 or as two bf16 terms (2^-17 each), joined at most thirty
times, 30 x 2^-17 / sqrt(3) = 1.3e-4 if all were of one sign and the past were never forgotten, sqrt(30) 2^-17 = 4.2e-5 of random sign;
bf16 outputs of the two differ where a value falls on the other side of a rounding: 2^-8 / sqrt(3) = 2.3e-3 at most, gradients, sums
of four such products, twice that.  fp32: the order of sums of up to 64 terms, 64 x 2^-24 = 4e-6, over three products in a row: 1.2e-5."""
import pytest
import torch

import state_space_model_scan_gb300 as pkg

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dinitial_states")


def rel(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm().clamp(min=1e-300))


def inputs(B, L, H, V, K, dtype, seqs=None, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    unit = lambda t: torch.nn.functional.normalize(t, dim=-1)  # noqa: E731
    return dict(q=unit(r(B, L, H, K)).to(dtype), k=unit(r(B, L, H, K)).to(dtype), v=r(B, L, H, V).to(dtype),
                g=-0.05 * torch.rand(B, L, H, generator=g, device="cuda"), beta=torch.rand(B, L, H, generator=g, device="cuda"),
                do=r(B, L, H, V).to(dtype), init=0.1 * r(seqs or B, H, V, K), df=0.1 * r(seqs or B, H, V, K))


def run(x, cu=None):
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, f, kept = pkg.gated_delta_forward(*a, initial_states=x["init"], cu_seqlens=cu, keep_chunk_states=True)
    o2, f2 = pkg.gated_delta_forward(*a, initial_states=x["init"], cu_seqlens=cu)
    assert torch.equal(o, o2) and torch.equal(f, f2)
    d = pkg.gated_delta_backward(*a, x["do"], initial_states=x["init"], dfinal_states=x["df"], cu_seqlens=cu, chunk_states=kept)
    return dict(o=o, f=f, **d)


def times(x, n):
    """The same heads n times over: a card full of chains, which are not cut."""
    return {k: v.repeat_interleave(n, 1 if k in ("init", "df") else 2) for k, v in x.items()}


@pytest.mark.parametrize("B,H,L,lens", [(1, 2, 64 * 21, None), (1, 1, 64 * 40 + 1, None), (1, 3, 64 * 33 + 63, None), (2, 1, 64 * 50, None),
                                        (1, 32, 64 * 40 - 5, None), (1, 2, 3000, [1700, 0, 64, 1, 1235]), (1, 1, 2600, [1, 2599]),
                                        (1, 4, 64 * 24, [64 * 12, 64 * 12])])
def test_segments_are_the_whole(B, H, L, lens):
    x = inputs(B, L, H, 128, 128, BF16, lens and len(lens))
    cu = None if lens is None else torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    n = -(-160 // ((len(lens) if lens else B) * H))
    a, b = run(x, cu), run(times(x, n), cu)
    for name in a:
        whole = b[name][:, ::n] if name in ("f", "dinitial_states") else b[name][:, :, ::n]
        assert rel(a[name], whole) <= (4.2e-5 if name == "f" else 2.3e-3 if name == "o" else 4.6e-3), name


@pytest.mark.parametrize("B,H,L,V,K", [(1, 1, 200, 96, 64), (3, 3, 130, 96, 64), (2, 6, 77, 72, 48), (1, 9, 65, 128, 128), (1, 2, 129, 33, 200), (1, 5, 64, 256, 33),
                                       (1, 1, 1, 1, 1)])
def test_few_heads_in_fp32_are_as_many(B, H, L, V, K):
    """Few values a block, gradients in shares of the keys: as in a full card."""
    x = inputs(B, L, H, V, K, F32)
    n = -(-400 // (B * H))
    a, b = run(x), run(times(x, n))
    for name in a:
        assert rel(a[name], b[name][:, ::n] if name in ("f", "dinitial_states") else b[name][:, :, ::n]) <= 1.2e-5, name


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_offsets_past_32_bits(dtype):
    L, step = 66, 1 << 26                                                  # the last token lies 4.3e9 elements on
    x = inputs(1, L, 2, 64, 64, dtype)
    base = torch.empty(L * step, dtype=dtype, device="cuda")
    far = dict(x)
    for i, n in enumerate(("q", "k", "v", "do")):
        far[n] = base.as_strided(x[n].shape, (L * step, step, 64, 1), 1024 * i)
        far[n].copy_(x[n])
    a, b = run(x), run(far)
    assert all(torch.equal(a[n], b[n]) for n in a)
    q, k = pkg.qk_norm_forward(far["q"], far["k"], mode="l2")
    q1, k1 = pkg.qk_norm_forward(x["q"], x["k"], mode="l2")
    assert torch.equal(q, q1) and torch.equal(k, k1)


@pytest.mark.parametrize("H,L", [(2, 64 * 24), (4, 200)])
def test_two_graphs_at_once(H, L):
    """Two captured steps of the same inputs (a reused one included), replayed on two streams at once, a hundred times."""
    x = inputs(1, L, H, 128, 128, BF16)
    want = run(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(side):
        run(x)
        torch.cuda.synchronize()
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            a = [x[n] for n in ("q", "k", "v", "g", "beta")]
            with torch.cuda.graph(g, stream=side):
                o, f, kept = pkg.gated_delta_forward(*a, initial_states=x["init"], keep_chunk_states=True)
                d = pkg.gated_delta_backward(*a, x["do"], initial_states=x["init"], dfinal_states=x["df"], chunk_states=kept)
            graphs.append(g)
            outs.append(dict(o=o, f=f, **d))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(100):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(t[n], want[n]) for t in outs for n in want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cu", [[0, 200, 100, 300], [-5, 40, 1000000, 300], [300, 0, 0, 0], [0, 0, 0, 0], [10, 20, 30, 40]])
def test_sequences_that_make_no_sense_stay_inside(cu, dtype):
    """What such a call gives is not defined, but it touches nothing else, and the next call is right."""
    x = inputs(1, 300, 2, 64, 64, dtype, seqs=3)
    good = torch.tensor([0, 100, 164, 300], dtype=torch.int32, device="cuda")
    want = run(x, good)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
    pkg.gated_delta_forward(*a, initial_states=x["init"], cu_seqlens=bad)
    pkg.gated_delta_backward(*a, x["do"], initial_states=x["init"], dfinal_states=x["df"], cu_seqlens=bad)
    torch.cuda.synchronize()
    got = run(x, good)
    assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("V,K", [(128, 128), (64, 64), (200, 40)])
def test_nan_outside_the_sequences_stays_there(V, K):
    """Rows behind the last sequence hold NaN and infinities: nothing of them is read."""
    x = inputs(1, 200, 2, V, K, BF16, seqs=2)
    y = {n: t.clone() for n, t in x.items()}
    for n in ("q", "k", "v", "g", "beta", "do"):
        y[n][:, 150:] = float("nan")
        y[n][:, 151] = float("inf")
    cu = torch.tensor([0, 70, 150], dtype=torch.int32, device="cuda")
    a, b = run(x, cu), run(y, cu)
    for n in a:
        s, t = (a[n], b[n]) if n in ("f", "dinitial_states") else (a[n][:, :150], b[n][:, :150])
        assert torch.equal(s, t), n


@pytest.mark.parametrize("V,K,dtype", [(128, 128, BF16), (40, 24, F32)])
def test_padding_gets_zeros(V, K, dtype):
    """Tokens before the first sequence and behind the last: zeros in outputs and gradients, also in memory that held something else."""
    x = inputs(1, 200, 2, V, K, dtype, seqs=2)
    cu = torch.tensor([7, 70, 150], dtype=torch.int32, device="cuda")
    del_me = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(8)]
    del del_me                                                             # what is allocated next holds NaN
    a = run(x, cu)
    for n in a:
        if n not in ("f", "dinitial_states"):
            assert not a[n][:, :7].any() and not a[n][:, 150:].any() and a[n][:, 7:150].any(), n


def test_rows_of_no_sequence_are_left_in_c():
    """Without zero_rest the C entry leaves them as they were."""
    import ctypes
    from state_space_model_scan_gb300 import _lib
    x = inputs(1, 200, 2, 128, 128, BF16, seqs=2)
    cu = torch.tensor([7, 70, 150], dtype=torch.int32, device="cuda")
    want = run(x, cu)
    lib = _lib.load()

    def desc(t):
        d = _lib.Tensor()
        d.ptr, d.dtype = t.data_ptr(), _lib.SSD_BF16 if t.dtype == BF16 else _lib.SSD_F32
        for i, s in enumerate(t.stride()):
            d.stride[i] = s
        return d

    p = _lib.DeltaProblem(1, 200, 2, 2, 128, 128, 2, 128 ** -0.5, _lib.SSD_BF16)
    f = _lib.DeltaArgs()
    o = torch.full_like(x["v"], 7.0)
    for n in ("q", "k", "v", "g", "beta"):
        setattr(f, n, desc(x[n]))
    f.o = desc(o)
    f.initial_states = desc(x["init"])
    f.cu_seqlens = cu.data_ptr()
    n = ctypes.c_size_t()
    assert lib.ssd_delta_fwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0
    ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.ssd_delta_fwd(ctypes.byref(p), ctypes.byref(f), ctypes.c_void_p(ws.data_ptr()), n, st) == 0
    assert torch.equal(o[:, 7:150], want["o"][:, 7:150])
    assert (o[:, :7] == 7).all() and (o[:, 150:] == 7).all()
    f.zero_rest = 1
    assert lib.ssd_delta_fwd(ctypes.byref(p), ctypes.byref(f), ctypes.c_void_p(ws.data_ptr()), n, st) == 0
    assert torch.equal(o, want["o"])


@pytest.mark.parametrize("case", [(1, 65, 2, 6, 128, 128, BF16, BF16, None, BF16), (2, 64, 2, 4, 128, 128, BF16, F32, None, F32), (3, 70, 1, 4, 33, 57, BF16, BF16, None, F32),
                                  (1, 150, 2, 8, 48, 96, BF16, F32, [150], None), (1, 129, 1, 6, 128, 72, BF16, F32, [1, 64, 64], BF16),
                                  (1, 257, 1, 1, 64, 64, BF16, BF16, None, F32), (1, 9, 1, 40, 128, 128, BF16, F32, None, F32), (1, 1, 8, 264, 128, 64, BF16, BF16, None, F32),
                                  (1, 300, 4, 12, 96, 48, BF16, BF16, [64, 0, 0, 235, 1], F32)])
@pytest.mark.parametrize("kept", [True, False])
def test_odd_sizes_of_more_heads(case, kept):
    """The tensor-core path at the sizes of the oracle's cases, with the heads that it takes; tolerances as there."""
    import test_gpu_delta as t
    B, L, G, H, V, K, dtype, gd, lens, init = case
    x = t.make(B, L, G, H, V, K, dtype, gd, lens and len(lens), init, train=True, seed=6)
    cu = None if lens is None else t.packed(lens)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, f, states = pkg.gated_delta_forward(*a, initial_states=x["init"], cu_seqlens=cu, state_dtype=F32, keep_chunk_states=True)
    d = pkg.gated_delta_backward(*a, x["do"], initial_states=x["init"], dfinal_states=x["dfinal"], cu_seqlens=cu, chunk_states=states if kept else None)
    w = t.want(x, K ** -0.5, None if cu is None else cu.tolist(), back=True)
    assert t.rel(o, w["o"]) <= t.OUT[BF16] and t.rel(f, w["final"]) <= t.OUT[F32]
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert t.rel(d[n], w[n]) <= t.GRAD[BF16], n
    if init is not None:
        assert t.rel(d["dinitial_states"], w["dinit"]) <= t.GRAD[BF16]


@pytest.mark.parametrize("L,H", [(1, 1), (1, 3), (2, 2), (7, 2), (20, 9), (64, 4), (5, 40)])
def test_few_tokens_are_as_right_as_their_rounding(L, H):
    """dg and dbeta of a few tokens are few numbers that may happen to be small: computed in fp32, each is off by its own rounding to
    bf16 (at most 2^-8 of it), and by 2e-5 of the terms that it is summed from, here up to a hundred times the norm."""
    import test_gpu_delta as t
    for seed in range(6):
        x = t.make(1, L, 1, H, 64, 64, BF16, BF16, None, F32 if seed % 2 else None, train=True, seed=seed)
        a = [x[n] for n in ("q", "k", "v", "g", "beta")]
        o, f, states = pkg.gated_delta_forward(*a, initial_states=x["init"], keep_chunk_states=True)
        d = pkg.gated_delta_backward(*a, x["do"], initial_states=x["init"], dfinal_states=x["dfinal"], chunk_states=states)
        w = t.want(x, 64 ** -0.5, back=True)
        for n, v in (("o", o), *d.items()):
            if n != "dinitial_states":
                assert t.rel(v, w[n]) <= 2.0 ** -8 + 2e-3, n
