"""How far bf16 outputs and gradients of the gated delta rule's tensor-core path are from the float64 oracle: no more than the roundings that
they are documented to go through.

A rounding to bf16 is off by at most half a step, uniformly, 2^-8 / sqrt(3) = 2.26e-3 in the mean square of values at the lower end of
a power of two (less above it).  n of them, of random sign, one after another or beside one another: sqrt(n) times that.
  o:   att, beta U, the output itself                                          3   3.91e-3
  dv:  att, the gradient itself (what is carried is held to 2^-17)             2   3.20e-3
  dq:  U and F, or the kept state; the gradient itself                         3   3.91e-3
  dk:  mu, U and E, or F's two, or a kept state and U; the gradient itself     4   4.52e-3
States go as the sum of two bf16 values: 2e-5, as in test_gpu_delta.py."""
import pytest
import torch

import state_space_model_scan_gb300 as pkg
import test_gpu_delta as t

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
BOUND = dict(o=3.91e-3, f=2e-5, dv=3.20e-3, dq=3.91e-3, dk=4.52e-3)


@pytest.mark.parametrize("kept", [True, False])
@pytest.mark.parametrize("B,L,G,H,V,K,lens", [(1, 320, 4, 8, 128, 128, None), (2, 256, 3, 3, 128, 64, None), (1, 500, 2, 4, 64, 128, [129, 1, 0, 370]),
                                              (1, 1408, 1, 2, 128, 128, None)])
def test_errors_are_those_of_the_roundings(B, L, G, H, V, K, lens, kept):
    x = t.make(B, L, G, H, V, K, BF16, F32, lens and len(lens), F32, seed=8, train=True)
    cu = None if lens is None else t.packed(lens)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, f, states = pkg.gated_delta_forward(*a, initial_states=x["init"], cu_seqlens=cu, keep_chunk_states=True)
    d = pkg.gated_delta_backward(*a, x["do"], initial_states=x["init"], dfinal_states=x["dfinal"], cu_seqlens=cu, chunk_states=states if kept else None)
    w = t.want(x, K ** -0.5, None if cu is None else cu.tolist(), back=True)
    got = dict(d, o=o, f=f)
    off = {n: t.rel(got[n], w["final" if n == "f" else n]) for n in BOUND}
    assert all(off[n] <= BOUND[n] for n in BOUND), off


@pytest.mark.parametrize("K", [1, 2, 3, 5, 7, 8])
@pytest.mark.parametrize("B,L,G,H,V,lens", [(1, 640, 4, 4, 64, None), (3, 65, 1, 3, 1, None), (1, 129, 3, 6, 128, [27, 13, 57, 6, 11, 8, 7])])
def test_few_features_of_the_keys(B, L, G, H, V, lens, K):
    """Keys that point the same way take back what the one before has written: outputs and gradients are differences.  The bounds are
    those of all sizes (test_gpu_delta.py)."""
    x = t.make(B, L, G, H, V, K, BF16, F32, lens and len(lens), F32, seed=3, train=True)
    cu = None if lens is None else t.packed(lens)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, f, states = pkg.gated_delta_forward(*a, initial_states=x["init"], cu_seqlens=cu, keep_chunk_states=True)
    d = pkg.gated_delta_backward(*a, x["do"], initial_states=x["init"], dfinal_states=x["dfinal"], cu_seqlens=cu, chunk_states=states)
    w = t.want(x, K ** -0.5, None if cu is None else cu.tolist(), back=True)
    assert t.rel(o, w["o"]) <= t.OUT[BF16] and t.rel(f, w["final"]) <= t.OUT[F32]
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert t.rel(d[n], w[n]) <= t.GRAD[BF16], n
    assert t.rel(d["dinitial_states"], w["dinit"]) <= t.GRAD[BF16]


@pytest.mark.parametrize("B,L,G,H,V,K,lens", [(1, 65, 1, 3, 128, 128, None), (2, 64, 2, 2, 128, 128, None), (1, 70, 1, 2, 33, 57, None), (1, 60, 2, 4, 128, 64, [1, 0, 59]),
                                              (1, 300, 2, 4, 64, 7, None), (1, 130, 1, 2, 160, 72, None)])
def test_calls_in_fp32_are_off_by_one_rounding(B, L, G, H, V, K, lens):
    """bf16 data of calls that the fp32 kernels take (few tokens and heads, few features, wide heads): outputs and gradients in bf16 are rounded
    once, 2.26e-3 in the mean square and fp32's own 2e-5; what is kept in fp32 is right to that."""
    x = t.make(B, L, G, H, V, K, BF16, F32, lens and len(lens), F32, seed=9, train=True)
    cu = None if lens is None else t.packed(lens)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, f, states = pkg.gated_delta_forward(*a, initial_states=x["init"], cu_seqlens=cu, keep_chunk_states=True)
    slots = L // 64 + len(lens) if lens else B * -(-L // 64)
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    assert states.numel() == up(slots * H * V * K * 4) + up(slots * H * 64 * V * 4)              # (states and values in fp32: that path)
    d = pkg.gated_delta_backward(*a, x["do"], initial_states=x["init"], dfinal_states=x["dfinal"], cu_seqlens=cu, chunk_states=states)
    w = t.want(x, K ** -0.5, None if cu is None else cu.tolist(), back=True)
    off = {n: t.rel(v, w[n]) for n, v in dict(d, o=o).items() if n != "dinitial_states"}
    assert all(off[n] <= 2.28e-3 for n in ("o", "dq", "dk", "dv")), off
    assert all(off[n] <= 2e-5 for n in ("dg", "dbeta")), off
    assert t.rel(f, w["final"]) <= 2e-5 and t.rel(d["dinitial_states"], w["dinit"]) <= 2e-5
