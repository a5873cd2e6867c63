"""The C ABI of the gated delta rule and of the norm and rotation of queries and keys on the CPU: every call here is refused
before anything reaches the device."""
import ctypes

import pytest

D = ctypes.c_void_p(0x100000)
Z = ctypes.c_size_t


@pytest.fixture(scope="module")
def m():
    from state_space_model_scan_gb300 import build, _lib
    build.build()
    _lib.load()
    return _lib


def fake(m, dtype, strides, ptr=0x100000):
    t = m.Tensor()
    t.ptr, t.dtype = ptr, dtype
    for i, s in enumerate(strides):
        t.stride[i] = s
    return t


def delta_case(m, B=2, L=70, G=2, H=4, V=24, K=40, packed=0, dtype=1):
    p = m.DeltaProblem(B, L, H, G, V, K, packed, 0.5, dtype)
    f, b = m.DeltaArgs(), m.DeltaBwdArgs()
    qk, vo, gb, st = [L * G * K, G * K, K, 1], [L * H * V, H * V, V, 1], [L * H, H, 1], [H * V * K, V * K, K, 1]
    for n in ("q", "k"):
        setattr(f, n, fake(m, dtype, qk))
        setattr(b, "d" + n, fake(m, dtype, qk))
    f.v, f.o, b.dO, b.dv = (fake(m, dtype, vo) for _ in range(4))
    f.g, f.beta, b.dg, b.dbeta = (fake(m, 0, gb) for _ in range(4))
    f.initial_states, f.final_states, b.dfinal_states, b.dinitial_states = (fake(m, 0, st) for _ in range(4))
    if packed:
        f.cu_seqlens = 0x200000
    b.fwd = f
    return p, f, b


def sizes(m, p):
    n = [Z(0) for _ in range(4)]
    rc = {m.load().ssd_delta_chunk_states_size(ctypes.byref(p), ctypes.byref(n[0])),
          m.load().ssd_delta_fwd_workspace_size(ctypes.byref(p), ctypes.byref(n[1])),
          m.load().ssd_delta_bwd_workspace_size(ctypes.byref(p), 0, ctypes.byref(n[2])),
          m.load().ssd_delta_bwd_workspace_size(ctypes.byref(p), 1, ctypes.byref(n[3]))}
    return rc, [v.value for v in n]


@pytest.mark.parametrize("mutate,code", [
    (lambda p, f: setattr(p, "ngroups", 3), 1),
    (lambda p, f: setattr(p, "batch", 0), 1),
    (lambda p, f: setattr(p, "seqlen", -1), 1),
    (lambda p, f: setattr(p, "dtype", 2), 1),
    (lambda p, f: setattr(p, "dstate", 0), 1),
    (lambda p, f: setattr(p, "dstate", 257), 2),
    (lambda p, f: setattr(p, "headdim", 257), 2),
    (lambda p, f: setattr(p, "seqlen", 1 << 31), 2),
    (lambda p, f: setattr(p, "batch", 1 << 25), 2),
    (lambda p, f: setattr(p, "nseqs", -1), 1),
    (lambda p, f: setattr(p, "nseqs", 2), 1),                      # packed rows come alone
    (lambda p, f: setattr(f, "cu_seqlens", 0x2000), 1),            # without nseqs
    (lambda p, f: setattr(f.q, "ptr", None), 1),
    (lambda p, f: setattr(f.k, "dtype", 0), 1),
    (lambda p, f: setattr(f.g, "dtype", 5), 1),
    (lambda p, f: setattr(f.beta, "ptr", None), 1),
    (lambda p, f: f.v.stride.__setitem__(3, 2), 1),
    (lambda p, f: f.v.stride.__setitem__(1, -1), 1),
    (lambda p, f: f.initial_states.stride.__setitem__(2, 41), 1),
    (lambda p, f: setattr(f.initial_states, "dtype", 3), 1),
    (lambda p, f: setattr(f.v, "ptr", 0x100001), 3),
    (lambda p, f: setattr(f.beta, "ptr", 0x100002), 3),
    (lambda p, f: setattr(f, "chunk_states", 0x100010), 3),
])
def test_delta_refusals(m, mutate, code):
    p, f, b = delta_case(m)
    assert sizes(m, p)[0] == {0}
    mutate(p, f)
    b.fwd = f
    assert m.load().ssd_delta_fwd(ctypes.byref(p), ctypes.byref(f), D, Z(1 << 40), None) == code
    assert m.load().ssd_delta_bwd(ctypes.byref(p), ctypes.byref(b), D, Z(1 << 40), None) == code


def test_delta_outputs_and_workspaces(m):
    p, f, b = delta_case(m)
    rc, (kept, fwd, bwd, bwd_kept) = sizes(m, p)
    assert bwd - bwd_kept == kept > 0 and fwd > 0
    run, back = m.load().ssd_delta_fwd, m.load().ssd_delta_bwd
    for ws, n, code in ((D, fwd - 1, 4), (None, fwd, 4), (ctypes.c_void_p(0x100010), fwd, 3)):
        assert run(ctypes.byref(p), ctypes.byref(f), ws, Z(n), None) == code
    for ws, n, code in ((D, bwd - 1, 4), (None, bwd, 4), (ctypes.c_void_p(0x100010), bwd, 3)):
        assert back(ctypes.byref(p), ctypes.byref(b), ws, Z(n), None) == code
    for k in ("dO", "dq", "dk", "dv", "dg", "dbeta", "dinitial_states"):
        p, f, b = delta_case(m)
        setattr(b, k, m.Tensor())
        assert back(ctypes.byref(p), ctypes.byref(b), D, Z(bwd), None) == 1, k
    p, f, b = delta_case(m)
    b.dg = fake(m, 1, [280, 4, 1])                                 # gradients have their inputs' types
    assert back(ctypes.byref(p), ctypes.byref(b), D, Z(bwd), None) == 1
    p, f, b = delta_case(m)
    f.o.stride[2] = 0                                              # what is written overlaps
    assert run(ctypes.byref(p), ctypes.byref(f), D, Z(fwd), None) == 1
    for arg in (None,):
        assert run(arg, ctypes.byref(f), D, Z(fwd), None) == 1 and back(ctypes.byref(p), arg, D, Z(bwd), None) == 1
    assert m.load().ssd_delta_chunk_states_size(ctypes.byref(p), None) == 1


def test_delta_packed_sizes(m):
    """A chunk for every 64 tokens, and one more for each packed sequence."""
    one = sizes(m, m.DeltaProblem(1, 64, 2, 1, 8, 8, 0, 1.0, 0))[1][0]
    assert sizes(m, m.DeltaProblem(1, 128 + 63, 2, 1, 8, 8, 5, 1.0, 0))[1][0] == 7 * one
    assert sizes(m, m.DeltaProblem(3, 65, 2, 1, 8, 8, 0, 1.0, 0))[1][0] == 6 * one
    assert sizes(m, m.DeltaProblem(3, 0, 2, 1, 8, 8, 0, 1.0, 0))[1][0] == 0


def step_case(m):
    return m.DeltaStepProblem(3, 5, 4, 2, 2, 16, 128, 32, 32, 8, 4, 4, 8, 1.0, 1, 0, 1, 0)


@pytest.mark.parametrize("mutate,code", [
    (lambda p: setattr(p, "ngroups", 3), 1),
    (lambda p: setattr(p, "nslots", -1), 1),
    (lambda p: setattr(p, "g_dtype", 3), 1),
    (lambda p: setattr(p, "state_dtype", 2), 1),
    (lambda p: setattr(p, "slot_stride", 127), 1),
    (lambda p: setattr(p, "q_stride", 31), 1),
    (lambda p: setattr(p, "o_stride", 7), 1),
    (lambda p: setattr(p, "beta_stride", 3), 1),
    (lambda p: setattr(p, "dstate", 257), 2),
    (lambda p: setattr(p, "batch", (1 << 20) + 1), 2),
])
def test_step_refusals(m, mutate, code):
    p = step_case(m)
    mutate(p)
    assert m.load().ssd_delta_step(ctypes.byref(p), D, None, *[D] * 6, None) == code


def test_step_addresses(m):
    run = m.load().ssd_delta_step
    for i in range(7):
        for bad, code in ((None, 1), (ctypes.c_void_p(0x100001), 3)):
            a = [D] * 7
            a[i] = bad
            assert run(ctypes.byref(step_case(m)), a[0], None, *a[1:], None) == code, i
    assert run(ctypes.byref(step_case(m)), D, ctypes.c_void_p(0x100002), *[D] * 6, None) == 3
    p = step_case(m)
    p.batch = 0
    assert run(ctypes.byref(p), None, None, *[None] * 6, None) == 0


def qk_case(m):
    p = m.QkProblem(2, 10, 4, 1, 24, 16, 30, 10, 1e-6, 0, 0, 0)
    f, b = m.QkArgs(), m.QkBwdArgs()
    q, k = [960, 96, 24, 1], [240, 24, 24, 1]
    f.q, f.q_out, b.dq, b.dq_out = (fake(m, 0, q) for _ in range(4))
    f.k, f.k_out, b.dk, b.dk_out = (fake(m, 0, k) for _ in range(4))
    f.cos = f.sin = f.positions = f.q_weight = f.k_weight = b.dq_weight = b.dk_weight = 0x100000
    b.fwd = f
    return p, f, b


@pytest.mark.parametrize("mutate,code", [
    (lambda p, f: setattr(p, "q_heads", 0), 1),
    (lambda p, f: setattr(p, "rotary", 15), 1),
    (lambda p, f: setattr(p, "rotary", 26), 1),
    (lambda p, f: setattr(p, "eps", -1.0), 1),
    (lambda p, f: setattr(p, "eps", float("nan")), 1),
    (lambda p, f: setattr(p, "mode", 2), 1),
    (lambda p, f: setattr(p, "interleaved", 2), 1),
    (lambda p, f: setattr(p, "dtype", 4), 1),
    (lambda p, f: setattr(p, "dim", 513), 2),
    (lambda p, f: setattr(p, "seqlen", 1 << 40), 2),
    (lambda p, f: setattr(f, "cos", None), 1),
    (lambda p, f: setattr(f.q, "ptr", None), 1),
    (lambda p, f: setattr(f.k, "dtype", 1), 1),
    (lambda p, f: f.q.stride.__setitem__(3, 2), 1),
    (lambda p, f: f.k.stride.__setitem__(1, -24), 1),
    (lambda p, f: setattr(f.q, "ptr", 0x100002), 3),
    (lambda p, f: setattr(f, "positions", 0x100002), 3),
    (lambda p, f: setattr(f, "k_weight", 0x100001), 3),
])
def test_qk_refusals(m, mutate, code):
    p, f, b = qk_case(m)
    mutate(p, f)
    b.fwd = f
    assert m.load().ssd_qk_norm_fwd(ctypes.byref(p), ctypes.byref(f), None) == code
    assert m.load().ssd_qk_norm_bwd(ctypes.byref(p), ctypes.byref(b), D, Z(1 << 40), None) == code


def test_qk_outputs_and_workspace(m):
    run, back = m.load().ssd_qk_norm_fwd, m.load().ssd_qk_norm_bwd
    for k in ("q_out", "k_out"):
        p, f, b = qk_case(m)
        setattr(f, k, m.Tensor())
        assert run(ctypes.byref(p), ctypes.byref(f), None) == 1
    p, f, b = qk_case(m)
    f.q_out.stride[1] = 0
    assert run(ctypes.byref(p), ctypes.byref(f), None) == 1
    n = Z(0)
    assert m.load().ssd_qk_norm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value > 0
    for ws, size, code in ((D, n.value - 1, 4), (None, n.value, 4), (ctypes.c_void_p(0x100010), n.value, 3)):
        p, f, b = qk_case(m)
        assert back(ctypes.byref(p), ctypes.byref(b), ws, Z(size), None) == code
    for k in ("dq", "dk", "dq_out", "dk_out"):
        p, f, b = qk_case(m)
        setattr(b, k, m.Tensor())
        assert back(ctypes.byref(p), ctypes.byref(b), D, n, None) == 1, k
    for k in ("dq_weight", "dk_weight"):
        p, f, b = qk_case(m)
        setattr(b, k, None)
        assert back(ctypes.byref(p), ctypes.byref(b), D, n, None) == 1, k
