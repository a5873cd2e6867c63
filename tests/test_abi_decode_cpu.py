"""The C ABI of the selective scan, the steps, the carried convolution and the snapshots on the CPU: every call here is
refused before anything reaches the device."""
import ctypes

import pytest

D = ctypes.c_void_p(0x100000)


def at(off):
    return ctypes.c_void_p(0x100000 + off)


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


def sel_case(m, Bt=2, L=40, Dm=24, G=2, N=12, packed=0):
    p = m.SelectiveProblem(Bt, L, Dm, G, N, packed)
    f = m.FwdArgs()
    tok, grp = [L * Dm, Dm, 1], [L * G * N, G * N, N, 1]
    for k in ("x", "dt", "z", "y"):
        setattr(f, k, fake(m, m.SSD_BF16, tok))
    for k in ("B", "C"):
        setattr(f, k, fake(m, m.SSD_BF16, grp))
    f.A = fake(m, m.SSD_F32, [N, 1])
    f.D, f.dt_bias = fake(m, m.SSD_F32, [1]), fake(m, m.SSD_F32, [1])
    f.final_states = fake(m, m.SSD_F32, [Dm * N, N, 1])
    if packed:
        f.cu_seqlens = 0x200000
    b = m.BwdArgs()
    b.fwd = f
    for k in ("dy", "dx", "ddt", "dz"):
        setattr(b, k, fake(m, m.SSD_BF16, tok))
    for k in ("dB", "dC"):
        setattr(b, k, fake(m, m.SSD_BF16, grp))
    b.dA = fake(m, m.SSD_F32, [N, 1])
    b.dD, b.ddt_bias = fake(m, m.SSD_F32, [1]), fake(m, m.SSD_F32, [1])
    return p, f, b


def bwd_size(m, p, b):
    n = ctypes.c_size_t(0)
    return m.load().ssd_selective_bwd_workspace_size(ctypes.byref(p), ctypes.byref(b), ctypes.byref(n)), n.value


@pytest.mark.parametrize("mutate,code", [
    (lambda p, f: setattr(p, "ngroups", 5), 1),
    (lambda p, f: setattr(p, "batch", 0), 1),
    (lambda p, f: setattr(p, "seqlen", -1), 1),
    (lambda p, f: setattr(p, "dstate", 0), 1),
    (lambda p, f: setattr(p, "dstate", 129), 2),
    (lambda p, f: setattr(p, "seqlen", 1 << 31), 2),
    (lambda p, f: setattr(p, "nseqs", 2), 1),                     # packed counts without cu_seqlens
    (lambda p, f: setattr(f, "cu_seqlens", 0x2000), 1),           # packed needs batch 1 and nseqs
    (lambda p, f: setattr(f.x, "ptr", None), 1),
    (lambda p, f: setattr(f.dt, "dtype", 7), 1),
    (lambda p, f: setattr(f.B, "dtype", 0), 1),
    (lambda p, f: setattr(f.A, "dtype", 1), 1),
    (lambda p, f: f.A.stride.__setitem__(0, 13), 1),
    (lambda p, f: f.x.stride.__setitem__(2, 2), 1),
    (lambda p, f: f.x.stride.__setitem__(1, 23), 1),              # tokens overlap
    (lambda p, f: f.x.stride.__setitem__(0, 39 * 24), 1),         # batch rows overlap
    (lambda p, f: f.C.stride.__setitem__(2, 11), 1),              # groups overlap
    (lambda p, f: setattr(f.z, "ptr", 0x100001), 3),
    (lambda p, f: setattr(f, "chunk_states", 0x100008), 3),
])
def test_selective_refusals(m, mutate, code):
    p, f, b = sel_case(m)
    assert bwd_size(m, p, b)[0] == 0
    mutate(p, f)
    b.fwd = f
    assert m.load().ssd_selective_fwd(ctypes.byref(p), ctypes.byref(f), None, ctypes.c_size_t(0), None) == code
    assert bwd_size(m, p, b)[0] == code


def test_selective_outputs_and_workspace(m):
    p, f, b = sel_case(m)
    f.y = m.Tensor()
    assert m.load().ssd_selective_fwd(ctypes.byref(p), ctypes.byref(f), None, ctypes.c_size_t(0), None) == 1
    p, f, b = sel_case(m)
    rc, n = bwd_size(m, p, b)
    assert rc == 0 and n > 0
    run = m.load().ssd_selective_bwd
    assert run(ctypes.byref(p), ctypes.byref(b), D, ctypes.c_size_t(n - 1), None) == 4
    assert run(ctypes.byref(p), ctypes.byref(b), None, ctypes.c_size_t(n), None) == 4
    assert run(ctypes.byref(p), ctypes.byref(b), at(16), ctypes.c_size_t(n), None) == 3
    b.fwd.chunk_states = 0x300000                                # kept states leave the workspace
    assert bwd_size(m, p, b)[1] < n
    for k in ("dy", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias"):
        p, f, b = sel_case(m)
        setattr(b, k, m.Tensor())
        assert bwd_size(m, p, b)[0] == 1, k
    p, f, b = sel_case(m)
    b.fwd.initial_states = fake(m, m.SSD_F32, [24 * 12, 12, 1])
    assert bwd_size(m, p, b)[0] == 1                             # dinitial_states missing


def test_selective_chunk_states_size(m):
    """f32 [chunk slots][channels][dstate padded]: a slot per 16 tokens; packed, one more per sequence."""
    def size(p):
        n = ctypes.c_size_t(0)
        assert m.load().ssd_selective_chunk_states_size(ctypes.byref(p), ctypes.byref(n)) == 0
        return n.value
    assert size(m.SelectiveProblem(2, 65, 24, 2, 12, 0)) == 2 * 5 * 24 * 16 * 4
    assert size(m.SelectiveProblem(1, 65, 24, 2, 17, 5)) == (4 + 5) * 24 * 32 * 4
    assert size(m.SelectiveProblem(2, 0, 24, 2, 12, 0)) == 0


def test_selective_forward_workspace(m):
    """None, but for a long sequence of few channels: f32 (dstate padded + 1) a segment and channel."""
    def size(p):
        n = ctypes.c_size_t(0)
        assert m.load().ssd_selective_fwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0
        return n.value
    assert size(m.SelectiveProblem(1, 2048, 4096, 1, 16, 0)) == 0 and size(m.SelectiveProblem(1, 300, 32, 1, 16, 0)) == 0
    p, f, b = sel_case(m, Bt=1, L=16000, Dm=24, G=2, N=16)
    n = size(p)
    assert n >= 3 * 24 * 17 * 4
    run = m.load().ssd_selective_fwd
    assert run(ctypes.byref(p), ctypes.byref(f), D, ctypes.c_size_t(n - 1), None) == 4
    assert run(ctypes.byref(p), ctypes.byref(f), None, ctypes.c_size_t(n), None) == 4
    assert run(ctypes.byref(p), ctypes.byref(f), at(16), ctypes.c_size_t(n), None) == 3


def step_problem(m, **k):
    v = dict(batch=2, nslots=3, nheads=4, headdim=8, ngroups=2, dstate=16, slot_stride=512, x_stride=32, dt_stride=4,
             z_stride=32, b_stride=32, c_stride=32, y_stride=32, dtype=1, dt_dtype=0, state_dtype=0, reserved=0)
    v.update(k)
    return m.StepProblem(*v.values())


@pytest.mark.parametrize("k,code", [
    (dict(nheads=5), 1), (dict(headdim=0), 1), (dict(batch=-1), 1), (dict(dstate=0), 1), (dict(dstate=257, slot_stride=1 << 20,
     b_stride=1 << 10, c_stride=1 << 10), 2), (dict(dtype=2), 1), (dict(state_dtype=2), 1), (dict(dt_dtype=1), 1),
    (dict(reserved=1), 1), (dict(slot_stride=511), 1), (dict(x_stride=31), 1), (dict(y_stride=31), 1), (dict(b_stride=31), 1),
    (dict(z_stride=31), 1), (dict(dt_stride=3), 1), (dict(batch=1 << 21), 2),
])
def test_step_refusals(m, k, code):
    p = step_problem(m, **k)
    f = m.load().ssd_step
    assert f(ctypes.byref(p), D, None, D, D, D, D, D, None, D, None, D, None) == code


def test_step_pointers(m):
    f, g = m.load().ssd_step, m.load().ssd_selective_step
    p = step_problem(m)
    args = [D, None, D, D, D, D, D, None, None, None, D]          # state, idx, x, dt, A, B, C, D, z, bias, y
    for k in (0, 2, 3, 4, 5, 6, 10):
        bad = list(args)
        bad[k] = None
        assert f(ctypes.byref(p), *bad, None) == 1, k
    for k, off in ((0, 2), (1, 2), (2, 1), (3, 2), (4, 1), (5, 1), (7, 2), (8, 1), (9, 2), (10, 1)):
        bad = list(args)
        bad[k] = at(off)
        assert f(ctypes.byref(p), *bad, None) == 3, k
    assert g(ctypes.byref(p), *args, None) == 1                   # the selective form has headdim 1
    p.batch = 0
    assert f(ctypes.byref(p), *([None] * 11), None) == 0          # nothing to do


def test_conv_window_refusals(m):
    p = m.ConvProblem(2, 5, 16, 4, 0, m.SSD_BF16, 1, 0, 0)
    f = m.load().ssd_conv1d_prompt

    def call(win=D, nslots=2, stride=48, idx=None, u=D, usl=16, w=D, out=D, cu=None):
        return f(ctypes.byref(p), u, 5 * usl, usl, w, None, cu, win, nslots, stride, idx, None, out, 80, 16, None)
    assert call(win=None) == 1 and call(nslots=-1) == 1 and call(stride=40) == 1 and call(stride=52) == 3
    assert call(win=at(8)) == 3 and call(idx=at(2)) == 3 and call(u=None) == 1 and call(w=None) == 1
    assert call(usl=20) == 3 and call(cu=D) == 1
    q = m.ConvProblem(2, 1, 16, 4, 0, m.SSD_BF16, 1, 0, 0)
    g = m.load().ssd_conv1d_step
    assert g(ctypes.byref(p), D, 16, D, None, D, 2, 48, None, D, 16, None) == 1          # seqlen is 1
    assert g(ctypes.byref(q), D, 16, D, None, None, 2, 48, None, D, 16, None) == 1
    assert g(ctypes.byref(q), D, 20, D, None, D, 2, 48, None, D, 16, None) == 3
    assert g(ctypes.byref(q), D, 16, None, None, D, 2, 48, None, D, 16, None) == 1
    q.batch = 1 << 31
    assert g(ctypes.byref(q), D, 16, D, None, D, 2, 48, None, D, 16, None) == 2


@pytest.mark.parametrize("k,code", [
    (dict(count=-1), 1), (dict(rows=0), 1), (dict(dstate=0), 1), (dict(dstate=1025, state_stride=1 << 20), 2),
    (dict(state_dtype=2), 1), (dict(reserved=1), 1), (dict(state_stride=95), 1), (dict(count=1 << 25), 2), (dict(count=0), 0),
])
def test_snapshot_refusals(m, k, code):
    v = dict(count=2, rows=6, dstate=16, nslots=3, nsnapshots=3, state_stride=96, state_dtype=0, reserved=0)
    v.update(k)
    p = m.SnapshotProblem(*v.values())
    assert m.load().ssd_snapshot_store(ctypes.byref(p), D, None, D, D, None, None) == code
    assert m.load().ssd_snapshot_load(ctypes.byref(p), D, D, None, D, None, None) == code
    if not k.get("count", 1):
        return
    q = m.SnapshotProblem(2, 6, 16, 3, 3, 96, 0, 0)
    assert m.load().ssd_snapshot_store(ctypes.byref(q), None, None, D, D, None, None) == 1
    assert m.load().ssd_snapshot_store(ctypes.byref(q), at(2), None, D, D, None, None) == 3
    assert m.load().ssd_snapshot_load(ctypes.byref(q), D, at(2), None, D, None, None) == 3


def test_step_too_many_blocks(m):
    """More blocks than a grid can have (rows of 33 states, two to a block): refused before the launch."""
    k = dict(batch=1 << 20, nheads=1536, headdim=4, ngroups=1, dstate=33, slot_stride=1 << 30, x_stride=6144, dt_stride=1536,
             z_stride=6144, b_stride=33, c_stride=33, y_stride=6144)
    p = step_problem(m, **k)
    f, g = m.load().ssd_step, m.load().ssd_selective_step
    assert f(ctypes.byref(p), D, None, D, D, D, D, D, None, D, None, D, None) == 2
    p = step_problem(m, **dict(k, nheads=6144, headdim=1, dt_stride=6144))
    assert g(ctypes.byref(p), D, None, D, D, D, D, D, None, D, None, D, None) == 2
