// binding.cpp -- Python's way to the entry points that are called for single tokens, where reading and checking a
// dozen tensors in Python would cost several times the kernel.  It checks that the tensors have the shapes,
// types and devices that the library assumes (the library itself sees addresses and strides), allocates the
// outputs with torch and calls the C ABI.  A failed check raises ValueError, a refusal SSDError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdarg.h>

#include <initializer_list>
#include <string>

#include "../../include/ssd.h"

namespace {

using at::Tensor;

// The library's functions, as _lib.py found them.
struct Lib {
    decltype(&ssd_step) step, selective_step;
    decltype(&ssd_conv1d_prompt) conv1d_prompt;
    decltype(&ssd_conv1d_step) conv1d_step;
    decltype(&ssd_snapshot_store) snapshot_store;
    decltype(&ssd_snapshot_load) snapshot_load;
    decltype(&ssd_selective_chunk_states_size) chunk_states_size;
    decltype(&ssd_selective_fwd_workspace_size) fwd_workspace_size;
    decltype(&ssd_selective_fwd) selective_fwd;
    decltype(&ssd_selective_bwd_workspace_size) bwd_workspace_size;
    decltype(&ssd_selective_bwd) selective_bwd;
} lib;
PyObject *ssd_error, *out_of_memory;   // the exception classes SSDError(code, where) and torch's

struct Raised {};      // a Python exception is set

[[noreturn]] void fail(PyObject *type, const char *fmt, ...) {
    va_list va;
    va_start(va, fmt);
    PyErr_FormatV(type, fmt, va);
    va_end(va);
    throw Raised();
}
#define NEED(cond, ...)                                      \
    do {                                                     \
        if (!(cond)) fail(PyExc_ValueError, __VA_ARGS__);    \
    } while (0)

void check(ssd_status s, const char *where) {
    if (s == SSD_OK) return;
    PyObject *e = PyObject_CallFunction(ssd_error, "is", (int)s, where);
    if (e) {
        PyErr_SetObject(ssd_error, e);
        Py_DECREF(e);
    }
    throw Raised();
}

// A tensor argument; None gives an undefined one where that is allowed.
const Tensor none;
const Tensor &arg(PyObject *o, const char *name, bool optional = false) {
    if (o == Py_None && optional) return none;
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s is not a tensor", name);
    return THPVariable_Unpack(o);
}

constexpr int F32 = 1, BF16 = 2, I32 = 4, I8 = 8, U8 = 16, BOOL = 32;   // sets of types
int type_of(const Tensor &t) {
    switch (t.scalar_type()) {
        case at::kFloat: return F32;
        case at::kBFloat16: return BF16;
        case at::kInt: return I32;
        case at::kChar: return I8;
        case at::kByte: return U8;
        case at::kBool: return BOOL;
        default: return 0;
    }
}
int code(const Tensor &t) { return t.scalar_type() == at::kBFloat16 ? SSD_BF16 : SSD_F32; }

// The tensor that fixes device and type of the others.
int lead(const char *name, const Tensor &t, int64_t dims) {
    NEED(t.dim() == dims, "%s has %lld dimensions, not %lld", name, (long long)t.dim(), (long long)dims);
    NEED(t.is_cuda(), "%s is not on a GPU", name);
    NEED(type_of(t) & (F32 | BF16), "%s is neither float32 nor bfloat16", name);
    return t.get_device();
}
// t has this shape, one of these types and this device, and its last `inner` dimensions are contiguous.
void like(const char *name, const Tensor &t, std::initializer_list<int64_t> shape, int types, int dev, int inner) {
    if (t.sizes() != at::IntArrayRef(shape)) {
        std::string has, wants;
        for (int64_t v : t.sizes()) has += (has.empty() ? "" : ", ") + std::to_string(v);
        for (int64_t v : shape) wants += (wants.empty() ? "" : ", ") + std::to_string(v);
        fail(PyExc_ValueError, "%s has shape [%s], not [%s]", name, has.c_str(), wants.c_str());
    }
    NEED(type_of(t) & types, "%s has the wrong type", name);
    NEED(t.is_cuda() && t.get_device() == dev, "%s is not on GPU %d", name, dev);
    int64_t n = 1;
    for (int64_t k = t.dim() - 1; k >= t.dim() - inner; --k) {
        NEED(t.size(k) == 1 || t.stride(k) == n, "%s: its last %d dimensions must be contiguous", name, inner);
        n *= t.size(k);
    }
}

void *ptr(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
template <typename P>
P *ptr_as(const Tensor &t) { return static_cast<P *>(ptr(t)); }
int64_t stride0(const Tensor &t) { return t.defined() ? t.stride(0) : 0; }

// The stream to launch on: a handle, or None for the device's current one.  While it lives the tensors' device is the current
// one (a null handle means the current device's default stream, and the library asks for the current device), and a given
// stream too, so that what is allocated comes from that stream's memory: a block that the caller's stream has freed may still be in
// use there.  The caller's stream, which will read the outputs, is noted for them.
struct Stream {
    void *handle;
    int dev;
    c10::cuda::CUDAGuard device;
    c10::cuda::CUDAStream caller;
    c10::cuda::OptionalCUDAStreamGuard guard;
    Stream(PyObject *o, int dev_) : dev(dev_), device((c10::DeviceIndex)dev_), caller(c10::cuda::getCurrentCUDAStream(dev_)) {
        handle = o != Py_None ? PyLong_AsVoidPtr(o) : (void *)caller.stream();
        if (PyErr_Occurred()) throw Raised();
        if (handle != caller.stream()) guard.reset_stream(c10::cuda::getStreamFromExternal((cudaStream_t)handle, (c10::DeviceIndex)dev));
    }
    Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
        return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
    }
    Tensor output(at::IntArrayRef shape, at::ScalarType type) const {
        Tensor t = empty(shape, type);
        if (guard.current_stream() && t.numel() > 0) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), caller);
        return t;
    }
    void used(const Tensor &t) const {                              // a tensor of the caller's that the call works in
        if (guard.current_stream() && t.numel() > 0)
            c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *guard.current_stream());
    }
};

// Tells autograd that a call has written t, as torch's own operations in place do (an inference tensor is not watched).
void written(const Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

PyObject *wrap(const Tensor &t) { return THPVariable_Wrap(t); }

// step(selective, state, x, dt, A, B, C, D, z, dt_bias, state_indices, stream)
PyObject *step(PyObject *const *a) {
    const bool sel = a[0] == Py_True;
    const Tensor &state = arg(a[1], "state"), &x = arg(a[2], "x"), &dt = arg(a[3], "dt"), &A = arg(a[4], "A"), &B = arg(a[5], "B"),
                 &C = arg(a[6], "C"), &D = arg(a[7], "D", true), &z = arg(a[8], "z", true), &bias = arg(a[9], "dt_bias", true),
                 &idx = arg(a[10], "state_indices", true);
    const int dev = lead("x", x, sel ? 2 : 3), own = type_of(x);
    NEED(B.dim() == 3, "B has shape [batch, ngroups, dstate]");
    NEED(state.dim() == x.dim() + 1, "state has shape [nslots, %s, dstate]", sel ? "channels" : "nheads, headdim");
    const int64_t n = x.size(0), H = x.size(1), P = sel ? 1 : x.size(2), G = B.size(1), N = B.size(2), slots = state.size(0);
    if (sel) {
        like("x", x, {n, H}, own, dev, 1);
        like("state", state, {slots, H, N}, F32 | BF16, dev, 2);
        like("A", A, {H, N}, F32, dev, 2);
        like("dt", dt, {n, H}, F32 | own, dev, 1);
        if (z.defined()) like("z", z, {n, H}, own, dev, 1);
    } else {
        like("x", x, {n, H, P}, own, dev, 2);
        like("state", state, {slots, H, P, N}, F32 | BF16, dev, 3);
        like("A", A, {H}, F32, dev, 1);
        like("dt", dt, {n, H}, F32, dev, 1);
        if (z.defined()) like("z", z, {n, H, P}, own, dev, 2);
    }
    like("B", B, {n, G, N}, own, dev, 2);
    like("C", C, {n, G, N}, own, dev, 2);
    if (D.defined()) like("D", D, {H}, F32, dev, 1);
    if (bias.defined()) like("dt_bias", bias, {H}, F32, dev, 1);
    if (idx.defined()) like("state_indices", idx, {n}, I32, dev, 1);
    else NEED(slots >= n, "the state pool has fewer slots than there are requests");
    const Stream st(a[11], dev);
    Tensor y = st.output(x.sizes(), x.scalar_type());
    const ssd_step_problem p{n, slots, H, P, G, N, state.stride(0), x.stride(0), dt.stride(0), stride0(z), B.stride(0), C.stride(0),
                             H * P, code(x), code(dt), code(state), 0};
    check((sel ? lib.selective_step : lib.step)(&p, ptr(state), ptr_as<int32_t>(idx), ptr(x), ptr(dt), ptr_as<float>(A), ptr(B), ptr(C),
                                                ptr_as<float>(D), ptr(z), ptr_as<float>(bias), ptr(y), st.handle),
          sel ? "ssd_selective_step" : "ssd_step");
    written(state);
    return wrap(y);
}

// What both forms of the convolution share; returns the width.
int64_t check_conv(const Tensor &u, const Tensor &w, const Tensor &bias, const Tensor &win, const Tensor &idx, int64_t n, int dev) {
    const int64_t Cn = u.size(-1);
    NEED(w.dim() == 2 && win.dim() == 3, "weight has shape [channels, width], conv_states [nslots, width - 1, channels]");
    const int64_t K = w.size(1);
    NEED(u.size(-1) == 1 || u.stride(-1) == 1, "xbc: its channels must be contiguous");
    like("weight", w, {Cn, K}, F32, dev, 2);
    if (bias.defined()) like("bias", bias, {Cn}, F32, dev, 1);
    like("conv_states", win, {win.size(0), K - 1, Cn}, type_of(u), dev, 2);
    if (idx.defined()) like("state_indices", idx, {n}, I32, dev, 1);
    else NEED(win.size(0) >= n, "conv_states has fewer slots than there are sequences");
    return K;
}

// conv1d_prompt(xbc, weight, bias, conv_states, cu_seqlens, state_indices, has_initial, silu, stream)
PyObject *conv1d_prompt(PyObject *const *a) {
    const Tensor &u = arg(a[0], "xbc"), &w = arg(a[1], "weight"), &bias = arg(a[2], "bias", true), &win = arg(a[3], "conv_states"),
                 &cu = arg(a[4], "cu_seqlens", true), &idx = arg(a[5], "state_indices", true), &has = arg(a[6], "has_initial", true);
    const int dev = lead("xbc", u, 3);
    const int64_t Bt = u.size(0), L = u.size(1), Cn = u.size(2), n = cu.defined() ? cu.numel() - 1 : Bt;
    const int64_t K = check_conv(u, w, bias, win, idx, n, dev);
    if (cu.defined()) {
        NEED(n >= 1, "cu_seqlens holds no sequence");
        like("cu_seqlens", cu, {n + 1}, I32, dev, 1);
    }
    if (has.defined()) like("has_initial", has, {n}, U8 | BOOL, dev, 1);
    const Stream st(a[8], dev);
    Tensor out = st.output({Bt, L, Cn}, u.scalar_type());
    const ssd_conv_problem p{Bt, L, Cn, K, cu.defined() ? n : 0, code(u), a[7] == Py_True, 0, 0};
    check(lib.conv1d_prompt(&p, ptr(u), u.stride(0), u.stride(1), ptr_as<float>(w), ptr_as<float>(bias), ptr_as<int32_t>(cu), ptr(win),
                            win.size(0), win.stride(0), ptr_as<int32_t>(idx), ptr_as<uint8_t>(has), ptr(out), L * Cn, Cn, st.handle),
          "ssd_conv1d_prompt");
    written(win);
    return wrap(out);
}

// conv1d_step(xbc, weight, bias, conv_states, state_indices, silu, stream)
PyObject *conv1d_step(PyObject *const *a) {
    const Tensor &u = arg(a[0], "xbc"), &w = arg(a[1], "weight"), &bias = arg(a[2], "bias", true), &win = arg(a[3], "conv_states"),
                 &idx = arg(a[4], "state_indices", true);
    const int dev = lead("xbc", u, 2);
    const int64_t n = u.size(0), Cn = u.size(1), K = check_conv(u, w, bias, win, idx, n, dev);
    const Stream st(a[6], dev);
    Tensor out = st.output({n, Cn}, u.scalar_type());
    if (n > 0) {
        const ssd_conv_problem p{n, 1, Cn, K, 0, code(u), a[5] == Py_True, 0, 0};
        check(lib.conv1d_step(&p, ptr(u), u.stride(0), ptr_as<float>(w), ptr_as<float>(bias), ptr(win), win.size(0), win.stride(0),
                              ptr_as<int32_t>(idx), ptr(out), Cn, st.handle),
              "ssd_conv1d_step");
        written(win);
    }
    return wrap(out);
}

// snapshot(store, states, snapshots, scales, state_indices, slots, stream)
PyObject *snapshot(PyObject *const *a) {
    const bool store = a[0] == Py_True;
    const Tensor &states = arg(a[1], "states"), &snaps = arg(a[2], "snapshots"), &scales = arg(a[3], "scales"),
                 &idx = arg(a[4], "state_indices", true), &slots = arg(a[5], "slots", true);
    const int64_t dims = states.dim();
    NEED(dims >= 2, "states has shape [nslots, ..., dstate]");
    const int dev = lead("states", states, dims);
    int64_t rows = 1, n1 = states.size(-1);
    NEED(states.stride(-1) == 1 || n1 == 1, "states: all dimensions but the first must be contiguous");
    for (int64_t k = dims - 2; k > 0; --k) {
        NEED(states.size(k) == 1 || states.stride(k) == n1 * rows, "states: all dimensions but the first must be contiguous");
        rows *= states.size(k);
    }
    NEED(snaps.dim() == dims && snaps.sizes().slice(1) == states.sizes().slice(1), "snapshots has the states' inner shape");
    NEED(scales.dim() == dims - 1 && scales.sizes() == snaps.sizes().slice(0, dims - 1), "scales has one value for each row of the snapshots");
    NEED(type_of(snaps) == I8 && type_of(scales) == F32, "snapshots is int8 and scales float32");
    NEED(snaps.is_contiguous() && scales.is_contiguous(), "snapshots and scales must be contiguous");
    NEED(snaps.is_cuda() && scales.is_cuda() && snaps.get_device() == dev && scales.get_device() == dev, "snapshots and scales are not on GPU %d", dev);
    const int64_t n = idx.defined() ? idx.numel() : slots.defined() ? slots.numel() : states.size(0);
    if (idx.defined()) like("state_indices", idx, {n}, I32, dev, 1);
    else NEED(states.size(0) >= n, "there are fewer states than slots");
    if (slots.defined()) like("slots", slots, {n}, I32, dev, 1);
    else NEED(snaps.size(0) >= n, "there are fewer snapshots than states");
    const Stream st(a[6], dev);
    const ssd_snapshot_problem p{n, rows, n1, states.size(0), snaps.size(0), states.stride(0), code(states), 0};
    if (store) {
        check(lib.snapshot_store(&p, ptr(states), ptr_as<int32_t>(idx), ptr_as<int8_t>(snaps), ptr_as<float>(scales), ptr_as<int32_t>(slots), st.handle),
              "ssd_snapshot_store");
        written(snaps);
        written(scales);
    } else {
        check(lib.snapshot_load(&p, ptr_as<int8_t>(snaps), ptr_as<float>(scales), ptr_as<int32_t>(slots), ptr(states), ptr_as<int32_t>(idx), st.handle),
              "ssd_snapshot_load");
        written(states);
    }
    Py_RETURN_NONE;
}

// An ssd_tensor; the last `inner` dimensions get the strides of contiguous ones, whatever torch notes for sizes of 1.
ssd_tensor desc(const Tensor &t, int inner) {
    ssd_tensor d{};
    if (!t.defined()) return d;
    d.ptr = t.data_ptr();
    d.dtype = code(t);
    int64_t n = 1;
    for (int64_t k = t.dim() - 1; k >= 0; --k) {
        d.stride[k] = t.dim() - k <= inner ? n : t.stride(k);
        n *= t.size(k);
    }
    return d;
}

struct Scan {
    int dev;
    int64_t S, Bt, L, Dm, G, N;
    ssd_selective_problem p;
    ssd_fwd_args f;
};
// The scan's inputs, in the order x, dt, A, B, C, D, z, dt_bias, initial_states, cu_seqlens.
Scan scan_inputs(const Tensor *const *t) {
    const Tensor &x = *t[0], &dt = *t[1], &A = *t[2], &B = *t[3], &C = *t[4], &D = *t[5], &z = *t[6], &bias = *t[7], &init = *t[8], &cu = *t[9];
    Scan s{};
    s.dev = lead("x", x, 3);
    NEED(B.dim() == 4, "B has shape [batch, seqlen, ngroups, dstate]");
    s.Bt = x.size(0); s.L = x.size(1); s.Dm = x.size(2); s.G = B.size(2); s.N = B.size(3);
    const int own = type_of(x), dev = s.dev;
    s.S = s.Bt;
    if (cu.defined()) {
        s.S = cu.numel() - 1;
        NEED(s.S >= 1, "cu_seqlens holds no sequence");
        like("cu_seqlens", cu, {s.S + 1}, I32, dev, 1);
    }
    like("x", x, {s.Bt, s.L, s.Dm}, own, dev, 1);
    like("dt", dt, {s.Bt, s.L, s.Dm}, F32 | own, dev, 1);
    like("A", A, {s.Dm, s.N}, F32, dev, 2);
    like("B", B, {s.Bt, s.L, s.G, s.N}, own, dev, 1);
    like("C", C, {s.Bt, s.L, s.G, s.N}, own, dev, 1);
    if (D.defined()) like("D", D, {s.Dm}, F32, dev, 1);
    if (z.defined()) like("z", z, {s.Bt, s.L, s.Dm}, own, dev, 1);
    if (bias.defined()) like("dt_bias", bias, {s.Dm}, F32, dev, 1);
    if (init.defined()) like("initial_states", init, {s.S, s.Dm, s.N}, F32 | BF16, dev, 3);
    s.p = {s.Bt, s.L, s.Dm, s.G, s.N, cu.defined() ? s.S : 0};
    s.f.x = desc(x, 1); s.f.dt = desc(dt, 1); s.f.A = desc(A, 2); s.f.B = desc(B, 1); s.f.C = desc(C, 1);
    s.f.D = desc(D, 1); s.f.z = desc(z, 1); s.f.dt_bias = desc(bias, 1); s.f.initial_states = desc(init, 3);
    s.f.cu_seqlens = ptr_as<int32_t>(cu);
    return s;
}
const char *const scan_names[10] = {"x", "dt", "A", "B", "C", "D", "z", "dt_bias", "initial_states", "cu_seqlens"};

// selective_fwd(the scan's inputs, return_final, state_dtype (-1: the initial states' or f32), keep, stream)
PyObject *selective_fwd(PyObject *const *a) {
    const Tensor *t[10];
    for (int i = 0; i < 10; ++i) t[i] = &arg(a[i], scan_names[i], i >= 5);
    Scan s = scan_inputs(t);
    const Tensor &x = *t[0], &init = *t[8];
    const bool want_final = a[10] == Py_True, keep = a[12] == Py_True;
    const long sd = PyLong_AsLong(a[11]);
    const Stream st(a[13], s.dev);
    Tensor y = st.output({s.Bt, s.L, s.Dm}, x.scalar_type()), final, kept;
    s.f.y = desc(y, 3);
    if (want_final) {
        const bool bf16 = sd < 0 ? init.defined() && init.scalar_type() == at::kBFloat16 : sd == SSD_BF16;
        final = st.output({s.S, s.Dm, s.N}, bf16 ? at::kBFloat16 : at::kFloat);
        s.f.final_states = desc(final, 3);
    }
    if (keep) {
        size_t n = 0;
        check(lib.chunk_states_size(&s.p, &n), "ssd_selective_chunk_states_size");
        kept = st.output({(int64_t)n}, at::kByte);
        s.f.chunk_states = kept.data_ptr();
    }
    size_t n = 0;
    check(lib.fwd_workspace_size(&s.p, &n), "ssd_selective_fwd_workspace_size");
    Tensor ws;
    if (n > 0) ws = st.empty({(int64_t)n}, at::kByte);
    check(lib.selective_fwd(&s.p, &s.f, ptr(ws), n, st.handle), "ssd_selective_fwd");
    PyObject *r = PyTuple_New(keep ? 3 : 2);
    if (!r) throw Raised();
    PyTuple_SET_ITEM(r, 0, wrap(y));
    PyTuple_SET_ITEM(r, 1, want_final ? wrap(final) : Py_NewRef(Py_None));
    if (keep) PyTuple_SET_ITEM(r, 2, wrap(kept));
    return r;
}

// selective_bwd(the scan's inputs, dy, dfinal_states, chunk_states, workspace, stream): workspace has get(bytes), or is None
PyObject *selective_bwd(PyObject *const *a) {
    const Tensor *t[10];
    for (int i = 0; i < 10; ++i) t[i] = &arg(a[i], scan_names[i], i >= 5);
    Scan s = scan_inputs(t);
    const Tensor &x = *t[0], &dt = *t[1], &D = *t[5], &z = *t[6], &bias = *t[7], &init = *t[8];
    const Tensor &dy = arg(a[10], "dy"), &dfinal = arg(a[11], "dfinal_states", true), &kept = arg(a[12], "chunk_states", true);
    like("dy", dy, {s.Bt, s.L, s.Dm}, type_of(x), s.dev, 1);
    if (dfinal.defined()) like("dfinal_states", dfinal, {s.S, s.Dm, s.N}, F32 | BF16, s.dev, 3);
    if (kept.defined()) {
        size_t n = 0;
        check(lib.chunk_states_size(&s.p, &n), "ssd_selective_chunk_states_size");
        NEED(kept.is_cuda() && kept.get_device() == s.dev && kept.is_contiguous(), "chunk_states: a contiguous buffer on GPU %d", s.dev);
        NEED(kept.nbytes() >= n, "chunk_states is smaller than %zu bytes", n);
        s.f.chunk_states = kept.data_ptr();
    }
    const Stream st(a[14], s.dev);
    const auto f32 = at::kFloat;
    ssd_bwd_args b{};
    b.fwd = s.f;
    b.dy = desc(dy, 1);
    b.dfinal_states = desc(dfinal, 3);
    PyObject *g = PyDict_New();
    if (!g) throw Raised();
    try {
        auto out = [&](const char *name, ssd_tensor &d, at::IntArrayRef shape, at::ScalarType type) {
            Tensor v = st.output(shape, type);
            d = desc(v, (int)v.dim());
            PyObject *o = wrap(v);
            const int rc = o ? PyDict_SetItemString(g, name, o) : -1;
            Py_XDECREF(o);
            if (rc) throw Raised();
        };
        out("dx", b.dx, {s.Bt, s.L, s.Dm}, x.scalar_type());
        out("ddt", b.ddt, {s.Bt, s.L, s.Dm}, dt.scalar_type());
        out("dA", b.dA, {s.Dm, s.N}, f32);
        out("dB", b.dB, {s.Bt, s.L, s.G, s.N}, x.scalar_type());
        out("dC", b.dC, {s.Bt, s.L, s.G, s.N}, x.scalar_type());
        if (D.defined()) out("dD", b.dD, {s.Dm}, f32);
        if (z.defined()) out("dz", b.dz, {s.Bt, s.L, s.Dm}, x.scalar_type());
        if (bias.defined()) out("ddt_bias", b.ddt_bias, {s.Dm}, f32);
        if (init.defined()) out("dinitial_states", b.dinitial_states, {s.S, s.Dm, s.N}, init.scalar_type());
        size_t n = 0;
        check(lib.bwd_workspace_size(&s.p, &b, &n), "ssd_selective_bwd_workspace_size");
        Tensor ws;
        if (a[13] != Py_None) {
            PyObject *o = PyObject_CallMethod(a[13], "get", "n", (Py_ssize_t)n);
            if (!o) throw Raised();
            const bool ok = THPVariable_Check(o);
            if (ok) ws = THPVariable_Unpack(o);
            Py_DECREF(o);
            NEED(ok && ws.is_cuda() && ws.get_device() == s.dev && ws.is_contiguous(), "workspace.get(bytes) gives a contiguous tensor on GPU %d", s.dev);
            st.used(ws);
        } else {
            ws = st.empty({(int64_t)(n < 256 ? 256 : n)}, at::kByte);
        }
        check(lib.selective_bwd(&s.p, &b, ws.data_ptr(), ws.nbytes(), st.handle), "ssd_selective_bwd");
    } catch (...) {
        Py_DECREF(g);
        throw;
    }
    return g;
}

// init(SSDError, torch.OutOfMemoryError, addresses of the library's functions in Lib's order)
PyObject *init(PyObject *const *a) {
    void **to = reinterpret_cast<void **>(&lib);
    for (size_t i = 0; i < sizeof(lib) / sizeof(void *); ++i) {
        to[i] = PyLong_AsVoidPtr(a[2 + i]);
        if (PyErr_Occurred()) throw Raised();
    }
    Py_XSETREF(ssd_error, Py_NewRef(a[0]));
    Py_XSETREF(out_of_memory, Py_NewRef(a[1]));
    Py_RETURN_NONE;
}

// No C++ exception passes into Python: torch's become RuntimeError.
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", n, N);
        return nullptr;
    }
    try {
        return F(a);
    } catch (const Raised &) {
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(out_of_memory ? out_of_memory : PyExc_MemoryError, e.what_without_backtrace());
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}
#define ENTRY(name, n) {#name, (PyCFunction)(void *)entry<name, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(step, 12),          ENTRY(conv1d_prompt, 9), ENTRY(conv1d_step, 7),
                         ENTRY(snapshot, 7),       ENTRY(selective_fwd, 14), ENTRY(selective_bwd, 15),
                         ENTRY(init, 2 + sizeof(Lib) / sizeof(void *)),      {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
