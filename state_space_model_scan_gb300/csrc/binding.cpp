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
#include <c10/core/AutogradState.h>
#include <ATen/ops/zeros_like.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/saved_variable.h>

#include <math.h>
#include <stdarg.h>

#include <array>
#include <initializer_list>
#include <memory>
#include <mutex>
#include <optional>
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
    decltype(&ssd_delta_chunk_states_size) delta_states_size;
    decltype(&ssd_delta_fwd_workspace_size) delta_fwd_workspace_size;
    decltype(&ssd_delta_fwd) delta_fwd;
    decltype(&ssd_delta_bwd_workspace_size) delta_bwd_workspace_size;
    decltype(&ssd_delta_bwd) delta_bwd;
    decltype(&ssd_delta_step) delta_step;
    decltype(&ssd_qk_norm_fwd) qk_fwd;
    decltype(&ssd_qk_norm_bwd_workspace_size) qk_bwd_workspace_size;
    decltype(&ssd_qk_norm_bwd) qk_bwd;
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

// ---- the gated delta rule
struct Delta {
    int dev;
    int64_t S, B, L, G, H, V, K;
    ssd_delta_problem p;
    ssd_delta_args f;
};
const char *const delta_names[7] = {"q", "k", "v", "g", "beta", "initial_states", "cu_seqlens"};

// A float argument; nothing where it is None.
std::optional<double> number(PyObject *o, const char *name) {
    if (o == Py_None) return std::nullopt;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        fail(PyExc_TypeError, "%s is not a number", name);
    }
    return v;
}

// q, k, v, g, beta, initial_states, cu_seqlens; scale: dstate^-0.5 where it is None
Delta delta_inputs(const Tensor *const *t, std::optional<double> scale) {
    const Tensor &q = *t[0], &k = *t[1], &v = *t[2], &g = *t[3], &beta = *t[4], &init = *t[5], &cu = *t[6];
    Delta s{};
    const int dev = s.dev = lead("v", v, 4), own = type_of(v);
    NEED(q.dim() == 4, "q has shape [batch, seqlen, ngroups, dstate]");
    s.B = v.size(0); s.L = v.size(1); s.H = v.size(2); s.V = v.size(3); s.G = q.size(2); s.K = q.size(3);
    s.S = s.B;
    if (cu.defined()) {
        s.S = cu.numel() - 1;
        NEED(s.S >= 1, "cu_seqlens holds no sequence");
        like("cu_seqlens", cu, {s.S + 1}, I32, dev, 1);
    }
    like("q", q, {s.B, s.L, s.G, s.K}, own, dev, 1);
    like("k", k, {s.B, s.L, s.G, s.K}, own, dev, 1);
    like("v", v, {s.B, s.L, s.H, s.V}, own, dev, 1);
    like("g", g, {s.B, s.L, s.H}, F32 | own, dev, 0);
    like("beta", beta, {s.B, s.L, s.H}, F32 | own, dev, 0);
    if (init.defined()) like("initial_states", init, {s.S, s.H, s.V, s.K}, F32 | BF16, dev, 4);
    s.p = {s.B, s.L, s.H, s.G, s.V, s.K, cu.defined() ? s.S : 0, (float)scale.value_or(s.K > 0 ? 1.0 / sqrt((double)s.K) : 1.0), code(v)};
    s.f.q = desc(q, 1); s.f.k = desc(k, 1); s.f.v = desc(v, 1); s.f.g = desc(g, 0); s.f.beta = desc(beta, 0);
    s.f.initial_states = desc(init, 4);
    s.f.cu_seqlens = ptr_as<int32_t>(cu);
    s.f.zero_rest = 1;                                      // (outputs are allocated here)
    return s;
}

struct DeltaOut {
    Tensor o, final, kept;
};
// state_dtype -1: the initial states' or f32
DeltaOut delta_forward(const Tensor *const *t, std::optional<double> scale, bool want_final, long state_dtype, bool keep, PyObject *stream) {
    Delta s = delta_inputs(t, scale);
    const Tensor &v = *t[2], &init = *t[5];
    const Stream st(stream, s.dev);
    DeltaOut r;
    r.o = st.output({s.B, s.L, s.H, s.V}, v.scalar_type());
    s.f.o = desc(r.o, 4);
    if (want_final) {
        const bool bf16 = state_dtype < 0 ? init.defined() && init.scalar_type() == at::kBFloat16 : state_dtype == SSD_BF16;
        r.final = st.output({s.S, s.H, s.V, s.K}, bf16 ? at::kBFloat16 : at::kFloat);
        s.f.final_states = desc(r.final, 4);
    }
    if (keep) {
        size_t n = 0;
        check(lib.delta_states_size(&s.p, &n), "ssd_delta_chunk_states_size");
        r.kept = st.output({(int64_t)n}, at::kByte);
        s.f.chunk_states = r.kept.data_ptr();
    }
    size_t n = 0;
    check(lib.delta_fwd_workspace_size(&s.p, &n), "ssd_delta_fwd_workspace_size");
    Tensor ws;
    if (n > 0) ws = st.empty({(int64_t)n}, at::kByte);
    check(lib.delta_fwd(&s.p, &s.f, ptr(ws), n, st.handle), "ssd_delta_fwd");
    return r;
}
PyObject *wrap_or_none(const Tensor &t) { return t.defined() ? wrap(t) : Py_NewRef(Py_None); }
template <int N>
void read(PyObject *const *a, const char *const (&names)[N], int required, const Tensor *(&t)[N]) {
    for (int i = 0; i < N; ++i) t[i] = &arg(a[i], names[i], i >= required);
}
// delta_fwd(the inputs, scale, return_final, state_dtype, keep, stream)
PyObject *delta_fwd(PyObject *const *a) {
    const Tensor *t[7];
    read(a, delta_names, 5, t);
    const bool keep = a[10] == Py_True;
    const DeltaOut out = delta_forward(t, number(a[7], "scale"), a[8] == Py_True, PyLong_AsLong(a[9]), keep, a[11]);
    PyObject *r = PyTuple_New(keep ? 3 : 2);
    if (!r) throw Raised();
    PyTuple_SET_ITEM(r, 0, wrap(out.o));
    PyTuple_SET_ITEM(r, 1, wrap_or_none(out.final));
    if (keep) PyTuple_SET_ITEM(r, 2, wrap(out.kept));
    return r;
}

// The tensors that are there, by name.
template <size_t N>
PyObject *dict_of(const std::array<Tensor, N> &t, const char *const (&names)[N]) {
    PyObject *g = PyDict_New();
    if (!g) throw Raised();
    for (size_t i = 0; i < N; ++i) {
        if (!t[i].defined()) continue;
        PyObject *o = wrap(t[i]);
        const int rc = o ? PyDict_SetItemString(g, names[i], o) : -1;
        Py_XDECREF(o);
        if (rc) {
            Py_DECREF(g);
            throw Raised();
        }
    }
    return g;
}
// The backward's workspace: from an object with get(bytes), or of its own.
Tensor workspace_of(PyObject *o, size_t n, const Stream &st) {
    if (o == Py_None) return st.empty({(int64_t)(n < 256 ? 256 : n)}, at::kByte);
    PyObject *r = PyObject_CallMethod(o, "get", "n", (Py_ssize_t)n);
    if (!r) throw Raised();
    const bool ok = THPVariable_Check(r);
    Tensor ws;
    if (ok) ws = THPVariable_Unpack(r);
    Py_DECREF(r);
    NEED(ok && ws.is_cuda() && ws.get_device() == st.dev && ws.is_contiguous(), "workspace.get(bytes) gives a contiguous tensor on GPU %d", st.dev);
    st.used(ws);
    return ws;
}

const char *const delta_grad_names[6] = {"dq", "dk", "dv", "dg", "dbeta", "dinitial_states"};
std::array<Tensor, 6> delta_backward(const Tensor *const *t, std::optional<double> scale, const Tensor &dO, const Tensor &dfinal, const Tensor &kept,
                                     PyObject *workspace, PyObject *stream) {
    Delta s = delta_inputs(t, scale);
    const Tensor &v = *t[2], &g = *t[3], &beta = *t[4], &init = *t[5];
    like("do", dO, {s.B, s.L, s.H, s.V}, type_of(v), s.dev, 1);
    if (dfinal.defined()) like("dfinal_states", dfinal, {s.S, s.H, s.V, s.K}, F32 | BF16, s.dev, 4);
    if (kept.defined()) {
        size_t n = 0;
        check(lib.delta_states_size(&s.p, &n), "ssd_delta_chunk_states_size");
        NEED(kept.is_cuda() && kept.get_device() == s.dev && kept.is_contiguous(), "chunk_states: a contiguous buffer on GPU %d", s.dev);
        NEED(kept.nbytes() >= n, "chunk_states is smaller than %zu bytes", n);
        s.f.chunk_states = kept.data_ptr();
    }
    const Stream st(stream, s.dev);
    ssd_delta_bwd_args b{};
    b.fwd = s.f;
    b.dO = desc(dO, 1);
    b.dfinal_states = desc(dfinal, 4);
    std::array<Tensor, 6> d = {st.output({s.B, s.L, s.G, s.K}, v.scalar_type()), st.output({s.B, s.L, s.G, s.K}, v.scalar_type()),
                               st.output({s.B, s.L, s.H, s.V}, v.scalar_type()), st.output({s.B, s.L, s.H}, g.scalar_type()),
                               st.output({s.B, s.L, s.H}, beta.scalar_type()), Tensor()};
    if (init.defined()) d[5] = st.output({s.S, s.H, s.V, s.K}, init.scalar_type());
    b.dq = desc(d[0], 4); b.dk = desc(d[1], 4); b.dv = desc(d[2], 4); b.dg = desc(d[3], 3); b.dbeta = desc(d[4], 3); b.dinitial_states = desc(d[5], 4);
    size_t n = 0;
    check(lib.delta_bwd_workspace_size(&s.p, kept.defined(), &n), "ssd_delta_bwd_workspace_size");
    Tensor ws = workspace_of(workspace, n, st);
    check(lib.delta_bwd(&s.p, &b, ws.data_ptr(), ws.nbytes(), st.handle), "ssd_delta_bwd");
    return d;
}
// delta_bwd(the inputs, scale, do, dfinal_states, chunk_states, workspace, stream)
PyObject *delta_bwd(PyObject *const *a) {
    const Tensor *t[7];
    read(a, delta_names, 5, t);
    return dict_of(delta_backward(t, number(a[7], "scale"), arg(a[8], "do"), arg(a[9], "dfinal_states", true), arg(a[10], "chunk_states", true), a[11], a[12]),
                   delta_grad_names);
}

// ---- autograd: nodes of their own, since a Python function's way into the graph and back takes 20 to 50 us of host time more a step
namespace ag = torch::autograd;

// What a node does under the interpreter's lock; a Python exception goes on as the engine carries those.
template <typename F>
auto locked(F f) {
    struct Lock {
        PyGILState_STATE s = PyGILState_Ensure();
        ~Lock() { PyGILState_Release(s); }
    } lock;
    try {
        return f();
    } catch (const Raised &) {
        python_error e;
        e.persist();
        throw std::move(e);
    }
}
// A backward's gradients: where a graph of them is asked for, one that refuses to be differentiated.
void refuse_second(ag::variable_list &d, ag::edge_list &&edges) {
    std::shared_ptr<ag::Node> no(new ag::Error("the gradients of this operator cannot be differentiated again", std::move(edges)), ag::deleteNode);
    for (Tensor &t : d)
        if (t.defined()) ag::set_history(t, no);
}
// An output's gradient with unit stride in its last dimension
Tensor unit(const Tensor &t) { return !t.defined() || t.stride(-1) == 1 ? t : t.contiguous(); }

// No operator here has a forward-mode derivative: a tensor that carries a tangent is refused, where an output without one would be wrong in
// silence.
void refuse_tangent(const Tensor &t, const char *name) {
    if (t.defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined())
        fail(PyExc_NotImplementedError, "%s carries a tangent: this operator has no forward-mode derivative", name);
}

// An operator's node: its N inputs (and one tensor more) saved.
template <size_t N>
struct OpNode : ag::Node {
    std::array<ag::SavedVariable, N> saved;
    void save(const Tensor *const *t) {
        for (size_t i = 0; i < N; ++i) saved[i] = ag::SavedVariable(*t[i], false);
    }
    void release_variables() override {
        const std::lock_guard<std::mutex> one(mutex_);       // (two threads may go through one graph)
        for (auto &v : saved) v.reset_data();
    }
    // f(inputs, gradients) -> gradients of the inputs, without a graph
    template <typename F>
    ag::variable_list run(ag::variable_list &&grads, F f) {
        std::array<Tensor, N> in;
        {
            const std::lock_guard<std::mutex> one(mutex_);
            for (size_t i = 0; i < N; ++i) in[i] = saved[i].unpack();
        }
        const bool again = at::GradMode::is_enabled();
        ag::variable_list d;
        {
            at::NoGradGuard off;
            const Tensor *t[N];
            for (size_t i = 0; i < N; ++i) t[i] = &in[i];
            d = locked([&] {
                for (const Tensor &g : grads) refuse_tangent(g, "an output's gradient");
                return f(t, grads);
            });
        }
        if (again) {
            ag::edge_list edges = ag::collect_next_edges(ag::variable_list(in.begin(), in.end()), grads);
            refuse_second(d, std::move(edges));
        }
        return d;
    }
};
bool graph_wanted(const Tensor *const *t, int n) {
    if (!at::GradMode::is_enabled()) return false;
    for (int i = 0; i < n; ++i)
        if (t[i]->defined() && t[i]->requires_grad()) return true;
    return false;
}

struct GatedDelta : OpNode<8> {                            // the seven inputs, what the forward kept
    std::optional<double> scale;
    std::string name() const override { return "GatedDelta"; }
    ag::variable_list apply(ag::variable_list &&grads) override {
        return run(std::move(grads), [this](const Tensor *const *t, const ag::variable_list &g) {
            const Tensor &v = *t[2];
            const Tensor dO = g[0].defined() ? unit(g[0]) : at::zeros_like(v, at::MemoryFormat::Contiguous);
            auto d = delta_backward(t, scale, dO, g[1].defined() ? g[1].contiguous() : g[1], *t[7], Py_None, Py_None);
            return ag::variable_list(d.begin(), d.end());
        });
    }
};
// delta_apply(the inputs, scale, keep) -> o, final_states in a graph
PyObject *delta_apply(PyObject *const *a) {
    const Tensor *t[8];
    for (int i = 0; i < 7; ++i) {
        t[i] = &arg(a[i], delta_names[i], i >= 5);
        refuse_tangent(*t[i], delta_names[i]);
    }
    const auto scale = number(a[7], "scale");
    const bool graph = graph_wanted(t, 6);
    const DeltaOut out = delta_forward(t, scale, true, -1, graph && a[8] == Py_True, Py_None);
    if (graph) {
        t[7] = &out.kept;
        std::shared_ptr<GatedDelta> node(new GatedDelta(), ag::deleteNode);
        node->scale = scale;
        node->set_next_edges(ag::collect_next_edges(*t[0], *t[1], *t[2], *t[3], *t[4], *t[5]));
        node->save(t);
        ag::set_history(out.o, node);
        ag::set_history(out.final, node);
    }
    PyObject *r = PyTuple_New(2);
    if (!r) throw Raised();
    PyTuple_SET_ITEM(r, 0, wrap(out.o));
    PyTuple_SET_ITEM(r, 1, wrap(out.final));
    return r;
}

// delta_step(state, q, k, v, g, beta, scale, state_indices, stream)
PyObject *delta_step(PyObject *const *a) {
    const Tensor &state = arg(a[0], "state"), &q = arg(a[1], "q"), &k = arg(a[2], "k"), &v = arg(a[3], "v"), &g = arg(a[4], "g"),
                 &beta = arg(a[5], "beta"), &idx = arg(a[7], "state_indices", true);
    const int dev = lead("v", v, 3), own = type_of(v);
    NEED(q.dim() == 3, "q has shape [batch, ngroups, dstate]");
    NEED(state.dim() == 4, "state has shape [nslots, nheads, headdim, dstate]");
    const int64_t n = v.size(0), H = v.size(1), V = v.size(2), G = q.size(1), K = q.size(2), slots = state.size(0);
    like("v", v, {n, H, V}, own, dev, 2);
    like("q", q, {n, G, K}, own, dev, 2);
    like("k", k, {n, G, K}, own, dev, 2);
    like("g", g, {n, H}, F32 | own, dev, 1);
    like("beta", beta, {n, H}, F32 | own, dev, 1);
    like("state", state, {slots, H, V, K}, F32 | BF16, dev, 3);
    if (idx.defined()) like("state_indices", idx, {n}, I32, dev, 1);
    else NEED(slots >= n, "the state pool has fewer slots than there are requests");
    const double scale = number(a[6], "scale").value_or(K > 0 ? 1.0 / sqrt((double)K) : 1.0);
    const Stream st(a[8], dev);
    Tensor o = st.output(v.sizes(), v.scalar_type());
    const ssd_delta_step_problem p{n, slots, H, V, G, K, state.stride(0), q.stride(0), k.stride(0), v.stride(0), g.stride(0), beta.stride(0),
                                   H * V, (float)scale, code(v), code(g), code(beta), code(state)};
    check(lib.delta_step(&p, ptr(state), ptr_as<int32_t>(idx), ptr(q), ptr(k), ptr(v), ptr(g), ptr(beta), ptr(o), st.handle), "ssd_delta_step");
    written(state);
    return wrap(o);
}

// ---- queries and keys: norm and rotation
struct Qk {
    int dev;
    int64_t B, L, Hq, Hk, D;
    ssd_qk_problem p;
    ssd_qk_args f;
};
const char *const qk_names[7] = {"q", "k", "q_weight", "k_weight", "cos", "sin", "positions"};
struct QkHow {
    int32_t mode;
    bool interleaved;
    float eps;
};
QkHow qk_how(PyObject *const *a) { return {(int32_t)PyLong_AsLong(a[0]), a[1] == Py_True, (float)number(a[2], "eps").value_or(1e-6)}; }
// q, k, q_weight, k_weight, cos, sin, positions
Qk qk_inputs(const Tensor *const *t, const QkHow &how) {
    const Tensor &q = *t[0], &k = *t[1], &wq = *t[2], &wk = *t[3], &cos = *t[4], &sin = *t[5], &pos = *t[6];
    Qk s{};
    const int dev = s.dev = lead("q", q, 4), own = type_of(q);
    s.B = q.size(0); s.L = q.size(1); s.Hq = q.size(2); s.D = q.size(3);
    s.Hk = 0;
    like("q", q, {s.B, s.L, s.Hq, s.D}, own, dev, 1);
    if (k.defined()) {
        NEED(k.dim() == 4, "k has shape [batch, seqlen, heads, dim]");
        s.Hk = k.size(2);
        like("k", k, {s.B, s.L, s.Hk, s.D}, own, dev, 1);
    }
    if (wq.defined()) like("q_weight", wq, {s.D}, F32, dev, 1);
    if (wk.defined()) {
        NEED(k.defined(), "k_weight without k");
        like("k_weight", wk, {s.D}, F32, dev, 1);
    }
    NEED(cos.defined() == sin.defined(), "cos and sin are given together");
    int64_t rotary = 0, rows = 0;
    if (cos.defined()) {
        NEED(cos.dim() == 2, "cos has shape [positions, rotary / 2]");
        rows = cos.size(0);
        rotary = 2 * cos.size(1);
        like("cos", cos, {rows, rotary / 2}, F32, dev, 2);
        like("sin", sin, {rows, rotary / 2}, F32, dev, 2);
        NEED(rotary <= s.D, "the rotation is wider than the heads");
    }
    if (pos.defined()) like("positions", pos, {s.B, s.L}, I32, dev, 1);
    s.p = {s.B, s.L, s.Hq, s.Hk, s.D, rotary, rows, pos.defined() ? pos.stride(0) : 0, how.eps, code(q), how.mode, how.interleaved};
    s.f.q = desc(q, 1); s.f.k = desc(k, 1);
    s.f.q_weight = ptr_as<float>(wq); s.f.k_weight = ptr_as<float>(wk); s.f.cos = ptr_as<float>(cos); s.f.sin = ptr_as<float>(sin);
    s.f.positions = ptr_as<int32_t>(pos);
    return s;
}

std::array<Tensor, 2> qk_forward(const Tensor *const *t, const QkHow &how, PyObject *stream) {
    Qk s = qk_inputs(t, how);
    const Stream st(stream, s.dev);
    std::array<Tensor, 2> out = {st.output({s.B, s.L, s.Hq, s.D}, t[0]->scalar_type()), Tensor()};
    s.f.q_out = desc(out[0], 4);
    if (t[1]->defined()) {
        out[1] = st.output({s.B, s.L, s.Hk, s.D}, t[0]->scalar_type());
        s.f.k_out = desc(out[1], 4);
    }
    check(lib.qk_fwd(&s.p, &s.f, st.handle), "ssd_qk_norm_fwd");
    return out;
}
PyObject *pair_of(const std::array<Tensor, 2> &t) {
    PyObject *r = PyTuple_New(2);
    if (!r) throw Raised();
    PyTuple_SET_ITEM(r, 0, wrap(t[0]));
    PyTuple_SET_ITEM(r, 1, wrap_or_none(t[1]));
    return r;
}
// qk_fwd(the inputs, mode, interleaved, eps, stream)
PyObject *qk_fwd(PyObject *const *a) {
    const Tensor *t[7];
    read(a, qk_names, 1, t);
    return pair_of(qk_forward(t, qk_how(a + 7), a[10]));
}

const char *const qk_grad_names[4] = {"dq", "dk", "dq_weight", "dk_weight"};
std::array<Tensor, 4> qk_backward(const Tensor *const *t, const QkHow &how, const Tensor &dq, const Tensor &dk, PyObject *workspace, PyObject *stream) {
    Qk s = qk_inputs(t, how);
    NEED(dk.defined() == t[1]->defined(), "dk is given where k is");
    like("dq", dq, {s.B, s.L, s.Hq, s.D}, type_of(*t[0]), s.dev, 1);
    if (dk.defined()) like("dk", dk, {s.B, s.L, s.Hk, s.D}, type_of(*t[0]), s.dev, 1);
    const Stream st(stream, s.dev);
    ssd_qk_bwd_args b{};
    b.fwd = s.f;
    b.dq_out = desc(dq, 1); b.dk_out = desc(dk, 1);
    std::array<Tensor, 4> d = {st.output({s.B, s.L, s.Hq, s.D}, t[0]->scalar_type()), Tensor(), Tensor(), Tensor()};
    if (dk.defined()) d[1] = st.output({s.B, s.L, s.Hk, s.D}, t[0]->scalar_type());
    if (t[2]->defined()) d[2] = st.output({s.D}, at::kFloat);
    if (t[3]->defined()) d[3] = st.output({s.D}, at::kFloat);
    b.dq = desc(d[0], 4); b.dk = desc(d[1], 4);
    b.dq_weight = ptr_as<float>(d[2]); b.dk_weight = ptr_as<float>(d[3]);
    size_t n = 0;
    check(lib.qk_bwd_workspace_size(&s.p, &n), "ssd_qk_norm_bwd_workspace_size");
    Tensor ws;
    if (b.dq_weight || b.dk_weight) ws = workspace_of(workspace, n, st);
    check(lib.qk_bwd(&s.p, &b, ptr(ws), ws.defined() ? ws.nbytes() : 0, st.handle), "ssd_qk_norm_bwd");
    return d;
}
// qk_bwd(the inputs, mode, interleaved, eps, dq_out, dk_out, workspace, stream)
PyObject *qk_bwd(PyObject *const *a) {
    const Tensor *t[7];
    read(a, qk_names, 1, t);
    return dict_of(qk_backward(t, qk_how(a + 7), arg(a[10], "dq"), arg(a[11], "dk", true), a[12], a[13]), qk_grad_names);
}

struct QKNorm : OpNode<7> {
    QkHow how;
    std::string name() const override { return "QKNorm"; }
    ag::variable_list apply(ag::variable_list &&grads) override {
        return run(std::move(grads), [this](const Tensor *const *t, const ag::variable_list &g) {
            Tensor d[2];                                     // an output that nothing came of: zeros
            for (int i = 0; i < 2; ++i)
                if (t[i]->defined()) d[i] = g[i].defined() ? unit(g[i]) : at::zeros_like(*t[i], at::MemoryFormat::Contiguous);
            auto r = qk_backward(t, how, d[0], d[1], Py_None, Py_None);
            return ag::variable_list(r.begin(), r.end());
        });
    }
};
// qk_apply(the inputs, mode, interleaved, eps) -> q_out, k_out in a graph
PyObject *qk_apply(PyObject *const *a) {
    const Tensor *t[7];
    read(a, qk_names, 1, t);
    for (int i = 0; i < 7; ++i) refuse_tangent(*t[i], qk_names[i]);
    const QkHow how = qk_how(a + 7);
    const auto out = qk_forward(t, how, Py_None);
    if (graph_wanted(t, 4)) {
        std::shared_ptr<QKNorm> node(new QKNorm(), ag::deleteNode);
        node->how = how;
        node->set_next_edges(ag::collect_next_edges(*t[0], *t[1], *t[2], *t[3]));
        node->save(t);
        for (const Tensor &o : out) ag::set_history(o, node);
    }
    return pair_of(out);
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
    } catch (python_error &e) {                              // (of a hook on saved tensors)
        e.restore();
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
                         ENTRY(delta_fwd, 12),     ENTRY(delta_bwd, 13),    ENTRY(delta_step, 9),
                         ENTRY(qk_fwd, 11),        ENTRY(qk_bwd, 14),
                         ENTRY(delta_apply, 9),    ENTRY(qk_apply, 10),
                         ENTRY(init, 2 + sizeof(Lib) / sizeof(void *)),      {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
