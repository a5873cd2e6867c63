// selective.cu -- the C entry points of the selective scan: validation, workspace, launches.
#include "selective.cuh"

using namespace ssd;

namespace {

bool al(const void *p, size_t n) { return (uintptr_t)p % n == 0; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
size_t esize(int dtype) { return dtype == SSD_BF16 ? 2 : 4; }
bool type_ok(int dtype) { return dtype == SSD_F32 || dtype == SSD_BF16; }

#define SEL_TRY(expr)                  \
    do {                               \
        ssd_status _s = (expr);        \
        if (_s != SSD_OK) return _s;   \
    } while (0)

ssd_status check_problem(const ssd_selective_problem *p, bool varlen) {
    if (p == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    if (p->batch < 1 || p->seqlen < 0 || p->channels < 1 || p->ngroups < 1 || p->dstate < 1) return SSD_ERR_INVALID_ARGUMENT;
    if (p->channels % p->ngroups != 0) return SSD_ERR_INVALID_ARGUMENT;
    if (varlen ? (p->batch != 1 || p->nseqs < 1) : p->nseqs != 0) return SSD_ERR_INVALID_ARGUMENT;
    if (p->dstate > 128) return SSD_ERR_UNSUPPORTED;
    // counters of tokens, chunks and blocks are 32-bit; element offsets are 64-bit
    const int64_t ns = varlen ? p->nseqs : p->batch;
    if (p->seqlen > ((int64_t)1 << 30) || p->channels > ((int64_t)1 << 22) || ns > ((int64_t)1 << 24) ||
        ns * ((p->channels + 3) / 4 + p->ngroups) > ((int64_t)1 << 30) ||
        (p->seqlen / SEL_Q + 1) * ns > ((int64_t)1 << 30) ||
        p->batch * p->seqlen * p->ngroups > ((int64_t)1 << 29))
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

int64_t chunk_slots(const ssd_selective_problem *p) {
    return p->nseqs ? p->seqlen / SEL_Q + p->nseqs : p->batch * ((p->seqlen + SEL_Q - 1) / SEL_Q);
}

// A token tensor [batch, seqlen, (groups,) inner] of `dtype`.
ssd_status check_tok(const ssd_selective_problem *p, const ssd_tensor &t, int dtype, bool grouped) {
    if (p->seqlen == 0) return SSD_OK;
    if (t.ptr == nullptr || t.dtype != dtype || !type_ok(dtype)) return SSD_ERR_INVALID_ARGUMENT;
    const int64_t inner = grouped ? p->dstate : p->channels;
    if (t.stride[grouped ? 3 : 2] != 1) return SSD_ERR_INVALID_ARGUMENT;
    if (p->seqlen > 1 && t.stride[1] >= ((int64_t)1 << 28)) return SSD_ERR_UNSUPPORTED;   // a token's bytes fit 31 bits
    if (grouped && p->ngroups > 1 && t.stride[2] < inner) return SSD_ERR_INVALID_ARGUMENT;
    const int64_t row = grouped ? (p->ngroups > 1 ? t.stride[2] * (p->ngroups - 1) : 0) + inner : inner;
    if (p->seqlen > 1 && t.stride[1] < row) return SSD_ERR_INVALID_ARGUMENT;
    if (p->batch > 1 && t.stride[0] < t.stride[1] * (p->seqlen - 1) + row) return SSD_ERR_INVALID_ARGUMENT;
    return al(t.ptr, esize(dtype)) ? SSD_OK : SSD_ERR_MISALIGNED;
}
ssd_status check_par(const ssd_tensor &t, bool required, bool matrix, const ssd_selective_problem *p) {
    if (t.ptr == nullptr) return required ? SSD_ERR_INVALID_ARGUMENT : SSD_OK;
    if (t.dtype != SSD_F32 || t.stride[matrix ? 1 : 0] != 1 || (matrix && t.stride[0] != p->dstate))
        return SSD_ERR_INVALID_ARGUMENT;
    return al(t.ptr, 4) ? SSD_OK : SSD_ERR_MISALIGNED;
}
ssd_status check_state(const ssd_tensor &t, const ssd_selective_problem *p) {
    if (t.ptr == nullptr) return SSD_OK;
    const int64_t ns = p->nseqs ? p->nseqs : p->batch;
    if (!type_ok(t.dtype) || t.stride[2] != 1 || t.stride[1] != p->dstate ||
        (ns > 1 && t.stride[0] != p->channels * p->dstate))
        return SSD_ERR_INVALID_ARGUMENT;
    return al(t.ptr, esize(t.dtype)) ? SSD_OK : SSD_ERR_MISALIGNED;
}

ssd_status check_inputs(const ssd_selective_problem *p, const ssd_fwd_args *a) {
    if (a == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    SEL_TRY(check_problem(p, a->cu_seqlens != nullptr));
    if (!type_ok(a->x.dtype)) return SSD_ERR_INVALID_ARGUMENT;
    if (a->dt.dtype != SSD_F32 && a->dt.dtype != a->x.dtype) return SSD_ERR_INVALID_ARGUMENT;
    SEL_TRY(check_tok(p, a->x, a->x.dtype, false));
    SEL_TRY(check_tok(p, a->dt, a->dt.dtype, false));
    SEL_TRY(check_tok(p, a->B, a->x.dtype, true));
    SEL_TRY(check_tok(p, a->C, a->x.dtype, true));
    if (a->z.ptr) SEL_TRY(check_tok(p, a->z, a->x.dtype, false));
    SEL_TRY(check_par(a->A, true, true, p));
    SEL_TRY(check_par(a->D, false, false, p));
    SEL_TRY(check_par(a->dt_bias, false, false, p));
    SEL_TRY(check_state(a->initial_states, p));
    if (a->chunk_states && !al(a->chunk_states, 16)) return SSD_ERR_MISALIGNED;
    return SSD_OK;
}

bool fours(const ssd_tensor &t, int dims) {
    if (t.ptr == nullptr) return true;
    for (int i = 0; i < dims; ++i)
        if (t.stride[i] % 4 != 0) return false;
    return al(t.ptr, 4 * esize(t.dtype));
}

SelArgs make_args(const ssd_selective_problem *p, const ssd_fwd_args *f) {
    SelArgs a{};
    a.x = f->x.ptr; a.xb = f->x.stride[0]; a.xt = f->x.stride[1];
    a.dt = f->dt.ptr; a.dtb = f->dt.stride[0]; a.dtt = f->dt.stride[1];
    a.B = f->B.ptr; a.Bb = f->B.stride[0]; a.Bt = f->B.stride[1]; a.Bg = f->B.stride[2];
    a.C = f->C.ptr; a.Cb = f->C.stride[0]; a.Ct = f->C.stride[1]; a.Cg = f->C.stride[2];
    a.z = f->z.ptr; a.zb = f->z.stride[0]; a.zt = f->z.stride[1];
    a.A = static_cast<const float *>(f->A.ptr);
    a.D = static_cast<const float *>(f->D.ptr);
    a.bias = static_cast<const float *>(f->dt_bias.ptr);
    a.init = f->initial_states.ptr;
    a.init_bf16 = f->initial_states.dtype == SSD_BF16;
    a.dt_f32 = f->dt.dtype == SSD_F32;
    a.cu = f->cu_seqlens;
    a.nbatch = (int)p->batch; a.seqlen = (int)p->seqlen; a.channels = (int)p->channels; a.ngroups = (int)p->ngroups;
    a.dpg = (int)(p->channels / p->ngroups);
    a.N = (int)p->dstate; a.NP = sel_pad(p->dstate);
    a.nseqs = (int)(p->nseqs ? p->nseqs : p->batch);
    a.nslots = (int)chunk_slots(p);
    a.states = static_cast<float *>(f->chunk_states);
    sel_segments(a.nseqs, p->channels, p->ngroups, p->seqlen, a.NP, &a.nseg, &a.seglen);
    a.vec = (p->ngroups == 1 || a.dpg % 4 == 0) && fours(f->x, 2) && fours(f->dt, 2) && fours(f->z, 2);
    a.vecA = p->dstate % 4 == 0 && al(f->A.ptr, 16);
    a.vecBC = fours(f->B, 3) && fours(f->C, 3);
    return a;
}

size_t states_bytes(const ssd_selective_problem *p) {
    return (size_t)chunk_slots(p) * (size_t)p->channels * (size_t)sel_pad(p->dstate) * sizeof(float);
}

// The segments' ends and sums of dt lie one after the other.
void set_segments(SelArgs &a, void *at) {
    a.segE = static_cast<float *>(at);
    a.segS = a.segE + (size_t)a.nseqs * a.nseg * a.channels * a.NP;
}
size_t seg_bytes(const ssd_selective_problem *p) {
    int nseg, seglen;
    const int64_t ns = p->nseqs ? p->nseqs : p->batch;
    sel_segments(ns, p->channels, p->ngroups, p->seqlen, sel_pad(p->dstate), &nseg, &seglen);
    return up256(sel_seg_bytes(ns, p->channels, nseg, sel_pad(p->dstate)));
}

// The backward's workspace: adjoints, shares of dA and (dD, ddt_bias), shares of dB and dC, segments, and
// the forward's kept states where the caller brings none.
struct BwdPlan {
    size_t adj, pA, pD, pBC, seg, states, total;
    int nsets, cps;
};
BwdPlan plan(const ssd_selective_problem *p, bool kept) {
    BwdPlan w;
    const int64_t slots = chunk_slots(p);
    sel_bwd_sets((int)p->channels, (int)p->ngroups, slots, &w.nsets, &w.cps);
    const size_t st = up256(states_bytes(p));
    w.adj = 0;
    w.pA = st;
    w.pD = 2 * st;
    w.pBC = w.pD + up256((size_t)slots * (size_t)p->channels * 2 * sizeof(float));
    w.seg = w.pBC + up256((size_t)w.nsets * 2 * (size_t)(p->batch * p->seqlen * p->ngroups) *
                             (size_t)sel_pad(p->dstate) * sizeof(float));
    w.states = w.seg + seg_bytes(p);
    w.total = w.states + (kept ? 0 : st);
    return w;
}

ssd_status check_bwd(const ssd_selective_problem *p, const ssd_bwd_args *b) {
    if (b == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    const ssd_fwd_args *f = &b->fwd;
    SEL_TRY(check_inputs(p, f));
    SEL_TRY(check_tok(p, b->dy, f->x.dtype, false));
    SEL_TRY(check_tok(p, b->dx, f->x.dtype, false));
    SEL_TRY(check_tok(p, b->ddt, f->dt.dtype, false));
    SEL_TRY(check_tok(p, b->dB, f->x.dtype, true));
    SEL_TRY(check_tok(p, b->dC, f->x.dtype, true));
    SEL_TRY(check_par(b->dA, true, true, p));
    if (f->z.ptr) SEL_TRY(check_tok(p, b->dz, f->x.dtype, false));
    SEL_TRY(check_par(b->dD, f->D.ptr != nullptr, false, p));
    SEL_TRY(check_par(b->ddt_bias, f->dt_bias.ptr != nullptr, false, p));
    SEL_TRY(check_state(b->dfinal_states, p));
    if (f->initial_states.ptr && b->dinitial_states.ptr == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    SEL_TRY(check_state(b->dinitial_states, p));
    const int64_t slots = chunk_slots(p);
    int nsets, cps;
    sel_bwd_sets((int)p->channels, (int)p->ngroups, slots, &nsets, &cps);
    if (slots * p->ngroups * nsets > ((int64_t)1 << 31) - 1) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

}  // namespace

extern "C" {

ssd_status ssd_selective_chunk_states_size(const ssd_selective_problem *p, size_t *bytes) {
    if (bytes == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    SEL_TRY(check_problem(p, p != nullptr && p->nseqs != 0));
    *bytes = states_bytes(p);
    return SSD_OK;
}

ssd_status ssd_selective_fwd_workspace_size(const ssd_selective_problem *p, size_t *bytes) {
    if (bytes == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    SEL_TRY(check_problem(p, p != nullptr && p->nseqs != 0));
    *bytes = seg_bytes(p);
    return SSD_OK;
}

ssd_status ssd_selective_fwd(const ssd_selective_problem *p, const ssd_fwd_args *f, void *workspace, size_t workspace_bytes,
                             void *stream) {
    SEL_TRY(check_inputs(p, f));
    SEL_TRY(check_tok(p, f->y, f->x.dtype, false));
    SEL_TRY(check_state(f->final_states, p));
    if (const size_t need = seg_bytes(p)) {
        if (workspace == nullptr || workspace_bytes < need) return SSD_ERR_WORKSPACE_TOO_SMALL;
        if (!al(workspace, 256)) return SSD_ERR_MISALIGNED;
    }
    if (p->seqlen == 0 && f->final_states.ptr == nullptr) return SSD_OK;
    SelArgs a = make_args(p, f);
    a.vec = a.vec && fours(f->y, 2);
    set_segments(a, workspace);
    a.y = f->y.ptr; a.yb = f->y.stride[0]; a.yt = f->y.stride[1];
    a.final = f->final_states.ptr;
    a.final_bf16 = f->final_states.dtype == SSD_BF16;
    return sel_launch_fwd(a, f->x.dtype == SSD_BF16, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_selective_bwd_workspace_size(const ssd_selective_problem *p, const ssd_bwd_args *b, size_t *bytes) {
    if (bytes == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    SEL_TRY(check_bwd(p, b));
    *bytes = plan(p, b->fwd.chunk_states != nullptr).total;
    return SSD_OK;
}

ssd_status ssd_selective_bwd(const ssd_selective_problem *p, const ssd_bwd_args *b, void *workspace,
                             size_t workspace_bytes, void *stream) {
    SEL_TRY(check_bwd(p, b));
    const ssd_fwd_args *f = &b->fwd;
    const BwdPlan w = plan(p, f->chunk_states != nullptr);
    if (w.total > 0) {
        if (workspace == nullptr || workspace_bytes < w.total) return SSD_ERR_WORKSPACE_TOO_SMALL;
        if (!al(workspace, 256)) return SSD_ERR_MISALIGNED;
    }
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    cudaStream_t st = (cudaStream_t)stream;
    const bool bf16 = f->x.dtype == SSD_BF16;
    SelArgs a = make_args(p, f);
    set_segments(a, ws + w.seg);
    if (a.states == nullptr && p->seqlen > 0) {       // the states entering the chunks, without an output
        a.states = reinterpret_cast<float *>(ws + w.states);
        if (sel_launch_fwd(a, bf16, st) != cudaSuccess) return SSD_ERR_CUDA;
    }
    a.adj = reinterpret_cast<float *>(ws + w.adj);
    a.pA = reinterpret_cast<float *>(ws + w.pA);
    a.pD = reinterpret_cast<float *>(ws + w.pD);
    a.pBC = reinterpret_cast<float *>(ws + w.pBC);
    a.nsets = w.nsets;
    a.cps = w.cps;
    a.dy = b->dy.ptr; a.dyb = b->dy.stride[0]; a.dyt = b->dy.stride[1];
    a.dx = b->dx.ptr; a.dxb = b->dx.stride[0]; a.dxt = b->dx.stride[1];
    a.ddt = b->ddt.ptr; a.ddtb = b->ddt.stride[0]; a.ddtt = b->ddt.stride[1];
    a.dz = b->dz.ptr; a.dzb = b->dz.stride[0]; a.dzt = b->dz.stride[1];
    a.dB = b->dB.ptr; a.dBb = b->dB.stride[0]; a.dBt = b->dB.stride[1]; a.dBg = b->dB.stride[2];
    a.dC = b->dC.ptr; a.dCb = b->dC.stride[0]; a.dCt = b->dC.stride[1]; a.dCg = b->dC.stride[2];
    a.vec = a.vec && fours(b->dy, 2);
    a.vec_out = (p->ngroups == 1 || a.dpg % 4 == 0) && fours(b->dx, 2) && fours(b->ddt, 2) && fours(b->dz, 2);
    a.dA = static_cast<float *>(b->dA.ptr);
    a.dD = f->D.ptr ? static_cast<float *>(b->dD.ptr) : nullptr;
    a.dbias = f->dt_bias.ptr ? static_cast<float *>(b->ddt_bias.ptr) : nullptr;
    a.dfinal = b->dfinal_states.ptr;
    a.dfinal_bf16 = b->dfinal_states.dtype == SSD_BF16;
    a.dinit = b->dinitial_states.ptr;
    a.dinit_bf16 = b->dinitial_states.dtype == SSD_BF16;
    return sel_launch_bwd(a, bf16, st) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
