// delta.cu -- the C entry points of the gated delta rule: validation, workspace, launches.
#include <initializer_list>

#include "delta_tc.cuh"

using namespace ssd;

namespace {

bool al(const void *p, size_t n) { return (uintptr_t)p % n == 0; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
size_t esize(int dtype) { return dtype == SSD_BF16 ? 2 : 4; }
bool type_ok(int dtype) { return dtype == SSD_F32 || dtype == SSD_BF16; }

#define DELTA_TRY(expr)                \
    do {                               \
        ssd_status _s = (expr);        \
        if (_s != SSD_OK) return _s;   \
    } while (0)

int64_t nstates(const ssd_delta_problem *p) { return p->nseqs ? p->nseqs : p->batch; }
int64_t slots(const ssd_delta_problem *p) {
    return p->seqlen == 0 ? 0 : p->nseqs ? p->seqlen / DQ + p->nseqs : p->batch * ((p->seqlen + DQ - 1) / DQ);
}

ssd_status check_problem(const ssd_delta_problem *p) {
    if (p == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    if (p->batch < 1 || p->seqlen < 0 || p->nheads < 1 || p->ngroups < 1 || p->headdim < 1 || p->dstate < 1 || p->nseqs < 0 ||
        p->nheads % p->ngroups != 0 || (p->nseqs > 0 && p->batch != 1) || !type_ok(p->dtype))
        return SSD_ERR_INVALID_ARGUMENT;
    if (p->headdim > 256 || p->dstate > 256) return SSD_ERR_UNSUPPORTED;
    // counters of tokens, chunks and blocks are 32-bit; element offsets are 64-bit
    if (p->batch > ((int64_t)1 << 24) || p->seqlen > ((int64_t)1 << 30) || p->nheads > ((int64_t)1 << 16) || p->nseqs > ((int64_t)1 << 24) ||
        nstates(p) * p->nheads > ((int64_t)1 << 27) || p->batch * (p->seqlen / DQ + 1) > ((int64_t)1 << 30) || slots(p) * p->nheads > ((int64_t)1 << 30))
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// A token tensor [batch, seqlen, n (, inner)].  What is read may have any strides but negative ones; what is written
// has rows that do not meet in any of its dimensions.
ssd_status check_tok(const ssd_delta_problem *p, const ssd_tensor &t, int dtype, int64_t n, int64_t inner, bool written) {
    if (p->seqlen == 0) return SSD_OK;
    if (t.ptr == nullptr || t.dtype != dtype || (inner > 1 && t.stride[3] != 1)) return SSD_ERR_INVALID_ARGUMENT;
    const int64_t size[3] = {p->batch, p->seqlen, n};
    for (int i = 0; i < 3; ++i)
        if (size[i] > 1 && t.stride[i] < (written ? inner : 0)) return SSD_ERR_INVALID_ARGUMENT;
    return al(t.ptr, esize(dtype)) ? SSD_OK : SSD_ERR_MISALIGNED;
}
ssd_status check_state(const ssd_delta_problem *p, const ssd_tensor &t) {
    if (t.ptr == nullptr) return SSD_OK;
    if (!type_ok(t.dtype) || (p->dstate > 1 && t.stride[3] != 1) || (p->headdim > 1 && t.stride[2] != p->dstate) ||
        (p->nheads > 1 && t.stride[1] != p->headdim * p->dstate) || (nstates(p) > 1 && t.stride[0] != p->nheads * p->headdim * p->dstate))
        return SSD_ERR_INVALID_ARGUMENT;
    return al(t.ptr, esize(t.dtype)) ? SSD_OK : SSD_ERR_MISALIGNED;
}
ssd_status check_inputs(const ssd_delta_problem *p, const ssd_delta_args *a) {
    DELTA_TRY(check_problem(p));
    if (a == nullptr || (a->cu_seqlens != nullptr) != (p->nseqs > 0)) return SSD_ERR_INVALID_ARGUMENT;
    for (const ssd_tensor *t : {&a->g, &a->beta})
        if (p->seqlen > 0 && t->dtype != SSD_F32 && t->dtype != p->dtype) return SSD_ERR_INVALID_ARGUMENT;
    DELTA_TRY(check_tok(p, a->q, p->dtype, p->ngroups, p->dstate, false));
    DELTA_TRY(check_tok(p, a->k, p->dtype, p->ngroups, p->dstate, false));
    DELTA_TRY(check_tok(p, a->v, p->dtype, p->nheads, p->headdim, false));
    DELTA_TRY(check_tok(p, a->g, a->g.dtype, p->nheads, 1, false));
    DELTA_TRY(check_tok(p, a->beta, a->beta.dtype, p->nheads, 1, false));
    DELTA_TRY(check_state(p, a->initial_states));
    if (!al(a->chunk_states, 256)) return SSD_ERR_MISALIGNED;
    if (!al(a->cu_seqlens, 4)) return SSD_ERR_MISALIGNED;
    return SSD_OK;
}

// The tensor-core path takes bf16 data of up to 128 values and keys; fp32 data is computed in fp32, and so are
// - calls of few tokens and heads: dg and dbeta are sums over a head's values and keys, and where there are only a few of them that happen
//   to be small, the roundings of bf16 operands do not average out.  (In 220 calls of 1 to 30000 tokens and heads dbeta or dg was off by
//   more than 5e-3, up to 1.3e-2, in three, of 3, 7 x 2 and 9; in fp32 by 2e-3, their own rounding.  The border lies well above those: of
//   425 calls of 1 to 60000 none was off by more than 4.0e-3 then.  A chunk of 128 x 128 on either side of it, forwards, and forwards and
//   backwards: one head 29 and 100 us in fp32, 32 heads 37 and 115, on the tensor cores 17 and 41.)
// - keys of fewer than eight features: what one token has taken up the next ones take back for the most part, the sums of att W cancel,
//   and their operands' roundings do not.  (o, dq and dg of 640 tokens, one feature: off by 1.0e-2, 1.1e-2, 1.3e-2; four: 5.9e-3, 5.9e-3,
//   5.3e-3; eight: 4.3e-3, 4.5e-3, 4.0e-3; from 64 on 2.8e-3.  8192 tokens of 32 heads x 128 values, four features, forward, and backward with
//   its forward: 1204 and 2082 us on the tensor cores, where no tensor map fills the tiles, 1109 and 2860 in fp32; eight features 234 and
//   646 on the tensor cores, 815 and 2391 as fp32 data.)
constexpr int64_t kFewTokens = 256, kFewKeys = 8;
bool on_tensor_cores(const ssd_delta_problem *p) {
    return p->dtype == SSD_BF16 && p->headdim <= 128 && p->dstate <= 128 && p->dstate >= kFewKeys && p->batch * p->seqlen * p->nheads > kFewTokens;
}

// What the forward keeps and the backward starts from: the state that enters each chunk, U, and on the tensor cores the chunks'
// matrices.
struct Kept {
    size_t S, U, tiles, total;
};
size_t state_bytes(const ssd_delta_problem *p) { return on_tensor_cores(p) ? dtc::STATE_BYTES : (size_t)p->headdim * p->dstate * 4; }
size_t value_bytes(const ssd_delta_problem *p) { return on_tensor_cores(p) ? dtc::VAL_BYTES : (size_t)DQ * p->headdim * 4; }
Kept kept_plan(const ssd_delta_problem *p) {
    const size_t ch = (size_t)slots(p) * p->nheads;
    Kept k;
    k.S = 0;
    k.U = up256(ch * state_bytes(p));
    k.tiles = k.U + up256(ch * value_bytes(p));
    k.total = k.tiles + (on_tensor_cores(p) ? up256(ch * dtc::OPS_BOTH) : 0);
    return k;
}
struct Plan {
    size_t hdr, gates, sys, att, a, tiles, seg, dS, mu, flow, part, kept, total;
    int nseg, seg0, seglen;
};
Plan plan(const ssd_delta_problem *p, bool back, bool kept) {
    const size_t ch = (size_t)slots(p) * p->nheads, mat = ch * DQ * DQ * 4;
    const bool tc = on_tensor_cores(p);
    Plan w{};
    size_t at = 0;
    auto take = [&](size_t n) { const size_t o = at; at += up256(n); return o; };
    w.hdr = take(HDR_WORDS * 4);
    if (tc) {
        w.tiles = take(back ? 0 : ch * dtc::OPS_BYTES);
        dtc::delta_segments(nstates(p), p->nheads, (p->seqlen + DQ - 1) / DQ, &w.nseg, &w.seg0, &w.seglen);
        w.seg = take(2 * (size_t)(w.nseg - 1) * nstates(p) * p->nheads * dtc::SEG_BYTES);
    } else {
        w.gates = take(ch * DGATES * 4);
        w.sys = take(mat);
        w.att = take(mat);
        if (back) w.a = take(mat);
    }
    if (back) {
        w.dS = take(ch * state_bytes(p));
        w.mu = take(ch * value_bytes(p));
        w.flow = take(tc ? 0 : ch * delta_grad_shares(slots(p), p->nheads, p->dstate) * DELTA_FLOW * 4);
        w.part = take(!tc && p->nheads > p->ngroups ? 2 * ch * DQ * p->dstate * 4 : 0);
        w.kept = take(kept ? 0 : kept_plan(p).total);
    }
    w.total = at;
    return w;
}

// Whether every row of a token tensor starts at 16 bytes.
bool aligned_rows(const ssd_delta_problem *p, const ssd_tensor &t, int64_t n) {
    const int64_t e = 16 / (int64_t)esize(p->dtype);
    return al(t.ptr, 16) && (p->batch == 1 || t.stride[0] % e == 0) && (p->seqlen == 1 || t.stride[1] % e == 0) && (n == 1 || t.stride[2] % e == 0);
}
void set3(int64_t *to, const ssd_tensor &t) {
    for (int i = 0; i < 3; ++i) to[i] = t.stride[i];
}
DeltaArgs make(const ssd_delta_problem *p, const ssd_delta_args *f, const Plan &w, uint8_t *ws) {
    DeltaArgs a{};
    a.q = f->q.ptr; a.k = f->k.ptr; a.v = f->v.ptr; a.g = f->g.ptr; a.beta = f->beta.ptr;
    set3(a.qs, f->q); set3(a.ks, f->k); set3(a.vs, f->v); set3(a.gs, f->g); set3(a.bs, f->beta);
    a.vq = aligned_rows(p, f->q, p->ngroups); a.vk = aligned_rows(p, f->k, p->ngroups); a.vv = aligned_rows(p, f->v, p->nheads);
    a.init = f->initial_states.ptr;
    a.init_bf16 = f->initial_states.dtype == SSD_BF16;
    a.g_f32 = f->g.dtype == SSD_F32; a.beta_f32 = f->beta.dtype == SSD_F32;
    a.cu = f->cu_seqlens;
    a.seqlen = (int)p->seqlen; a.H = (int)p->nheads; a.G = (int)p->ngroups; a.V = (int)p->headdim; a.K = (int)p->dstate;
    a.nseqs = (int)nstates(p); a.nslots = (int)slots(p);
    a.scale = p->scale;
    a.hdr = reinterpret_cast<int32_t *>(ws + w.hdr);
    a.tiles = ws + w.tiles;
    a.nseg = w.nseg; a.seg0 = w.seg0; a.seglen = w.seglen;
    a.segB = ws + w.seg;
    a.segM = ws + w.seg + (size_t)(w.nseg > 1 ? w.nseg - 1 : 0) * nstates(p) * p->nheads * dtc::SEG_BYTES;
    a.gates = reinterpret_cast<float *>(ws + w.gates);
    a.sys = reinterpret_cast<float *>(ws + w.sys);
    a.att = reinterpret_cast<float *>(ws + w.att);
    a.a = reinterpret_cast<float *>(ws + w.a);
    return a;
}
void set_kept(DeltaArgs &a, const ssd_delta_problem *p, void *at) {
    const Kept k = kept_plan(p);
    a.S = static_cast<uint8_t *>(at) + k.S;
    a.U = static_cast<uint8_t *>(at) + k.U;
    if (on_tensor_cores(p)) {
        a.tiles = static_cast<uint8_t *>(at) + k.tiles;
        a.both = true;
    }
}
ssd_status check_workspace(const void *ws, size_t bytes, size_t need) {
    if (need == 0) return SSD_OK;
    if (ws == nullptr || bytes < need) return SSD_ERR_WORKSPACE_TOO_SMALL;
    return al(ws, 256) ? SSD_OK : SSD_ERR_MISALIGNED;
}
DeltaMaps maps(const ssd_delta_problem *p, const ssd_delta_args *f, const DeltaArgs &a, const ssd_delta_bwd_args *b, const ssd_tensor &out) {
    DeltaMaps m{};
    m.has_q = delta_map(&m.q, f->q.ptr, p->dstate, p->ngroups, p->seqlen, p->batch, f->q.stride);
    m.has_k = delta_map(&m.k, f->k.ptr, p->dstate, p->ngroups, p->seqlen, p->batch, f->k.stride);
    m.has_v = delta_map(&m.v, f->v.ptr, p->headdim, p->nheads, p->seqlen, p->batch, f->v.stride);
    m.has_out = out.ptr != nullptr && delta_map(&m.out, out.ptr, p->headdim, p->nheads, p->seqlen, p->batch, out.stride, true);
    if (b != nullptr) {
        m.has_dO = delta_map(&m.dO, b->dO.ptr, p->headdim, p->nheads, p->seqlen, p->batch, b->dO.stride);
        m.has_dqk = delta_map(&m.dq, b->dq.ptr, p->dstate, p->ngroups, p->seqlen, p->batch, b->dq.stride) &&
                    delta_map(&m.dk, b->dk.ptr, p->dstate, p->ngroups, p->seqlen, p->batch, b->dk.stride);
        const int64_t rows[3] = {0, 128, DQ * 128}, ch = (int64_t)a.nslots * a.H;
        m.has_vals = delta_map(&m.U, a.U, 128, ch, DQ, 1, rows) && delta_map(&m.mu, a.mu, 128, ch, DQ, 1, rows);
    }
    return m;
}
cudaError_t run_fwd(const ssd_delta_problem *p, const ssd_delta_args *f, const DeltaArgs &a, const ssd_tensor &o, cudaStream_t st) {
    return on_tensor_cores(p) && a.nslots > 0 ? delta_tc_fwd(a, maps(p, f, a, nullptr, o), st) : delta_simt_fwd(a, p->dtype == SSD_BF16, st);
}
// ---- rows of tokens that lie in no sequence
struct Rest {
    struct {
        void *p;
        int64_t s[3];
        int heads, inner, bytes;
    } t[5];
    int n, nseqs, seqlen;
    const int32_t *cu;
};
__global__ void k_rest(const Rest a) {
    after_previous();
    const int first = min(max(a.cu[0], 0), a.seqlen), last = max(first, min(max(a.cu[a.nseqs], 0), a.seqlen));
    const int rows = first + a.seqlen - last;
    for (int k = 0; k < a.n; ++k) {
        const auto &t = a.t[k];
        for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < (int64_t)rows * t.heads * t.inner; e += (int64_t)gridDim.x * blockDim.x) {
            const int64_t r = e / ((int64_t)t.heads * t.inner), rest = e - r * t.heads * t.inner;
            const int64_t at = (r < first ? r : last + r - first) * t.s[1] + rest / t.inner * t.s[2] + rest % t.inner;
            if (t.bytes == 2) static_cast<uint16_t *>(t.p)[at] = 0;
            else static_cast<float *>(t.p)[at] = 0.f;
        }
    }
}
ssd_status zero_rest(const ssd_delta_problem *p, const ssd_delta_args *f, std::initializer_list<const ssd_tensor *> tensors, cudaStream_t st) {
    if (!f->zero_rest || f->cu_seqlens == nullptr || p->seqlen == 0) return SSD_OK;
    Rest a{};
    a.nseqs = (int)p->nseqs; a.seqlen = (int)p->seqlen; a.cu = f->cu_seqlens;
    int k = 0;
    for (const ssd_tensor *t : tensors) {                    // o, or dq, dk, dv, dg, dbeta
        auto &to = a.t[a.n++];
        to.p = t->ptr;
        set3(to.s, *t);
        to.heads = (int)(tensors.size() > 1 && k < 2 ? p->ngroups : p->nheads);
        to.inner = (int)(k >= 3 ? 1 : tensors.size() > 1 && k < 2 ? p->dstate : p->headdim);
        to.bytes = (int)esize(t->dtype);
        ++k;
    }
    return launch_early(k_rest, 64u, 256u, 0, st, a) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
ssd_status of_cuda(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

}  // namespace

extern "C" {

ssd_status ssd_delta_chunk_states_size(const ssd_delta_problem *p, size_t *bytes) {
    if (bytes == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    DELTA_TRY(check_problem(p));
    *bytes = kept_plan(p).total;
    return SSD_OK;
}
ssd_status ssd_delta_fwd_workspace_size(const ssd_delta_problem *p, size_t *bytes) {
    if (bytes == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    DELTA_TRY(check_problem(p));
    *bytes = plan(p, false, false).total;
    return SSD_OK;
}
ssd_status ssd_delta_bwd_workspace_size(const ssd_delta_problem *p, int32_t kept, size_t *bytes) {
    if (bytes == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    DELTA_TRY(check_problem(p));
    *bytes = plan(p, true, kept != 0).total;
    return SSD_OK;
}

ssd_status ssd_delta_fwd(const ssd_delta_problem *p, const ssd_delta_args *f, void *workspace, size_t workspace_bytes, void *stream) {
    DELTA_TRY(check_inputs(p, f));
    DELTA_TRY(check_tok(p, f->o, p->dtype, p->nheads, p->headdim, true));
    DELTA_TRY(check_state(p, f->final_states));
    const Plan w = plan(p, false, false);
    DELTA_TRY(check_workspace(workspace, workspace_bytes, w.total));
    DeltaArgs a = make(p, f, w, static_cast<uint8_t *>(workspace));
    a.o = f->o.ptr;
    set3(a.os, f->o);
    a.final = f->final_states.ptr;
    a.final_bf16 = f->final_states.dtype == SSD_BF16;
    if (f->chunk_states) set_kept(a, p, f->chunk_states);
    DELTA_TRY(of_cuda(run_fwd(p, f, a, f->o, (cudaStream_t)stream)));
    return zero_rest(p, f, {&f->o}, (cudaStream_t)stream);
}

ssd_status ssd_delta_bwd(const ssd_delta_problem *p, const ssd_delta_bwd_args *b, void *workspace, size_t workspace_bytes, void *stream) {
    if (b == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    const ssd_delta_args *f = &b->fwd;
    DELTA_TRY(check_inputs(p, f));
    DELTA_TRY(check_tok(p, b->dO, p->dtype, p->nheads, p->headdim, false));
    DELTA_TRY(check_tok(p, b->dq, p->dtype, p->ngroups, p->dstate, true));
    DELTA_TRY(check_tok(p, b->dk, p->dtype, p->ngroups, p->dstate, true));
    DELTA_TRY(check_tok(p, b->dv, p->dtype, p->nheads, p->headdim, true));
    DELTA_TRY(check_tok(p, b->dg, f->g.dtype, p->nheads, 1, true));
    DELTA_TRY(check_tok(p, b->dbeta, f->beta.dtype, p->nheads, 1, true));
    DELTA_TRY(check_state(p, b->dfinal_states));
    if (f->initial_states.ptr && b->dinitial_states.ptr == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    DELTA_TRY(check_state(p, b->dinitial_states));
    const bool kept = f->chunk_states != nullptr;
    const Plan w = plan(p, true, kept);
    DELTA_TRY(check_workspace(workspace, workspace_bytes, w.total));
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    cudaStream_t st = (cudaStream_t)stream;
    DeltaArgs a = make(p, f, w, ws);
    set_kept(a, p, kept ? f->chunk_states : ws + w.kept);
    a.fresh = kept;
    if (!kept && p->seqlen > 0) DELTA_TRY(of_cuda(run_fwd(p, f, a, ssd_tensor{}, st)));
    a.dO = b->dO.ptr; set3(a.dos, b->dO);
    a.vo = aligned_rows(p, b->dO, p->nheads);
    a.dq = b->dq.ptr; set3(a.dqs, b->dq);
    a.dk = b->dk.ptr; set3(a.dks, b->dk);
    a.dv = b->dv.ptr; set3(a.dvs, b->dv);
    a.dg = b->dg.ptr; set3(a.dgs, b->dg);
    a.dbeta = b->dbeta.ptr; set3(a.dbs, b->dbeta);
    a.dfinal = b->dfinal_states.ptr; a.dfinal_bf16 = b->dfinal_states.dtype == SSD_BF16;
    a.dinit = b->dinitial_states.ptr; a.dinit_bf16 = b->dinitial_states.dtype == SSD_BF16;
    a.dS = ws + w.dS;
    a.mu = ws + w.mu;
    a.flow = reinterpret_cast<float *>(ws + w.flow);
    a.part = !on_tensor_cores(p) && p->nheads > p->ngroups ? reinterpret_cast<float *>(ws + w.part) : nullptr;
    DELTA_TRY(of_cuda(on_tensor_cores(p) && a.nslots > 0 ? delta_tc_bwd(a, maps(p, f, a, b, b->dv), st) : delta_simt_bwd(a, p->dtype == SSD_BF16, st)));
    return zero_rest(p, f, {&b->dq, &b->dk, &b->dv, &b->dg, &b->dbeta}, st);
}

}  // extern "C"
