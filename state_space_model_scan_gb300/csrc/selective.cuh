// selective.cuh -- what the selective scan's kernels share: packed fp32 pairs, the exponential and
// softplus, the chunk grid of its kept states, and the arguments of a call.
#pragma once

#include <algorithm>

#include "f32x2.cuh"

namespace ssd {

// Chunk of the kept states: the state entering every SEL_Q-th token of a sequence is what the
// forward keeps and the backward starts from.  Sequence s's chunks lie at slots
// slot0(s) .. slot0(s) + ceil(len / SEL_Q) - 1.
constexpr int SEL_Q = 16;
constexpr int kSMs = 152;   // of a GB300

// dstate padded to the sizes that the kernels are compiled for.
__host__ __device__ inline int sel_pad(int64_t n) { return n <= 16 ? 16 : n <= 32 ? 32 : n <= 64 ? 64 : 128; }

struct SelArgs {
    const void *x, *dt, *B, *C, *z, *dy;
    int64_t xb, xt, dtb, dtt, Bb, Bt, Bg, Cb, Ct, Cg, zb, zt, dyb, dyt;   // element strides: batch row, token (, group)
    const float *A, *D, *bias;
    const void *init, *dfinal;
    // four elements at places divisible by four are aligned to their size, in the channel tensors / in B and C / in A
    bool vec, vecBC, vecA, vec_out;    // (vec_out: the gradients' channel tensors)
    bool dt_f32, init_bf16, final_bf16, dfinal_bf16, dinit_bf16;
    const int32_t *cu;                 // packed sequences (batch 1) or NULL
    int nbatch, seqlen, channels, ngroups, dpg, N, NP, nseqs, nslots;     // dpg: channels per group; nseqs: batch or packed
    // forward
    void *y, *final;
    int64_t yb, yt;
    float *states;                     // [nslots][channels][NP]: the state entering each chunk, or NULL
    // a long sequence of few channels is cut into nseg segments of seglen tokens (a multiple of every tile); a first
    // launch (ends) takes each from zero and leaves its end [nseqs][nseg][channels][NP] and sum of dt [nseqs][nseg][channels]
    int nseg, seglen;
    bool ends;
    float *segE, *segS;
    // backward
    void *dx, *ddt, *dz, *dB, *dC, *dinit;
    int64_t dxb, dxt, ddtb, ddtt, dzb, dzt, dBb, dBt, dBg, dCb, dCt, dCg;
    float *dA, *dD, *dbias;
    float *adj;                        // [nslots][channels][NP]: the adjoint leaving each chunk to the right
    float *pA, *pD;                    // [nslots][channels][NP], [nslots][channels][2]: shares of dA and of (dD, ddt_bias)
    float *pBC;                        // [nsets][2][rows of B][NP]: shares of dB and dC
    int nsets, cps;                    // channel sets per group, channels per set
};

// Sequence s: batch row, first token in the row, length, first chunk slot.  Whatever cu_seqlens
// holds, the tokens lie inside the row.
struct SelSeq {
    int b, t0, len, slot0;
};
__device__ __forceinline__ SelSeq sel_seq(const SelArgs &a, int s) {
    SelSeq q;
    if (a.cu == nullptr) {
        q.b = s; q.t0 = 0; q.len = a.seqlen;
        q.slot0 = s * ((a.seqlen + SEL_Q - 1) / SEL_Q);
    } else {
        q.b = 0;
        q.t0 = min(max(a.cu[s], 0), a.seqlen);
        q.len = min(max(a.cu[s + 1], q.t0), a.seqlen) - q.t0;
        q.slot0 = q.t0 / SEL_Q + s;    // floor(end / Q) + 1 slots on: enough for ceil(len / Q) chunks
    }
    return q;
}

// Segment k of a sequence: its tokens (none, where the sequence is shorter) and first chunk slot.
__device__ __forceinline__ SelSeq sel_segment(const SelArgs &a, SelSeq q, int k) {
    if (a.nseg > 1) {
        const int at = min(k * a.seglen, q.len);
        q.slot0 += at / SEL_Q;
        q.t0 += at;
        q.len = min(q.len - at, a.seglen);
    }
    return q;
}

__device__ __forceinline__ f32x2 ex2x2(f32x2 v) {
    float lo, hi;
    up2(v, lo, hi);
    return pk2(ex2f(lo), ex2f(hi));
}

// A log2(e), kept finite: a rate of -inf (or near fp32's lowest value) forgets all of a state in any step, and a step of
// 0, which stands for the tokens past a sequence's end, leaves it as it is instead of making it 0 x inf.
__device__ __forceinline__ float sel_rate(float A) {
    const float v = A * kLog2e;
    return v < -3.402823466e38f ? -3.402823466e38f : v;
}
// softplus(v) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1].  log1p(e) = 2 atanh(s) with
// s = e / (2 + e) <= 1/3; 2 atanh(s) / s is a polynomial of degree 4 in s^2 there, fitted to
// its smallest largest relative error, 8e-9 with the rounded coefficients.  No cancellation: small steps keep their relative accuracy.
__device__ __forceinline__ float sel_softplus(float v) {
    const float e = ex2f(-kLog2e * fabsf(v));
    const float s = e * rcpf(2.f + e), q = s * s;
    float p = 0.28178334f;
    p = fmaf(p, q, 0.27960601f);
    p = fmaf(p, q, 0.40024909f);
    p = fmaf(p, q, 0.66666317f);
    p = fmaf(p, q, 2.f);
    return fmaf(s, p, fmaxf(v, 0.f));   // a NaN comes through s
}

// v silu(z) = v z / (1 + exp(-z)): for bf16 data the reciprocal's approximation, for fp32 data the full divide and
// exponential.  Not (1 + tanh(z / 2)) / 2, which costs one operation of the multi-function unit less: for z
// far below 0 the approximate tanh is -1, and the gate 0.
template <typename T>
__device__ __forceinline__ float sel_gate(float v, float z) {
    if (sizeof(T) == 2) return v * z * rcpf(1.f + ex2f(-kLog2e * z));
    return v * z / (1.f + expf(-z));
}

// ---- four neighbouring elements: a thread's share of a row in the elementwise steps.  vec: the rows'
// addresses allow one access for all four; n: how many of them exist.
template <int BYTES>
__device__ __forceinline__ void cp_async_small(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// to shared memory in the background (one by one and at once where four do not go)
template <typename U>
__device__ __forceinline__ void fetch4(U *dst, const U *src, int n, bool vec) {
    if (n == 4 && vec) {
        cp_async_small<4 * sizeof(U)>(dst, src);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) dst[i] = src[i];
    }
}
// Rows whose addresses do not allow that, to shared memory: R rows of W neighbouring elements by NT threads,
// element by element, neighbours by neighbours.  fp32 goes in the background at load(); bf16 (no
// asynchronous copy is that small) waits in registers for store().  Row r's elements are src + r `bytes`
// bytes on; nr rows and nw elements exist (one of each at least; for the others the last one's are read,
// so that no load waits for a branch).
template <int R, int W, int NT, typename U>
struct Rows {
    static constexpr int E = (R * W + NT - 1) / NT;
    U v[sizeof(U) == 4 ? 1 : E];
    __device__ __forceinline__ void load(U *dst, const U *src, int bytes, int nr, int nw, int tid) {
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const int i = tid + k * NT, r = i / W, c = i % W;
            if constexpr (sizeof(U) == 4) {
                if (r < nr && c < nw)
                    cp_async_small<4>(dst + i, reinterpret_cast<const U *>(reinterpret_cast<uintptr_t>(src + c) + (int64_t)r * bytes));
            } else {
                v[k] = *reinterpret_cast<const U *>(reinterpret_cast<uintptr_t>(src + min(c, nw - 1)) + (int64_t)min(r, nr - 1) * bytes);
            }
        }
    }
    __device__ __forceinline__ void store(U *dst, int nr, int nw, int tid) const {
        if constexpr (sizeof(U) != 4) {
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const int i = tid + k * NT;
                if (i / W < nr && i % W < nw) dst[i] = v[k];
            }
        }
    }
};
// both at once, eight elements at a time
template <int R, int W, int NT, typename U>
__device__ __forceinline__ void fetch_rows(U *dst, const U *src, int bytes, int nr, int nw, int tid) {
    constexpr int B = 8 * NT >= W && (8 * NT) % W == 0 && R % (8 * NT / W) == 0 ? 8 * NT / W : R;   // rows at a time
#pragma unroll 1
    for (int r = 0; r < R && r < nr; r += B) {
        Rows<B, W, NT, U> g;
        const U *p = reinterpret_cast<const U *>(reinterpret_cast<uintptr_t>(src) + (int64_t)r * bytes);
        g.load(dst + r * W, p, bytes, min(nr - r, B), nw, tid);
        g.store(dst + r * W, min(nr - r, B), nw, tid);
    }
}
// as they lie in memory (two bf16 to a register)
template <typename U>
struct Raw4;
template <>
struct Raw4<float> {
    float4 v;
    __device__ __forceinline__ void f(float (&o)[4]) const { o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w; }
    __device__ __forceinline__ void load(const float *p, int n, bool vec) {
        if (n == 4 && vec) v = *reinterpret_cast<const float4 *>(p);
        else v = make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
    }
};
template <>
struct Raw4<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ void f(float (&o)[4]) const {
        o[0] = __uint_as_float(v.x << 16); o[1] = __uint_as_float(v.x & 0xffff0000u);
        o[2] = __uint_as_float(v.y << 16); o[3] = __uint_as_float(v.y & 0xffff0000u);
    }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, int n, bool vec) {
        if (n == 4 && vec) {
            v = *reinterpret_cast<const uint2 *>(p);
        } else {
            const unsigned short *u = reinterpret_cast<const unsigned short *>(p);
            v.x = (n > 0 ? u[0] : 0u) | (n > 1 ? (uint32_t)u[1] << 16 : 0u);
            v.y = (n > 2 ? u[2] : 0u) | (n > 3 ? (uint32_t)u[3] << 16 : 0u);
        }
    }
};
__device__ __forceinline__ void put4(float *p, const float (&v)[4]) { *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void put4(__nv_bfloat16 *p, const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}
template <typename U>
__device__ __forceinline__ void store4(U *p, const float (&v)[4], int n, bool vec) {
    if (n == 4 && vec) {
        put4(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = from_f<U>(v[i]);
    }
}
// p moved on by t rows of `bytes` bytes (one wide multiply-add; the library bounds the strides)
template <typename U>
__device__ __forceinline__ U *row(U *p, int t, int bytes) {
    return reinterpret_cast<U *>(reinterpret_cast<uintptr_t>(p) + (int64_t)t * bytes);
}

__device__ __forceinline__ float ld_st(const void *p, bool bf16, int64_t at) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[at]) : static_cast<const float *>(p)[at];
}
__device__ __forceinline__ void st_st(void *p, bool bf16, int64_t at, float v) {
    if (bf16) static_cast<__nv_bfloat16 *>(p)[at] = __float2bfloat16_rn(v);
    else static_cast<float *>(p)[at] = v;
}

// Sums v[0..R-1] over the R lanes of an aligned group (R a power of two): lane q of the group
// returns the sum of everybody's v[q].  R - 1 shuffles for R sums.
template <int R>
__device__ __forceinline__ float reduce_scatter(float (&v)[R], int q) {
#pragma unroll
    for (int o = R / 2; o > 0; o >>= 1) {
        const bool up = q & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return v[0];
}

// Tokens of a tile and channels of a block where the sequences are split over time, by padded dstate.
__host__ __device__ constexpr int sel_tile(int NP) { return NP <= 32 ? 128 : 64; }
__host__ __device__ constexpr int sel_block(int NP) { return NP <= 32 ? 16 : NP == 64 ? 8 : 4; }

// Segments: where a third of the card or less would be busy (two blocks to an SM), enough of them to fill
// it, of two tiles at least.  Both launches together do half as much again as one, so that two segments
// do not pay.  Measured at 4000 tokens, dstate 16, bf16, cut against whole: 768 channels 58 / 117 us,
// 1024 72 / 124, 1536 121 / 131, 2048 158 / 131.
inline void sel_segments(int64_t nseqs, int64_t channels, int64_t ngroups, int64_t seqlen, int NP, int *nseg, int *seglen) {
    const int64_t cb = sel_block(NP), blocks = nseqs * ngroups * ((channels / ngroups + cb - 1) / cb), slots = 2 * kSMs;
    *nseg = 1;
    *seglen = (int)seqlen;
    if (blocks * 3 > slots) return;
    const int64_t t = sel_tile(NP), want = (slots + blocks - 1) / blocks, tiles = (seqlen + t - 1) / t;
    const int64_t per = std::max<int64_t>(2, (tiles + want - 1) / want), n = (tiles + per - 1) / per;
    if (n < 3) return;
    *nseg = (int)n;
    *seglen = (int)(per * t);
}
inline size_t sel_seg_bytes(int64_t nseqs, int64_t channels, int nseg, int NP) {
    return nseg > 1 ? (size_t)nseqs * nseg * channels * (NP + 1) * sizeof(float) : 0;
}

// selective_fwd.cu: the scan, or with y == NULL its kept states alone
cudaError_t sel_launch_fwd(SelArgs a, bool bf16, cudaStream_t st);
// selective_bwd.cu
cudaError_t sel_launch_bwd(SelArgs a, bool bf16, cudaStream_t st);
void sel_bwd_sets(int channels, int ngroups, int64_t nslots, int *nsets, int *cps);

}  // namespace ssd
