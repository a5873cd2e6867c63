// selective.cuh -- what the selective scan's kernels share: packed fp32 pairs, the exponential and
// softplus, the chunk grid of its kept states, and the arguments of a call.
#pragma once

#include "common.cuh"

namespace ssd {

// Chunk of the kept states: the state entering every SEL_Q-th token of a sequence is what the
// forward keeps and the backward starts from.  Sequence s's chunks lie at slots
// slot0(s) .. slot0(s) + ceil(len / SEL_Q) - 1.
constexpr int SEL_Q = 32;

// dstate padded to the sizes that the kernels are compiled for.
__host__ __device__ inline int sel_pad(int64_t n) { return n <= 16 ? 16 : n <= 32 ? 32 : n <= 64 ? 64 : 128; }

struct SelArgs {
    const void *x, *dt, *B, *C, *z, *dy;
    int64_t xb, xt, dtb, dtt, Bb, Bt, Bg, Cb, Ct, Cg, zb, zt, dyb, dyt;   // element strides: batch row, token (, group)
    const float *A, *D, *bias;
    const void *init, *dfinal;
    bool dt_f32, init_bf16, final_bf16, dfinal_bf16, dinit_bf16;
    const int32_t *cu;                 // packed sequences (batch 1) or NULL
    int nbatch, seqlen, channels, ngroups, dpg, N, NP, nseqs, nslots;     // dpg: channels per group; nseqs: batch or packed
    // forward
    void *y, *final;
    int64_t yb, yt;
    float *states;                     // [nslots][channels][NP]: the state entering each chunk, or NULL
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

// ---- two fp32 lanes in a 64-bit register: one issue slot for two multiply-adds
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pk2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void up2(f32x2 v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum2(f32x2 v) {
    float lo, hi;
    up2(v, lo, hi);
    return lo + hi;
}
// 2^v on the multi-function unit (relative error about 2^-22; results below 2^-126 flush to zero,
// which a decay of that size is)
__device__ __forceinline__ float ex2f(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ f32x2 ex2x2(f32x2 v) {
    float lo, hi;
    up2(v, lo, hi);
    return pk2(ex2f(lo), ex2f(hi));
}

constexpr float kLog2e = 1.4426950408889634f;

// softplus(v) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1].  log1p(e) = 2 atanh(s) with
// s = e / (2 + e) <= 1/3, by atanh's power series s + s^3/3 + ... + s^15/15 (the rest is below
// 2^-27 of the sum); no cancellation, so small steps keep their relative accuracy.
__device__ __forceinline__ float sel_softplus(float v) {
    const float e = expf(-fabsf(v));
    const float s = __fdividef(e, 2.f + e), q = s * s;
    float p = 1.f / 15.f;
    p = fmaf(p, q, 1.f / 13.f);
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    p = fmaf(p, q, 1.f);
    const float r = fmaf(2.f * s, p, fmaxf(v, 0.f));
    return v == v ? r : v;   // fmaxf would drop a NaN
}

// The gate's logistic function: for bf16 data one tanh.approx (relative error 2^-11, below the
// data's own rounding of 2^-9), for fp32 data the full exponential and divide.
template <typename T>
__device__ __forceinline__ float sel_sigmoid(float v) {
    if (sizeof(T) == 2) {
        float t;
        asm("tanh.approx.f32 %0, %1;" : "=f"(t) : "f"(0.5f * v));
        return fmaf(0.5f, t, 0.5f);
    }
    return 1.f / (1.f + expf(-v));
}

__device__ __forceinline__ float ld_dt(const SelArgs &a, int64_t at) {
    return a.dt_f32 ? static_cast<const float *>(a.dt)[at] : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.dt)[at]);
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

// selective_fwd.cu: the scan, or with y == NULL its kept states alone
cudaError_t sel_launch_fwd(const SelArgs &a, bool bf16, cudaStream_t st);
// selective_bwd.cu
cudaError_t sel_launch_bwd(const SelArgs &a, bool bf16, cudaStream_t st);
void sel_bwd_sets(int channels, int ngroups, int64_t nslots, int *nsets, int *cps);

}  // namespace ssd
