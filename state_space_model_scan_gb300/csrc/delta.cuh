// delta.cuh -- what the gated delta rule's kernels share: the arguments of a call, the chunks of its sequences, the
// gates of a chunk and the inverse of its triangular system.
//
// Per value head, with a state S [headdim][dstate] and k, q of the head's group:
//
//   S <- e^g S,  u = beta (v - S k),  S <- S + u k^T,  o = scale S q
//
// In chunks of 64 tokens, G the sum of g from the chunk's first token on, S the state that enters it, and
// a_ij = e^(G_i - G_j) k_i.k_j below the diagonal (rows of K, Q, V are tokens):
//
//   U = (I + a diag(beta))^-1 (V - e^G K S^T),  W = beta U,  O = scale (e^G Q S^T + att W),  att_ij = e^(G_i - G_j) q_i.k_j, j <= i
//   S' = e^Gc S + (e^(Gc - G) W)^T K
//
// and backwards, from dS' and dO:
//
//   N = scale att^T dO + e^(Gc - G) K dS'^T,  mu = (I + diag(beta) a)^-T N,  lam = beta mu
//   dS = e^Gc dS' + (scale e^G dO)^T Q - (e^G lam)^T K
//   E_ij = -e^(G_i - G_j) lam_i.W_j (j < i),  F_ij = scale e^(G_i - G_j) dO_i.W_j (j <= i)
//   dQ = F K + scale e^G dO S,  dK = (E + E^T) K + F^T Q - e^G lam S + e^(Gc - G) W dS',  dV = lam,  dbeta = mu.U
//   dg_t = sum over i >= t > j of (F_ij q_i.k_j + E_ij k_i.k_j)            (what crosses token t inside the chunk)
//        + sum over i >= t of (scale e^G_i q_i.(dO S)_i - e^G_i k_i.(lam S)_i)       (what comes from before it)
//        + sum over j < t of e^(Gc - G_j) k_j.(W dS')_j + e^Gc <dS', S>               (what leaves it, and what passes)
//
// Both ways the sequential part (the chain) is the same: a product with the state, a product with the inverse, a
// product with K onto the state.
#pragma once

#include "f32x2.cuh"

namespace ssd {

constexpr int DQ = 64;          // tokens of a chunk
constexpr int DGATES = 6 * DQ;  // of a chunk and head: e^G, e^(Gc - G), beta, G as the sum of two floats, -e^G

struct DeltaArgs {
    const void *q, *k, *v, *g, *beta, *dO;
    int64_t qs[3], ks[3], vs[3], gs[3], bs[3], dos[3];   // element strides: batch row, token, group or head
    const void *init, *dfinal;
    void *o, *final, *dq, *dk, *dv, *dg, *dbeta, *dinit;
    int64_t os[3], dqs[3], dks[3], dvs[3], dgs[3], dbs[3];
    bool vq, vk, vv, vo;        // SIMT: rows of q, k, v, dO start at 16 bytes
    bool g_f32, beta_f32, init_bf16, final_bf16, dfinal_bf16, dinit_bf16;
    const int32_t *cu;          // packed sequences (batch 1) or NULL
    int seqlen, H, G, V, K, nseqs, nslots;   // nseqs: batch or packed; nslots: chunks of all sequences, at most
    float scale;
    // workspace and kept states
    int32_t *hdr;               // the workspace's first words (HeaderWord): the status of bounded waits
    float *gates;               // [nslots][H][DGATES]
    float *sys, *att, *a;       // SIMT: [nslots][H][64][64] each: the inverse, att, and (backward) a
    // state entering each chunk and U (kept by a training forward), gradient of the state leaving each chunk and mu: SIMT
    // [nslots][H][V][K] and [nslots][H][64][V] fp32, tensor-core path [nslots][H] operand images of 32 KB and [64][128] bf16
    void *S, *U, *dS, *mu;
    float *flow;                // SIMT backward: [nslots][H][shares][DELTA_FLOW]: what dg is made of
    float *part;                // [2][nslots][H][64][K]: dq and dk of each value head, where heads share a group
    void *tiles;                // tensor-core path: operand images of every chunk and head, `both` for a backward too
    bool both, fresh;           // fresh: a backward's first launch clears the header
    // tensor-core path: a chain of few heads is cut into nseg segments (see delta_segments), the first of seg0 chunks, those between of
    // seglen; a first launch leaves, for all but the last, the end from a zero state (the first's from its own) [nseqs][H][nseg - 1][128][128]
    // fp32 and, for those between, what it makes of a state (as two terms, 64 KB each)
    int nseg, seg0, seglen;
    void *segB, *segM;
};

// Sequence s: batch row, first token in the row, length, first chunk.  Whatever cu_seqlens holds, the
// tokens lie inside the row and the chunks inside [0, nslots).
struct DeltaSeq {
    int b, t0, len, slot0;
};
__device__ __forceinline__ DeltaSeq delta_seq(const DeltaArgs &a, int s) {
    DeltaSeq q;
    if (a.cu == nullptr) {
        q.b = s; q.t0 = 0; q.len = a.seqlen;
        q.slot0 = s * ((a.seqlen + DQ - 1) / DQ);
    } else {
        q.b = 0;
        q.t0 = min(max(a.cu[s], 0), a.seqlen);
        q.len = min(max(a.cu[s + 1], q.t0), a.seqlen) - q.t0;
        q.slot0 = q.t0 / DQ + s;       // floor(end / 64) + 1 slots on: enough for ceil(len / 64) chunks
    }
    return q;
}
// Chunk of a slot: batch row, first token, tokens (0: nothing lies in the slot).  Slots of packed sequences
// ascend, so the sequence is found by halving; one that does not ascend leaves slots empty or taken twice,
// inside the row all the same.
struct DeltaChunk {
    int b, t0, len;
};
__device__ __forceinline__ DeltaChunk delta_chunk(const DeltaArgs &a, int slot) {
    DeltaChunk c;
    int at;
    DeltaSeq q;
    if (a.cu == nullptr) {
        const int n = (a.seqlen + DQ - 1) / DQ;
        q = delta_seq(a, slot / n);
        at = slot % n;
    } else {
        int lo = 0, hi = a.nseqs - 1;  // the last sequence whose first slot is at most `slot`
        while (lo < hi) {
            const int m = (lo + hi + 1) / 2;
            if (min(max(a.cu[m], 0), a.seqlen) / DQ + m <= slot) lo = m;
            else hi = m - 1;
        }
        q = delta_seq(a, lo);
        at = slot - q.slot0;
    }
    c.b = q.b;
    c.t0 = q.t0 + at * DQ;
    c.len = at < 0 ? 0 : max(0, min(DQ, q.len - at * DQ));
    return c;
}

__device__ __forceinline__ float delta_ld(const void *p, bool f32, int64_t at) {
    return f32 ? static_cast<const float *>(p)[at] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[at]);
}
__device__ __forceinline__ void delta_st(void *p, bool f32, int64_t at, float v) {
    if (f32) static_cast<float *>(p)[at] = v;
    else static_cast<__nv_bfloat16 *>(p)[at] = __float2bfloat16_rn(v);
}

// e^(G_i - G_j) of two sums that are each held as two floats: next to a token that forgets nearly everything (g of
// -300, say) a difference of single floats would be off by 2e-5, and so would every decay after it.
__device__ __forceinline__ float delta_decay(float hi_i, float lo_i, float hi_j, float lo_j) {
    return expf((hi_i - hi_j) + (lo_i - lo_j));
}

// The gates of a chunk by its first warp (lane l: tokens 2l and 2l + 1), into `to` [DGATES].  Tokens past the
// chunk's end keep the state as it is (g = 0) and write nothing (beta = 0).  A g below -200, -inf among
// them, is taken as -200: its exponential is 0 in fp32 either way, and sums of such stay finite.
__device__ __forceinline__ void delta_gates(const DeltaArgs &a, const DeltaChunk &c, int h, float *to, int lane) {
    double g[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e;
        float v = 0.f, b = 0.f;
        if (i < c.len) {
            v = delta_ld(a.g, a.g_f32, c.b * a.gs[0] + (int64_t)(c.t0 + i) * a.gs[1] + h * a.gs[2]);
            b = delta_ld(a.beta, a.beta_f32, c.b * a.bs[0] + (int64_t)(c.t0 + i) * a.bs[1] + h * a.bs[2]);
        }
        g[e] = v < -200.f ? -200.f : v;
        to[2 * DQ + i] = b;
    }
    g[1] += g[0];
    double sum = g[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double t = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += t;
    }
    const double before = sum - g[1], all = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e;
        const double G = before + g[e];
        const float hi = (float)G;
        to[i] = expf((float)G);
        to[5 * DQ + i] = -to[i];
        to[DQ + i] = expf((float)(all - G));
        to[3 * DQ + i] = hi;
        to[4 * DQ + i] = (float)(G - (double)hi);
    }
}

constexpr int DELTA_ML = 68;    // row stride of a 64 x 64 matrix in shared memory: rows of 16-byte pieces, four banks apart

// Inverse of I + M, M strictly lower triangular 64 x 64, in place in shared memory, by NT threads: the four 16 x 16 blocks on the
// diagonal by substitution, a thread a column; then twice the block below the diagonal of a pair, -T22 M21 T11, a thread four
// neighbouring columns of a row (t: 32 x 36 floats of scratch).  Of the blocks above the diagonal, those in the pairs of 32 are set
// to zero, the other is neither read nor written.
template <int NT>
__device__ __forceinline__ void delta_invert(float *M, float *t, int tid) {
    constexpr int MLD = DELTA_ML;
    if (tid < 64) {
        const int o = tid / 16 * 16, j = tid & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == j ? 1.f : 0.f;
#pragma unroll
            for (int l = 0; l < i; l += 4) {
                const float4 m = *reinterpret_cast<const float4 *>(M + (o + i) * MLD + o + l);
                s = fmaf(-m.x, x[l], s);
                if (l + 1 < i) s = fmaf(-m.y, x[l + 1], s);
                if (l + 2 < i) s = fmaf(-m.z, x[l + 2], s);
                if (l + 3 < i) s = fmaf(-m.w, x[l + 3], s);
            }
            x[i] = s;
        }
        __syncwarp();                                        // a block's sixteen threads are in one warp
#pragma unroll
        for (int i = 0; i < 16; ++i) M[(o + i) * MLD + o + j] = x[i];
    }
    if (tid < 128) {                                         // the blocks of 16 above a pair's diagonal: zeros, for the pair of 32
        const int o = tid / 64 * 32;
        *reinterpret_cast<float4 *>(M + (o + tid % 64 / 4) * MLD + o + 16 + tid % 4 * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
#pragma unroll
    for (int n = 16; n <= 32; n *= 2) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {               // t = M21 T11, then M21 = -T22 t
#pragma unroll 1
            for (int it = tid; it < 8 * n; it += NT) {
                const int per = n * n / 4, p = it / per, i = it % per / (n / 4), j = it % (n / 4) * 4, o = p * 2 * n;
                f32x2 s0 = 0, s1 = 0;
                const float *A = M + (o + n + i) * MLD + o + (half ? n : 0), *B = half ? t + p * n * 36 + j : M + o * MLD + o + j;
                const int ldb = half ? 36 : MLD;
#pragma unroll 2
                for (int l = 0; l < n; l += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(A + l);
                    const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const ulonglong2 y = *reinterpret_cast<const ulonglong2 *>(B + (l + e) * ldb);
                        const f32x2 xx = pk2(xs[e], xs[e]);
                        s0 = fma2(xx, y.x, s0);
                        s1 = fma2(xx, y.y, s1);
                    }
                }
                float4 r;
                up2(s0, r.x, r.y);
                up2(s1, r.z, r.w);
                if (half) *reinterpret_cast<float4 *>(M + (o + n + i) * MLD + o + j) = make_float4(-r.x, -r.y, -r.z, -r.w);
                else *reinterpret_cast<float4 *>(t + (p * n + i) * 36 + j) = r;
            }
            __syncthreads();
        }
    }
}

// Into how many shares of its keys (slices of 32) a chunk's gradients are cut, so that the blocks fill the SMs; every share
// computes the chunk's matrices again, a fifth of a block's work at 64 keys.
constexpr int DELTA_FLOW = 3 * DQ + 1;
constexpr int64_t kDeltaSMs = 152;
inline int delta_grad_shares(int64_t nslots, int64_t H, int64_t K) {
    const int64_t n = nslots * H, most = (K + 31) / 32, fit = n > 0 ? kDeltaSMs / n : 1;
    return (int)(fit < 1 ? 1 : fit < most ? fit : most);
}

// delta_simt.cu: any type and size.  states: leave a.S and a.U (and no o, where a.o is NULL).
cudaError_t delta_simt_fwd(const DeltaArgs &a, bool bf16, cudaStream_t st);
cudaError_t delta_simt_bwd(const DeltaArgs &a, bool bf16, cudaStream_t st);

}  // namespace ssd
