// delta_simt.cu -- the gated delta rule in plain fp32 arithmetic, for every type and size that the tensor-core path
// does not take (fp32 data among them, which is computed in fp32 throughout).
//
// Four kernels (formulas in delta.cuh): k_prep, a block a chunk and head: the triangular system's inverse and att;
// k_chain, a block a sequence, head and 8, 16 or 32 values, from chunk to chunk with its rows of the state in shared memory,
// forwards (o, states, U) or backwards (mu, dS); k_grads, a block a chunk, head and share of the keys: everything else of the
// gradients; k_finish, what is summed over those blocks.  Products go through shared memory in slices of 32,
// a thread a few rows and columns of the result, and its reads are what bounds the chain: 75% of its cycles with 32 values.  A chunk of 64 tokens
// at dstate 64 takes 6 us with 8 values a block, 11 with 32, whatever the number of heads, until the card is full.
#include "delta.cuh"

namespace ssd {

namespace {

constexpr int NT = 256;
constexpr int LD = 36;              // row stride of a slice of 32: rows of 16-byte pieces, four banks apart
constexpr int MLD = DELTA_ML;

// rows [0, 64) of a slice of 32 columns from column k0 of a chunk's rows (row stride `step` elements); zeros past the chunk and past n
template <int N, typename T>
__device__ __forceinline__ void load_slice(float *to, const T *p, int64_t step, int len, int k0, int n, int tid) {
    for (int e = tid; e < 64 * 32; e += N) {
        const int i = e / 32, c = e % 32;
        to[i * LD + c] = i < len && k0 + c < n ? to_f(p[i * step + k0 + c]) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ const T *rows_of(const void *p, const int64_t *s, const DeltaChunk &c, int h) {
    return static_cast<const T *>(p) + c.b * s[0] + c.t0 * s[1] + h * s[2];
}
// R x 2 of a product over a slice of n: rows 64 / R r + ty of A, columns 2 tx and 2 tx + 1 of B [n][ldb]
template <int R>
__device__ __forceinline__ void fma_slice(float (&acc)[R][2], const float *A, int lda, const float *B, int ldb, int n, int ty, int tx) {
#pragma unroll 4
    for (int l = 0; l < n; l += 4) {
        float2 b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = *reinterpret_cast<const float2 *>(B + (l + e) * ldb + 2 * tx);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float4 x = *reinterpret_cast<const float4 *>(A + (64 / R * r + ty) * lda + l);
            const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[r][0] = fmaf(xs[e], b[e].x, acc[r][0]);
                acc[r][1] = fmaf(xs[e], b[e].y, acc[r][1]);
            }
        }
    }
}
// the same with A given by columns: A^T [n][lda]
template <int R>
__device__ __forceinline__ void fma_slice_t(float (&acc)[R][2], const float *A, int lda, const float *B, int ldb, int n, int ty, int tx) {
#pragma unroll 8
    for (int l = 0; l < n; ++l) {
        const float2 b = *reinterpret_cast<const float2 *>(B + l * ldb + 2 * tx);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float x = A[l * lda + 64 / R * r + ty];
            acc[r][0] = fmaf(x, b.x, acc[r][0]);
            acc[r][1] = fmaf(x, b.y, acc[r][1]);
        }
    }
}
// x[r][s] += rows 64 / R r + ty of A times rows 16 s + tx of B, y of A2 (all [64][LD], a slice of 32)
template <int R>
__device__ __forceinline__ void mul_rows(float (&x)[R][4], float (&y)[R][4], const float *A, const float *A2, const float *B, int ty, int tx) {
#pragma unroll 2
    for (int l = 0; l < 32; l += 4) {
        float4 b[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) b[s] = *reinterpret_cast<const float4 *>(B + (16 * s + tx) * LD + l);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float4 u = *reinterpret_cast<const float4 *>(A + (64 / R * r + ty) * LD + l), v = *reinterpret_cast<const float4 *>(A2 + (64 / R * r + ty) * LD + l);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                x[r][s] = fmaf(u.x, b[s].x, fmaf(u.y, b[s].y, fmaf(u.z, b[s].z, fmaf(u.w, b[s].w, x[r][s]))));
                y[r][s] = fmaf(v.x, b[s].x, fmaf(v.y, b[s].y, fmaf(v.z, b[s].z, fmaf(v.w, b[s].w, y[r][s]))));
            }
        }
    }
}

// ---- the chunk's matrices: sys = (I + a diag(beta))^-1 or, backwards, (I + diag(beta) a)^-1; att; a.
template <typename T>
__global__ void __launch_bounds__(NT) k_prep(const DeltaArgs a, const bool back) {
    after_previous();
    __shared__ __align__(16) float Ks[64 * LD], Qs[64 * LD], M[64 * MLD], gate[DGATES];
    const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x;
    if (blockIdx.x == 0 && tid < HDR_WORDS) a.hdr[tid] = 0;
    const DeltaChunk c = delta_chunk(a, slot);
    if (c.len == 0) return;
    const int grp = h / (a.H / a.G);
    if (tid < 32) delta_gates(a, c, h, gate, tid);
    const T *q = rows_of<T>(a.q, a.qs, c, grp), *k = rows_of<T>(a.k, a.ks, c, grp);
    const int ty = tid / 16, tx = tid % 16;
    float kk[4][4], qk[4][4];          // rows 16 r + ty, columns 16 s + tx
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int s = 0; s < 4; ++s) kk[r][s] = qk[r][s] = 0.f;
    for (int k0 = 0; k0 < a.K; k0 += 32) {
        __syncthreads();
        load_slice<NT>(Ks, k, a.ks[1], c.len, k0, a.K, tid);
        load_slice<NT>(Qs, q, a.qs[1], c.len, k0, a.K, tid);
        __syncthreads();
        mul_rows(kk, qk, Ks, Qs, Ks, ty, tx);
    }
    const int64_t at = ((int64_t)slot * a.H + h) * 4096;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int i = 16 * r + ty, j = 16 * s + tx;
            const float d = j <= i ? delta_decay(gate[3 * DQ + i], gate[4 * DQ + i], gate[3 * DQ + j], gate[4 * DQ + j]) : 0.f;
            a.att[at + i * 64 + j] = j <= i ? d * qk[r][s] : 0.f;
            const float low = j < i ? d * kk[r][s] : 0.f;
            if (back) a.a[at + i * 64 + j] = low;
            M[i * MLD + j] = j < i ? low * gate[2 * DQ + (back ? i : j)] : 0.f;
        }
    if (tid < DQ)
#pragma unroll
        for (int e = 0; e < DGATES / DQ; ++e) a.gates[((int64_t)slot * a.H + h) * DGATES + e * DQ + tid] = gate[e * DQ + tid];
    __syncthreads();
    delta_invert<NT>(M, Ks, tid);
    for (int e = tid; e < 4096; e += NT) a.sys[at + e] = e % 64 / 16 <= e / 64 / 16 ? M[e / 64 * MLD + e % 64] : 0.f;
}

// ---- the chain.  Shared memory, in floats: the state's rows [VS][KL]; Y, Z [64][XL] of this block's values; and one or two stages (two
// where they fit) of what a chunk needs: K and Q [64][KL], V or dO [64][XL], the inverse and att [64][ML], the gates.
// 16 threads for each of a block's VS values: two rows and two values a thread.
constexpr int ML = DELTA_ML;                  // rows of 16-byte pieces, four banks apart; XL of VS values: an odd number of pieces
constexpr int chain_threads(int VS) { return 16 * VS; }
constexpr int chain_row(int VS) { return VS + 4; }
struct ChainSizes {
    int KP, KL, stage, stages, bytes;
};
__host__ __device__ inline ChainSizes chain_sizes(int K, int VS) {
    ChainSizes z;
    const int XL = chain_row(VS);
    z.KP = (K + 3) / 4 * 4;
    z.KL = z.KP + (z.KP % 8 == 0 ? 4 : 8);     // an odd number of pieces
    z.stage = 2 * 64 * z.KL + 64 * XL + 2 * 64 * ML + DGATES;
    const int fix = VS * z.KL + 2 * 64 * XL;
    z.stages = (fix + 2 * z.stage) * 4 <= 227 * 1024 ? 2 : 1;
    z.bytes = (fix + z.stages * z.stage) * 4;
    return z;
}
__device__ __forceinline__ void copy_async(float *to, const float *from, int n) {   // n of 4 floats, zeros after them
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from), "r"(4 * n) : "memory");
}
__device__ __forceinline__ void copy_async1(float *to, const float *from, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from), "r"(in ? 4 : 0) : "memory");
}
// rows [0, 64) x columns [c0, c0 + W), W a multiple of 4, of a token tensor of n columns, zeros past `len` rows and n.  fp32 in the background.
template <int N, typename T>
__device__ __forceinline__ void load_tile(float *to, int ld, const T *p, int64_t step, int len, int c0, int W, int n, bool vec, int tid) {
    if constexpr (sizeof(T) == 4) {
        if (vec) {
            for (int e = tid; e < 64 * (W / 4); e += N) {
                const int i = e / (W / 4), c = e % (W / 4) * 4, left = i < len ? min(4, max(0, n - c0 - c)) : 0;
                copy_async(to + i * ld + c, left > 0 ? p + i * step + c0 + c : p, left);
            }
        } else {
            for (int e = tid; e < 64 * W; e += N) {
                const int i = e / W, c = e % W;
                const bool in = i < len && c0 + c < n;
                copy_async1(to + i * ld + c, in ? p + i * step + c0 + c : p, in);
            }
        }
    } else {
        for (int e = tid; e < 64 * W; e += N) {
            const int i = e / W, c = e % W;
            to[i * ld + c] = i < len && c0 + c < n ? to_f(p[i * step + c0 + c]) : 0.f;
        }
    }
}
// C[i][v] += sum over j <= i of A[i][j] B[j][v]: rows i = ig + 32 r, columns v = 2 vg, 2 vg + 1
template <int XL>
__device__ __forceinline__ void mul_lower(float (&C)[2][2], const float *A, const float *B, int ig, int vg) {
    const int ib = ig / 16;                                 // (the same for a warp's threads)
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
        if (jb > 2 + ib) break;
#pragma unroll
        for (int j = 16 * jb; j < 16 * jb + 16; j += 4) {
            float2 b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = *reinterpret_cast<const float2 *>(B + (j + e) * XL + 2 * vg);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if (r == 0 && jb > ib) continue;
                const float4 x = *reinterpret_cast<const float4 *>(A + (ig + 32 * r) * ML + j);
                const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    C[r][0] = fmaf(xs[e], b[e].x, C[r][0]);
                    C[r][1] = fmaf(xs[e], b[e].y, C[r][1]);
                }
            }
        }
    }
}
// C[j][v] += sum over i >= j of A[i][j] B[i][v]: rows j = 2 ig + r
template <int XL>
__device__ __forceinline__ void mul_lower_t(float (&C)[2][2], const float *A, const float *B, int ig, int vg) {
#pragma unroll 8
    for (int i = ig / 8 * 16; i < 64; ++i) {
        const float2 x = *reinterpret_cast<const float2 *>(A + i * ML + 2 * ig);
        const float2 b = *reinterpret_cast<const float2 *>(B + i * XL + 2 * vg);
        C[0][0] = fmaf(x.x, b.x, C[0][0]);
        C[0][1] = fmaf(x.x, b.y, C[0][1]);
        C[1][0] = fmaf(x.y, b.x, C[1][0]);
        C[1][1] = fmaf(x.y, b.y, C[1][1]);
    }
}
// D[v][k] += sum over i of W[i][v] K[i][k]: TV values from v0 on, four keys
template <int TV, int XL>
__device__ __forceinline__ void mul_state(float (&D)[TV][4], const float *W, const float *K, int KL) {
#pragma unroll 8
    for (int i = 0; i < 64; ++i) {
        const float4 k = *reinterpret_cast<const float4 *>(K + i * KL);
        float w[TV];
#pragma unroll
        for (int e = 0; e < TV; ++e) w[e] = W[i * XL + e];
#pragma unroll
        for (int e = 0; e < TV; ++e) {
            D[e][0] = fmaf(w[e], k.x, D[e][0]);
            D[e][1] = fmaf(w[e], k.y, D[e][1]);
            D[e][2] = fmaf(w[e], k.z, D[e][2]);
            D[e][3] = fmaf(w[e], k.w, D[e][3]);
        }
    }
}
// S[v][k] = whole S + W^T K (+ Z^T Q), tiles of TV values x 4 keys
template <int TV, int VS, bool BACK>
__device__ __forceinline__ void update_state(float *S, const float *W, const float *Z, const float *K, const float *Q, float whole, int KP, int KL, int tid) {
    for (int t = tid; t < VS / TV * (KP / 4); t += chain_threads(VS)) {
        const int v0 = t % (VS / TV) * TV, k0 = t / (VS / TV) * 4;
        float D[TV][4] = {};
        mul_state<TV, chain_row(VS)>(D, W + v0, K + k0, KL);
        if (BACK) mul_state<TV, chain_row(VS)>(D, Z + v0, Q + k0, KL);
#pragma unroll
        for (int e = 0; e < TV; ++e) {
            float4 *p = reinterpret_cast<float4 *>(S + (v0 + e) * KL + k0);
            const float4 x = *p;
            *p = make_float4(fmaf(whole, x.x, D[e][0]), fmaf(whole, x.y, D[e][1]), fmaf(whole, x.z, D[e][2]), fmaf(whole, x.w, D[e][3]));
        }
    }
}

template <typename T, bool BACK, int VS>
__global__ void __launch_bounds__(chain_threads(VS), 1) k_chain(const DeltaArgs a) {
    constexpr int XL = chain_row(VS), N_ = chain_threads(VS);
    after_previous();
    extern __shared__ float sm[];
    const ChainSizes z = chain_sizes(a.K, VS);
    const int KP = z.KP, KL = z.KL;
    float *S = sm, *Y = S + VS * KL, *Z = Y + 64 * XL, *stages = Z + 64 * XL;
    const int nv = (a.V + VS - 1) / VS, tid = threadIdx.x, ig = tid / (VS / 2), vg = tid % (VS / 2);
    const int v0 = blockIdx.x % nv * VS, h = blockIdx.x / nv % a.H, s = blockIdx.x / nv / a.H, grp = h / (a.H / a.G);
    if (a.nslots == 0 && blockIdx.x == 0 && tid < HDR_WORDS) a.hdr[tid] = 0;   // (of a call without tokens this is the first launch)
    const DeltaSeq q = delta_seq(a, s);
    const int64_t sat = ((int64_t)s * a.H + h) * a.V * a.K;
    const int nch = (q.len + DQ - 1) / DQ;
    auto issue = [&](int n) {                               // what step n needs
        const int ci = BACK ? nch - 1 - n : n;
        const DeltaChunk c{q.b, q.t0 + ci * DQ, min(DQ, q.len - ci * DQ)};
        const int64_t ch = (int64_t)(q.slot0 + ci) * a.H + h;
        float *st = stages + (z.stages == 2 ? n & 1 : 0) * z.stage;
        load_tile<N_>(st, KL, rows_of<T>(a.k, a.ks, c, grp), a.ks[1], c.len, 0, KP, a.K, a.vk, tid);
        if (BACK || a.o) load_tile<N_>(st + 64 * KL, KL, rows_of<T>(a.q, a.qs, c, grp), a.qs[1], c.len, 0, KP, a.K, a.vq, tid);
        if (BACK) load_tile<N_>(st + 128 * KL, XL, rows_of<T>(a.dO, a.dos, c, h), a.dos[1], c.len, v0, VS, a.V, a.vo, tid);
        else load_tile<N_>(st + 128 * KL, XL, rows_of<T>(a.v, a.vs, c, h), a.vs[1], c.len, v0, VS, a.V, a.vv, tid);
        float *M = st + 128 * KL + 64 * XL;
        for (int e = tid; e < 64 * 16; e += N_) {
            copy_async(M + e / 16 * ML + e % 16 * 4, a.sys + ch * 4096 + e * 4, 4);
            copy_async(M + 64 * ML + e / 16 * ML + e % 16 * 4, a.att + ch * 4096 + e * 4, 4);
        }
        for (int e = tid; e < DGATES / 4; e += N_) copy_async(M + 2 * 64 * ML + e * 4, a.gates + ch * DGATES + e * 4, 4);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (nch > 0) issue(0);
    const void *in = BACK ? a.dfinal : a.init;
    const bool in16 = BACK ? a.dfinal_bf16 : a.init_bf16;
    for (int e = tid; e < VS * KP; e += N_) {
        const int v = e / KP, k = e % KP;
        S[v * KL + k] = in && v0 + v < a.V && k < a.K ? delta_ld(in, !in16, sat + (int64_t)(v0 + v) * a.K + k) : 0.f;
    }
    float *kept = static_cast<float *>(BACK ? a.dS : a.S), *vals = static_cast<float *>(BACK ? a.mu : a.U);
    for (int n = 0; n < nch; ++n) {
        const int ci = BACK ? nch - 1 - n : n;
        const DeltaChunk c{q.b, q.t0 + ci * DQ, min(DQ, q.len - ci * DQ)};
        const int64_t ch = (int64_t)(q.slot0 + ci) * a.H + h;
        if (z.stages == 2 && n + 1 < nch) {                 // (every thread is done with the other stage since the last sync)
            issue(n + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        const float *Ks = stages + (z.stages == 2 ? n & 1 : 0) * z.stage, *Qs = Ks + 64 * KL, *Xs = Qs + 64 * KL, *Ms = Xs + 64 * XL, *Ma = Ms + 64 * ML, *gate = Ma + 64 * ML;
        if (kept)
            for (int e = tid; e < VS * KP; e += N_) {
                const int v = e / KP, k = e % KP;
                if (v0 + v < a.V && k < a.K) kept[(ch * a.V + v0 + v) * a.K + k] = S[v * KL + k];
            }
        // P = K S^T and, forwards, Q S^T: rows ig + 32 r (backwards 2 ig + r), columns 2 vg, 2 vg + 1
        float P[2][2] = {}, O[2][2] = {};
        const bool outs = !BACK && a.o;
        auto rw = [&](int r) { return BACK ? 2 * ig + r : ig + 32 * r; };
#pragma unroll 2
        for (int l = 0; l < KP; l += 4) {
            float4 b[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) b[e] = *reinterpret_cast<const float4 *>(S + (2 * vg + e) * KL + l);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float4 x = *reinterpret_cast<const float4 *>(Ks + rw(r) * KL + l);
#pragma unroll
                for (int e = 0; e < 2; ++e) P[r][e] = fmaf(x.x, b[e].x, fmaf(x.y, b[e].y, fmaf(x.z, b[e].z, fmaf(x.w, b[e].w, P[r][e]))));
                if (outs) {
                    const float4 y = *reinterpret_cast<const float4 *>(Qs + rw(r) * KL + l);
#pragma unroll
                    for (int e = 0; e < 2; ++e) O[r][e] = fmaf(y.x, b[e].x, fmaf(y.y, b[e].y, fmaf(y.z, b[e].z, fmaf(y.w, b[e].w, O[r][e]))));
                }
            }
        }
        float N[2][2] = {};
        if (BACK) mul_lower_t<XL>(N, Ma, Xs, ig, vg);           // N = scale att^T dO + e^(Gc - G) P
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int i = rw(r);
            float2 y;
            if (BACK) {
                y = make_float2(fmaf(gate[DQ + i], P[r][0], a.scale * N[r][0]), fmaf(gate[DQ + i], P[r][1], a.scale * N[r][1]));
            } else {
                const float2 v = *reinterpret_cast<const float2 *>(Xs + i * XL + 2 * vg);
                y = make_float2(fmaf(-gate[i], P[r][0], v.x), fmaf(-gate[i], P[r][1], v.y));
            }
            *reinterpret_cast<float2 *>(Y + i * XL + 2 * vg) = y;
        }
        __syncthreads();
        float U[2][2] = {};
        if (BACK) mul_lower_t<XL>(U, Ms, Y, ig, vg);
        else mul_lower<XL>(U, Ms, Y, ig, vg);
        __syncthreads();
        // W = beta U, or lam; what goes to the state: e^(Gc - G) W in Z, backwards -e^G lam in Y and scale e^G dO in Z
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int i = rw(r);
            if (vals)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (v0 + 2 * vg + e < a.V) vals[(ch * 64 + i) * a.V + v0 + 2 * vg + e] = U[r][e];
            const float w0 = gate[2 * DQ + i] * U[r][0], w1 = gate[2 * DQ + i] * U[r][1];
            if (BACK) {
                *reinterpret_cast<float2 *>(Y + i * XL + 2 * vg) = make_float2(-gate[i] * w0, -gate[i] * w1);
                const float2 v = *reinterpret_cast<const float2 *>(Xs + i * XL + 2 * vg);
                *reinterpret_cast<float2 *>(Z + i * XL + 2 * vg) = make_float2(a.scale * gate[i] * v.x, a.scale * gate[i] * v.y);
            } else {
                *reinterpret_cast<float2 *>(Y + i * XL + 2 * vg) = make_float2(w0, w1);
                *reinterpret_cast<float2 *>(Z + i * XL + 2 * vg) = make_float2(gate[DQ + i] * w0, gate[DQ + i] * w1);
            }
        }
        __syncthreads();
        const float whole = gate[DQ - 1];
        if (outs) {
            float A[2][2] = {};
            mul_lower<XL>(A, Ma, Y, ig, vg);
            T *op = static_cast<T *>(a.o) + c.b * a.os[0] + c.t0 * a.os[1] + h * a.os[2] + v0;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = ig + 32 * r, v = 2 * vg + e;
                    if (i < c.len && v0 + v < a.V) op[i * a.os[1] + v] = from_f<T>(a.scale * fmaf(gate[i], O[r][e], A[r][e]));
                }
        }
        if (KP > 64) update_state<2, VS, BACK>(S, BACK ? Y : Z, Z, Ks, Qs, whole, KP, KL, tid);
        else update_state<1, VS, BACK>(S, BACK ? Y : Z, Z, Ks, Qs, whole, KP, KL, tid);
        __syncthreads();
        if (z.stages == 1 && n + 1 < nch) issue(n + 1);
    }
    __syncthreads();
    void *out = BACK ? a.dinit : a.final;
    const bool out16 = BACK ? a.dinit_bf16 : a.final_bf16;
    if (out)
        for (int e = tid; e < VS * KP; e += N_) {
            const int v = e / KP, k = e % KP;
            if (v0 + v < a.V && k < a.K) delta_st(out, !out16, sat + (int64_t)(v0 + v) * a.K + k, S[v * KL + k]);
        }
}

// rows [0, 64) x 32 columns from column c0 of a contiguous fp32 matrix of n columns, row i times f[i]
__device__ __forceinline__ void load_plain(float *to, const float *p, int rows, int c0, int n, const float *f, int tid) {
    for (int e = tid; e < 64 * 32; e += NT) {
        const int i = e / 32, c = e % 32;
        to[i * LD + c] = i < rows && c0 + c < n ? p[(int64_t)i * n + c0 + c] * (f ? f[i] : 1.f) : 0.f;
    }
}
__device__ __forceinline__ float row16(float v) {                  // sum over the 16 threads that share a row
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---- a chunk's gradients, a block a chunk, head and share of the keys (slices of 32, one after the other).  Shared memory: E + E^T and F
// (64 x 64), four slices, the gates, sums per row.  What goes into dg is left for the last launch: of the first share what crosses each token
// inside the chunk, of each share the sums of its keys, and its part of <dS', S>.
constexpr int GRADS_FLOATS = 2 * 64 * MLD + 4 * 64 * LD + DGATES + 4 * 64 + 64 + 64 + NT / 32;
constexpr int FLOW = DELTA_FLOW;        // floats left by a share: flow, X, R, <dS', S>

template <typename T>
__global__ void __launch_bounds__(NT) k_grads(const DeltaArgs a, const int shares) {
    after_previous();
    extern __shared__ float sm[];
    float *E = sm, *F = E + 64 * MLD, *s0 = F + 64 * MLD, *s1 = s0 + 64 * LD, *s2 = s1 + 64 * LD, *s3 = s2 + 64 * LD;
    float *gate = s3 + 64 * LD, *R = gate + DGATES, *X = R + 64, *fg = X + 64, *fd = fg + 64, *fl = fd + 64, *red = fl + 64;
    const int share = blockIdx.x % shares, h = blockIdx.x / shares % a.H, slot = blockIdx.x / shares / a.H, grp = h / (a.H / a.G), tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    const DeltaChunk c = delta_chunk(a, slot);
    if (c.len == 0) return;
    const int64_t ch = (int64_t)slot * a.H + h;
    const float *U = static_cast<const float *>(a.U) + ch * 64 * a.V, *mu = static_cast<const float *>(a.mu) + ch * 64 * a.V;
    const float *S = static_cast<const float *>(a.S) + ch * a.V * a.K, *dS = static_cast<const float *>(a.dS) + ch * a.V * a.K;
    const T *dop = rows_of<T>(a.dO, a.dos, c, h), *kp = rows_of<T>(a.k, a.ks, c, grp), *qp = rows_of<T>(a.q, a.qs, c, grp);
    for (int e = tid; e < DGATES; e += NT) gate[e] = a.gates[ch * DGATES + e];
    __syncthreads();
    const float *beta = gate + 2 * DQ;
    if (tid < 64) {
        R[tid] = X[tid] = 0.f;
        fg[tid] = a.scale * gate[tid];                              // scale e^G
        fd[tid] = beta[tid] * gate[DQ + tid];                       // e^(Gc - G) beta
        fl[tid] = -gate[tid] * beta[tid];                           // -e^G beta
    }
    // lam_i.W_j and dO_i.W_j; dV = lam; dbeta = mu.U
    float lw[4][4], ow[4][4];
    float db[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int s = 0; s < 4; ++s) lw[r][s] = ow[r][s] = 0.f;
    for (int v0 = 0; v0 < a.V; v0 += 32) {
        __syncthreads();
        load_plain(s0, U, 64, v0, a.V, beta, tid);
        load_plain(s1, mu, 64, v0, a.V, beta, tid);
        load_slice<NT>(s2, dop, a.dos[1], c.len, v0, a.V, tid);
        __syncthreads();
        T *dv = static_cast<T *>(a.dv) + c.b * a.dvs[0] + c.t0 * a.dvs[1] + h * a.dvs[2];
        for (int e = tid; e < 64 * 32 && share == 0; e += NT) {
            const int i = e / 32, v = e % 32;
            if (i < c.len && v0 + v < a.V) dv[i * a.dvs[1] + v0 + v] = from_f<T>(s1[i * LD + v]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int v = v0 + 2 * tx + e, i = 16 * r + ty;
                if (v < a.V) db[r] = fmaf(mu[(int64_t)i * a.V + v], U[(int64_t)i * a.V + v], db[r]);
            }
        mul_rows(lw, ow, s1, s2, s0, ty, tx);
    }
    // F, E, and what crosses the tokens: W_ij = F_ij q_i.k_j + E_ij k_i.k_j below the diagonal
    float W[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        db[r] = row16(db[r]);
        const int i = 16 * r + ty;
        if (share == 0 && tx == 0 && i < c.len) delta_st(a.dbeta, a.beta_f32, c.b * a.dbs[0] + (int64_t)(c.t0 + i) * a.dbs[1] + h * a.dbs[2], db[r]);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int j = 16 * s + tx;
            const float d = j <= i ? delta_decay(gate[3 * DQ + i], gate[4 * DQ + i], gate[3 * DQ + j], gate[4 * DQ + j]) : 0.f;
            F[i * MLD + j] = j <= i ? a.scale * ow[r][s] * d : 0.f;
            E[i * MLD + j] = j < i ? -lw[r][s] * d : 0.f;
            W[r][s] = j < i ? a.scale * ow[r][s] * a.att[ch * 4096 + i * 64 + j] - lw[r][s] * a.a[ch * 4096 + i * 64 + j] : 0.f;
        }
    }
    // the slices' memory holds W meanwhile; then flow_t = sum over i >= t > j of W_ij
    float *left = a.flow + (ch * shares + share) * FLOW;
    __syncthreads();
    if (share == 0) {
    float *Wm = s0;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int s = 0; s < 4; ++s) Wm[(16 * r + ty) * MLD + 16 * s + tx] = W[r][s];
    __syncthreads();
    if (tid < 64) {                                                  // along each row: sums before the column
        float run = 0.f;
        for (int j = 0; j < 64; ++j) {
            const float w = Wm[tid * MLD + j];
            Wm[tid * MLD + j] = run;
            run += w;
        }
    }
    __syncthreads();
    if (tid < 64) {
        float f = 0.f;
        for (int i = tid; i < 64; ++i) f += Wm[i * MLD + tid];
        left[tid] = f;
    }
    }
    __syncthreads();
    // E + E^T
    for (int e = tid; e < 4096; e += NT) {
        const int i = e / 64, j = e % 64;
        if (j < i) E[j * MLD + i] = E[i * MLD + j];
    }
    float SS = 0.f;
    T *dqp = static_cast<T *>(a.dq) + c.b * a.dqs[0] + c.t0 * a.dqs[1] + grp * a.dqs[2];
    T *dkp = static_cast<T *>(a.dk) + c.b * a.dks[0] + c.t0 * a.dks[1] + grp * a.dks[2];
    for (int k0 = 32 * share; k0 < a.K; k0 += 32 * shares) {
        float dq[4][2] = {}, kr[4][2] = {}, kw[4][2] = {};
        for (int v0 = 0; v0 < a.V; v0 += 32) {
            // scale e^G dO S, -e^G lam S
            __syncthreads();
            load_slice<NT>(s0, dop, a.dos[1], c.len, v0, a.V, tid);
            load_plain(s1, mu, 64, v0, a.V, fl, tid);
            for (int e = tid; e < 32 * 32; e += NT) {
                const int v = e / 32, k = e % 32;
                const bool in = v0 + v < a.V && k0 + k < a.K;
                const float x = in ? S[(int64_t)(v0 + v) * a.K + k0 + k] : 0.f, y = in ? dS[(int64_t)(v0 + v) * a.K + k0 + k] : 0.f;
                s2[v * LD + k] = x;
                s2[(32 + v) * LD + k] = y;
                SS = fmaf(x, y, SS);
            }
            load_plain(s3, U, 64, v0, a.V, fd, tid);
            __syncthreads();
            fma_slice(dq, s0, LD, s2, LD, 32, ty, tx);
            fma_slice(kr, s1, LD, s2, LD, 32, ty, tx);
            fma_slice(kw, s3, LD, s2 + 32 * LD, LD, 32, ty, tx);
        }
        __syncthreads();
        load_slice<NT>(s0, kp, a.ks[1], c.len, k0, a.K, tid);
        load_slice<NT>(s1, qp, a.qs[1], c.len, k0, a.K, tid);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * r + ty;
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float kv = s0[i * LD + 2 * tx + e], qv = s1[i * LD + 2 * tx + e];
                dq[r][e] *= fg[i];
                x += qv * dq[r][e] + kv * kr[r][e];
                y += kv * kw[r][e];
                kr[r][e] += kw[r][e];
            }
            x = row16(x);
            y = row16(y);
            if (tx == 0) {
                R[i] += x;
                X[i] += y;
            }
        }
        fma_slice(dq, F, MLD, s0, LD, 64, ty, tx);
        fma_slice(kr, E, MLD, s0, LD, 64, ty, tx);
        fma_slice_t(kr, F, MLD, s1, LD, 64, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 16 * r + ty, k = k0 + 2 * tx + e;
                if (i >= c.len || k >= a.K) continue;
                if (a.part) {
                    a.part[(ch * 64 + i) * a.K + k] = dq[r][e];
                    a.part[(((int64_t)a.nslots * a.H + ch) * 64 + i) * a.K + k] = kr[r][e];
                } else {
                    dqp[i * a.dqs[1] + k] = from_f<T>(dq[r][e]);
                    dkp[i * a.dks[1] + k] = from_f<T>(kr[r][e]);
                }
            }
    }
    SS = warp_sum(SS);
    if (tid % 32 == 0) red[tid / 32] = SS;
    __syncthreads();
    if (tid < 64) {
        left[64 + tid] = X[tid];
        left[128 + tid] = R[tid];
    }
    if (tid < 32) {
        const float all = warp_sum(tid < NT / 32 ? red[tid] : 0.f);
        if (tid == 0) left[192] = gate[DQ - 1] * all;
    }
}

// The last launch, a block a chunk and group: dq and dk, the sums over the group's heads in their order; and dg of each head by a warp,
// lane l tokens 2l and 2l + 1: what crosses the token, what left the tokens before it, what passes all, what came from before it.
template <typename T>
__global__ void __launch_bounds__(NT) k_finish(const DeltaArgs a, const int shares) {
    after_previous();
    const int slot = blockIdx.x / a.G, grp = blockIdx.x % a.G, per = a.H / a.G, lane = threadIdx.x % 32;
    const DeltaChunk c = delta_chunk(a, slot);
    if (c.len == 0) return;
    for (int h = grp * per + threadIdx.x / 32; h < (grp + 1) * per; h += NT / 32) {
        const float *left = a.flow + ((int64_t)slot * a.H + h) * shares * FLOW;
        float x[2] = {}, r[2] = {}, all = 0.f;
        for (int p = 0; p < shares; ++p) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                x[e] += left[p * FLOW + 64 + 2 * lane + e];
                r[e] += left[p * FLOW + 128 + 2 * lane + e];
            }
            all += left[p * FLOW + 192];
        }
        float before = x[0] + x[1], after = r[0] + r[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float u = __shfl_up_sync(0xffffffffu, before, o), d = __shfl_down_sync(0xffffffffu, after, o);
            if (lane >= o) before += u;
            if (lane + o < 32) after += d;
        }
        before = __shfl_up_sync(0xffffffffu, before, 1);
        after = __shfl_down_sync(0xffffffffu, after, 1);
        if (lane == 0) before = 0.f;
        if (lane == 31) after = 0.f;
        after += r[1];
        const float d[2] = {left[2 * lane] + before + all + (after + r[0]), left[2 * lane + 1] + (before + x[0]) + all + after};
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (2 * lane + e < c.len) delta_st(a.dg, a.g_f32, c.b * a.dgs[0] + (int64_t)(c.t0 + 2 * lane + e) * a.dgs[1] + h * a.dgs[2], d[e]);
    }
    if (a.part == nullptr) return;
    T *dqp = static_cast<T *>(a.dq) + c.b * a.dqs[0] + c.t0 * a.dqs[1] + grp * a.dqs[2];
    T *dkp = static_cast<T *>(a.dk) + c.b * a.dks[0] + c.t0 * a.dks[1] + grp * a.dks[2];
    const int64_t other = (int64_t)a.nslots * a.H * 64 * a.K;
    for (int e = threadIdx.x; e < c.len * a.K; e += NT) {
        const int i = e / a.K, k = e % a.K;
        float x = 0.f, y = 0.f;
        for (int r = 0; r < per; ++r) {
            const int64_t at = (((int64_t)slot * a.H + grp * per + r) * 64 + i) * a.K + k;
            x += a.part[at];
            y += a.part[other + at];
        }
        dqp[i * a.dqs[1] + k] = from_f<T>(x);
        dkp[i * a.dks[1] + k] = from_f<T>(y);
    }
}

template <typename T, bool BACK, int VS>
cudaError_t launch_chain(const DeltaArgs &a, cudaStream_t st) {
    static int set[64] = {};
    const int bytes = chain_sizes(a.K, VS).bytes;
    if (cudaError_t e = ensure_smem_attr(k_chain<T, BACK, VS>, bytes, set); e != cudaSuccess) return e;
    return launch_early(k_chain<T, BACK, VS>, (unsigned)(a.nseqs * (int64_t)a.H * ((a.V + VS - 1) / VS)), chain_threads(VS), bytes, st, a);
}
// The fewest values a block whose blocks still have an SM each: a block is bound by its reads of shared memory, which go with
// its values.  6 chunks of 9 sequences and heads of 96 x 64: 32 / 16 / 8 values 66 / 47 / 38 us; 8 chunks of 12 of 128 x 128:
// 129 / 88 / 131 (192 blocks); of 20: 129 / 165 / 193; 32 chunks of 64: 966 / 1228 / 1720.
template <typename T, bool BACK>
cudaError_t chain(const DeltaArgs &a, cudaStream_t st) {
    auto fits = [&](int VS) { return a.nseqs * (int64_t)a.H * ((a.V + VS - 1) / VS) <= kDeltaSMs; };
    return fits(8) ? launch_chain<T, BACK, 8>(a, st) : fits(16) ? launch_chain<T, BACK, 16>(a, st) : launch_chain<T, BACK, 32>(a, st);
}

template <typename T>
cudaError_t fwd(const DeltaArgs &a, cudaStream_t st) {
    if (a.nslots > 0)
        if (cudaError_t e = launch_early(k_prep<T>, (unsigned)((int64_t)a.nslots * a.H), NT, 0, st, a, false); e != cudaSuccess) return e;
    return chain<T, false>(a, st);
}
template <typename T>
cudaError_t bwd(const DeltaArgs &a, cudaStream_t st) {
    if (a.nslots > 0)
        if (cudaError_t e = launch_early(k_prep<T>, (unsigned)((int64_t)a.nslots * a.H), NT, 0, st, a, true); e != cudaSuccess) return e;
    if (cudaError_t e = chain<T, true>(a, st); e != cudaSuccess) return e;
    if (a.nslots == 0) return cudaSuccess;
    static int set[64] = {};
    const int bytes = GRADS_FLOATS * (int)sizeof(float);
    if (cudaError_t e = ensure_smem_attr(k_grads<T>, bytes, set); e != cudaSuccess) return e;
    const int shares = delta_grad_shares(a.nslots, a.H, a.K);
    if (cudaError_t e = launch_early(k_grads<T>, (unsigned)((int64_t)a.nslots * a.H * shares), NT, bytes, st, a, shares); e != cudaSuccess) return e;
    return launch_early(k_finish<T>, (unsigned)((int64_t)a.nslots * a.G), NT, 0, st, a, shares);
}

}  // namespace

cudaError_t delta_simt_fwd(const DeltaArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? fwd<__nv_bfloat16>(a, st) : fwd<float>(a, st);
}
cudaError_t delta_simt_bwd(const DeltaArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? bwd<__nv_bfloat16>(a, st) : bwd<float>(a, st);
}

}  // namespace ssd
