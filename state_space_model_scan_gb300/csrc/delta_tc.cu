// delta_tc.cu -- the gated delta rule on tcgen05 tensor cores: bf16 data, headdim and dstate up to 128 (smaller ones as
// the zero-extended part of 128).  Formulas in delta.cuh.
//
// Two kernels forwards.  k_prep, a block a chunk and head: K K^T and Q K^T in one product (K's rows and Q's rows as the 128
// rows of A), the gates, the triangular system, its inverse (fp32, by blocks) and att, left as operand images.  k_chain, a block a
// sequence and head (or a segment of one), walks the chunks.  It works on transposed matrices, so that the
// 128 TMEM lanes are the values: lane v holds row v of the state S [values][keys], and every product
//
//     P^T = S K^T   [v][i]        Y = V^T - e^G P^T     U^T = Y sys^T  [v][i]      S' = e^Gc S + (e^(Gc - G) beta U)^T K   [v][k]
//
// has its left operand in tensor memory, put there from registers by the threads that own the lane, and its right one (K,
// sys, att, Q as they lie) in shared memory: between two products of the chain there is one tcgen05.ld, a
// little arithmetic and one tcgen05.st, and no shared memory is written.  The state stays in registers, in fp32.
// What is carried (S, Y, e^(Gc - G) beta U, sys) enters a product as the sum of two bf16 values (2^-17), two or three products of
// which the small ones are the cheaper price than tf32's single one of half the rate and 2^-11; what only leaves as bf16
// (att, beta U in o) as one: o is off by 2.6e-3, of which its own rounding is 1.7e-3 (beta U as two took 6% more time for 2.2e-3).  Where keys point
// much the same way and little is forgotten, a token's U takes back what the ones before have written, att W is a sum that cancels, and those
// roundings count for more: 5.8e-3 at a mean cosine of 0.5, 8.9e-3 at 0.95 (by arithmetic in 64 bits: 6e-3 with beta U or att as two, 1.7e-3 with both).
// Backwards the same chain runs from the last chunk to the first, with dS in S's place and the transposed inverse in sys's: k_prep
// leaves both for it, which come of one substitution, and nothing of the chunks is computed twice.
//
// Warps of a chain block: eight with two threads a lane, each half of the columns (four threads a lane were 13% slower: a thread's
// second quarter is what runs beside the products of the first); four with one thread a lane for what is off
// the chain; two that load the next chunk, one that stores; one thread that issues every product.  A product of 128 x 64 x 16 takes as
// long as one of 128 x 128 x 16 (64 cycles), so that K's and
// Q's rows, and both terms of sys, go as one right operand of 128 rows.  All waits are bounded.
//
// Bound by latency: a step of a chunk is three products in a row with arithmetic between them, about 2.6 us, of which the products are 40% and the
// rest are splits, loads and stores of tensor memory at two warps a scheduler; the launch's first step comes 7 us late (first
// copies, tensor memory, cold code).  8192 tokens of 32 heads, 128 x 128: k_prep 50 us, chains 117 + 67 (34.6 GF, 204 MB: 18 and 30 us);
// 2 x 2048 tokens forwards 31 + 96 us, backwards 102, k_grads 80 (294 MB, 3.7 TB/s).
#include <cudaTypedefs.h>

#include <algorithm>

#include "delta_tc.cuh"

namespace ssd {

namespace {

using namespace dtc;

// ---------------------------------------------------------------------------------------- the chunk's matrices
// Bound by instructions and by the waits between its steps, six blocks on an SM (shared memory): issue 61%, shared memory 63%.
constexpr int PREP_NT = 128;
constexpr int MLD = DELTA_ML;
// K's and Q's rows; once their product is out, the system and scratch lie over them
constexpr int TLD = 40;         // of the scratch matrix: its columns are read four rows at a time, eight banks apart
constexpr uint32_t P_A = 0, P_M = 0, P_T = 64 * MLD * 4, P_ATT = 3 * HALF, P_GATE = 4 * HALF, P_COLS = P_GATE + GATE_BYTES, P_MISC = P_COLS + DQ * 4, P_BYTES = P_MISC + 64 + 1024;

// e^(G_i - G_j), as delta_decay, by the multi-function unit: off by 2^-22 and by 2^-24 of the exponent
__device__ __forceinline__ float decay_of(float hi_i, float lo_i, float hi_j, float lo_j) {
    return ex2f(kLog2e * ((hi_i - hi_j) + (lo_i - lo_j)));
}
// D += A B for A 16 x 8 (rows), B 8 x 8, by a warp; fp32 entries of which the tensor core takes the leading 11 bits
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&x)[4], const uint32_t (&y)[2]) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(y[0]), "r"(y[1]));
}
// v as the sum of its leading 11 bits and the rest (exact)
__device__ __forceinline__ void split_tf32(float v, uint32_t &hi, uint32_t &lo) {
    hi = __float_as_uint(v) & 0xffffe000u;
    lo = __float_as_uint(v - __uint_as_float(hi));
}
// acc = A diag(f) B for 16 rows of A (rows lda apart; f NULL: 1) and 8 COLS columns of B (rows MLD or TLD apart), inner length N: every
// entry as two terms of 11 bits, three of the four products (off by 2^-20 of each).  At N = 8 there are eight rows, taken twice.
template <int N, int COLS>
__device__ __forceinline__ void small_product(float (&acc)[COLS][4], const float *A, const float *f, const float *B, int ldb, int lane) {
    const int r = lane >> 2, c = lane & 3, r2 = N == 8 ? r : r + 8;
#pragma unroll
    for (int t = 0; t < COLS; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
#pragma unroll
    for (int l = 0; l < N; l += 8) {
        float x[4] = {A[r * MLD + l + c], A[r2 * MLD + l + c], A[r * MLD + l + c + 4], A[r2 * MLD + l + c + 4]};
        if (f != nullptr) {
            const float f0 = f[l + c], f1 = f[l + c + 4];
            x[0] *= f0; x[1] *= f0; x[2] *= f1; x[3] *= f1;
        }
        uint32_t xh[4], xl[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_tf32(x[e], xh[e], xl[e]);
#pragma unroll
        for (int t = 0; t < COLS; ++t) {
            uint32_t yh[2], yl[2];
            split_tf32(B[(l + c) * ldb + 8 * t + r], yh[0], yl[0]);
            split_tf32(B[(l + c + 4) * ldb + 8 * t + r], yh[1], yl[1]);
            mma_tf32(acc[t], xl, yh);
            mma_tf32(acc[t], xh, yl);
            mma_tf32(acc[t], xh, yh);
        }
    }
}
// The block X21 below the diagonal of a pair of N x N blocks, from a21 in its place, with t = a21 - a21 B1 X11:
// X21 = t - X22 B2 t (T: scratch for B2 t).  At N = 8 a warp takes each of the four pairs, at 16 two each of two, at 32 four the one; a
// warp 16 rows (at 8 eight).
template <int N>
__device__ __forceinline__ void join_pair(float *M, float *T, const float *beta, int w, int lane) {
    constexpr int COLS = N == 32 ? 2 : 1, ROWS = N == 8 ? 1 : 2;
    const int o = N == 8 ? w * 16 : N == 16 ? (w >> 1) * 32 : 0, i = N == 32 ? (w >> 1) * 16 : 0, j = N == 8 ? 0 : (w & 1) * (N / 2), r = lane >> 2, c = 2 * (lane & 3);
    float *own = M + (o + N + i) * MLD + o + j, *scr = T + o / 2 * TLD, *t = scr + i * TLD + j, acc[COLS][4], d[COLS][4];
    small_product<N, COLS>(acc, M + (o + N + i) * MLD + o, beta + o, M + o * MLD + o + j, MLD, lane);
#pragma unroll
    for (int k = 0; k < COLS; ++k)
#pragma unroll
        for (int e = 0; e < ROWS; ++e) {
            const int row = r + 8 * e, col = 8 * k + c;
            const float2 u = *reinterpret_cast<const float2 *>(own + row * MLD + col);
            const float f = beta[o + N + i + row];
            d[k][2 * e] = u.x - acc[k][2 * e];
            d[k][2 * e + 1] = u.y - acc[k][2 * e + 1];
            *reinterpret_cast<float2 *>(t + row * TLD + col) = make_float2(f * d[k][2 * e], f * d[k][2 * e + 1]);
        }
    if (N == 8) __syncwarp();
    else __syncthreads();
    small_product<N, COLS>(acc, M + (o + N + i) * MLD + o + N, nullptr, scr + j, TLD, lane);
#pragma unroll
    for (int k = 0; k < COLS; ++k)
#pragma unroll
        for (int e = 0; e < ROWS; ++e)
            *reinterpret_cast<float2 *>(own + (r + 8 * e) * MLD + 8 * k + c) = make_float2(d[k][2 * e] - acc[k][2 * e], d[k][2 * e + 1] - acc[k][2 * e + 1]);
    __syncthreads();
}
// X = (I + a B)^-1 a = a (I + B a)^-1 for a strictly lower triangular 64 x 64, B = diag(beta), in place (rows MLD apart), by PREP_NT
// threads.  Both inverses that are needed are in it: (I + a B)^-1 = I - X B and (I + B a)^-1 = I - B X.  A warp a block of 16 on the
// diagonal: its two blocks of 8 by substitution, a thread a column, and what lies below them as a join; then twice the join of
// a pair.  Those products are of 8, 16 and 32: too small for a tile of tcgen05, whose operands would have to be laid out anew for each.
// By FMAs out of shared memory they were three quarters of the kernel's shared-memory traffic, which bounded it.  Blocks above the
// diagonal: those in the pairs of 16 and 32 are set to zero, the other is neither read nor written.
__device__ __forceinline__ void solve(float *M, float *T, const float *beta, int tid) {
    const int w = tid >> 5, lane = tid & 31;
    {
        const int o = w * 16 + (lane & 8), j = lane & 7;
        if (lane < 16) {
            float x[8], xb[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float s = i > j ? M[(o + i) * MLD + o + j] : 0.f;
#pragma unroll
                for (int l = 0; l < i; l += 4) {
                    const float4 m = *reinterpret_cast<const float4 *>(M + (o + i) * MLD + o + l);
                    s = fmaf(-m.x, xb[l], s);
                    if (l + 1 < i) s = fmaf(-m.y, xb[l + 1], s);
                    if (l + 2 < i) s = fmaf(-m.z, xb[l + 2], s);
                    if (l + 3 < i) s = fmaf(-m.w, xb[l + 3], s);
                }
                x[i] = s;
                xb[i] = beta[o + i] * s;
            }
            __syncwarp(0xffffu);                             // a block's threads are in one warp
#pragma unroll
            for (int i = 0; i < 8; ++i) M[(o + i) * MLD + o + j] = x[i];
        } else {                                             // zeros above: 8 x 8 of this warp's block, and half of a pair's 16 x 16
            const int e = lane - 16, p = (w >> 1) * 32;
            *reinterpret_cast<float4 *>(M + (w * 16 + e / 2) * MLD + w * 16 + 8 + e % 2 * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                *reinterpret_cast<float4 *>(M + (p + (w & 1) * 8 + k * 4 + e / 4) * MLD + p + 16 + e % 4 * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    __syncwarp();
    join_pair<8>(M, T, beta, w, lane);
    join_pair<16>(M, T, beta, w, lane);
    join_pair<32>(M, T, beta, w, lane);
}

// a block a chunk and head
template <bool BOTH>
__global__ void __launch_bounds__(PREP_NT, 6) k_prep(const DeltaArgs a, const __grid_constant__ DeltaMaps m) {
    after_previous();
    extern __shared__ uint8_t raw[];
    uint8_t *sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    float *M = reinterpret_cast<float *>(sm + P_M), *T = reinterpret_cast<float *>(sm + P_T), *gate = reinterpret_cast<float *>(sm + P_GATE);
    float *cols = reinterpret_cast<float *>(sm + P_COLS);   // e^(G_end - G_j), end the last token of j's block of 16
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + P_MISC);
    uint32_t *tm = reinterpret_cast<uint32_t *>(sm + P_MISC + 16);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0 && tid < HDR_WORDS) a.hdr[tid] = 0;
    const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H, grp = h / (a.H / a.G);
    const DeltaChunk c = delta_chunk(a, slot);
    if (c.len == 0) return;
    // a whole chunk that comes by TMA needs nobody but one thread until its product is out, while another warp computes the gates
    const bool quick = m.has_k && m.has_q && c.len == DQ;
    const uint32_t base = smem_u32(sm + P_A);
    auto product = [&] {
#pragma unroll
        for (int k = 0; k < 8; ++k) umma_bf16(*tm, kmaj(base, k, 2 * HALF), kmaj(base, k, 2 * HALF), idesc_bf16(128, 64, 0, 0), k > 0);
        umma_commit(bar + 1);
    };
    bool ok = true;
    if (w == 0) {
        tmem_alloc(tm, 64);
        __syncwarp();
        if (lane == 0) {
            mbar_init(bar, 1);
            mbar_init(bar + 1, 1);
            fence_mbar_init();
            if (m.has_k || m.has_q) {
                mbar_expect_tx(bar, (m.has_k + m.has_q) * TOK_BYTES);
                if (m.has_k) tma_rows(sm + P_A, 2 * HALF, &m.k, bar, c, grp);
                if (m.has_q) tma_rows(sm + P_A + HALF, 2 * HALF, &m.q, bar, c, grp);
            }
            if (quick) {
                ok = mbar_wait(bar, 0);
                product();
            }
        }
        __syncwarp();
    } else if (w == 3) {
        delta_gates(a, c, h, gate, lane);
    }
    if (!quick) {
        if (!m.has_k) load_rows<PREP_NT>(sm + P_A, 2 * HALF, tok_rows(a.k, a.ks, c, grp), a.ks[1], c.len, a.K, tid);
        if (!m.has_q) load_rows<PREP_NT>(sm + P_A + HALF, 2 * HALF, tok_rows(a.q, a.qs, c, grp), a.qs[1], c.len, a.K, tid);
        __syncthreads();
        if (m.has_k || m.has_q) {
            ok = mbar_wait(bar, 0);
            if (m.has_k && c.len < DQ) zero_rows<PREP_NT>(sm + P_A, 2 * HALF, c.len, tid);
            if (m.has_q && c.len < DQ) zero_rows<PREP_NT>(sm + P_A + HALF, 2 * HALF, c.len, tid);
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) product();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tm;
    uint8_t *ops = static_cast<uint8_t *>(a.tiles) + ((int64_t)slot * a.H + h) * (BOTH ? OPS_BOTH : OPS_BYTES);
    if (tid >= 64) {                                         // (warps 2 and 3: while the product runs)
        const int j = tid - 64, e = j | 15;
        const float f = decay_of(gate[3 * DQ + e], gate[4 * DQ + e], gate[3 * DQ + j], gate[4 * DQ + j]);
        cols[j] = f;
    }
    ok = mbar_wait(bar + 1, 0) && ok;
    __syncthreads();
    if (!ok && tid == 0) set_status(a.hdr, SSD_ERR_DEVICE_TIMEOUT);
    tc_fence_after();
    // Row of K K^T (warps 0, 1) or of Q K^T (2, 3); columns in blocks of 16, as far as the warp's rows reach.  In the block on the
    // diagonal every decay is an exponential of its own; left of it e^(G_i - G_j) is the product of one of the row
    // (from the end of j's block on) and one of the column (to that end), each at most 1.
    const int i = tid & 63, ib = i >> 4, nb = 2 * (w & 1) + 2;
    const float ghi = gate[3 * DQ + i], glo = gate[4 * DQ + i];
#pragma unroll 1
    for (int jb = 0; jb < 4; ++jb) {                         // (unrolled, this loop and the next cost 4 us of 56 by their fetches)
        float x[16];
        if (jb < nb) {
            tmem_ld16(tmem + ((uint32_t)w << 21) + 16 * jb, x);
            tmem_wait_ld();
            if (jb < ib) {
                const float f = decay_of(ghi, glo, gate[3 * DQ + 16 * jb + 15], gate[4 * DQ + 16 * jb + 15]);
                const float *col = cols + 16 * jb;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(col + e);
                    x[e] *= f * v.x; x[e + 1] *= f * v.y; x[e + 2] *= f * v.z; x[e + 3] *= f * v.w;
                }
            } else if (jb == ib) {
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 h4 = *reinterpret_cast<const float4 *>(gate + 3 * DQ + 16 * jb + e), l4 = *reinterpret_cast<const float4 *>(gate + 4 * DQ + 16 * jb + e);
                    const float hs[4] = {h4.x, h4.y, h4.z, h4.w}, ls[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const int j = 16 * jb + e + d;
                        const float f = decay_of(ghi, glo, hs[d], ls[d]) * x[e + d];
                        x[e + d] = (w < 2 ? j < i : j <= i) ? f : 0.f;
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = 0.f;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = 0.f;
        }
        if (w < 2) {
            if (jb < nb)
#pragma unroll
                for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4 *>(M + i * MLD + 16 * jb + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                *reinterpret_cast<uint4 *>(sm + P_ATT + i * 128 + (((2 * jb + q) ^ (i & 7)) << 4)) =
                    make_uint4(pack_bf16(x[8 * q], x[8 * q + 1]), pack_bf16(x[8 * q + 2], x[8 * q + 3]), pack_bf16(x[8 * q + 4], x[8 * q + 5]),
                               pack_bf16(x[8 * q + 6], x[8 * q + 7]));
        }
    }
    tc_fence_before();
    fence_proxy_async_smem();
    __syncthreads();
    if (w == 0) {
        if (!ok) mbar_wait(bar + 1, 0);                      // the product is not on its way when the tensor memory is given up
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 64);
    }
    if (tid == PREP_NT - 1) {                                // (not of the warp that gives the tensor memory back)
        bulk_store(ops + ATT, sm + P_ATT, MAT_BYTES);
        bulk_store(ops + GATES, gate, GATE_BYTES);
        bulk_commit();
    }
    __syncwarp();
    const float *beta = gate + 2 * DQ;
    solve(M, T, beta, tid);
    // Rows of the right operands, N index n, K index k: (I + a B)^-1, eight threads a row, so that a warp's pieces are whole lines; and
    // of the transposed (I + B a)^-1, where lanes are rows, so that what they read lies in different banks.
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        uint32_t hi[4] = {0u, 0u, 0u, 0u}, lo[4] = {0u, 0u, 0u, 0u};
        const int n = q * 16 + (tid >> 3), k0 = (tid & 7) * 8;
        uint8_t *to = ops + n * 128 + (((k0 / 8) ^ (n & 7)) << 4);
        if (k0 / 16 <= n / 16)
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(M + n * MLD + k0 + e), f = *reinterpret_cast<const float4 *>(beta + k0 + e);
                split2((k0 + e == n ? 1.f : 0.f) - x.x * f.x, (k0 + e + 1 == n ? 1.f : 0.f) - x.y * f.y, hi[e / 2], lo[e / 2]);
                split2((k0 + e + 2 == n ? 1.f : 0.f) - x.z * f.z, (k0 + e + 3 == n ? 1.f : 0.f) - x.w * f.w, hi[e / 2 + 1], lo[e / 2 + 1]);
            }
        *reinterpret_cast<uint4 *>(to + SYS_HI) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(to + SYS_LO) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    if (BOTH) {
        const int n = tid >> 1;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
            uint32_t hi[4] = {0u, 0u, 0u, 0u}, lo[4] = {0u, 0u, 0u, 0u};
            const int k0 = 16 * q + 8 * (tid & 1);           // (a sector of 32 bytes for two threads)
            uint8_t *to = ops + n * 128 + (((k0 / 8) ^ (n & 7)) << 4);
            if (q >= n / 16)
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    split2((k0 + e == n ? 1.f : 0.f) - beta[k0 + e] * M[(k0 + e) * MLD + n], (k0 + e + 1 == n ? 1.f : 0.f) - beta[k0 + e + 1] * M[(k0 + e + 1) * MLD + n],
                           hi[e / 2], lo[e / 2]);
            *reinterpret_cast<uint4 *>(to + SYS_T) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(to + SYS_T + MAT_BYTES) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
    if (tid == PREP_NT - 1) bulk_wait0();
    if (tid == 0 && !ok && (m.has_k || m.has_q)) mbar_wait(bar, 0);   // (no copy is on its way when the block ends)
}

// ---------------------------------------------------------------------------------------- the chain
// warps: of the lanes, four more of the lanes for what is off the chain (o, backwards scale e^G dO), of the loads, one that stores, one for the products
constexpr int CH_CW = 8, CH_EW = 4, CH_LW = 2, CH_NT = (CH_CW + CH_EW + CH_LW + 2) * 32;
constexpr int CH_L = CH_LW * 32, CH_L0 = (CH_CW + CH_EW) * 32;
// a stage: K and Q (two images of 128 rows: K's, Q's), V (backwards dO), operands
constexpr uint32_t ST_KQ = 0, ST_X = 2 * TOK_BYTES, ST_OPS = 3 * TOK_BYTES, ST_BYTES = (ST_OPS + OPS_BYTES + 1023) / 1024 * 1024;
// and what leaves by bulk copies (and, before that, the state that comes in): two tiles [64][128], plain, of o (backwards dV) and U (mu), the state's image; and a copy of e^G for each warp that computes o
constexpr uint32_t CH_O = 2 * ST_BYTES, CH_V = CH_O + VAL_BYTES, CH_S = CH_V + VAL_BYTES, CH_EG = CH_S + STATE_BYTES, CH_MISC = CH_EG + CH_EW * DQ * 4, CH_BYTES = CH_MISC + 256 + 1024;
// TMEM columns.  A lane's columns of each belong to two threads, two of its quarters each, taken one after the other; a quarter of
// an operand lies over the quarter that its thread has read, both terms one after the other.
//   S   state (its operand; then what is added to it)
//   P   K S, then Y, then forwards att W          R   Q S; backwards att^T dO
//   U   sys Y, its two shares in U and W; then what goes to the state in U, and W = beta U in W
//   X   backwards scale e^G dO
// Forwards P and R are there twice, for even and odd chunks: o is read from them while the next chunk runs.
template <bool BACK>
struct Cols {
    static constexpr uint32_t S = 0, U = BACK ? 256 : 384, W = U + 64, X = 384;
    static __device__ __forceinline__ uint32_t P(int c) { return BACK ? 128 : 128 + 128 * (c & 1); }
    static __device__ __forceinline__ uint32_t R(int c) { return P(c) + 64; }
};
// Barriers.  A wait tells the completions of a barrier apart by their parity: nothing completes twice before every waiter has seen the
// first, because a waiter's own next step is needed for the second; where that is two steps off there is one barrier
// for even chunks (or joins) and one for odd.
enum { B_FULL0, B_FULL1, B_TMA0, B_TMA1, B_O0, B_O1, B_WO0, B_WO1, B_EG0, B_EG1, B_P, B_U, B_S, B_END, B_AF, B_WV, B_WS, B_FO, B_FV, B_FS, B_JM0, B_JM1, B_JD0, B_JD1,
       B_AY, B_AW = B_AY + 2, B_AS = B_AW + 2, NB = B_AS + 2 };   // (one for each thread's first quarter, one for its second)

// a column of 16 tokens of one value, two to a register, into a plain tile
__device__ __forceinline__ void tile_column(unsigned short *to, const uint32_t (&y)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        to[2 * e * 128] = (unsigned short)y[e];
        to[(2 * e + 1) * 128] = (unsigned short)(y[e] >> 16);
    }
}
// and to rows `step` elements apart, `left` of them
__device__ __forceinline__ void st_column(__nv_bfloat16 *p, int64_t step, const uint32_t (&y)[8], int left) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        if (e < left) *reinterpret_cast<unsigned short *>(p) = (unsigned short)(y[e >> 1] >> (16 * (e & 1)));
        p += step;
    }
}

struct ChainBars {
    uint64_t bar[NB];
    uint32_t tmem;
    int abort_;
};
static_assert(sizeof(ChainBars) <= 256, "the barriers' place in shared memory");

__device__ __forceinline__ void tmem_st8(uint32_t at, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                 "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// two values as the sums of two bf16 each (split2 on a pair)
__device__ __forceinline__ void split_pair(f32x2 v, uint32_t &hi, uint32_t &lo) {
    float x, y;
    up2(v, x, y);
    hi = pack_bf16(x, y);
    up2(fma2(pk2(bf_lo(hi), bf_hi(hi)), pk2(-1.f, -1.f), v), x, y);
    lo = pack_bf16(x, y);
}
// a thread's 16 values as both terms of an operand at its quarter
__device__ __forceinline__ void put_terms(uint32_t at, const f32x2 (&y)[8]) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) split_pair(y[e], hi[e], lo[e]);
    tmem_st8(at, hi);
    tmem_st8(at + 8, lo);
}
__device__ __forceinline__ void tmem_ld16x2(uint32_t at, f32x2 (&v)[8]) {
    float x[16];
    tmem_ld16(at, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = pk2(x[2 * e], x[2 * e + 1]);
}
// gates of tokens 4e .. 4e + 3 as two pairs (shared memory, the same for all lanes)
__device__ __forceinline__ void ld_gates(f32x2 &g0, f32x2 &g1, const float *p) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p);
    g0 = v.x;
    g1 = v.y;
}
// A state in shared memory, fp32: piece p (four keys) of row v lies at p ^ (v & 31), so that a thread's row and a warp's pieces of one row are
// in different banks.  Rows w, w + 8, .. by a warp, from and to memory, where a row's pieces are neighbours.
__device__ __forceinline__ float4 *state_piece(uint8_t *buf, int v, int p) { return reinterpret_cast<float4 *>(buf) + v * 32 + (p ^ (v & 31)); }
__device__ __forceinline__ void state_rows(uint8_t *buf, const void *in, bool f32, int64_t at, int V, int K, int w, int lane) {
    const bool wide = (K & 3) == 0 && (reinterpret_cast<uintptr_t>(in) & 15) == 0;   // (a head's rows start at a multiple of four elements)
    const int k = 4 * lane;
#pragma unroll 4
    for (int r = w; r < 128; r += CH_CW) {
        float x[4] = {};
        if (r < V && k < K) {
            const int64_t e = at + (int64_t)r * K + k;
            if (wide && f32) {
                const float4 u = *reinterpret_cast<const float4 *>(static_cast<const float *>(in) + e);
                x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
            } else if (wide) {
                const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(in) + e);
                x[0] = bf_lo(u.x); x[1] = bf_hi(u.x); x[2] = bf_lo(u.y); x[3] = bf_hi(u.y);
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (k + d < K) x[d] = delta_ld(in, f32, e + d);
            }
        }
        *state_piece(buf, r, lane) = make_float4(x[0], x[1], x[2], x[3]);
    }
}
__device__ __forceinline__ void rows_state(uint8_t *buf, void *out, bool f32, int64_t at, int V, int K, int w, int lane) {
    const bool wide = (K & 3) == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    const int k = 4 * lane;
#pragma unroll 4
    for (int r = w; r < V; r += CH_CW) {
        const float4 x = *state_piece(buf, r, lane);
        const int64_t e = at + (int64_t)r * K + k;
        if (k >= K) continue;
        if (wide && f32) {
            *reinterpret_cast<float4 *>(static_cast<float *>(out) + e) = x;
        } else if (wide) {
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(out) + e) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
        } else {
            const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int d = 0; d < 4; ++d)
                if (k + d < K) delta_st(out, f32, e + d, y[d]);
        }
    }
}
// a barrier of the lanes' warps, where each of them comes by whatever has run out before
__device__ __forceinline__ void lanes_meet() { asm volatile("bar.sync 1, %0;" ::"n"(CH_CW * 32) : "memory"); }
// KEEP: U, or mu, and the states are left for the gradients; OUT: o (backwards dV) is computed; ENDS: the first launch of chains that
// are cut into segments: the first segment as it is, of the others but the last the end from a zero state and the matrix, and nothing else
template <bool BACK, bool KEEP, bool OUT, bool ENDS>
__global__ void __launch_bounds__(CH_NT, 1) k_chain(const DeltaArgs a, const __grid_constant__ DeltaMaps m) {
    after_previous();
    extern __shared__ uint8_t raw[];
    uint8_t *sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    ChainBars *ms = reinterpret_cast<ChainBars *>(sm + CH_MISC);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    // unit: sequence and head; segment; of a segment's two, its end or (mat) what it makes of the state before it, S -> S M.  The longest first.
    const int units = a.nseqs * a.H, unit = blockIdx.x % units, part = blockIdx.x / units, s = unit / a.H, h = unit % a.H, grp = h / (a.H / a.G);
    const bool mat = ENDS && part > a.nseg - 2;
    const int seg = mat ? part - (a.nseg - 2) : ENDS ? part : a.nseg - 1 - part;
    const bool run = !ENDS || seg == 0, keeps = KEEP && run, outs = OUT && run;
    if (BACK && a.fresh && (ENDS || a.nseg == 1) && blockIdx.x == 0 && tid < HDR_WORDS) a.hdr[tid] = 0;
    const DeltaSeq q = delta_seq(a, s);
    const int all = (q.len + DQ - 1) / DQ, c0 = seg == 0 ? 0 : a.seg0 + (seg - 1) * a.seglen;   // chunks of the sequence; the segment's first step
    if (seg > 0 && c0 + (ENDS ? a.seglen : 0) >= all) return;              // no segment follows; nothing in it
    const int n = a.nseg > 1 && seg < a.nseg - 1 ? min(seg == 0 ? a.seg0 : a.seglen, all - c0) : all - c0, joins = ENDS ? 0 : max(0, seg - 1);
    if (tid == 0) {
        for (int b : {B_FULL0, B_FULL1}) mbar_init(&ms->bar[b], CH_LW);
        for (int b : {B_O0, B_O1, B_P, B_U, B_S, B_END, B_FO, B_FV, B_FS, B_JM0, B_JM1, B_JD0, B_JD1}) mbar_init(&ms->bar[b], 1);
        for (int b : {B_WV, B_WS}) mbar_init(&ms->bar[b], CH_CW);
        for (int b = B_AY; b < NB; ++b) mbar_init(&ms->bar[b], CH_CW);
        for (int b : {B_AF, B_EG0, B_EG1}) mbar_init(&ms->bar[b], CH_EW);
        for (int b : {B_WO0, B_WO1}) mbar_init(&ms->bar[b], BACK ? CH_CW : CH_EW);
        ms->abort_ = 0;
        fence_mbar_init();
    }
    auto stage = [&](int c) { return sm + (c & 1) * ST_BYTES; };
    auto idx = [&](int c) { return BACK ? all - 1 - c0 - c : c0 + c; };    // the chunk of step c
    // Q and, backwards, dO are needed for the state's sake too
    const bool outputs = BACK ? !mat : outs, values = !mat;
    const CUtensorMap *mx = BACK ? &m.dO : &m.v;
    const bool has_x = values && (BACK ? m.has_dO : m.has_v);
    auto chunk = [&](int c) {
        const int ci = idx(c);
        return DeltaChunk{q.b, q.t0 + ci * DQ, min(DQ, q.len - ci * DQ)};
    };
    auto issue_copies = [&](int c) {                        // by one thread
        const DeltaChunk k = chunk(c);
        uint8_t *st = stage(c);
        uint64_t *bar = &ms->bar[B_TMA0 + (c & 1)];
        mbar_expect_tx(bar, OPS_BYTES + (m.has_k + has_x + (m.has_q && outputs)) * TOK_BYTES);
        if (m.has_k) tma_rows(st + ST_KQ, 2 * HALF, &m.k, bar, k, grp);
        if (has_x) tma_rows(st + ST_X, HALF, mx, bar, k, h);
        const uint8_t *ops = static_cast<const uint8_t *>(a.tiles) + (((int64_t)q.slot0 + idx(c)) * a.H + h) * (a.both ? OPS_BOTH : OPS_BYTES);
        if (BACK) {                                  // the other inverse in its place
            bulk_load(st + ST_OPS, ops + SYS_T, 2 * MAT_BYTES, bar);
            bulk_load(st + ST_OPS + ATT, ops + ATT, OPS_BYTES - ATT, bar);
        } else {
            bulk_load(st + ST_OPS, ops, OPS_BYTES, bar);
        }
        if (m.has_q && outputs) tma_rows(st + ST_KQ + HALF, 2 * HALF, &m.q, bar, k, grp);
    };
    // the first chunks' copies, before anything else is set up
    if (tid == CH_L0) {
        for (int b : {B_TMA0, B_TMA1}) mbar_init(&ms->bar[b], 1);
        fence_mbar_init();
        if (joins == 0)
            for (int c = 0; c < min(n, 2); ++c) issue_copies(c);
        if (outs && m.has_out) prefetch_tmap(&m.out);
    }
    if (w == 0) tmem_alloc(&ms->tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms->tmem;
    volatile int *ab = &ms->abort_;
    auto wait = [&](int b, int c) { return mbar_wait_abort(&ms->bar[b], c & 1, ab); };   // the (c + 1)-th completion
    auto wait2 = [&](int b, int c) { return mbar_wait_abort(&ms->bar[b + (c & 1)], (c >> 1) & 1, ab); };   // of a pair
    auto full = [&](int c) { return wait2(B_FULL0, c); };
    // a warp's one arrival, after what its lanes have written
    auto arrive = [&](int b) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms->bar[b]);
    };
    using C = Cols<BACK>;

    if (w < CH_CW) {
        // ------------------------------------------------------------ two threads a lane: quarters 2 hf and 2 hf + 1 of the columns
        const int hf = w >> 2, v = (w & 3) * 32 + lane;
        const uint32_t at = tmem + ((uint32_t)(w & 3) << 21);
        const bool mine = v < a.V;
        f32x2 S[32];                                         // row v, keys 64 hf ..
        const int64_t row = ((int64_t)s * a.H + h) * a.V * a.K;
        const float4 *ends = static_cast<const float4 *>(a.segB) + (int64_t)unit * (a.nseg - 1) * 4096 + 16 * hf * 128 + v;   // [piece of four keys][value]
        if (!ENDS && seg > 0) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                const float4 x = ends[e / 2 * 128];
                S[e] = pk2(x.x, x.y);
                S[e + 1] = pk2(x.z, x.w);
            }
        } else if (ENDS && (mat || seg > 0)) {
#pragma unroll
            for (int e = 0; e < 32; ++e) S[e] = pk2(mat && v == 64 * hf + 2 * e ? 1.f : 0.f, mat && v == 64 * hf + 2 * e + 1 ? 1.f : 0.f);
        } else {
            const void *in = BACK ? a.dfinal : a.init;
            if (in) {                                        // (nothing else is there yet)
                state_rows(sm + CH_O, in, BACK ? !a.dfinal_bf16 : !a.init_bf16, row, a.V, a.K, w, lane);
                lanes_meet();
            }
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                const float4 x = in ? *state_piece(sm + CH_O, v, 16 * hf + e / 2) : make_float4(0.f, 0.f, 0.f, 0.f);
                S[e] = pk2(x.x, x.y);
                S[e + 1] = pk2(x.z, x.w);
            }
            if (in) lanes_meet();                            // (the tile of kept states lies over rows that other warps read)
        }
        // quarter 2 hf + g of the state as chunk c's operand, and kept as the state that enters it (backwards: whose gradient leaves it)
        auto publish = [&](int c, int g, bool keep) {
            uint32_t hi[16];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                uint32_t h8[8], lo[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    split_pair(S[16 * g + 8 * d + e], h8[e], lo[e]);
                    hi[8 * d + e] = h8[e];
                }
                tmem_st8(at + C::S + 64 * hf + 32 * g + 16 * d, h8);
                tmem_st8(at + C::S + 64 * hf + 32 * g + 16 * d + 8, lo);
            }
            tmem_wait_st();
            arrive(B_AS + g);
            if (keeps && keep) {
                if (g == 0 && c > 0) wait(B_FS, c - 1);
                uint8_t *to = sm + CH_S + hf * (STATE_BYTES / 2) + v * 128;
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    *reinterpret_cast<uint4 *>(to + (((4 * g + p) ^ (v & 7)) << 4)) = make_uint4(hi[4 * p], hi[4 * p + 1], hi[4 * p + 2], hi[4 * p + 3]);
                if (g == 1) {
                    fence_proxy_async_smem();
                    arrive(B_WS);
                }
            }
        };
        // the state that enters the segment: from segment to segment S <- S M + end
        bool go = true;
        for (int j = 0; j < joins; ++j) {
            publish(0, 0, false);
            publish(0, 1, false);
            ends += 4096;                                    // (the state is in tensor memory now: the next end takes its registers)
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                const float4 x = ends[e / 2 * 128];
                S[e] = pk2(x.x, x.y);
                S[e + 1] = pk2(x.z, x.w);
            }
            if (!(go = wait2(B_JD0, j))) break;
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                f32x2 x[8];
                tmem_ld16x2(at + C::U + 64 * hf + 16 * g, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) S[8 * g + e] = add2(x[e], S[8 * g + e]);
            }
        }
        if (n > 0) {
            publish(0, 0, true);
            publish(0, 1, true);
        }
        const f32x2 sc = pk2(a.scale, a.scale);
        for (int c = 0; c < n && go; ++c) {
            const int ci = idx(c);
            const float *gates = reinterpret_cast<const float *>(stage(c) + ST_OPS + GATES);
            if (!full(c)) break;
            const float whole = gates[DQ - 1];
            f32x2 x[8], y[8], g0, g1;
            // ---- Y = -e^G P (V's part of U is a product of its own); backwards N = scale att^T dO + e^(Gc - G) P
            if (!wait(B_P, c)) break;
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int i0 = 32 * hf + 16 * g;             // 16 tokens
                tmem_ld16x2(at + C::P(c) + i0, x);
                if (BACK && values) tmem_ld16x2(at + C::R(c) + i0, y);
                tmem_wait_ld();
                if (BACK && !values)
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = 0;
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    ld_gates(g0, g1, gates + (BACK ? 1 : 5) * DQ + i0 + 2 * e);
                    y[e] = BACK ? fma2(g0, x[e], mul2(sc, y[e])) : mul2(g0, x[e]);
                    y[e + 1] = BACK ? fma2(g1, x[e + 1], mul2(sc, y[e + 1])) : mul2(g1, x[e + 1]);
                }
                put_terms(at + C::P(c) + i0, y);
                tmem_wait_st();
                arrive(B_AY + g);
            }
            // ---- U (backwards mu)
            if (!wait(B_U, c)) break;
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int i0 = 32 * hf + 16 * g;
                tmem_ld16x2(at + C::U + i0, x);
                tmem_ld16x2(at + C::W + i0, y);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = add2(x[e], y[e]);
                uint32_t hi[8], lo[8], wb[8];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    f32x2 d0, d1;
                    ld_gates(g0, g1, gates + 2 * DQ + i0 + 2 * e);
                    ld_gates(d0, d1, gates + (BACK ? 5 * DQ : DQ) + i0 + 2 * e);
                    g0 = mul2(g0, x[e]);                     // W = beta U, lam = beta mu
                    g1 = mul2(g1, x[e + 1]);
                    float p, o;
                    up2(g0, p, o);
                    wb[e] = pack_bf16(p, o);
                    up2(g1, p, o);
                    wb[e + 1] = pack_bf16(p, o);
                    split_pair(mul2(d0, g0), hi[e], lo[e]);
                    split_pair(mul2(d1, g1), hi[e + 1], lo[e + 1]);
                }
                tmem_st8(at + C::U + i0, hi);
                tmem_st8(at + C::U + i0 + 8, lo);
                if (!BACK) tmem_st8(at + C::W + i0, wb);
                tmem_wait_st();
                arrive(B_AW + g);
                if (keeps) {
                    if (g == 0 && c > 0) go = wait(B_FV, c - 1);
                    if (!go) break;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float p, o;
                        up2(x[e], p, o);
                        hi[e] = pack_bf16(p, o);
                    }
                    tile_column(reinterpret_cast<unsigned short *>(sm + CH_V) + i0 * 128 + v, hi);
                    if (g == 1) {
                        fence_proxy_async_smem();
                        arrive(B_WV);
                    }
                }
                if (BACK && outs) {                           // dV: a whole chunk through a tile, as one copy; another by itself
                    if (g == 0 && c > 0) go = wait(B_FO, c - 1);
                    if (!go) break;
                    if (m.has_out && q.len - ci * DQ >= DQ) {
                        tile_column(reinterpret_cast<unsigned short *>(sm + CH_O) + i0 * 128 + v, wb);
                        if (g == 1) fence_proxy_async_smem();
                    } else if (mine) {
                        st_column(static_cast<__nv_bfloat16 *>(a.dv) + q.b * a.dvs[0] + (q.t0 + ci * DQ + i0) * a.dvs[1] + h * a.dvs[2] + v, a.dvs[1], wb, q.len - ci * DQ - i0);
                    }
                    if (g == 1) arrive(B_WO0 + (c & 1));
                }
            }
            // ---- the state
            if (!go || !wait(B_S, c)) break;
            tc_fence_after();
            const f32x2 wh = pk2(whole, whole);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                tmem_ld16x2(at + C::S + 64 * hf + 32 * g, x);
                tmem_ld16x2(at + C::S + 64 * hf + 32 * g + 16, y);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    S[16 * g + e] = fma2(wh, S[16 * g + e], x[e]);
                    S[16 * g + 8 + e] = fma2(wh, S[16 * g + 8 + e], y[e]);
                }
                if (c + 1 < n) publish(c + 1, g, true);
            }
        }
        void *out = !run || c0 + n < all ? nullptr : BACK ? a.dinit : a.final;
        const bool f32 = BACK ? !a.dinit_bf16 : !a.final_bf16;
        if (ENDS && !mat && c0 + n < all) {
            float4 *to = const_cast<float4 *>(ends) + seg * 4096;
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                float4 x;
                up2(S[e], x.x, x.y);
                up2(S[e + 1], x.z, x.w);
                to[e / 2 * 128] = x;
            }
        } else if (ENDS && mat) {
            uint8_t *to = static_cast<uint8_t *>(a.segM) + ((int64_t)unit * (a.nseg - 1) + seg) * SEG_BYTES + hf * (STATE_BYTES / 2) + v * 128;
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split_pair(S[4 * p + e], hi[e], lo[e]);
                *reinterpret_cast<uint4 *>(to + ((p ^ (v & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(to + STATE_BYTES + ((p ^ (v & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
        if (out) {
            // Chunk n - 2 was the last with anything in that stage, and its products are done.  Its gates, which the warps of o may still have to copy, lie
            // behind the state.
            static_assert(128 * 128 * 4 <= ST_OPS + GATES, "the state is staged in front of a stage's gates");
            uint8_t *buf = stage(n);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                float4 x;
                up2(S[e], x.x, x.y);
                up2(S[e + 1], x.z, x.w);
                *state_piece(buf, v, 16 * hf + e / 2) = x;
            }
            lanes_meet();
            rows_state(buf, out, f32, row, a.V, a.K, w, lane);
        }
        tc_fence_before();
    } else if (w < CH_CW + CH_EW) {
        // ------------------------------------------------------------ one thread a lane, off the chain
        const int v = (w & 3) * 32 + lane;
        const uint32_t at = tmem + ((uint32_t)(w & 3) << 21);
        const f32x2 sc = pk2(a.scale, a.scale);
        if (BACK && values) {
            for (int c = 0; c < n; ++c) {                    // scale e^G dO
                if (!full(c) || (c > 0 && !wait2(B_O0, c - 1))) break;
                const float *gate = reinterpret_cast<const float *>(stage(c) + ST_OPS + GATES);
                const uint8_t *xs = stage(c) + ST_X + (v >> 6) * HALF + (v & 7) * 2;
                tc_fence_after();
#pragma unroll
                for (int qu = 0; qu < 4; ++qu) {
                    f32x2 y[8], g0, g1;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int i = 16 * qu + 2 * e;
                        const uint32_t u0 = *reinterpret_cast<const unsigned short *>(xs + i * 128 + ((((v & 63) >> 3) ^ (i & 7)) << 4));
                        const uint32_t u1 = *reinterpret_cast<const unsigned short *>(xs + (i + 1) * 128 + ((((v & 63) >> 3) ^ ((i + 1) & 7)) << 4));
                        y[e] = mul2(sc, pk2(bf_lo(u0), bf_lo(u1)));
                    }
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        ld_gates(g0, g1, gate + 16 * qu + 2 * e);
                        y[e] = mul2(g0, y[e]);
                        y[e + 1] = mul2(g1, y[e + 1]);
                    }
                    put_terms(at + C::X + 16 * qu, y);
                }
                tmem_wait_st();
                arrive(B_AF);
            }
        } else if (!BACK && outs) {
            float *eg = reinterpret_cast<float *>(sm + CH_EG) + (w & 3) * DQ;
            for (int c = 0; c < n; ++c) {                    // o = scale (e^G Q S + att W)
                if (!full(c)) break;
                __syncwarp();
                const float *gate = reinterpret_cast<const float *>(stage(c) + ST_OPS + GATES);
                eg[lane] = gate[lane];                       // (the stage is filled anew once the products are done with it)
                eg[32 + lane] = gate[32 + lane];
                arrive(B_EG0 + (c & 1));
                const int t0 = idx(c) * DQ;
                const bool tile = m.has_out && q.len - t0 >= DQ;
                if (!wait2(B_O0, c) || (c > 0 && !wait(B_FO, c - 1))) break;
                tc_fence_after();
                __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + q.b * a.os[0] + (q.t0 + (int64_t)t0) * a.os[1] + h * a.os[2] + v;
                unsigned short *to = reinterpret_cast<unsigned short *>(sm + CH_O) + v;
#pragma unroll 1
                for (int qu = 0; qu < 4; ++qu) {
                    f32x2 x[8], r[8], g0, g1;
                    tmem_ld16x2(at + C::P(c) + 16 * qu, x);
                    tmem_ld16x2(at + C::R(c) + 16 * qu, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        ld_gates(g0, g1, eg + 16 * qu + 2 * e);
                        x[e] = mul2(sc, fma2(g0, r[e], x[e]));
                        x[e + 1] = mul2(sc, fma2(g1, r[e + 1], x[e + 1]));
                    }
                    uint32_t b2[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float p, o2;
                        up2(x[e], p, o2);
                        b2[e] = pack_bf16(p, o2);
                    }
                    if (tile) tile_column(to + 16 * qu * 128, b2);
                    else if (v < a.V) st_column(o + 16 * qu * a.os[1], a.os[1], b2, q.len - t0 - 16 * qu);
                }
                if (tile) fence_proxy_async_smem();
                arrive(B_WO0 + (c & 1));                                // (and the columns may be written again)
            }
        }
        tc_fence_before();
    } else if (w < CH_CW + CH_EW + CH_LW) {
        // ------------------------------------------------------------ loads
        const int t = tid - CH_L0;
        auto issue_rows = [&](int c) {
            const DeltaChunk k = chunk(c);
            uint8_t *st = stage(c);
            if (!m.has_k) load_rows<CH_L>(st + ST_KQ, 2 * HALF, tok_rows(a.k, a.ks, k, grp), a.ks[1], k.len, a.K, t);
            if (!has_x && values) {
                if (BACK) load_rows<CH_L>(st + ST_X, HALF, tok_rows(a.dO, a.dos, k, h), a.dos[1], k.len, a.V, t);
                else load_rows<CH_L>(st + ST_X, HALF, tok_rows(a.v, a.vs, k, h), a.vs[1], k.len, a.V, t);
            }
            if (!m.has_q && outputs) load_rows<CH_L>(st + ST_KQ + HALF, 2 * HALF, tok_rows(a.q, a.qs, k, grp), a.qs[1], k.len, a.K, t);
        };
        auto issue = [&](int c) {
            if (t == 0) issue_copies(c);
            issue_rows(c);
        };
        bool go = true;
        int matrices = 0, sent = joins == 0 ? min(n, 2) : 0, seen = 0;   // copies on their way, and those that have come
        for (int j = 0; j < joins && go; ++j) {              // the matrices of the segments between, in either stage's memory in turn
            if (j > 1 && !(go = wait2(B_JD0, j - 2))) break;
            matrices = j + 1;
            if (t == 0) {
                uint64_t *bar = &ms->bar[B_JM0 + (j & 1)];
                mbar_expect_tx(bar, SEG_BYTES);
                bulk_load(stage(j), static_cast<const uint8_t *>(a.segM) + ((int64_t)unit * (a.nseg - 1) + 1 + j) * SEG_BYTES, SEG_BYTES, bar);
            }
        }
        if (joins > 1 && go) go = wait2(B_JD0, joins - 2);
        if (joins > 0 && go) go = wait2(B_JD0, joins - 1);
        for (int c = 0; c < min(n, 2) && go; ++c) {
            if (joins > 0 && t == 0) issue_copies(c);
            sent = c + 1;
            issue_rows(c);
        }
        for (int c = 0; c < n && go; ++c) {
            if (!wait2(B_TMA0, c)) break;
            seen = c + 1;
            if (const int len = chunk(c).len; len < DQ) {    // the next sequence's tokens
                if (m.has_k) zero_rows<CH_L>(stage(c) + ST_KQ, 2 * HALF, len, t);
                if (has_x) zero_rows<CH_L>(stage(c) + ST_X, HALF, len, t);
                if (m.has_q && outputs) zero_rows<CH_L>(stage(c) + ST_KQ + HALF, 2 * HALF, len, t);
            }
            fence_proxy_async_smem();
            arrive(B_FULL0 + (c & 1));
            // chunk c has been announced; chunk c - 1's products are done with its stage (and so is every lane): chunk c + 1
            if (c > 0 && c + 1 < n) {
                if (!wait2(B_O0, c - 1) || (!BACK && outs && !wait2(B_EG0, c - 1))) break;
                issue(c + 1);
                sent = c + 2;
            }
        }
        if (t == 0 && *ab) {                                 // a wait has run out: no copy is on its way when the block ends
            for (int j = max(0, matrices - 2); j < matrices; ++j) mbar_wait(&ms->bar[B_JM0 + (j & 1)], (j >> 1) & 1);
            for (int c = seen; c < sent; ++c) mbar_wait(&ms->bar[B_TMA0 + (c & 1)], (c >> 1) & 1);
        }
    } else if (w == CH_CW + CH_EW + CH_LW) {
        // ------------------------------------------------------------ tiles that leave
        if (lane == 0) {
            uint8_t *vals = static_cast<uint8_t *>(BACK ? a.mu : a.U), *kept = static_cast<uint8_t *>(BACK ? a.dS : a.S);
            for (int c = 0; c < n; ++c) {
                const int ci = idx(c);
                if (keeps) {
                    if (!wait(B_WS, c)) break;
                    bulk_store(kept + (((int64_t)q.slot0 + ci) * a.H + h) * STATE_BYTES, sm + CH_S, STATE_BYTES);
                    bulk_commit();
                    bulk_wait_read0();
                    mbar_arrive(&ms->bar[B_FS]);
                    if (!wait(B_WV, c)) break;
                    bulk_store(vals + (((int64_t)q.slot0 + ci) * a.H + h) * VAL_BYTES, sm + CH_V, VAL_BYTES);
                    bulk_commit();
                    bulk_wait_read0();
                    mbar_arrive(&ms->bar[B_FV]);
                }
                if (outs) {
                    if (!wait2(B_WO0, c)) break;
                    if (m.has_out && q.len - ci * DQ >= DQ) {
                        tma_store_4d(&m.out, sm + CH_O, 0, h, q.t0 + ci * DQ, q.b);
                        bulk_commit();
                        bulk_wait_read0();
                    }
                    mbar_arrive(&ms->bar[B_FO]);
                }
            }
            bulk_wait0();
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ the products
        if (lane == 0) {
            const uint32_t s0 = smem_u32(sm);
            constexpr uint32_t id64 = idesc_bf16(128, 64, 0, 0), id128 = idesc_bf16(128, 128, 0, 0), id128t = idesc_bf16(128, 128, 0, 1);
            bool go = true;
            for (int j = 0; j < joins && go; ++j) {          // S M, both terms of each but the product of the small ones, into U and W (R may be written before it has been read)
                if (!(go = wait2(B_JM0, j) && wait(B_AS, j) && wait(B_AS + 1, j))) break;
                tc_fence_after();
                const uint32_t M = s0 + (j & 1) * ST_BYTES;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t A = tmem + C::S + 16 * k;
                    umma_bf16_ta(tmem + C::U, A, mnmaj(M, k, STATE_BYTES / 2), id128t, k > 0);
                    umma_bf16_ta(tmem + C::U, A + 8, mnmaj(M, k, STATE_BYTES / 2), id128t, 1);
                    umma_bf16_ta(tmem + C::U, A, mnmaj(M + STATE_BYTES, k, STATE_BYTES / 2), id128t, 1);
                }
                umma_commit(&ms->bar[B_JD0 + (j & 1)]);
            }
            for (int c = 0; c < n && go; ++c) {
                const uint32_t st = s0 + (c & 1) * ST_BYTES, K = st + ST_KQ, Q = K + HALF, X = st + ST_X, ops = st + ST_OPS;
                if (!full(c)) break;
                if (BACK && values) {                        // att^T dO: dO by columns, att by columns
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_bf16(tmem + C::R(c), mnmaj(X, k, HALF), mnmaj(ops + ATT, k, HALF), idesc_bf16(128, 64, 1, 1), k > 0);
                }
                go = BACK || !outs || c < 2 || wait2(B_WO0, c - 2);   // o of the chunk before last has been read
                // K S and Q S in one: their rows are the 128 rows of the right operand.  Each thread's first quarter
                // while it still writes the second; so with the other products.
#pragma unroll
                for (int g = 0; g < 2 && go; ++g) {
                    if (!(go = wait(B_AS + g, joins + c))) break;
                    tc_fence_after();
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const int k = 4 * (d >> 1) + 2 * g + (d & 1);
                        const uint32_t A = tmem + C::S + 16 * k;
                        umma_bf16_ta(tmem + C::P(c), A, kmaj(K, k, 2 * HALF), BACK ? id64 : id128, g || d);
                        umma_bf16_ta(tmem + C::P(c), A + 8, kmaj(K, k, 2 * HALF), BACK ? id64 : id128, 1);
                    }
                }
                if (!go) break;
                umma_commit(&ms->bar[B_P]);
                if (!BACK && values) {                       // V's part of U: V by columns, both terms of sys
                    if (c > 0 && !wait2(B_O0, c - 1)) break;   // (att W has read its operand there)
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_bf16(tmem + C::U, mnmaj(X, k, HALF), kmaj(ops + SYS_HI, k, 0), idesc_bf16(128, 128, 1, 0), k > 0);
                }
                auto from_o = [&](int term) {                // (scale e^G dO)^T Q
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_bf16_ta(tmem + C::S, tmem + C::X + 16 * k + 8 * term, mnmaj(Q, k, 2 * HALF), id128t, term || k > 0);
                };
                if (BACK && values) {
                    if (!wait(B_AF, c) || !wait(B_P, c)) break;   // P is done with the columns that are written now
                    tc_fence_after();
                    from_o(0);
                }
                // both terms of sys in one: its images are the 128 rows of the right operand
#pragma unroll
                for (int g = 0; g < 2 && go; ++g) {
                    if (!(go = wait(B_AY + g, c))) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = g; k < 4; k += 2) {
                        umma_bf16_ta(tmem + C::U, tmem + C::P(c) + 16 * k, kmaj(ops + SYS_HI, k, 0), id128, (!BACK && values) || k > 0);
                        umma_bf16_ta(tmem + C::U, tmem + C::P(c) + 16 * k + 8, kmaj(ops + SYS_HI, k, 0), id128, 1);
                    }
                }
                if (!go) break;
                umma_commit(&ms->bar[B_U]);
                if (BACK && values) from_o(1);
#pragma unroll
                for (int g = 0; g < 2 && go; ++g) {
                    if (!(go = wait(B_AW + g, c))) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = g; k < 4; k += 2) {
                        umma_bf16_ta(tmem + C::S, tmem + C::U + 16 * k, mnmaj(K, k, 2 * HALF), id128t, (BACK && values) || k > 0);
                        umma_bf16_ta(tmem + C::S, tmem + C::U + 16 * k + 8, mnmaj(K, k, 2 * HALF), id128t, 1);
                    }
                }
                if (!go) break;
                umma_commit(&ms->bar[B_S]);
                if (!BACK && outs)
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma_bf16_ta(tmem + C::P(c), tmem + C::W + 16 * k, kmaj(ops + ATT, k, 0), id64, k > 0);
                umma_commit(&ms->bar[B_O0 + (c & 1)]);
            }
            // nothing is in flight when the tensor memory is given up, also where a wait has given up
            umma_commit(&ms->bar[B_END]);
            mbar_wait(&ms->bar[B_END], 0);
        }
        __syncwarp();
    }
    __syncthreads();
    if (tid == 0 && *ab) set_status(a.hdr, SSD_ERR_DEVICE_TIMEOUT);
    if (w == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------------------- a chunk's gradients
// Persistent blocks over the chunks and groups, a group's heads one after the other (their dQ and dK are added up in registers, in
// fp32).  Rows 0..63 of the 128 TMEM lanes are K's side of a token, rows 64..127 Q's:
//
//   D0 = [K; Q] K^T        D1 = [mu; dO] U^T        D2 = [mu; dO] S       D3 = mu's rows: U dS
//   D4 = [E; F] K + [E^T K + F^T Q; 0]              dK, dQ = f D2 + D4 (+ f D3)
//
// Every operand is a tile as it lies in memory or was left by the chains; factors of a token (beta, e^G, scale) go into E and F or
// multiply a row of the result, in fp32.  dbeta is D1's diagonal.  dg adds up, for each token, what crosses it inside
// the chunk (E and F times D0: sums before the column along a row, then down the columns), and rows of D2 and D3 times K, Q.
// Four threads a row, a quarter of the columns each.  The next head's tiles (115 KB) are on their way as soon as the products with
// this one's are done.  Bound by the work and the waits between the products, a block alone on its SM.
constexpr int GR_NT = 512;
constexpr uint32_t G_KQ = 0, G_A = G_KQ + 8 * HALF, G_U = G_A + 4 * HALF, G_S = G_U + TOK_BYTES, G_DS = G_S + STATE_BYTES, G_EF = G_DS + STATE_BYTES,
                   G_Z = G_EF + 2 * HALF, G_GATE = G_Z + HALF, G_COLS = G_GATE + GATE_BYTES, G_SUM = G_COLS + DQ * 4,
                   G_MISC = G_SUM + (2 * (16 * 16 + 4 * 128 + 4 * 64 + 16) + 4 * 128) * 4, G_BYTES = G_MISC + 64 + 1024;
constexpr uint32_t T_D0 = 0, T_D1 = 64, T_D2 = 128, T_D3 = 256, T_D4 = 384;

// 8 features from piece q on of row r of a tile's image
__device__ __forceinline__ void ld_row(const uint8_t *tile, int r, int q, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(tile + r * 128 + ((q ^ (r & 7)) << 4));
    v[0] = bf_lo(u.x); v[1] = bf_hi(u.x); v[2] = bf_lo(u.y); v[3] = bf_hi(u.y);
    v[4] = bf_lo(u.z); v[5] = bf_hi(u.z); v[6] = bf_lo(u.w); v[7] = bf_hi(u.w);
}
// sums over a warp's lanes of v[e], for lanes e and e + 16
__device__ __forceinline__ float warp_columns(float (&v)[16], int lane) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

__global__ void __launch_bounds__(GR_NT, 1) k_grads(const DeltaArgs a, const __grid_constant__ DeltaMaps m) {
    after_previous();
    extern __shared__ uint8_t raw[];
    uint8_t *sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    float *gate = reinterpret_cast<float *>(sm + G_GATE), *cols = reinterpret_cast<float *>(sm + G_COLS), *colsum = reinterpret_cast<float *>(sm + G_SUM);
    // sums by quarter, warp: two sets of all but the first
    constexpr int SUMS = 16 * 16 + 4 * 128 + 4 * 64 + 16;
    float *R = colsum + 16 * 16, *X = R + 4 * 128, *SSw = X + 4 * 64, *sofar = colsum + 2 * SUMS;
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + G_MISC);
    uint32_t *tm = reinterpret_cast<uint32_t *>(sm + G_MISC + 48);
    enum { L_KQ, L_HEAD, L_D1, L_D2, L_D4 };
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int per = a.H / a.G, units = a.nslots * a.G;
    // the block's next chunk and group from u on that holds tokens
    DeltaChunk c{}, c2{};
    auto find = [&](int u, DeltaChunk &to) {
        for (; u < units; u += gridDim.x)
            if (to = delta_chunk(a, u / a.G); to.len > 0) break;
        return u;
    };
    int unit = find(blockIdx.x, c);
    if (unit >= units) return;
    if (w == 0) tmem_alloc(tm, 512);
    if (tid == 0) {
        for (int i = 0; i < 5; ++i) mbar_init(bar + i, i == L_KQ ? 2 : i == L_HEAD ? 5 : 1);
        tm[1] = 0;
        fence_mbar_init();
    }
    for (int e = tid; e < (int)HALF / 16; e += GR_NT) reinterpret_cast<uint4 *>(sm + G_Z)[e] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    // A copy takes the thread that issues it some 180 cycles: they are spread over warps of Q's side, which has less to do.
    const bool one = lane == 0;
    auto issue_kq = [&](const DeltaChunk &k, int grp, uint8_t *kq) {
        if (one && (w == 11 || w == 14)) {
            const bool has = w == 11 ? m.has_k : m.has_q;
            mbar_expect_tx(bar + L_KQ, has ? TOK_BYTES : 0);
            if (has) tma_rows(w == 11 ? kq : kq + HALF, 2 * HALF, w == 11 ? &m.k : &m.q, bar + L_KQ, k, grp);
        }
        if (!m.has_k) load_rows<GR_NT>(kq, 2 * HALF, tok_rows(a.k, a.ks, k, grp), a.ks[1], k.len, a.K, tid);
        if (!m.has_q) load_rows<GR_NT>(kq + HALF, 2 * HALF, tok_rows(a.q, a.qs, k, grp), a.qs[1], k.len, a.K, tid);
    };
    auto issue = [&](const DeltaChunk &k, int slot, int h) {   // a head's operands
        const int64_t ch = (int64_t)slot * a.H + h;
        const DeltaChunk vals{0, 0, DQ};
        uint64_t *b = bar + L_HEAD;
        if (one && w == 2) {
            mbar_expect_tx(b, VAL_BYTES);
            tma_rows(sm + G_A, 2 * HALF, &m.mu, b, vals, (int)ch);
        } else if (one && w == 3) {
            mbar_expect_tx(b, m.has_dO ? TOK_BYTES : 0);
            if (m.has_dO) tma_rows(sm + G_A + HALF, 2 * HALF, &m.dO, b, k, h);
        } else if (one && w == 6) {
            mbar_expect_tx(b, VAL_BYTES);
            tma_rows(sm + G_U, HALF, &m.U, b, vals, (int)ch);
        } else if (one && w == 7) {
            mbar_expect_tx(b, GATE_BYTES + STATE_BYTES);
            bulk_load(sm + G_GATE, static_cast<const uint8_t *>(a.tiles) + ch * OPS_BOTH + GATES, GATE_BYTES, b);
            bulk_load(sm + G_S, static_cast<const uint8_t *>(a.S) + ch * STATE_BYTES, STATE_BYTES, b);
        } else if (one && w == 10) {
            mbar_expect_tx(b, STATE_BYTES);
            bulk_load(sm + G_DS, static_cast<const uint8_t *>(a.dS) + ch * STATE_BYTES, STATE_BYTES, b);
        }
        if (!m.has_dO) load_rows<GR_NT>(sm + G_A + HALF, 2 * HALF, tok_rows(a.dO, a.dos, k, h), a.dos[1], k.len, a.V, tid);
    };
    issue_kq(c, unit % a.G, sm + G_KQ);
    issue(c, unit / a.G, unit % a.G * per);
    // After a wait has run out the block leaves both loops at the next head's start.  (The word beside the tensor memory's address is written
    // before one barrier and read behind it, by all threads alike: 80 us where none left took 78, and a barrier that gathers it with waits that look at it 90.)
    bool ok = true, left = false;
    const uint32_t base = smem_u32(sm), A = base + G_A, U = base + G_U, S = base + G_S, dS = base + G_DS, EF = base + G_EF, Z = base + G_Z;
    const int row = (w & 3) * 32 + lane, i = row & 63, qu = w >> 2, j0 = 16 * qu;
    const bool qside = row >= 64;
    const uint32_t lanes = (uint32_t)(w & 3) << 21;
    uint32_t tmem = 0;
    // dg of the head before, whose sums are complete (two sets of them in turn): by the first two warps, while the next head's first
    // products run
    DeltaChunk was{};
    int was_h = 0;
    float was_whole = 0.f;
    auto write_dg = [&](int set) {
        const float *cs = colsum + set * SUMS, *Rs = R + set * SUMS, *Xs = X + set * SUMS, *ss = SSw + set * SUMS;
        float f = lane < 14 ? ss[2 + lane] : 0.f;
        f = warp_sum(f) * was_whole;
        float rs = 0.f, xs = 0.f, other = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f += cs[((tid >> 4) * 4 + k) * 16 + (tid & 15)];
            rs += Rs[k * 128 + tid] + Rs[k * 128 + 64 + tid];
            xs += Xs[k * 64 + tid];
            other += tid < 32 ? Rs[k * 128 + 32 + lane] + Rs[k * 128 + 96 + lane] : Xs[k * 64 + lane];
        }
        float pr = rs, px = xs;                              // inclusive sums: of reads from the end, of writes from the start
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float u = __shfl_down_sync(0xffffffffu, pr, o), v = __shfl_up_sync(0xffffffffu, px, o);
            if (lane + o < 32) pr += u;
            if (lane >= o) px += v;
        }
        // and the other 32 tokens': their reads come after the first ones, their writes before the last
        f += pr + (px - xs) + warp_sum(other);
        if (tid < was.len) delta_st(a.dg, a.g_f32, was.b * a.dgs[0] + (int64_t)(was.t0 + tid) * a.dgs[1] + was_h * a.dgs[2], f);
    };
    int it = 0, nu = 0;
    for (; unit < units; ++nu) {
        const int grp = unit % a.G;
        const int next = find(unit + gridDim.x, c2);
        uint8_t *kqt = sm + G_KQ + (nu & 1) * 4 * HALF;
        const uint32_t KQ = smem_u32(kqt);
        ok = mbar_wait(bar + L_KQ, nu & 1) && ok;
        if (c.len < DQ) {
            if (m.has_k) zero_rows<GR_NT>(kqt, 2 * HALF, c.len, tid);
            if (m.has_q) zero_rows<GR_NT>(kqt + HALF, 2 * HALF, c.len, tid);
        }
        float acc[32];                                       // dK's, dQ's row: keys 32 qu ..
#pragma unroll
        for (int e = 0; e < 32; ++e) acc[e] = 0.f;
        for (int r = 0; r < per; ++r, ++it) {
            const int h = grp * per + r;
            ok = mbar_wait(bar + L_HEAD, it & 1) && ok;
            if (c.len < DQ && m.has_dO) zero_rows<GR_NT>(sm + G_A + HALF, 2 * HALF, c.len, tid);
            if (tid < DQ) {                                  // beta_j e^(G_end - G_j), end the last token of j's block of 16
                const int e = tid | 15;
                cols[tid] = gate[2 * DQ + tid] * ex2f(kLog2e * ((gate[3 * DQ + e] - gate[3 * DQ + tid]) + (gate[4 * DQ + e] - gate[4 * DQ + tid])));
            }
            fence_proxy_async_smem();
            tc_fence_before();
            if (!ok) tm[1] = 1;
            __syncthreads();
            tc_fence_after();
            const uint2 words = *reinterpret_cast<const uint2 *>(tm);
            tmem = words.x;
            if ((left = words.y != 0)) break;
            if (tid == 15 * 32) {
                if (r == 0)
#pragma unroll
                    for (int k = 0; k < 8; ++k) umma_bf16(tmem + T_D0, kmaj(KQ, k, 2 * HALF), kmaj(KQ, k, 2 * HALF), idesc_bf16(128, 64, 0, 0), k > 0);
#pragma unroll
                for (int k = 0; k < 8; ++k) umma_bf16(tmem + T_D1, kmaj(A, k, 2 * HALF), kmaj(U, k, HALF), idesc_bf16(128, 64, 0, 0), k > 0);
                umma_commit(bar + L_D1);
#pragma unroll
                for (int k = 0; k < 8; ++k) umma_bf16(tmem + T_D2, kmaj(A, k, 2 * HALF), mnmaj(S, k, STATE_BYTES / 2), idesc_bf16(128, 128, 0, 1), k > 0);
                // (rows 64..127 of this left operand are the state's first rows: nothing reads what comes of them)
#pragma unroll
                for (int k = 0; k < 8; ++k) umma_bf16(tmem + T_D3, kmaj(U, k, HALF), mnmaj(dS, k, STATE_BYTES / 2), idesc_bf16(128, 128, 0, 1), k > 0);
                umma_commit(bar + L_D2);
            }
            // <S, dS> meanwhile, by the warps that have no dg to write
            const int set = (it & 1) * SUMS;
            if (w >= 2) {
                float ss = 0.f;
#pragma unroll 2
                for (int e = tid - 64; e < (int)STATE_BYTES / 16; e += GR_NT - 64) {
                    const uint4 x = reinterpret_cast<const uint4 *>(sm + G_S)[e], y = reinterpret_cast<const uint4 *>(sm + G_DS)[e];
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        ss = fmaf(bf_lo(xs[d]), bf_lo(ys[d]), ss);
                        ss = fmaf(bf_hi(xs[d]), bf_hi(ys[d]), ss);
                    }
                }
                ss = warp_sum(ss);
                if (lane == 0) SSw[set + w] = ss;
            } else if (it > 0) {
                write_dg(~it & 1);
            }
            // ---- E, F: this thread's row, tokens j0 .. j0 + 15
            const float ghi = gate[3 * DQ + i], glo = gate[4 * DQ + i], bi = gate[2 * DQ + i], eg = gate[i];
            const float fd = gate[DQ + i] * bi, whole = gate[DQ - 1], f1 = qside ? a.scale : -bi, f2 = qside ? a.scale * eg : -eg * bi;
            float flow[16], x[16], before = 0.f;             // before: sum of the row's w_ij so far
            ok = mbar_wait(bar + L_D1, it & 1) && ok;
            tc_fence_after();
            tmem_ld16(tmem + lanes + T_D1 + j0, x);
            tmem_ld16(tmem + lanes + T_D0 + j0, flow);
            tmem_wait_ld();
            {
                // the warp's rows lie in two blocks of 16: columns left of both have e^(G_i - G_j) as a product (as in k_prep), those
                // of either one by one, those right of both are zero
                const int b0 = 2 * (w & 1);
                float diag = 0.f;
                if (qu < b0) {
                    const float left = f1 * ex2f(kLog2e * ((ghi - gate[3 * DQ + j0 + 15]) + (glo - gate[4 * DQ + j0 + 15])));
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 col = *reinterpret_cast<const float4 *>(cols + j0 + e);
                        x[e] *= left * col.x; x[e + 1] *= left * col.y; x[e + 2] *= left * col.z; x[e + 3] *= left * col.w;
                    }
                } else if (qu <= b0 + 1) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 h4 = *reinterpret_cast<const float4 *>(gate + 3 * DQ + j0 + e), l4 = *reinterpret_cast<const float4 *>(gate + 4 * DQ + j0 + e);
                        const float4 b4 = *reinterpret_cast<const float4 *>(gate + 2 * DQ + j0 + e);
                        const float hs[4] = {h4.x, h4.y, h4.z, h4.w}, ls[4] = {l4.x, l4.y, l4.z, l4.w}, bs[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int j = j0 + e + k;
                            const float d = x[e + k];
                            diag = j == i ? d : diag;
                            const float v = f1 * bs[k] * ex2f(kLog2e * ((ghi - hs[k]) + (glo - ls[k]))) * d;
                            x[e + k] = j > i || (!qside && j == i) ? 0.f : v;
                        }
                    }
                    if (!qside && (i >> 4) == qu && i < c.len)
                        delta_st(a.dbeta, a.beta_f32, c.b * a.dbs[0] + (int64_t)(c.t0 + i) * a.dbs[1] + h * a.dbs[2], diag);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int j = j0 + e;
                    const float wij = j < i ? x[e] * flow[e] : 0.f;
                    flow[e] = j <= i ? before : 0.f;         // what comes from before j, if it reaches i
                    before += wij;
                }
                uint8_t *to = sm + G_EF + row * 128;
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    *reinterpret_cast<uint4 *>(to + (((2 * qu + q) ^ (row & 7)) << 4)) = make_uint4(pack_bf16(x[8 * q], x[8 * q + 1]), pack_bf16(x[8 * q + 2], x[8 * q + 3]),
                                                                                                  pack_bf16(x[8 * q + 4], x[8 * q + 5]), pack_bf16(x[8 * q + 6], x[8 * q + 7]));
            }
            sofar[qu * 128 + row] = before;
            fence_proxy_async_smem();
            tc_fence_before();
            ok = mbar_wait(bar + L_D2, it & 1) && ok;
            if (one && (w == 11 || w == 14)) bulk_wait_read0();   // the chunk before this one has left its tile, which may be filled anew now by all threads
            __syncthreads();
            tc_fence_after();
            if (tid == 15 * 32) {
#pragma unroll
                for (int k = 0; k < 4; ++k) umma_bf16(tmem + T_D4, kmaj(EF, k, 0), mnmaj(KQ, k, 2 * HALF), idesc_bf16(128, 128, 0, 1), k > 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) umma_bf16(tmem + T_D4, mnmaj(EF, k, Z - EF), mnmaj(KQ, k, 2 * HALF), idesc_bf16(128, 128, 1, 1), 1);
#pragma unroll
                for (int k = 0; k < 4; ++k) umma_bf16(tmem + T_D4, mnmaj(EF + HALF, k, Z - EF - HALF), mnmaj(KQ + HALF, k, 2 * HALF), idesc_bf16(128, 128, 1, 1), 1);
                umma_commit(bar + L_D4);
            }
            // this head's tiles and gates have been read: the next head's may come, or the next chunk's
            if (r + 1 < per) {
                issue(c, unit / a.G, h + 1);
            } else if (next < units) {
                issue_kq(c2, next % a.G, sm + G_KQ + (~nu & 1) * 4 * HALF);
                issue(c2, next / a.G, next % a.G * per);
            }
            {
                float mine = 0.f;
                for (int k = 0; k < qu; ++k) mine += sofar[k * 128 + row];
#pragma unroll
                for (int e = 0; e < 16; ++e) flow[e] += j0 + e <= i ? mine : 0.f;
                const float sum = warp_columns(flow, lane);
                if (lane < 16) colsum[set + w * 16 + lane] = sum;
            }
            // ---- rows of D2, D3 times K or Q, and their sum; keys 32 qu ..
            const uint8_t *kq = kqt + (qu >> 1) * 2 * HALF;
            float dot = 0.f, dotx = 0.f;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                float y[16];
                tmem_ld16(tmem + lanes + T_D2 + 32 * qu + 16 * g, x);
                if (!qside) tmem_ld16(tmem + lanes + T_D3 + 32 * qu + 16 * g, y);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float z[8];
                    ld_row(kq, row, 4 * (qu & 1) + 2 * g + q, z);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        dot = fmaf(x[8 * q + e], z[e], dot);
                        acc[16 * g + 8 * q + e] = fmaf(f2, x[8 * q + e], acc[16 * g + 8 * q + e]);
                        if (!qside) {
                            dotx = fmaf(y[8 * q + e], z[e], dotx);
                            acc[16 * g + 8 * q + e] = fmaf(fd, y[8 * q + e], acc[16 * g + 8 * q + e]);
                        }
                    }
                }
            }
            R[set + qu * 128 + row] = f2 * dot;                    // a token's reads, by K's and by Q's rows
            if (!qside) X[set + qu * 64 + i] = fd * dotx;          // and its writes
            ok = mbar_wait(bar + L_D4, it & 1) && ok;
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                tmem_ld16(tmem + lanes + T_D4 + 32 * qu + 16 * g, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[16 * g + e] += x[e];
            }
            tc_fence_before();
            __syncthreads();
            was = c;
            was_h = h;
            was_whole = whole;
        }
        if (left) break;
        // dK's and dQ's rows: a whole chunk through K's and Q's tile, which nothing reads any more, as one copy
        uint32_t out[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) out[e] = pack_bf16(acc[2 * e], acc[2 * e + 1]);
        if (m.has_dqk && c.len == DQ) {
            uint8_t *to = kqt + (qu >> 1) * 2 * HALF + row * 128;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint4 *>(to + (((4 * (qu & 1) + q) ^ (row & 7)) << 4)) = make_uint4(out[4 * q], out[4 * q + 1], out[4 * q + 2], out[4 * q + 3]);
            fence_proxy_async_smem();
            __syncthreads();
            if (one && (w == 11 || w == 14)) {
                for (int x = 0; x < 2; ++x) tma_store_4d(w == 11 ? &m.dk : &m.dq, kqt + x * 2 * HALF + (w == 11 ? 0 : HALF), 64 * x, grp, c.t0, c.b);
                bulk_commit();
            }
        } else if (i < c.len) {
            unsigned short *to = qside ? static_cast<unsigned short *>(a.dq) + c.b * a.dqs[0] + (int64_t)(c.t0 + i) * a.dqs[1] + grp * a.dqs[2]
                                       : static_cast<unsigned short *>(a.dk) + c.b * a.dks[0] + (int64_t)(c.t0 + i) * a.dks[1] + grp * a.dks[2];
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (32 * qu + e < a.K) to[32 * qu + e] = (unsigned short)(out[e >> 1] >> (16 * (e & 1)));
        }
        unit = next;
        c = c2;
    }
    if (w < 2) write_dg(~it & 1);
    bulk_wait0();
    if (__syncthreads_or(!ok) && w == 0) {                   // no copy and no product is on its way when the block ends
        if (lane == 0) set_status(a.hdr, SSD_ERR_DEVICE_TIMEOUT);
        mbar_wait(bar + L_KQ, (left ? nu : nu - 1) & 1);
        mbar_wait(bar + L_HEAD, (left ? it : it - 1) & 1);
        if (it > 0) mbar_wait(bar + L_D4, (it - 1) & 1);
        __syncwarp();
    }
    if (w == 0) {
        tc_fence_after();
        tmem_dealloc(*tm, 512);
    }
}

template <bool BOTH>
cudaError_t prep(const DeltaArgs &a, const DeltaMaps &m, cudaStream_t st) {
    static int set[64] = {};
    if (cudaError_t e = ensure_smem_attr(k_prep<BOTH>, (int)P_BYTES, set); e != cudaSuccess) return e;
    return launch_early(k_prep<BOTH>, (unsigned)((int64_t)a.nslots * a.H), PREP_NT, P_BYTES, st, a, m);
}
template <bool BACK, bool KEEP, bool OUT, bool ENDS>
cudaError_t launch_chain(const DeltaArgs &a, const DeltaMaps &m, int parts, cudaStream_t st) {
    static int set[64] = {};
    if (cudaError_t e = ensure_smem_attr(k_chain<BACK, KEEP, OUT, ENDS>, (int)CH_BYTES, set); e != cudaSuccess) return e;
    return launch_early(k_chain<BACK, KEEP, OUT, ENDS>, (unsigned)(a.nseqs * (int64_t)a.H * parts), CH_NT, CH_BYTES, st, a, m);
}
template <bool BACK, bool KEEP, bool OUT>
cudaError_t chain(const DeltaArgs &a, const DeltaMaps &m, cudaStream_t st) {
    if (a.nseg > 1)
        if (cudaError_t e = launch_chain<BACK, KEEP, OUT, true>(a, m, 2 * a.nseg - 3, st); e != cudaSuccess) return e;
    return launch_chain<BACK, KEEP, OUT, false>(a, m, std::max(1, a.nseg - 1), st);
}

}  // namespace

bool delta_map(CUtensorMap *m, const void *p, int64_t inner, int64_t heads, int64_t tokens, int64_t batch, const int64_t *strides, bool out) {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f)
                   : nullptr;
    }();
    // the encoder wants the device's context current, which a thread that has made no other call yet (autograd's) has not
    static thread_local int bound = -1;
    if (int dev = 0; cudaGetDevice(&dev) == cudaSuccess && dev != bound && cudaSetDevice(dev) == cudaSuccess) bound = dev;
    const int64_t n[3] = {heads, tokens, batch}, s[3] = {strides[2], strides[1], strides[0]};
    if (encode == nullptr || (uintptr_t)p % 16 != 0 || inner % 8 != 0) return false;
    cuuint64_t dims[4] = {(cuuint64_t)inner, (cuuint64_t)heads, (cuuint64_t)tokens, (cuuint64_t)batch}, by[3];
    for (int i = 0; i < 3; ++i) {
        if (n[i] > 1 && (s[i] % 8 != 0 || s[i] < inner || s[i] >= ((int64_t)1 << 38))) return false;
        by[i] = (cuuint64_t)(n[i] > 1 ? s[i] : inner) * 2;
    }
    const cuuint32_t box[4] = {out ? 128u : 64u, 1, (cuuint32_t)DQ, 1}, step[4] = {1, 1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, by, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  out ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t delta_tc_fwd(const DeltaArgs &a, const DeltaMaps &m, cudaStream_t st) {
    if (cudaError_t e = a.both ? prep<true>(a, m, st) : prep<false>(a, m, st); e != cudaSuccess) return e;
    return a.S == nullptr ? chain<false, false, true>(a, m, st) : a.o != nullptr ? chain<false, true, true>(a, m, st) : chain<false, true, false>(a, m, st);
}
cudaError_t delta_tc_bwd(const DeltaArgs &a, const DeltaMaps &m, cudaStream_t st) {
    if (!m.has_vals) return cudaErrorNotSupported;
    if (cudaError_t e = chain<true, true, true>(a, m, st); e != cudaSuccess) return e;
    static int set[64] = {};
    if (cudaError_t e = ensure_smem_attr(k_grads, (int)G_BYTES, set); e != cudaSuccess) return e;
    return launch_early(k_grads, (unsigned)std::min<int64_t>((int64_t)a.nslots * a.G, 152), GR_NT, G_BYTES, st, a, m);
}

}  // namespace ssd
