// selective_bwd.cu -- the selective scan, backward.  With dyp = dy silu(z) the gradient of the
// pre-gate output, the adjoint of the state runs from the end of each sequence,
//
//   g[t] = C[t] dyp[t] + u[t+1],   u[t] = a[t] g[t],   a[t] = exp(dt[t] A),   u[len] = dfinal
//
// and every gradient is a sum over it (h[-1] the initial state):
//
//   dB[t,n] = sum_d g dt x        dC[t,n] = sum_d h[t] dyp       dinit = u[0]
//   dA[d,n] = sum_t u[t] h[t-1] dt[t]
//   e[t,d] = sum_n g B            f[t,d] = sum_n u[t] h[t-1] A
//   dx = D dyp + e dt             d dt = e x + f, through the softplus        dD = sum_t dyp x
//   dz = dy (C.h + D x) silu'(z)
//
// k_sel_rev walks each sequence backwards and keeps u at the right end of every SEL_Q-token chunk,
// as the forward keeps the state at its left end.  With both ends known the chunks are
// independent: k_sel_grad takes (chunk, set of channels) pairs, and keeps the chunk's dB and dC in
// registers while it goes through its channels, so that the sums over channels cost one
// multiply-add each and no exchange.  The shares of the channel sets and of the chunks are
// added in a fixed order at the end: results are bitwise reproducible.
#include <algorithm>

#include "selective.cuh"

namespace ssd {

namespace {

// the gate's logistic function to about 1e-6: dA, dD and the others keep 32 bits
__device__ __forceinline__ float sigf(float v) { return __fdividef(1.f, 1.f + ex2f(-kLog2e * v)); }

// ---- the adjoint at the chunks' right ends
template <int S_, int TPC_, int CW_, int TW_, int TK_>
struct RevCfg {
    static constexpr int S = S_, TPC = TPC_, CW = CW_, TW = TW_, TK = TK_;
    static constexpr int NP = S * TPC, CPW = 32 / TPC, CB = CW * CPW, TT = TW * TK, NT = 32 * CW * TW;
    static constexpr size_t smem = (size_t)TT * CB * 8 + (size_t)TT * NP * 4 + (size_t)(TW + 1) * CB * NP * 4 +
                                   (size_t)TW * CB * 4;
};

template <typename T, typename F>
__global__ void __launch_bounds__(F::NT, 2) k_sel_rev(const SelArgs a, int cblocks) {
    constexpr int S = F::S, TPC = F::TPC, NP = F::NP, CB = F::CB, TT = F::TT, TK = F::TK, TW = F::TW, NT = F::NT;
    extern __shared__ __align__(16) uint8_t sel_sm[];
    float2 *dd = reinterpret_cast<float2 *>(sel_sm);                // [TT][CB]: (dt, dyp)
    float *Cs = reinterpret_cast<float *>(dd + TT * CB);            // [TT][NP]
    float *E = Cs + TT * NP;                                        // [TW][CB][NP]: what each warp passes on; then the carry
    float *Sd = E + (TW + 1) * CB * NP;                             // [TW][CB]: sums of dt
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int w = wid % TW, cw = wid / TW;
    const int q = lane % TPC, cl = cw * F::CPW + lane / TPC;
    const int cb = blockIdx.x % cblocks, s = blockIdx.x / cblocks;
    const int bpg = cblocks / a.ngroups, g = cb / bpg;
    const int d0 = g * a.dpg + (cb % bpg) * CB, dend = (g + 1) * a.dpg, d = d0 + cl;
    const SelSeq sq = sel_seq(a, s);
    const int N = a.N;
    const T *dy = static_cast<const T *>(a.dy) + sq.b * a.dyb + sq.t0 * a.dyt;
    const T *z = a.z ? static_cast<const T *>(a.z) + sq.b * a.zb + sq.t0 * a.zt : nullptr;
    const T *C = static_cast<const T *>(a.C) + sq.b * a.Cb + sq.t0 * a.Ct + g * a.Cg;
    const int64_t dt0 = sq.b * a.dtb + sq.t0 * a.dtt;
    f32x2 A2[S / 2];
#pragma unroll
    for (int i = 0; i < S / 2; ++i) {
        float v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int n = q * S + 2 * i + e;
            v[e] = d < dend && n < N ? a.A[(int64_t)d * N + n] * kLog2e : 0.f;
        }
        A2[i] = pk2(v[0], v[1]);
    }
    for (int i = tid; i < CB * NP; i += NT) {
        const int c = i / NP, n = i % NP;
        E[TW * CB * NP + i] = (a.dfinal && d0 + c < dend && n < N)
                                  ? ld_st(a.dfinal, a.dfinal_bf16, ((int64_t)s * a.channels + d0 + c) * N + n) : 0.f;
    }
    for (int t0 = sq.len > 0 ? (sq.len - 1) / TT * TT : -1; t0 >= 0; t0 -= TT) {
        __syncthreads();
        for (int i = tid; i < TT * CB; i += NT) {
            const int t = t0 + i / CB, dc = d0 + i % CB;
            float dt = 0.f, v = 0.f;
            if (t < sq.len && dc < dend) {
                dt = sel_softplus(ld_dt(a, dt0 + t * a.dtt + dc) + (a.bias ? a.bias[dc] : 0.f));
                v = to_f(dy[t * a.dyt + dc]);
                if (z) {
                    const float zv = to_f(z[t * a.zt + dc]);
                    v *= zv * sigf(zv);
                }
            }
            dd[i] = make_float2(dt, v);
        }
        for (int i = tid; i < TT * NP; i += NT) {
            const int t = t0 + i / NP, n = i % NP;
            Cs[i] = t < sq.len && n < N ? to_f(C[t * a.Ct + n]) : 0.f;
        }
        __syncthreads();
        f32x2 u[S / 2];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < S / 2; ++i) u[i] = 0;
        if (t0 + w * TK < sq.len) {
            const float2 *dp = dd + w * TK * CB + cl;
            const float *cp = Cs + w * TK * NP + q * S;
#pragma unroll 4
            for (int t = TK - 1; t >= 0; --t) {
                const float2 v = dp[t * CB];
                sum += v.x;
                const f32x2 dt2 = pk2(v.x, v.x), dy2 = pk2(v.y, v.y);
                const ulonglong2 *c = reinterpret_cast<const ulonglong2 *>(cp + t * NP);
#pragma unroll
                for (int i = 0; i < S / 4; ++i) {
                    const ulonglong2 cv = c[i];
                    u[2 * i] = mul2(ex2x2(mul2(dt2, A2[2 * i])), fma2(cv.x, dy2, u[2 * i]));
                    u[2 * i + 1] = mul2(ex2x2(mul2(dt2, A2[2 * i + 1])), fma2(cv.y, dy2, u[2 * i + 1]));
                }
            }
        }
        ulonglong2 *ep = reinterpret_cast<ulonglong2 *>(E + (w * CB + cl) * NP + q * S);
#pragma unroll
        for (int i = 0; i < S / 4; ++i) ep[i] = make_ulonglong2(u[2 * i], u[2 * i + 1]);
        if (q == 0) Sd[w * CB + cl] = sum;
        __syncthreads();
        for (int i = tid; i < CB * NP; i += NT) {
            const int c = i / NP, n = i % NP, dc = d0 + c;
            const float An = dc < dend && n < N ? a.A[(int64_t)dc * N + n] * kLog2e : 0.f;
            float uc = E[TW * CB * NP + i];
#pragma unroll
            for (int k = TW - 1; k >= 0; --k) {
                const int te = t0 + (k + 1) * TK;                   // the k-th warp's tokens end here
                if (te % SEL_Q == 0 && te - SEL_Q < sq.len && dc < dend) {
                    const int slot = sq.slot0 + te / SEL_Q - 1;
                    if (slot < a.nslots) a.adj[((int64_t)slot * a.channels + dc) * NP + n] = uc;
                }
                uc = fmaf(ex2f(An * Sd[k * CB + c]), uc, E[k * CB * NP + i]);
            }
            E[TW * CB * NP + i] = uc;
        }
    }
    if (a.dinit == nullptr) return;
    __syncthreads();
    for (int i = tid; i < CB * NP; i += NT) {
        const int c = i / NP, n = i % NP;
        if (d0 + c < dend && n < N)
            st_st(a.dinit, a.dinit_bf16, ((int64_t)s * a.channels + d0 + c) * N + n, E[TW * CB * NP + i]);
    }
}

// ---- the gradients.  A block takes one chunk of SEL_Q tokens and a set of channels: warp w has the
// w-th GT tokens, and the block goes through its channels 128 / NP at a time, a thread with four
// states of one channel.
constexpr int GT = 4, GW = SEL_Q / GT, GNT = 32 * GW, GC = 32;   // tokens a warp, warps, threads, channels staged at once

template <int NP>
constexpr size_t grad_smem() {
    return (size_t)2 * SEL_Q * NP * 4 + (size_t)SEL_Q * GC * 16 + (size_t)3 * SEL_Q * GC * 4 + (size_t)GC * NP * 4 +
           (size_t)3 * GW * 128 * 4 + (size_t)GW * 32 * 4 + (size_t)GW * GC * 8;
}

template <typename T, int NP>
__global__ void __launch_bounds__(GNT, 2) k_sel_grad(const SelArgs a) {
    constexpr int TPC = NP / 4, CPW = 32 / TPC;
    extern __shared__ __align__(16) uint8_t sel_sm[];
    float4 *sv = reinterpret_cast<float4 *>(sel_sm);                // [SEL_Q][GC]: (dt, dt x, dyp, -)
    float *Bs = reinterpret_cast<float *>(sv + SEL_Q * GC);         // [SEL_Q][NP]
    float *Cs = Bs + SEL_Q * NP;                                    // [SEL_Q][NP]
    float *As = Cs + SEL_Q * NP;                                    // [GC][NP]: A log2(e)
    float *EX = As + GC * NP;                                       // [2][GW][128]: ends, then entering values
    float *DA = EX + 2 * GW * 128;                                  // [GW][128]: shares of dA
    float *ov = DA + GW * 128;                                      // [3][SEL_Q][GC]: sums over the states
    float *Sd = ov + 3 * SEL_Q * GC;                                // [GW][32]: sums of dt
    float2 *red = reinterpret_cast<float2 *>(Sd + GW * 32);         // [GW][GC]
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, q = lane % TPC, cw = lane / TPC;
    const int set = blockIdx.x % a.nsets, g = blockIdx.x / a.nsets % a.ngroups, slot = blockIdx.x / a.nsets / a.ngroups;
    const int N = a.N;
    const int c_lo = g * a.dpg + set * a.cps, c_hi = min(c_lo + a.cps, (g + 1) * a.dpg);

    int s, j;
    if (a.cu == nullptr) {
        const int nc = (a.seqlen + SEL_Q - 1) / SEL_Q;
        s = slot / nc;
        j = slot % nc;
    } else {
        int lo = 0, hi = a.nseqs - 1;                               // the last sequence whose chunks start at or before slot
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (sel_seq(a, mid).slot0 <= slot) lo = mid; else hi = mid - 1;
        }
        s = lo;
        j = slot - sel_seq(a, s).slot0;
    }
    const SelSeq sq = sel_seq(a, s);
    const int tb = j * SEL_Q, n_tok = min(SEL_Q, sq.len - tb);
    if (j < 0 || n_tok <= 0) {                                      // a slot without a chunk: no shares
        for (int64_t i = (int64_t)c_lo * NP + tid; i < (int64_t)c_hi * NP; i += GNT) a.pA[(int64_t)slot * a.channels * NP + i] = 0.f;
        for (int i = c_lo * 2 + tid; i < c_hi * 2; i += GNT) a.pD[(int64_t)slot * a.channels * 2 + i] = 0.f;
        return;
    }
    const int64_t r0 = sq.t0 + tb;                                  // the chunk's first token in its row
    const T *x = static_cast<const T *>(a.x) + sq.b * a.xb + r0 * a.xt;
    const T *dy = static_cast<const T *>(a.dy) + sq.b * a.dyb + r0 * a.dyt;
    const T *z = a.z ? static_cast<const T *>(a.z) + sq.b * a.zb + r0 * a.zt : nullptr;
    const T *B = static_cast<const T *>(a.B) + sq.b * a.Bb + r0 * a.Bt + g * a.Bg;
    const T *C = static_cast<const T *>(a.C) + sq.b * a.Cb + r0 * a.Ct + g * a.Cg;
    T *dx = static_cast<T *>(a.dx) + sq.b * a.dxb + r0 * a.dxt;
    T *dz = a.z ? static_cast<T *>(a.dz) + sq.b * a.dzb + r0 * a.dzt : nullptr;
    const int64_t dt0 = sq.b * a.dtb + r0 * a.dtt, ddt0 = sq.b * a.ddtb + r0 * a.ddtt;
    for (int i = tid; i < SEL_Q * NP; i += GNT) {
        const int t = i / NP, n = i % NP;
        const bool in = t < n_tok && n < N;
        Bs[i] = in ? to_f(B[t * a.Bt + n]) : 0.f;
        Cs[i] = in ? to_f(C[t * a.Ct + n]) : 0.f;
    }
    f32x2 aB[GT][2], aC[GT][2];                                     // this thread's dB and dC
#pragma unroll
    for (int t = 0; t < GT; ++t) aB[t][0] = aB[t][1] = aC[t][0] = aC[t][1] = 0;

    for (int cb = c_lo; cb < c_hi; cb += GC) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < SEL_Q * GC / GNT; ++k) {
            const int i = tid + k * GNT, t = i / GC, c = i % GC, dc = cb + c;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t < n_tok && dc < c_hi) {
                v.x = sel_softplus(ld_dt(a, dt0 + t * a.dtt + dc) + (a.bias ? a.bias[dc] : 0.f));
                v.y = v.x * to_f(x[t * a.xt + dc]);
                v.z = to_f(dy[t * a.dyt + dc]);
                if (z) {
                    const float zv = to_f(z[t * a.zt + dc]);
                    v.z *= zv * sigf(zv);
                }
            }
            sv[i] = v;
        }
        for (int i = tid; i < GC * NP; i += GNT) {
            const int c = i / NP, n = i % NP;
            As[i] = cb + c < c_hi && n < N ? a.A[(int64_t)(cb + c) * N + n] * kLog2e : 0.f;
        }
        __syncthreads();
        for (int it = 0; it < TPC; ++it) {                          // CPW channels at a time
            const int c = it * CPW + cw;
            // what enters the chunk, for the joining below: threads 0..127 the state, 128..255 the adjoint
            const int dir = tid >> 7, p = tid & 127, pc = it * CPW + p / NP, pn = p % NP;
            const bool pin = cb + pc < c_hi;
            const float *src = dir ? a.adj : a.states;
            float carry = pin ? src[((int64_t)slot * a.channels + cb + pc) * NP + pn] : 0.f;

            const ulonglong2 av = *reinterpret_cast<const ulonglong2 *>(As + c * NP + q * 4);
            const float4 *vp = sv + w * GT * GC + c;
            const float *bp = Bs + w * GT * NP + q * 4, *cp = Cs + w * GT * NP + q * 4;
            f32x2 al[GT][2], h[GT + 1][2], u[2];
            h[0][0] = h[0][1] = u[0] = u[1] = 0;
            float sum = 0.f;
#pragma unroll
            for (int t = 0; t < GT; ++t) {
                const float4 v = vp[t * GC];
                const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(bp + t * NP);
                const f32x2 dt2 = pk2(v.x, v.x), dx2 = pk2(v.y, v.y);
                sum += v.x;
                al[t][0] = ex2x2(mul2(dt2, av.x));
                al[t][1] = ex2x2(mul2(dt2, av.y));
                h[0][0] = fma2(al[t][0], h[0][0], mul2(dx2, b.x));
                h[0][1] = fma2(al[t][1], h[0][1], mul2(dx2, b.y));
            }
#pragma unroll
            for (int t = GT - 1; t >= 0; --t) {
                const float v = vp[t * GC].z;
                const ulonglong2 cv = *reinterpret_cast<const ulonglong2 *>(cp + t * NP);
                const f32x2 dy2 = pk2(v, v);
                u[0] = mul2(al[t][0], fma2(cv.x, dy2, u[0]));
                u[1] = mul2(al[t][1], fma2(cv.y, dy2, u[1]));
            }
            *reinterpret_cast<ulonglong2 *>(EX + w * 128 + lane * 4) = make_ulonglong2(h[0][0], h[0][1]);
            *reinterpret_cast<ulonglong2 *>(EX + (GW + w) * 128 + lane * 4) = make_ulonglong2(u[0], u[1]);
            if (q == 0) Sd[w * 32 + cw] = sum;
            __syncthreads();
            {
                const float An = As[pc * NP + pn];
                const float *sd = Sd + p / NP;
                if (dir == 0) {
#pragma unroll
                    for (int k = 0; k < GW; ++k) {
                        const float end = EX[k * 128 + p];
                        EX[k * 128 + p] = carry;
                        carry = fmaf(ex2f(An * sd[k * 32]), carry, end);
                    }
                } else {
#pragma unroll
                    for (int k = GW - 1; k >= 0; --k) {
                        const float end = EX[(GW + k) * 128 + p];
                        EX[(GW + k) * 128 + p] = carry;
                        carry = fmaf(ex2f(An * sd[k * 32]), carry, end);
                    }
                    if (it > 0 && cb + pc - CPW < c_hi) {           // the last channels' dA, over the warps
                        float v = 0.f;
#pragma unroll
                        for (int k = 0; k < GW; ++k) v += DA[k * 128 + p];
                        a.pA[((int64_t)slot * a.channels + cb + pc - CPW) * NP + pn] = v;
                    }
                }
            }
            __syncthreads();
            {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(EX + w * 128 + lane * 4);
                h[0][0] = v.x; h[0][1] = v.y;
                const ulonglong2 e = *reinterpret_cast<const ulonglong2 *>(EX + (GW + w) * 128 + lane * 4);
                u[0] = e.x; u[1] = e.y;
            }
            float ys[GT], es[GT], fs[GT];
#pragma unroll
            for (int t = 0; t < GT; ++t) {
                const float4 v = vp[t * GC];
                const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(bp + t * NP);
                const ulonglong2 cv = *reinterpret_cast<const ulonglong2 *>(cp + t * NP);
                const f32x2 dx2 = pk2(v.y, v.y), dy2 = pk2(v.z, v.z);
                h[t + 1][0] = fma2(al[t][0], h[t][0], mul2(dx2, b.x));
                h[t + 1][1] = fma2(al[t][1], h[t][1], mul2(dx2, b.y));
                ys[t] = sum2(fma2(h[t + 1][1], cv.y, mul2(h[t + 1][0], cv.x)));
                aC[t][0] = fma2(h[t + 1][0], dy2, aC[t][0]);
                aC[t][1] = fma2(h[t + 1][1], dy2, aC[t][1]);
            }
            f32x2 dA[2] = {0, 0};
#pragma unroll
            for (int t = GT - 1; t >= 0; --t) {
                const float4 v = vp[t * GC];
                const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(bp + t * NP);
                const ulonglong2 cv = *reinterpret_cast<const ulonglong2 *>(cp + t * NP);
                const f32x2 dt2 = pk2(v.x, v.x), dx2 = pk2(v.y, v.y), dy2 = pk2(v.z, v.z);
                const f32x2 g0 = fma2(cv.x, dy2, u[0]), g1 = fma2(cv.y, dy2, u[1]);
                aB[t][0] = fma2(g0, dx2, aB[t][0]);
                aB[t][1] = fma2(g1, dx2, aB[t][1]);
                es[t] = sum2(fma2(g1, b.y, mul2(g0, b.x)));
                u[0] = mul2(al[t][0], g0);
                u[1] = mul2(al[t][1], g1);
                const f32x2 k0 = mul2(u[0], h[t][0]), k1 = mul2(u[1], h[t][1]);
                dA[0] = fma2(k0, dt2, dA[0]);
                dA[1] = fma2(k1, dt2, dA[1]);
                fs[t] = sum2(fma2(k1, av.y, mul2(k0, av.x)));
            }
            float yq = reduce_scatter<GT>(ys, q % GT), eq = reduce_scatter<GT>(es, q % GT), fq = reduce_scatter<GT>(fs, q % GT);
#pragma unroll
            for (int o = GT; o < TPC; o <<= 1) {
                yq += __shfl_xor_sync(0xffffffffu, yq, o);
                eq += __shfl_xor_sync(0xffffffffu, eq, o);
                fq += __shfl_xor_sync(0xffffffffu, fq, o);
            }
            if (q < GT) {
                const int at = (w * GT + q) * GC + c;
                ov[at] = yq;
                ov[SEL_Q * GC + at] = eq;
                ov[2 * SEL_Q * GC + at] = fq * 0.6931471805599453f;   // av holds A log2(e)
            }
            *reinterpret_cast<ulonglong2 *>(DA + w * 128 + lane * 4) = make_ulonglong2(dA[0], dA[1]);
        }
        __syncthreads();
        if (tid < 128) {
            const int pc = (TPC - 1) * CPW + tid / NP, pn = tid % NP;
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < GW; ++k) v += DA[k * 128 + tid];
            if (cb + pc < c_hi) a.pA[((int64_t)slot * a.channels + cb + pc) * NP + pn] = v;
        }
        float sD = 0.f, sb = 0.f;
        const int c = tid % GC, dc = cb + c;
        if (dc < c_hi) {
            const float Dv = a.D ? a.D[dc] : 0.f, bias = a.bias ? a.bias[dc] : 0.f;
#pragma unroll
            for (int k = 0; k < SEL_Q * GC / GNT; ++k) {
                const int i = tid + k * GNT, t = i / GC;
                if (t >= n_tok) continue;
                const float4 v = sv[i];
                const float xv = to_f(x[t * a.xt + dc]), e = ov[SEL_Q * GC + i];
                const float raw = ld_dt(a, dt0 + t * a.dtt + dc) + bias;
                const float dr = fmaf(e, xv, ov[2 * SEL_Q * GC + i]) * sigf(raw);
                dx[t * a.dxt + dc] = from_f<T>(fmaf(e, v.x, Dv * v.z));
                if (a.dt_f32) static_cast<float *>(a.ddt)[ddt0 + t * a.ddtt + dc] = dr;
                else static_cast<__nv_bfloat16 *>(a.ddt)[ddt0 + t * a.ddtt + dc] = __float2bfloat16_rn(dr);
                if (z) {
                    const float zv = to_f(z[t * a.zt + dc]), sg = sigf(zv);
                    dz[t * a.dzt + dc] = from_f<T>(to_f(dy[t * a.dyt + dc]) * fmaf(Dv, xv, ov[i]) * sg * (1.f + zv * (1.f - sg)));
                }
                sD = fmaf(v.z, xv, sD);
                sb += dr;
            }
        }
        red[w * GC + c] = make_float2(sD, sb);                      // thread (w, c) had tokens w, w + 8, ...
        __syncthreads();
        if (tid < GC && cb + tid < c_hi) {
            float2 v = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < GW; ++k) {
                v.x += red[k * GC + tid].x;
                v.y += red[k * GC + tid].y;
            }
            reinterpret_cast<float2 *>(a.pD)[(int64_t)slot * a.channels + cb + tid] = v;
        }
    }
    // dB and dC of this channel set: over the warp's channels, then one row of NP values a token
    const int64_t rows = (int64_t)a.nbatch * a.seqlen * a.ngroups;
#pragma unroll
    for (int t = 0; t < GT; ++t) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int o = TPC; o < 32; o <<= 1) {
                aB[t][k] = add2(aB[t][k], __shfl_xor_sync(0xffffffffu, aB[t][k], o));
                aC[t][k] = add2(aC[t][k], __shfl_xor_sync(0xffffffffu, aC[t][k], o));
            }
        }
        const int tt = w * GT + t;
        if (cw == 0 && tt < n_tok) {
            const int64_t row = ((int64_t)sq.b * a.seqlen + r0 + tt) * a.ngroups + g;
            float *pb = a.pBC + ((int64_t)set * 2 * rows + row) * NP + q * 4;
            *reinterpret_cast<ulonglong2 *>(pb) = make_ulonglong2(aB[t][0], aB[t][1]);
            *reinterpret_cast<ulonglong2 *>(pb + rows * NP) = make_ulonglong2(aC[t][0], aC[t][1]);
        }
    }
}

// dB and dC: the channel sets' shares in order
template <typename T>
__global__ void __launch_bounds__(256) k_sel_dbc(const SelArgs a) {
    const int64_t rows = (int64_t)a.nbatch * a.seqlen * a.ngroups, per = rows * a.NP;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= 2 * per) return;
    const int64_t row = i % per / a.NP;
    const int n = (int)(i % a.NP), which = i >= per;
    if (n >= a.N) return;
    float v = 0.f;
    for (int k = 0; k < a.nsets; ++k) v += a.pBC[k * 2 * per + i];
    const int g = (int)(row % a.ngroups);
    const int64_t tok = row / a.ngroups, b = tok / a.seqlen, t = tok % a.seqlen;
    if (which) static_cast<T *>(a.dC)[b * a.dCb + t * a.dCt + g * a.dCg + n] = from_f<T>(v);
    else static_cast<T *>(a.dB)[b * a.dBb + t * a.dBt + g * a.dBg + n] = from_f<T>(v);
}

// dA, dD and ddt_bias: sums of the chunks' shares over the slots.  A block takes 32 columns; warp w
// sums slots w, w + 8, ... in order, and the eight sums are added in order.
__global__ void __launch_bounds__(256) k_sel_cols(const SelArgs a, int64_t blocksA) {
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const bool isA = blockIdx.x < blocksA;
    const int64_t cols = isA ? (int64_t)a.channels * a.NP : (int64_t)a.channels * 2;
    const int64_t col = (blockIdx.x - (isA ? 0 : blocksA)) * 32 + lane;
    const float *src = isA ? a.pA : a.pD;
    float v = 0.f;
    if (col < cols) {
#pragma unroll 4
        for (int k = w; k < a.nslots; k += 8) v += src[k * cols + col];
    }
    red[w][lane] = v;
    __syncthreads();
    if (w != 0 || col >= cols) return;
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += red[k][lane];
    if (isA) {
        const int n = (int)(col % a.NP);
        if (n < a.N) a.dA[col / a.NP * a.N + n] = v;
    } else if (col % 2 == 0) {
        if (a.dD) a.dD[col / 2] = v;
    } else if (a.dbias) {
        a.dbias[col / 2] = v;
    }
}

template <typename T, typename F>
cudaError_t launch_rev(const SelArgs &a, cudaStream_t st) {
    static int attr[64] = {0};
    cudaError_t e = ensure_smem_attr(k_sel_rev<T, F>, (int)F::smem, attr);
    if (e != cudaSuccess) return e;
    const int cblocks = a.ngroups * ((a.dpg + F::CB - 1) / F::CB);
    k_sel_rev<T, F><<<(unsigned)((int64_t)a.nseqs * cblocks), F::NT, F::smem, st>>>(a, cblocks);
    return cudaGetLastError();
}
template <typename T, int NP>
cudaError_t launch_grad(const SelArgs &a, cudaStream_t st) {
    static int attr[64] = {0};
    cudaError_t e = ensure_smem_attr(k_sel_grad<T, NP>, (int)grad_smem<NP>(), attr);
    if (e != cudaSuccess) return e;
    k_sel_grad<T, NP><<<(unsigned)((int64_t)a.nslots * a.ngroups * a.nsets), GNT, grad_smem<NP>(), st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t run_bwd(const SelArgs &a, cudaStream_t st) {
    cudaError_t e;
    switch (a.NP) {
        case 16: e = launch_rev<T, RevCfg<8, 2, 2, 8, 16>>(a, st); break;
        case 32: e = launch_rev<T, RevCfg<8, 4, 4, 4, 16>>(a, st); break;
        case 64: e = launch_rev<T, RevCfg<8, 8, 4, 4, 16>>(a, st); break;
        default: e = launch_rev<T, RevCfg<8, 16, 4, 4, 16>>(a, st);
    }
    if (e != cudaSuccess) return e;
    if (a.nslots > 0) {
        switch (a.NP) {
            case 16: e = launch_grad<T, 16>(a, st); break;
            case 32: e = launch_grad<T, 32>(a, st); break;
            case 64: e = launch_grad<T, 64>(a, st); break;
            default: e = launch_grad<T, 128>(a, st);
        }
        if (e != cudaSuccess) return e;
    }
    const int64_t n = (int64_t)2 * a.nbatch * a.seqlen * a.ngroups * a.NP;
    if (n > 0) k_sel_dbc<T><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(a);
    const int64_t bA = ((int64_t)a.channels * a.NP + 31) / 32, bD = ((int64_t)a.channels * 2 + 31) / 32;
    k_sel_cols<<<(unsigned)(bA + bD), 256, 0, st>>>(a, bA);
    return cudaGetLastError();
}

}  // namespace

// Channels per set: as many as leave a few blocks per SM (each set writes its own shares of dB and dC).
void sel_bwd_sets(int channels, int ngroups, int64_t nslots, int *nsets, int *cps) {
    const int dpg = channels / ngroups;
    int c = 256;
    while (c > GC && nslots * ngroups * ((dpg + c - 1) / c) < 1216) c >>= 1;
    *cps = c;
    *nsets = (dpg + c - 1) / c;
}

cudaError_t sel_launch_bwd(const SelArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? run_bwd<__nv_bfloat16>(a, st) : run_bwd<float>(a, st);
}

}  // namespace ssd
