// selective_fwd.cu -- the selective scan, forward: a state-space scan with a decay rate per channel
// and state,
//
//   dt[t,d] = softplus(dt_raw[t,d] + dt_bias[d])
//   h[t,d,n] = exp(dt[t,d] A[d,n]) h[t-1,d,n] + dt[t,d] x[t,d] B[t,n]
//   y[t,d] = (sum_n C[t,n] h[t,d,n] + D[d] x[t,d]) silu(z[t,d])
//
// No contraction is shared between channels, so nothing of it is a matrix product: every (token,
// channel, state) costs one exponential and four fp32 operations.  A block owns CB channels of one
// sequence and goes through its tokens in tiles of TW x TK: warp (w, cw) has the w-th TK tokens of
// the tile and the cw-th 32 / TPC channels, a thread S states of one channel.  Where TW > 1 the tile is
// split over time as well: each warp first takes its tokens from a zero state, then the warps'
// end states are joined in order (h <- exp(A sum dt) h + end), and each warp goes through its
// tokens again from the state that really enters them.
#include <algorithm>

#include "selective.cuh"

namespace ssd {

namespace {

template <int S_, int TPC_, int CW_, int TW_, int TK_>
struct Cfg {
    static constexpr int S = S_, TPC = TPC_, CW = CW_, TW = TW_, TK = TK_;
    static constexpr int NP = S * TPC, CPW = 32 / TPC, CB = CW * CPW, TT = TW * TK, NT = 32 * CW * TW;
    static constexpr size_t smem = (size_t)TT * CB * 8 + (size_t)TT * NP * 8 +
                                   (TW > 1 ? (size_t)(TW + 1) * CB * NP * 4 + (size_t)TW * CB * 4 : 0);
    static_assert(TK % TPC == 0 && SEL_Q % TK == 0 && TT % SEL_Q == 0 && S % 4 == 0, "tile shape");
};

template <typename T, typename F>
__global__ void __launch_bounds__(F::NT, F::NT <= 512 ? 2 : 1) k_sel_fwd(const SelArgs a, int cblocks) {
    constexpr int S = F::S, TPC = F::TPC, NP = F::NP, CB = F::CB, TT = F::TT, TK = F::TK, TW = F::TW, NT = F::NT;
    extern __shared__ __align__(16) uint8_t sel_sm[];
    float2 *dd = reinterpret_cast<float2 *>(sel_sm);                // [TT][CB]: (dt, dt x), then (dt, sum C h)
    float *Bs = reinterpret_cast<float *>(dd + TT * CB);            // [TT][NP]
    float *Cs = Bs + TT * NP;                                       // [TT][NP]
    float *E = Cs + TT * NP;                                        // [TW + 1][CB][NP]: end states, then entering states
    float *Sd = E + (TW + 1) * CB * NP;                             // [TW][CB]: sums of dt
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int w = wid % TW, cw = wid / TW;
    const int q = lane % TPC, cl = cw * F::CPW + lane / TPC;        // this thread's states [q S, q S + S) of channel cl
    const int cb = blockIdx.x % cblocks, s = blockIdx.x / cblocks;
    const int bpg = cblocks / a.ngroups, g = cb / bpg;
    const int d0 = g * a.dpg + (cb % bpg) * CB, dend = (g + 1) * a.dpg;
    const SelSeq sq = sel_seq(a, s);
    const int N = a.N;
    const T *x = static_cast<const T *>(a.x) + sq.b * a.xb + sq.t0 * a.xt;
    const T *z = a.z ? static_cast<const T *>(a.z) + sq.b * a.zb + sq.t0 * a.zt : nullptr;
    const T *B = static_cast<const T *>(a.B) + sq.b * a.Bb + sq.t0 * a.Bt + g * a.Bg;
    const T *C = static_cast<const T *>(a.C) + sq.b * a.Cb + sq.t0 * a.Ct + g * a.Cg;
    T *y = a.y ? static_cast<T *>(a.y) + sq.b * a.yb + sq.t0 * a.yt : nullptr;
    const int64_t dt0 = sq.b * a.dtb + sq.t0 * a.dtt;

    f32x2 A2[S / 2], h[S / 2];                                      // A log2(e); the running state
    const int d = d0 + cl;
#pragma unroll
    for (int i = 0; i < S / 2; ++i) {
        float v[2], hv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int n = q * S + 2 * i + e;
            const bool in = d < dend && n < N;
            v[e] = in ? a.A[(int64_t)d * N + n] * kLog2e : 0.f;
            hv[e] = (TW == 1 && in && a.init) ? ld_st(a.init, a.init_bf16, ((int64_t)s * a.channels + d) * N + n) : 0.f;
        }
        A2[i] = pk2(v[0], v[1]);
        h[i] = pk2(hv[0], hv[1]);
    }
    if (TW > 1) {
        for (int i = tid; i < CB * NP; i += NT) {
            const int c = i / NP, n = i % NP;
            E[TW * CB * NP + i] = (a.init && d0 + c < dend && n < N)
                                      ? ld_st(a.init, a.init_bf16, ((int64_t)s * a.channels + d0 + c) * N + n) : 0.f;
        }
    }
    for (int t0 = 0; t0 < sq.len; t0 += TT) {
        __syncthreads();   // the last tile's epilogue has read dd
        for (int i = tid; i < TT * CB; i += NT) {
            const int t = t0 + i / CB, dc = d0 + i % CB;
            float dt = 0.f, xv = 0.f;                               // past the end: decay 1, no input
            if (t < sq.len && dc < dend) {
                const float raw = ld_dt(a, dt0 + t * a.dtt + dc) + (a.bias ? a.bias[dc] : 0.f);
                xv = to_f(x[t * a.xt + dc]);
                dt = sel_softplus(raw);
            }
            dd[i] = make_float2(dt, dt * xv);
        }
        for (int i = tid; i < TT * NP; i += NT) {
            const int t = t0 + i / NP, n = i % NP;
            const bool in = t < sq.len && n < N;
            Bs[i] = in ? to_f(B[t * a.Bt + n]) : 0.f;
            Cs[i] = in ? to_f(C[t * a.Ct + n]) : 0.f;
        }
        __syncthreads();
        const bool live = t0 + w * TK < sq.len;                     // this warp has tokens
        const float2 *dp = dd + w * TK * CB + cl;
        const float *bp = Bs + w * TK * NP + q * S, *cp = Cs + w * TK * NP + q * S;
        if (TW > 1) {
            f32x2 e[S / 2];
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < S / 2; ++i) e[i] = 0;
            if (live) {
#pragma unroll 4
                for (int t = 0; t < TK; ++t) {
                    const float2 v = dp[t * CB];
                    sum += v.x;
                    const f32x2 dt2 = pk2(v.x, v.x), dx2 = pk2(v.y, v.y);
                    const ulonglong2 *b = reinterpret_cast<const ulonglong2 *>(bp + t * NP);
#pragma unroll
                    for (int i = 0; i < S / 4; ++i) {
                        const ulonglong2 bv = b[i];
                        e[2 * i] = fma2(ex2x2(mul2(dt2, A2[2 * i])), e[2 * i], mul2(dx2, bv.x));
                        e[2 * i + 1] = fma2(ex2x2(mul2(dt2, A2[2 * i + 1])), e[2 * i + 1], mul2(dx2, bv.y));
                    }
                }
            }
            ulonglong2 *ep = reinterpret_cast<ulonglong2 *>(E + (w * CB + cl) * NP + q * S);
#pragma unroll
            for (int i = 0; i < S / 4; ++i) ep[i] = make_ulonglong2(e[2 * i], e[2 * i + 1]);
            if (q == 0) Sd[w * CB + cl] = sum;
            __syncthreads();
            for (int i = tid; i < CB * NP; i += NT) {               // (channel, state): the warps' ends in order
                const int c = i / NP, n = i % NP, dc = d0 + c;
                const bool in = dc < dend && n < N;
                const float An = in ? a.A[(int64_t)dc * N + n] * kLog2e : 0.f;
                float hc = E[TW * CB * NP + i];
#pragma unroll
                for (int k = 0; k < TW; ++k) {
                    const int tk = t0 + k * TK;
                    if (a.states && tk % SEL_Q == 0 && tk < sq.len && dc < dend) {
                        const int slot = sq.slot0 + tk / SEL_Q;
                        if (slot < a.nslots) a.states[((int64_t)slot * a.channels + dc) * NP + n] = hc;
                    }
                    const float end = E[k * CB * NP + i];
                    E[k * CB * NP + i] = hc;
                    hc = fmaf(ex2f(An * Sd[k * CB + c]), hc, end);
                }
                E[TW * CB * NP + i] = hc;
            }
            __syncthreads();
            if (y == nullptr) continue;
#pragma unroll
            for (int i = 0; i < S / 4; ++i) {
                const ulonglong2 v = ep[i];
                h[2 * i] = v.x;
                h[2 * i + 1] = v.y;
            }
        } else if (a.states && d < dend && t0 % SEL_Q == 0) {
            const int slot = sq.slot0 + t0 / SEL_Q;
            if (slot < a.nslots) {
                ulonglong2 *sp = reinterpret_cast<ulonglong2 *>(a.states + ((int64_t)slot * a.channels + d) * NP + q * S);
#pragma unroll
                for (int i = 0; i < S / 4; ++i) sp[i] = make_ulonglong2(h[2 * i], h[2 * i + 1]);
            }
        }
        if (live) {
#pragma unroll
            for (int t = 0; t < TK; t += TPC) {
                float yv[TPC];
#pragma unroll
                for (int u = 0; u < TPC; ++u) {
                    const float2 v = dp[(t + u) * CB];
                    const f32x2 dt2 = pk2(v.x, v.x), dx2 = pk2(v.y, v.y);
                    const ulonglong2 *b = reinterpret_cast<const ulonglong2 *>(bp + (t + u) * NP);
                    const ulonglong2 *c = reinterpret_cast<const ulonglong2 *>(cp + (t + u) * NP);
                    f32x2 acc = 0;
#pragma unroll
                    for (int i = 0; i < S / 4; ++i) {
                        const ulonglong2 bv = b[i], cv = c[i];
                        h[2 * i] = fma2(ex2x2(mul2(dt2, A2[2 * i])), h[2 * i], mul2(dx2, bv.x));
                        acc = fma2(h[2 * i], cv.x, acc);
                        h[2 * i + 1] = fma2(ex2x2(mul2(dt2, A2[2 * i + 1])), h[2 * i + 1], mul2(dx2, bv.y));
                        acc = fma2(h[2 * i + 1], cv.y, acc);
                    }
                    yv[u] = sum2(acc);
                }
                const float ys = reduce_scatter<TPC>(yv, q);        // token t + q
                dd[(w * TK + t + q) * CB + cl].y = ys;
            }
        }
        __syncthreads();
        for (int i = tid; i < TT * CB; i += NT) {
            const int t = t0 + i / CB, dc = d0 + i % CB;
            if (t >= sq.len || dc >= dend) continue;
            float v = dd[i].y;
            if (a.D) v = fmaf(a.D[dc], to_f(x[t * a.xt + dc]), v);
            if (z) {
                const float zv = to_f(z[t * a.zt + dc]);
                v *= zv * sel_sigmoid<T>(zv);
            }
            y[t * a.yt + dc] = from_f<T>(v);
        }
    }
    if (a.final == nullptr) return;
    const int64_t f0 = ((int64_t)s * a.channels + d0) * N;
    if (TW > 1) {
        __syncthreads();
        for (int i = tid; i < CB * NP; i += NT) {
            const int c = i / NP, n = i % NP;
            if (d0 + c < dend && n < N) st_st(a.final, a.final_bf16, f0 + c * N + n, E[TW * CB * NP + i]);
        }
    } else if (d < dend) {
#pragma unroll
        for (int i = 0; i < S / 2; ++i) {
            float v[2];
            up2(h[i], v[0], v[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = q * S + 2 * i + e;
                if (n < N) st_st(a.final, a.final_bf16, f0 + cl * N + n, v[e]);
            }
        }
    }
}

template <typename T, typename F>
cudaError_t launch(const SelArgs &a, cudaStream_t st) {
    static int attr[64] = {0};
    cudaError_t e = ensure_smem_attr(k_sel_fwd<T, F>, (int)F::smem, attr);
    if (e != cudaSuccess) return e;
    const int cblocks = a.ngroups * ((a.dpg + F::CB - 1) / F::CB);
    k_sel_fwd<T, F><<<(unsigned)((int64_t)a.nseqs * cblocks), F::NT, F::smem, st>>>(a, cblocks);
    return cudaGetLastError();
}

template <typename T>
cudaError_t pick(const SelArgs &a, cudaStream_t st) {
    switch (a.NP) {
        case 16: return launch<T, Cfg<8, 2, 2, 8, 16>>(a, st);
        case 32: return launch<T, Cfg<8, 4, 4, 4, 16>>(a, st);
        case 64: return launch<T, Cfg<8, 8, 4, 4, 16>>(a, st);
        default: return launch<T, Cfg<8, 16, 4, 4, 16>>(a, st);
    }
}

}  // namespace

cudaError_t sel_launch_fwd(const SelArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? pick<__nv_bfloat16>(a, st) : pick<float>(a, st);
}

}  // namespace ssd
