// selective_fwd.cu -- the selective scan, forward: a state-space scan with a decay rate per channel
// and state,
//
//   dt[t,d] = softplus(dt_raw[t,d] + dt_bias[d])
//   h[t,d,n] = exp(dt[t,d] A[d,n]) h[t-1,d,n] + dt[t,d] x[t,d] B[t,n]
//   y[t,d] = (sum_n C[t,n] h[t,d,n] + D[d] x[t,d]) silu(z[t,d])
//
// No contraction is shared between channels, so nothing of it is a matrix product: every (token,
// channel, state) costs one exponential and four fp32 operations, which pair up two to an
// instruction.  A block owns CB channels of one sequence and goes through its tokens in tiles of
// TW x TK: warp (w, cw) has the w-th TK tokens of the tile and the cw-th 64 / TPC channels, a thread
// S states of two neighbouring channels (shared memory hands a thread one value a cycle whatever
// the width of the load, so B and C are read once for both).  Where TW > 1 the tile is split over time
// as well: each warp first takes its tokens from a zero state, then the warps' end states are
// joined in order (h <- exp(A sum dt) h + end), and each warp goes through its tokens again from the
// state that really enters them.  A warp brings in, converts and finishes its own tokens (the next
// tile's in the background), so that nothing but the joining needs the block's barriers.
//
// Bytes do not bound it: 2048 tokens x 4096 channels, dstate 16, bf16 (68 MB, 10 us of HBM) take 94 us,
// two sweeps of 134 million exponentials, 13 us each at the multi-function units' 32 a clock and SM.
// Instructions issue in 56% of the cycles with 13 warps an SM, shared memory is busy for 58%, the
// multi-function unit for 36%: latency between the few warps that 128 registers a thread leave.
// Three blocks an SM (80 registers, spills) took 108 us, 12 and 16 warps a block 112 and 131; a
// thread for one channel, which reads B and C twice as often, 100.
#include <algorithm>

#include "selective.cuh"

namespace ssd {

namespace {

template <int S_, int TPC_, int CW_, int TW_, int TK_, int OCC_>
struct Cfg {
    static constexpr int S = S_, TPC = TPC_, CW = CW_, TW = TW_, TK = TK_, OCC = OCC_;   // OCC: blocks per SM asked for
    static constexpr int NP = S * TPC, CPW = 64 / TPC, CB = CW * CPW, TT = TW * TK, NT = 32 * CW * TW;
    static constexpr int U = TPC / 2;                                                    // tokens summed over lanes at once
    // fours of a warp's x and of its B: rows a pass of the warp covers, passes
    static constexpr int RX = 128 / CPW, PX = (TK + RX - 1) / RX, RB = NP < 128 ? 128 / NP : 1, PB = (TK + RB - 1) / RB;
    static_assert(TPC >= 2 && TK % U == 0 && (TW == 1 ? TK % SEL_Q == 0 : SEL_Q % TK == 0) && TT % SEL_Q == 0 && S % 4 == 0, "tile shape");
    static_assert(TW == 1 || (CB * NP / 4 <= NT && TT == sel_tile(NP) && CB == sel_block(NP)), "the joining takes a thread for four states");
    // where the n-th four of channel c's states lies: a warp's threads write one of two neighbouring channels at a
    // time, and every other pair has them swapped, so that eight threads meet eight different bank groups
    static __device__ __forceinline__ int at(int c, int n) { return (c ^ (c >> 1 & 1)) * (NP / 4) + n; }
    // bytes a warp keeps: (dt, dt x), B, C, and the next tile as it comes
    static constexpr size_t wsmem(size_t ts, size_t ds) {
        return ((size_t)TK * CPW * 8 + (size_t)TK * NP * 8 + (size_t)TK * CPW * (ts + ds) + (size_t)TK * NP * 2 * ts);
    }
    template <typename T>
    static size_t smem(bool dt_f32) {
        return CW * TW * wsmem(sizeof(T), dt_f32 ? 4 : sizeof(T)) +
               (TW > 1 ? (size_t)TW * CB * NP * 4 + (size_t)TW * CB * 4 : 0);
    }
};

// VEC: every row allows four elements an access.
template <typename T, typename F, bool VEC>
__global__ void __launch_bounds__(F::NT, F::OCC) k_sel_fwd(const SelArgs a, int cblocks) {
    after_previous();
    constexpr int S = F::S, TPC = F::TPC, NP = F::NP, CB = F::CB, CPW = F::CPW, TT = F::TT, TK = F::TK, TW = F::TW, U = F::U;
    extern __shared__ __align__(16) uint8_t sel_sm[];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int w = wid % TW, cw = wid / TW;
    const size_t wbytes = F::wsmem(sizeof(T), a.dt_f32 ? 4 : sizeof(T));
    float4 *dd = reinterpret_cast<float4 *>(sel_sm + wid * wbytes); // [TK][CPW / 2]: (dt, dt x) of two channels; then (dt, sum C h)
    float *Bs = reinterpret_cast<float *>(dd + TK * CPW / 2);       // [TK][NP]
    float *Cs = Bs + TK * NP;                                       // [TK][NP]
    float *rD = Cs + TK * NP;                                       // the next tile as it came: dt [TK][CPW], fp32 or T
    T *rX = reinterpret_cast<T *>(rD + TK * CPW / (a.dt_f32 ? 1 : 4 / (int)sizeof(T)));   // x [TK][CPW]
    T *rB = rX + TK * CPW, *rC = rB + TK * NP;                      // B, C [TK][NP]
    float *E = reinterpret_cast<float *>(sel_sm + F::CW * TW * wbytes);   // [TW][CB][NP / 4] fours of end states, then entering states, placed by at()
    float *Sd = E + TW * CB * NP;                                   // [TW][CB]: sums of dt
    const int q = lane % TPC, cp0 = 2 * (lane / TPC), cl = cw * CPW + cp0;   // this thread's states [q S, q S + S) of channels cl, cl + 1
    const int cb = blockIdx.x % cblocks, s = blockIdx.x / cblocks / a.nseg, seg = blockIdx.x / cblocks % a.nseg;
    const int bpg = cblocks / a.ngroups, g = cb / bpg;
    const int d0 = g * a.dpg + (cb % bpg) * CB, dend = (g + 1) * a.dpg, d = d0 + cl;
    const SelSeq whole = sel_seq(a, s), sq = sel_segment(a, whole, seg);
    const int N = a.N, len = sq.len;
    // for the elementwise steps: this thread's four channels (the first is e0) and first token, and of B and C
    const int pc = 4 * (lane % (CPW / 4)), pt = lane / (CPW / 4), e0 = d0 + cw * CPW + pc, nc = min(max(dend - e0, 0), 4);
    const int pn = 4 * (lane % (NP / 4)), pbt = lane / (NP / 4), nn = min(max(N - pn, 0), 4);
    const bool vec = VEC || a.vec, vecBC = VEC || a.vecBC;
    const int xs = (int)a.xt * (int)sizeof(T), zs = (int)a.zt * (int)sizeof(T), ys = (int)a.yt * (int)sizeof(T);
    const int es = a.dt_f32 ? 4 : (int)sizeof(T), ds = (int)a.dtt * es;
    const int bs = (int)a.Bt * (int)sizeof(T), cs = (int)a.Ct * (int)sizeof(T);
    const T *x = static_cast<const T *>(a.x) + sq.b * a.xb + sq.t0 * a.xt + e0;
    const T *z = a.z ? static_cast<const T *>(a.z) + sq.b * a.zb + sq.t0 * a.zt + e0 : nullptr;
    T *y = a.y ? static_cast<T *>(a.y) + sq.b * a.yb + sq.t0 * a.yt + e0 : nullptr;
    const uint8_t *dtp = static_cast<const uint8_t *>(a.dt) + (sq.b * a.dtb + sq.t0 * a.dtt + e0) * es;
    const T *B = static_cast<const T *>(a.B) + sq.b * a.Bb + sq.t0 * a.Bt + g * a.Bg + pn;
    const T *C = static_cast<const T *>(a.C) + sq.b * a.Cb + sq.t0 * a.Ct + g * a.Cg + pn;
    float bias[4], Dv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bias[i] = a.bias && i < nc ? a.bias[e0 + i] : 0.f;
        Dv[i] = a.D && i < nc ? a.D[e0 + i] : 0.f;
    }

    // the channels and states of the warp that exist, and its rows' first elements, for rows taken element by element
    const int nch = min(dend - d0 - cw * CPW, CPW);
    const T *x0 = x - pc, *z0 = z - pc, *B0 = B - pn, *C0 = C - pn;
    auto fetch = [&](int t0) {                                      // the warp's tokens of a tile, in the background
        const int tw = t0 + w * TK, nr = len - tw;
        if (vec) {
#pragma unroll
            for (int k = 0; k < F::PX; ++k) {
                const int tl = pt + k * F::RX, t = tw + tl;
                if ((F::RX * F::PX == TK || tl < TK) && t < len) {
                    fetch4(rX + tl * CPW + pc, row(x, t, xs), nc, vec);
                    if (a.dt_f32) fetch4(rD + tl * CPW + pc, reinterpret_cast<const float *>(row(dtp, t, ds)), nc, vec);
                    else fetch4(reinterpret_cast<T *>(rD) + tl * CPW + pc, reinterpret_cast<const T *>(row(dtp, t, ds)), nc, vec);
                }
            }
        } else if (nr > 0 && nch > 0) {
            fetch_rows<TK, CPW, 32>(rX, row(x0, tw, xs), xs, nr, nch, lane);
            const uint8_t *dt0 = dtp - pc * es;
            if (a.dt_f32) fetch_rows<TK, CPW, 32>(rD, reinterpret_cast<const float *>(row(dt0, tw, ds)), ds, nr, nch, lane);
            else fetch_rows<TK, CPW, 32>(reinterpret_cast<T *>(rD), reinterpret_cast<const T *>(row(dt0, tw, ds)), ds, nr, nch, lane);
        }
        if (vecBC) {
#pragma unroll 4
            for (int k = 0; k < F::PB; ++k) {
                const int tl = pbt + k * F::RB, t = tw + tl;
                if (t < len) {
                    fetch4(rB + tl * NP + pn, row(B, t, bs), nn, vecBC);
                    fetch4(rC + tl * NP + pn, row(C, t, cs), nn, vecBC);
                }
            }
        } else if (nr > 0) {
            fetch_rows<TK, NP, 32>(rB, row(B0, tw, bs), bs, nr, N, lane);
            fetch_rows<TK, NP, 32>(rC, row(C0, tw, cs), cs, nr, N, lane);
        }
        cp_async_commit();
    };

    f32x2 A2[2][S / 2], h[2][S / 2];                                // A log2(e); the running states
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < S / 2; ++i) {
            float v[2], hv[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = q * S + 2 * i + e;
                const bool in = d + c < dend && n < N;
                v[e] = in ? sel_rate(a.A[(int64_t)(d + c) * N + n]) : 0.f;
                hv[e] = (TW == 1 && in && a.init) ? ld_st(a.init, a.init_bf16, ((int64_t)s * a.channels + d + c) * N + n) : 0.f;
            }
            A2[c][i] = pk2(v[0], v[1]);
            h[c][i] = pk2(hv[0], hv[1]);
        }
    // the joining over the warps: a thread takes four states of one channel, and carries them on
    const int jc = tid / (NP / 4), jn = 4 * (tid % (NP / 4));
    const bool joins = TW > 1 && tid < CB * NP / 4;
    f32x2 jA[2] = {0, 0}, jh[2] = {0, 0};
    float jsum = 0.f;
    if (joins) {
        float v[4], hv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = d0 + jc < dend && jn + e < N;
            v[e] = in ? sel_rate(a.A[(int64_t)(d0 + jc) * N + jn + e]) : 0.f;
            hv[e] = in && a.init && !a.ends ? ld_st(a.init, a.init_bf16, ((int64_t)s * a.channels + d0 + jc) * N + jn + e) : 0.f;
        }
        jA[0] = pk2(v[0], v[1]); jA[1] = pk2(v[2], v[3]);
        jh[0] = pk2(hv[0], hv[1]); jh[1] = pk2(hv[2], hv[3]);
        if (!a.ends && d0 + jc < dend) {                            // what the segments before this one leave
            const int64_t at = (int64_t)s * a.nseg * a.channels + d0 + jc;
#pragma unroll 4
            for (int k = 0; k < seg; ++k) {
                const float sd = a.segS[at + (int64_t)k * a.channels];
                const ulonglong2 e = *reinterpret_cast<const ulonglong2 *>(a.segE + (at + (int64_t)k * a.channels) * NP + jn);
                const f32x2 sd2 = pk2(sd, sd);
                jh[0] = fma2(ex2x2(mul2(sd2, jA[0])), jh[0], e.x);
                jh[1] = fma2(ex2x2(mul2(sd2, jA[1])), jh[1], e.y);
            }
        }
    }
    fetch(0);
    for (int t0 = 0; t0 < len; t0 += TT) {
        cp_async_wait_all();
        __syncwarp();      // the tokens have come; the last ones' epilogue has read dd
        const int tw = t0 + w * TK;                                 // the warp's first token
        const bool live = tw < len;
        if (live) {
#pragma unroll
            for (int k = 0; k < F::PX; ++k) {
                const int tl = pt + k * F::RX;
                if (F::RX * F::PX != TK && tl >= TK) break;
                float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};   // past the end: decay 1, no input
                if (tw + tl < len) {
                    float xv[4], r[4];
                    Raw4<T> r0;
                    r0.load(rX + tl * CPW + pc, 4, true);
                    r0.f(xv);
                    if (a.dt_f32) {
                        Raw4<float> rd;
                        rd.load(rD + tl * CPW + pc, 4, true);
                        rd.f(r);
                    } else {
                        Raw4<T> rd;
                        rd.load(reinterpret_cast<T *>(rD) + tl * CPW + pc, 4, true);
                        rd.f(r);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float dt = sel_softplus(r[i] + bias[i]);
                        if (i < nc) {
                            v[2 * i] = dt;
                            v[2 * i + 1] = dt * xv[i];
                        }
                    }
                }
                float4 *o = dd + tl * (CPW / 2);                    // (odd tokens have neighbouring pairs swapped, off the banks)
                o[pc / 2 ^ (tl & 1)] = make_float4(v[0], v[1], v[2], v[3]);
                o[pc / 2 + 1 ^ (tl & 1)] = make_float4(v[4], v[5], v[6], v[7]);
            }
#pragma unroll 4
            for (int k = 0; k < F::PB; ++k) {
                const int tl = pbt + k * F::RB;
                float b[4] = {0.f, 0.f, 0.f, 0.f}, c[4] = {0.f, 0.f, 0.f, 0.f};
                if (tw + tl < len) {
                    float rb[4], rc[4];
                    Raw4<T> r;
                    r.load(rB + tl * NP + pn, 4, true);
                    r.f(rb);
                    r.load(rC + tl * NP + pn, 4, true);
                    r.f(rc);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < nn) {
                            b[i] = rb[i];
                            c[i] = rc[i];
                        }
                }
                put4(Bs + tl * NP + pn, b);
                put4(Cs + tl * NP + pn, c);
            }
        }
        __syncwarp();
        if (t0 + TT < len) fetch(t0 + TT);
        const float4 *dp[2] = {dd + cp0 / 2, dd + (cp0 / 2 ^ 1)};   // even and odd tokens
        const float *bp = Bs + q * S, *cp = Cs + q * S;
        Raw4<T> rx[F::PX], rz[F::PX];                               // for the epilogue
        auto early = [&]() {
            if (y == nullptr || !vec) return;
#pragma unroll
            for (int k = 0; k < F::PX; ++k) {
                const int tl = pt + k * F::RX, t = tw + tl;
                if ((F::RX * F::PX == TK || tl < TK) && t < len) {
                    rx[k].load(row(x, t, xs), nc, vec);
                    if (z) rz[k].load(row(z, t, zs), nc, vec);
                }
            }
        };
        if (TW > 1) {
            f32x2 e[2][S / 2];
            float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
            for (int i = 0; i < S / 2; ++i) e[0][i] = e[1][i] = 0;
            if (live) {
#pragma unroll 4
                for (int t = 0; t < TK; ++t) {
                    const float4 v = dp[t & 1][t * (CPW / 2)];
                    sum0 += v.x;
                    sum1 += v.z;
                    const f32x2 dt0 = pk2(v.x, v.x), dx0 = pk2(v.y, v.y), dt1 = pk2(v.z, v.z), dx1 = pk2(v.w, v.w);
                    const ulonglong2 *b = reinterpret_cast<const ulonglong2 *>(bp + t * NP);
#pragma unroll
                    for (int i = 0; i < S / 4; ++i) {
                        const ulonglong2 bv = b[i];
                        e[0][2 * i] = fma2(ex2x2(mul2(dt0, A2[0][2 * i])), e[0][2 * i], mul2(dx0, bv.x));
                        e[0][2 * i + 1] = fma2(ex2x2(mul2(dt0, A2[0][2 * i + 1])), e[0][2 * i + 1], mul2(dx0, bv.y));
                        e[1][2 * i] = fma2(ex2x2(mul2(dt1, A2[1][2 * i])), e[1][2 * i], mul2(dx1, bv.x));
                        e[1][2 * i + 1] = fma2(ex2x2(mul2(dt1, A2[1][2 * i + 1])), e[1][2 * i + 1], mul2(dx1, bv.y));
                    }
                }
            }
            ulonglong2 *ep = reinterpret_cast<ulonglong2 *>(E) + w * CB * (NP / 4);
#pragma unroll
            for (int i = 0; i < S / 4; ++i) {
                ep[F::at(cl, q * (S / 4) + i)] = make_ulonglong2(e[0][2 * i], e[0][2 * i + 1]);
                ep[F::at(cl + 1, q * (S / 4) + i)] = make_ulonglong2(e[1][2 * i], e[1][2 * i + 1]);
            }
            if (q == 0) *reinterpret_cast<float2 *>(Sd + w * CB + cl) = make_float2(sum0, sum1);
            early();
            __syncthreads();
            if (joins) {
                ulonglong2 end[TW];
                float sd[TW];
#pragma unroll
                for (int k = 0; k < TW; ++k) {
                    end[k] = *(reinterpret_cast<const ulonglong2 *>(E) + k * CB * (NP / 4) + F::at(jc, jn / 4));
                    sd[k] = Sd[k * CB + jc];
                }
#pragma unroll
                for (int k = 0; k < TW; ++k) {
                    const int tk = t0 + k * TK;
                    if (a.states && tk % SEL_Q == 0 && tk < len && d0 + jc < dend) {
                        const int slot = sq.slot0 + tk / SEL_Q;
                        if (slot < a.nslots)
                            *reinterpret_cast<ulonglong2 *>(a.states + ((int64_t)slot * a.channels + d0 + jc) * NP + jn) =
                                make_ulonglong2(jh[0], jh[1]);
                    }
                    const f32x2 sd2 = pk2(sd[k], sd[k]);
                    jsum += sd[k];
                    *(reinterpret_cast<ulonglong2 *>(E) + k * CB * (NP / 4) + F::at(jc, jn / 4)) = make_ulonglong2(jh[0], jh[1]);
                    jh[0] = fma2(ex2x2(mul2(sd2, jA[0])), jh[0], end[k].x);
                    jh[1] = fma2(ex2x2(mul2(sd2, jA[1])), jh[1], end[k].y);
                }
            }
            __syncthreads();
            if (y == nullptr) continue;
#pragma unroll
            for (int i = 0; i < S / 4; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const ulonglong2 v = ep[F::at(cl + c, q * (S / 4) + i)];
                    h[c][2 * i] = v.x;
                    h[c][2 * i + 1] = v.y;
                }
        }
        if (TW == 1) early();
        if (live) {
            // The sums stay in registers over SB batches of tokens: a store after each would hold up the
            // next tokens' loads (the compiler cannot tell that they differ), and with them everything.
            constexpr int SB = SEL_Q / U < 4 ? SEL_Q / U : 4;
            static_assert(SEL_Q % (SB * U) == 0 && TK % (SB * U) == 0 && SB * U % 2 == 0, "chunks start at batches, batches at even tokens");
#pragma unroll 1
            for (int t0s = 0; t0s < TK; t0s += SB * U) {
                if (TW == 1 && a.states && t0s % SEL_Q == 0 && tw + t0s < len) {
                    const int slot = sq.slot0 + (tw + t0s) / SEL_Q;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        if (d + c < dend && slot < a.nslots) {
                            ulonglong2 *sp = reinterpret_cast<ulonglong2 *>(a.states + ((int64_t)slot * a.channels + d + c) * NP + q * S);
#pragma unroll
                            for (int i = 0; i < S / 4; ++i) sp[i] = make_ulonglong2(h[c][2 * i], h[c][2 * i + 1]);
                        }
                }
                float yq[SB];
#pragma unroll
                for (int sb = 0; sb < SB; ++sb) {
                    const int t = t0s + sb * U;
                    float yv[TPC];                                  // [token][channel]
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const float4 v = dp[(sb * U + u) & 1][(t + u) * (CPW / 2)];
                        const f32x2 dt0 = pk2(v.x, v.x), dx0 = pk2(v.y, v.y), dt1 = pk2(v.z, v.z), dx1 = pk2(v.w, v.w);
                        const ulonglong2 *b = reinterpret_cast<const ulonglong2 *>(bp + (t + u) * NP);
                        const ulonglong2 *c = reinterpret_cast<const ulonglong2 *>(cp + (t + u) * NP);
                        f32x2 y0 = 0, y1 = 0;
#pragma unroll
                        for (int i = 0; i < S / 4; ++i) {
                            const ulonglong2 bv = b[i], cv = c[i];
                            h[0][2 * i] = fma2(ex2x2(mul2(dt0, A2[0][2 * i])), h[0][2 * i], mul2(dx0, bv.x));
                            h[1][2 * i] = fma2(ex2x2(mul2(dt1, A2[1][2 * i])), h[1][2 * i], mul2(dx1, bv.x));
                            h[0][2 * i + 1] = fma2(ex2x2(mul2(dt0, A2[0][2 * i + 1])), h[0][2 * i + 1], mul2(dx0, bv.y));
                            h[1][2 * i + 1] = fma2(ex2x2(mul2(dt1, A2[1][2 * i + 1])), h[1][2 * i + 1], mul2(dx1, bv.y));
                            y0 = i == 0 ? mul2(h[0][0], cv.x) : fma2(h[0][2 * i], cv.x, y0);
                            y1 = i == 0 ? mul2(h[1][0], cv.x) : fma2(h[1][2 * i], cv.x, y1);
                            y0 = fma2(h[0][2 * i + 1], cv.y, y0);
                            y1 = fma2(h[1][2 * i + 1], cv.y, y1);
                        }
                        yv[2 * u] = sum2(y0);
                        yv[2 * u + 1] = sum2(y1);
                    }
                    yq[sb] = reduce_scatter<TPC>(yv, q);            // token t + q / 2, channel cl + q % 2
                }
#pragma unroll
                for (int sb = 0; sb < SB; ++sb)
                    reinterpret_cast<float *>(dd + (t0s + sb * U + q / 2) * (CPW / 2) + (cp0 / 2 ^ ((sb * U + q / 2) & 1)))[q % 2 * 2 + 1] = yq[sb];
            }
        }
        if (y == nullptr) continue;
        __syncwarp();
        if (!vec) {                                                 // element by element, eight of x and z at a time
            if (!live || nch <= 0) continue;
            constexpr int E = TK * CPW / 32, EB = E < 8 ? E : 8;
            const int c = lane % CPW, rr = lane / CPW;
            const bool in = c < nch;
            const float Dc = a.D && in ? a.D[d0 + cw * CPW + c] : 0.f;
#pragma unroll 1
            for (int k0 = 0; k0 < E; k0 += EB) {
                T xv[EB], zv[EB];
#pragma unroll
                for (int k = 0; k < EB; ++k) {
                    const int t = min(tw + (k0 + k) * (32 / CPW) + rr, len - 1), e = min(c, nch - 1);   // (no load waits for a branch)
                    xv[k] = row(x0, t, xs)[e];
                    zv[k] = z ? row(z0, t, zs)[e] : xv[k];
                }
#pragma unroll
                for (int k = 0; k < EB; ++k) {
                    const int tl = (k0 + k) * (32 / CPW) + rr, t = tw + tl;
                    if (in && t < len) {
                        float v = reinterpret_cast<const float *>(dd + tl * (CPW / 2) + (c / 2 ^ (tl & 1)))[c % 2 * 2 + 1];
                        if (a.D) v = fmaf(Dc, to_f(xv[k]), v);
                        if (z) v = sel_gate<T>(v, to_f(zv[k]));
                        row(y - pc, t, ys)[c] = from_f<T>(v);
                    }
                }
            }
            continue;
        }
#pragma unroll
        for (int k = 0; k < F::PX; ++k) {
            const int tl = pt + k * F::RX, t = tw + tl;
            if ((F::RX * F::PX == TK || tl < TK) && t < len) {
                const float4 *o4 = dd + tl * (CPW / 2);
                const float4 v0 = o4[pc / 2 ^ (tl & 1)], v1 = o4[pc / 2 + 1 ^ (tl & 1)];
                float o[4] = {v0.y, v0.w, v1.y, v1.w}, f[4];
                if (a.D) {
                    rx[k].f(f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = fmaf(Dv[i], f[i], o[i]);
                }
                if (z) {
                    rz[k].f(f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = sel_gate<T>(o[i], f[i]);
                }
                store4(row(y, t, ys), o, nc, vec);
            }
        }
    }
    if (TW > 1 && a.ends) {
        if (joins && d0 + jc < dend) {
            const int64_t at = ((int64_t)s * a.nseg + seg) * a.channels + d0 + jc;
            *reinterpret_cast<ulonglong2 *>(a.segE + at * NP + jn) = make_ulonglong2(jh[0], jh[1]);
            if (jn == 0) a.segS[at] = jsum;
        }
        return;
    }
    // the segment that holds the sequence's last token (the first one, where there is none) has the final state
    if (a.final == nullptr || sq.t0 + len != whole.t0 + whole.len || (len == 0 && seg > 0)) return;
    auto put = [&](int c, int n0, f32x2 lo, f32x2 hi) {             // states n0 .. n0 + 3 of channel d0 + c
        if (d0 + c >= dend) return;
        float v[4];
        up2(lo, v[0], v[1]);
        up2(hi, v[2], v[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n0 + e < N) st_st(a.final, a.final_bf16, ((int64_t)s * a.channels + d0 + c) * N + n0 + e, v[e]);
    };
    if (TW > 1) {
        if (joins) put(jc, jn, jh[0], jh[1]);
    } else {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < S / 4; ++i) put(cl + c, q * S + 4 * i, h[c][2 * i], h[c][2 * i + 1]);
    }
}

template <typename T, typename F, bool VEC>
cudaError_t launch_rows(const SelArgs &a, cudaStream_t st) {
    static int attr[64] = {0};
    const size_t sm = F::template smem<T>(a.dt_f32);
    cudaError_t e = ensure_smem_attr(k_sel_fwd<T, F, VEC>, (int)sm, attr);
    if (e != cudaSuccess) return e;
    const int cblocks = a.ngroups * ((a.dpg + F::CB - 1) / F::CB);
    return launch_early(k_sel_fwd<T, F, VEC>, (unsigned)((int64_t)a.nseqs * a.nseg * cblocks), F::NT, sm, st, a, cblocks);
}
template <typename T, typename F>
cudaError_t launch(const SelArgs &a, cudaStream_t st) {
    return a.vec && a.vecBC ? launch_rows<T, F, true>(a, st) : launch_rows<T, F, false>(a, st);
}

// Without a split over time nothing is computed twice, but a sequence's tokens follow one another at
// some 200 cycles each, so it takes many (sequence, channel) pairs to fill the card.  Measured at dstate
// 16, bf16, split against whole: 4 x 2048 tokens x 2048 channels 185 / 279 us, 2 x 2048 x 8192 326 / 326,
// 16 x 1024 x 4096 610 / 434.  Of packed sequences the host knows the number and not the lengths.  Its limit is
// right where the lengths are alike: x 4096 channels, 16 of 500 tokens 317 / 221, 64 of 64 295 / 124, 64 of 1 217 / 54; 9 of mixed
// lengths, 16111 tokens, 614 / 724 (below the limit).  It is wrong for one long sequence among many short
// ones: 8000 tokens and 14 single ones (split) take 358 us, and 15 (whole) 1080 where split they would take 359.
template <typename T>
cudaError_t pick(const SelArgs &a, cudaStream_t st) {
    if (a.nseg == 1 && (int64_t)a.nseqs * a.channels >= (a.cu ? 65536 : 16384)) {
        switch (a.NP) {
            case 16: return launch<T, Cfg<4, 4, 4, 1, 32, 4>>(a, st);
            case 32: return launch<T, Cfg<8, 4, 4, 1, 32, 3>>(a, st);
            case 64: return launch<T, Cfg<8, 8, 2, 1, 32, 4>>(a, st);
            default: return launch<T, Cfg<8, 16, 1, 1, 32, 4>>(a, st);
        }
    }
    switch (a.NP) {
        case 16: return launch<T, Cfg<4, 4, 1, 8, 16, 2>>(a, st);
        case 32: return launch<T, Cfg<8, 4, 1, 8, 16, 2>>(a, st);
        case 64: return launch<T, Cfg<8, 8, 1, 4, 16, 3>>(a, st);
        default: return launch<T, Cfg<8, 16, 1, 4, 16, 2>>(a, st);
    }
}

}  // namespace

cudaError_t sel_launch_fwd(SelArgs a, bool bf16, cudaStream_t st) {
    if (a.nseg > 1) {                                               // the segments' ends from zero
        SelArgs e = a;
        e.ends = true;
        e.y = nullptr;
        e.states = nullptr;
        const cudaError_t rc = bf16 ? pick<__nv_bfloat16>(e, st) : pick<float>(e, st);
        if (rc != cudaSuccess) return rc;
    }
    return bf16 ? pick<__nv_bfloat16>(a, st) : pick<float>(a, st);
}

}  // namespace ssd
