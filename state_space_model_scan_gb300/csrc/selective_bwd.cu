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

// ---- the adjoint at the chunks' right ends: the forward's first sweep, backwards.  Warp (w, cw) has the w-th TK
// tokens of a tile and the cw-th 64 / TPC channels, a thread S states of two channels; the warps' folds are
// joined from the last to the first while the next tile is on its way.  Bound as the forward: 2 x 2048 tokens x
// 4096 channels, dstate 16, bf16 take 101 us (139 MB, 20 us of HBM); one sweep with states kept at the end.
template <int S_, int TPC_, int CW_, int TW_, int TK_, int OCC_>
struct RevCfg {
    static constexpr int S = S_, TPC = TPC_, CW = CW_, TW = TW_, TK = TK_, OCC = OCC_;
    static constexpr int NP = S * TPC, CPW = 64 / TPC, CB = CW * CPW, TT = TW * TK, NT = 32 * CW * TW;
    static constexpr int RX = 128 / CPW, PX = (TK + RX - 1) / RX, RB = NP < 128 ? 128 / NP : 1, PB = (TK + RB - 1) / RB;
    static_assert(SEL_Q % TK == 0 && TT == sel_tile(NP) && CB == sel_block(NP) && S % 4 == 0 && CB * NP / 4 <= NT, "tile shape");
    // where the n-th four of channel c's states lies (as in the forward, off the banks)
    static __device__ __forceinline__ int at(int c, int n) { return (c ^ (c >> 1 & 1)) * (NP / 4) + n; }
    // bytes a warp keeps: (dt, dyp), C, and the next tile's dt, dy, z and C as they come
    static constexpr size_t wsmem(size_t ts, size_t ds) {
        return (size_t)TK * CPW * 8 + (size_t)TK * NP * 4 + (size_t)TK * CPW * (2 * ts + ds) + (size_t)TK * NP * ts;
    }
    template <typename T>
    static size_t smem(bool dt_f32) {
        return CW * TW * wsmem(sizeof(T), dt_f32 ? 4 : sizeof(T)) + 2 * ((size_t)TW * CB * NP * 4 + (size_t)TW * CB * 4);
    }
};

// VEC: every row allows four elements an access.
template <typename T, typename F, bool VEC>
__global__ void __launch_bounds__(F::NT, F::OCC) k_sel_rev(const SelArgs a, int cblocks) {
    after_previous();
    constexpr int S = F::S, TPC = F::TPC, NP = F::NP, CB = F::CB, CPW = F::CPW, TT = F::TT, TK = F::TK, TW = F::TW;
    extern __shared__ __align__(16) uint8_t sel_sm[];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int w = wid % TW, cw = wid / TW;
    const size_t wbytes = F::wsmem(sizeof(T), a.dt_f32 ? 4 : sizeof(T));
    float4 *dd = reinterpret_cast<float4 *>(sel_sm + wid * wbytes);  // [TK][CPW / 2]: (dt, dyp) of two channels
    float *Cs = reinterpret_cast<float *>(dd + TK * CPW / 2);        // [TK][NP]
    float *rD = Cs + TK * NP;                                        // dt [TK][CPW], fp32 or T
    T *rY = reinterpret_cast<T *>(rD + TK * CPW / (a.dt_f32 ? 1 : 4 / (int)sizeof(T)));   // dy, z [TK][CPW]
    T *rZ = rY + TK * CPW, *rC = rZ + TK * CPW;                      // C [TK][NP]
    float *E = reinterpret_cast<float *>(sel_sm + F::CW * TW * wbytes);   // two of [TW][CB][NP / 4] fours, placed by at(): what each warp passes on
    float *Sd = E + 2 * TW * CB * NP;                                // two of [TW][CB]: sums of dt
    const int q = lane % TPC, cp0 = 2 * (lane / TPC), cl = cw * CPW + cp0;
    const int cb = blockIdx.x % cblocks, s = blockIdx.x / cblocks / a.nseg, seg = blockIdx.x / cblocks % a.nseg;
    const int bpg = cblocks / a.ngroups, g = cb / bpg;
    const int d0 = g * a.dpg + (cb % bpg) * CB, dend = (g + 1) * a.dpg, d = d0 + cl;
    const SelSeq sq = sel_segment(a, sel_seq(a, s), seg);
    const int N = a.N, len = sq.len;
    const int pc = 4 * (lane % (CPW / 4)), pt = lane / (CPW / 4), e0 = d0 + cw * CPW + pc, nc = min(max(dend - e0, 0), 4);
    const int pn = 4 * (lane % (NP / 4)), pbt = lane / (NP / 4), nn = min(max(N - pn, 0), 4);
    const bool vec = VEC || a.vec, vecBC = VEC || a.vecBC, gated = a.z != nullptr;
    const int es = a.dt_f32 ? 4 : (int)sizeof(T), ds = (int)a.dtt * es;
    const int ys = (int)a.dyt * (int)sizeof(T), zs = (int)a.zt * (int)sizeof(T), cs = (int)a.Ct * (int)sizeof(T);
    const T *dy = static_cast<const T *>(a.dy) + sq.b * a.dyb + sq.t0 * a.dyt + e0;
    const T *z = gated ? static_cast<const T *>(a.z) + sq.b * a.zb + sq.t0 * a.zt + e0 : nullptr;
    const uint8_t *dtp = static_cast<const uint8_t *>(a.dt) + (sq.b * a.dtb + sq.t0 * a.dtt + e0) * es;
    const T *C = static_cast<const T *>(a.C) + sq.b * a.Cb + sq.t0 * a.Ct + g * a.Cg + pn;
    float bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] = a.bias && i < nc ? a.bias[e0 + i] : 0.f;

    const int nch = min(dend - d0 - cw * CPW, CPW);
    Rows<TK, CPW, 32, T> ld, ly, lz;
    Rows<TK, CPW, 32, float> lf;
    auto fetch = [&](int t0) {
        const int tw = t0 + w * TK, nr = len - tw;
        if (vec) {
#pragma unroll
            for (int k = 0; k < F::PX; ++k) {
                const int tl = pt + k * F::RX, t = tw + tl;
                if ((F::RX * F::PX == TK || tl < TK) && t < len) {
                    if (a.dt_f32) fetch4(rD + tl * CPW + pc, reinterpret_cast<const float *>(row(dtp, t, ds)), nc, vec);
                    else fetch4(reinterpret_cast<T *>(rD) + tl * CPW + pc, reinterpret_cast<const T *>(row(dtp, t, ds)), nc, vec);
                    fetch4(rY + tl * CPW + pc, row(dy, t, ys), nc, vec);
                    if (gated) fetch4(rZ + tl * CPW + pc, row(z, t, zs), nc, vec);
                }
            }
        } else if (nr > 0 && nch > 0) {                              // (element by element; the copies end in put())
            const uint8_t *dt0 = dtp - pc * es;
            if (a.dt_f32) lf.load(rD, reinterpret_cast<const float *>(row(dt0, tw, ds)), ds, nr, nch, lane);
            else ld.load(reinterpret_cast<T *>(rD), reinterpret_cast<const T *>(row(dt0, tw, ds)), ds, nr, nch, lane);
            ly.load(rY, row(dy - pc, tw, ys), ys, nr, nch, lane);
            if (gated) lz.load(rZ, row(z - pc, tw, zs), zs, nr, nch, lane);
        }
        if (vecBC) {
#pragma unroll 4
            for (int k = 0; k < F::PB; ++k) {
                const int tl = pbt + k * F::RB, t = tw + tl;
                if (t < len) fetch4(rC + tl * NP + pn, row(C, t, cs), nn, vecBC);
            }
        } else if (nr > 0) {
            fetch_rows<TK, NP, 32>(rC, row(C - pn, tw, cs), cs, nr, N, lane);
        }
        cp_async_commit();
    };
    auto put = [&](int t0) {
        const int nr = len - t0 - w * TK;
        if (vec || nr <= 0 || nch <= 0) return;
        if (!a.dt_f32) ld.store(reinterpret_cast<T *>(rD), nr, nch, lane);
        ly.store(rY, nr, nch, lane);
        if (gated) lz.store(rZ, nr, nch, lane);
    };

    f32x2 A2[2][S / 2];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < S / 2; ++i) {
            float v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = q * S + 2 * i + e;
                v[e] = d + c < dend && n < N ? sel_rate(a.A[(int64_t)(d + c) * N + n]) : 0.f;
            }
            A2[c][i] = pk2(v[0], v[1]);
        }
    const int jc = tid / (NP / 4), jn = 4 * (tid % (NP / 4));
    const bool joins = tid < CB * NP / 4;
    f32x2 jA[2] = {0, 0}, ju[2] = {0, 0};
    if (joins) {
        float v[4], uv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = d0 + jc < dend && jn + e < N;
            v[e] = in ? sel_rate(a.A[(int64_t)(d0 + jc) * N + jn + e]) : 0.f;
            uv[e] = in && a.dfinal && !a.ends ? ld_st(a.dfinal, a.dfinal_bf16, ((int64_t)s * a.channels + d0 + jc) * N + jn + e) : 0.f;
        }
        jA[0] = pk2(v[0], v[1]); jA[1] = pk2(v[2], v[3]);
        ju[0] = pk2(uv[0], uv[1]); ju[1] = pk2(uv[2], uv[3]);
        if (!a.ends && d0 + jc < dend) {                             // what the segments after this one pass on
            const int64_t at = (int64_t)s * a.nseg * a.channels + d0 + jc;
#pragma unroll 4
            for (int k = a.nseg - 1; k > seg; --k) {
                const float sd = a.segS[at + (int64_t)k * a.channels];
                const ulonglong2 e = *reinterpret_cast<const ulonglong2 *>(a.segE + (at + (int64_t)k * a.channels) * NP + jn);
                const f32x2 sd2 = pk2(sd, sd);
                ju[0] = fma2(ex2x2(mul2(sd2, jA[0])), ju[0], e.x);
                ju[1] = fma2(ex2x2(mul2(sd2, jA[1])), ju[1], e.y);
            }
        }
    }
    float jsum = 0.f;
    const int last = len > 0 ? (len - 1) / TT * TT : -1;
    if (last >= 0) {
        fetch(last);
        put(last);
    }
    int buf = 0;
    for (int t0 = last; t0 >= 0; t0 -= TT, buf ^= 1) {
        cp_async_wait_all();
        __syncwarp();
        const int tw = t0 + w * TK;
        f32x2 u[2][S / 2];
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int i = 0; i < S / 2; ++i) u[0][i] = u[1][i] = 0;
        if (tw < len) {
#pragma unroll
            for (int k = 0; k < F::PX; ++k) {
                const int tl = pt + k * F::RX;
                if (F::RX * F::PX != TK && tl >= TK) break;
                float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};   // past the end: decay 1, no gradient
                if (tw + tl < len) {
                    float yv[4], zv[4], r[4];
                    Raw4<T> r0;
                    r0.load(rY + tl * CPW + pc, 4, true);
                    r0.f(yv);
                    if (a.dt_f32) {
                        Raw4<float> rd;
                        rd.load(rD + tl * CPW + pc, 4, true);
                        rd.f(r);
                    } else {
                        Raw4<T> rd;
                        rd.load(reinterpret_cast<T *>(rD) + tl * CPW + pc, 4, true);
                        rd.f(r);
                    }
                    if (gated) {
                        r0.load(rZ + tl * CPW + pc, 4, true);
                        r0.f(zv);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < nc) {
                            v[2 * i] = sel_softplus(r[i] + bias[i]);
                            v[2 * i + 1] = gated ? yv[i] * zv[i] * sigf(zv[i]) : yv[i];
                        }
                }
                float4 *o = dd + tl * (CPW / 2);                    // (odd tokens have neighbouring pairs swapped, off the banks)
                o[pc / 2 ^ (tl & 1)] = make_float4(v[0], v[1], v[2], v[3]);
                o[pc / 2 + 1 ^ (tl & 1)] = make_float4(v[4], v[5], v[6], v[7]);
            }
#pragma unroll 4
            for (int k = 0; k < F::PB; ++k) {
                const int tl = pbt + k * F::RB;
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                if (tw + tl < len) {
                    float rc[4];
                    Raw4<T> r;
                    r.load(rC + tl * NP + pn, 4, true);
                    r.f(rc);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < nn) c[i] = rc[i];
                }
                put4(Cs + tl * NP + pn, c);
            }
        }
        __syncwarp();
        if (t0 > 0) fetch(t0 - TT);
        if (tw < len) {
            const float4 *dp[2] = {dd + cp0 / 2, dd + (cp0 / 2 ^ 1)};   // even and odd tokens
            const float *cp = Cs + q * S;
#pragma unroll 4
            for (int t = TK - 1; t >= 0; --t) {
                const float4 v = dp[t & 1][t * (CPW / 2)];
                sum0 += v.x;
                sum1 += v.z;
                const f32x2 dt0 = pk2(v.x, v.x), y0 = pk2(v.y, v.y), dt1 = pk2(v.z, v.z), y1 = pk2(v.w, v.w);
                const ulonglong2 *c = reinterpret_cast<const ulonglong2 *>(cp + t * NP);
#pragma unroll
                for (int i = 0; i < S / 4; ++i) {
                    const ulonglong2 cv = c[i];
                    u[0][2 * i] = mul2(ex2x2(mul2(dt0, A2[0][2 * i])), fma2(cv.x, y0, u[0][2 * i]));
                    u[1][2 * i] = mul2(ex2x2(mul2(dt1, A2[1][2 * i])), fma2(cv.x, y1, u[1][2 * i]));
                    u[0][2 * i + 1] = mul2(ex2x2(mul2(dt0, A2[0][2 * i + 1])), fma2(cv.y, y0, u[0][2 * i + 1]));
                    u[1][2 * i + 1] = mul2(ex2x2(mul2(dt1, A2[1][2 * i + 1])), fma2(cv.y, y1, u[1][2 * i + 1]));
                }
            }
        }
        if (t0 > 0) put(t0 - TT);
        ulonglong2 *ep = reinterpret_cast<ulonglong2 *>(E) + (buf * TW + w) * CB * (NP / 4);
#pragma unroll
        for (int i = 0; i < S / 4; ++i) {
            ep[F::at(cl, q * (S / 4) + i)] = make_ulonglong2(u[0][2 * i], u[0][2 * i + 1]);
            ep[F::at(cl + 1, q * (S / 4) + i)] = make_ulonglong2(u[1][2 * i], u[1][2 * i + 1]);
        }
        if (q == 0) *reinterpret_cast<float2 *>(Sd + (buf * TW + w) * CB + cl) = make_float2(sum0, sum1);
        __syncthreads();   // (the other buffer's joining is over: its threads are here)
        if (joins) {
            ulonglong2 fold[TW];
            float sd[TW];
#pragma unroll
            for (int k = 0; k < TW; ++k) {
                fold[k] = *(reinterpret_cast<const ulonglong2 *>(E) + (buf * TW + k) * CB * (NP / 4) + F::at(jc, jn / 4));
                sd[k] = Sd[(buf * TW + k) * CB + jc];
            }
#pragma unroll
            for (int k = TW - 1; k >= 0; --k) {
                const int te = t0 + (k + 1) * TK;                   // the k-th warp's tokens end here
                if (!a.ends && te % SEL_Q == 0 && te - SEL_Q < len && d0 + jc < dend) {
                    const int slot = sq.slot0 + te / SEL_Q - 1;
                    if (slot < a.nslots)
                        *reinterpret_cast<ulonglong2 *>(a.adj + ((int64_t)slot * a.channels + d0 + jc) * NP + jn) =
                            make_ulonglong2(ju[0], ju[1]);
                }
                const f32x2 sd2 = pk2(sd[k], sd[k]);
                jsum += sd[k];
                ju[0] = fma2(ex2x2(mul2(sd2, jA[0])), ju[0], fold[k].x);
                ju[1] = fma2(ex2x2(mul2(sd2, jA[1])), ju[1], fold[k].y);
            }
        }
    }
    if (!joins || d0 + jc >= dend) return;
    if (a.ends) {
        const int64_t at = ((int64_t)s * a.nseg + seg) * a.channels + d0 + jc;
        *reinterpret_cast<ulonglong2 *>(a.segE + at * NP + jn) = make_ulonglong2(ju[0], ju[1]);
        if (jn == 0) a.segS[at] = jsum;
        return;
    }
    if (a.dinit == nullptr || seg > 0) return;
    float v[4];
    up2(ju[0], v[0], v[1]);
    up2(ju[1], v[2], v[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (jn + e < N) st_st(a.dinit, a.dinit_bf16, ((int64_t)s * a.channels + d0 + jc) * N + jn + e, v[e]);
}

// ---- the gradients.  A block takes one chunk of SEL_Q tokens and a set of channels: warp w has the
// w-th GT tokens, a thread four states of one channel, and the block goes through its channels GC at a
// time, in IT steps of 128 / NP.  The thread's B, C, dB and dC (GT tokens x four states of each) stay in
// registers for the block's life: shared memory hands a thread one value a cycle, and would be the
// bound.  For each GC channels the warps first sweep their tokens from zero (the state forwards, the
// adjoint backwards), the ends are joined with what enters the chunk, and then the warps sweep again
// from what really enters their tokens; the next channels' inputs come in the background.
// 2 x 2048 tokens x 4096 channels, dstate 16, bf16: 393 us for 420 MB (62 us of HBM), instructions in 55% of
// the cycles with 12 warps an SM (168 registers a thread), shared memory busy for 55%.  One step between
// barriers instead of four took 900 us for the whole training step, instead of 743; dB and dC in shared memory 1009.
constexpr int GT = 4, GW = SEL_Q / GT, GNT = 32 * GW, IT = 4;   // tokens a warp, warps, threads, steps
constexpr int GOCC = 3;   // blocks per SM: the whole backward and forward at the size above took 795 us with two, 727 with three, 927 with four (spills)
template <typename T, int NP>
struct Grad {
    static constexpr int TPC = NP / 4, CPW = 32 / TPC, GC = IT * CPW, OP = GC + (CPW > 4 ? CPW : 4);   // (OP: row of the sums, off the banks)
    float4 sv[SEL_Q * GC];             // dt, dt x, dyp, softplus' of (token, channel), four channels of a row swapped by place()
    float As[GC * NP];                 // A log2(e)
    float EX[2][IT][GW][128];          // state and adjoint: what the warps end with, then what enters their tokens
    float DA[IT][GW][128];             // shares of dA
    float ov[3][SEL_Q * OP];           // the sums over the states: C.h, e, f
    float Sd[IT][GW][32];              // sums of dt
    float2 red[2][GW][GC];             // shares of dD and ddt_bias, of this and the last channels
    T rx[2][SEL_Q * GC], ry[2][SEL_Q * GC], rz[2][SEL_Q * GC];   // the inputs as they come, of these and the next channels
    float rd[2][SEL_Q * GC];           // dt: fp32 or T
    float rA[2][GC * NP], rh[2][GC * NP], ru[2][GC * NP];   // A, and the state and adjoint that enter the chunk
    // where channel c of a token lies: a thread writes four neighbours, eight threads neighbouring fours
    static __device__ __forceinline__ int place(int c) { return c ^ (c >> 3 & 3); }
};

template <typename T, int NP, bool VEC>
__global__ void __launch_bounds__(GNT, GOCC) k_sel_grad(const SelArgs a) {
    after_previous();
    using G = Grad<T, NP>;
    constexpr int TPC = G::TPC, CPW = G::CPW, GC = G::GC, OP = G::OP;
    extern __shared__ __align__(16) uint8_t sel_sm[];
    G &m = *reinterpret_cast<G *>(sel_sm);
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
    // the elementwise steps: this thread's token and first channel of those staged
    const int pt = tid / (GC / 4), pc = 4 * (tid % (GC / 4)), po = pt * GC + pc;
    const bool tok = pt < n_tok, vec = VEC || a.vec, gated = a.z != nullptr;
    const int64_t rt = r0 + (tok ? pt : 0);
    const T *x = static_cast<const T *>(a.x) + sq.b * a.xb + rt * a.xt + pc;
    const T *dy = static_cast<const T *>(a.dy) + sq.b * a.dyb + rt * a.dyt + pc;
    const T *z = gated ? static_cast<const T *>(a.z) + sq.b * a.zb + rt * a.zt + pc : nullptr;
    T *dx = static_cast<T *>(a.dx) + sq.b * a.dxb + rt * a.dxt + pc;
    T *dz = gated ? static_cast<T *>(a.dz) + sq.b * a.dzb + rt * a.dzt + pc : nullptr;
    const int64_t dt0 = sq.b * a.dtb + rt * a.dtt + pc, ddt0 = sq.b * a.ddtb + rt * a.ddtt + pc;
    const int64_t e0 = (int64_t)slot * a.channels * NP + tid * 4;   // this thread's four (channel, state) of IT x 32 fours

    f32x2 Bv[GT][2], Cv[GT][2], aB[GT][2], aC[GT][2];               // B and C, and this thread's dB and dC
#pragma unroll
    for (int t = 0; t < GT; ++t) {
        const bool in = w * GT + t < n_tok;
        const int64_t row = r0 + w * GT + t;
        float b[4], c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = q * 4 + e;
            b[e] = in && n < N ? to_f(static_cast<const T *>(a.B)[sq.b * a.Bb + row * a.Bt + g * a.Bg + n]) : 0.f;
            c[e] = in && n < N ? to_f(static_cast<const T *>(a.C)[sq.b * a.Cb + row * a.Ct + g * a.Cg + n]) : 0.f;
        }
        Bv[t][0] = pk2(b[0], b[1]); Bv[t][1] = pk2(b[2], b[3]);
        Cv[t][0] = pk2(c[0], c[1]); Cv[t][1] = pk2(c[2], c[3]);
        aB[t][0] = aB[t][1] = aC[t][0] = aC[t][1] = 0;
    }
    auto count = [&](int cb) { return tok ? min(max(c_hi - cb - pc, 0), 4) : 0; };
    const int xs = (int)a.xt * (int)sizeof(T), ys = (int)a.dyt * (int)sizeof(T), zs = (int)a.zt * (int)sizeof(T);
    const int ds = (int)a.dtt * (a.dt_f32 ? 4 : (int)sizeof(T));
    Rows<SEL_Q, GC, GNT, T> lx, ly, lz, ld;
    Rows<SEL_Q, GC, GNT, float> lf;
    auto fetch = [&](int cb, int k) {                               // the inputs of channels cb.., in the background
        const int nc = count(cb);
        if (!vec) {                                                 // (element by element; the copies end in put())
            const int nw = min(c_hi - cb, GC);
            const T *x0 = static_cast<const T *>(a.x) + sq.b * a.xb + r0 * a.xt + cb, *y0 = static_cast<const T *>(a.dy) + sq.b * a.dyb + r0 * a.dyt + cb;
            lx.load(m.rx[k], x0, xs, n_tok, nw, tid);
            ly.load(m.ry[k], y0, ys, n_tok, nw, tid);
            if (gated) lz.load(m.rz[k], static_cast<const T *>(a.z) + sq.b * a.zb + r0 * a.zt + cb, zs, n_tok, nw, tid);
            const int64_t d0 = sq.b * a.dtb + r0 * a.dtt + cb;
            if (a.dt_f32) lf.load(m.rd[k], static_cast<const float *>(a.dt) + d0, ds, n_tok, nw, tid);
            else ld.load(reinterpret_cast<T *>(m.rd[k]), static_cast<const T *>(a.dt) + d0, ds, n_tok, nw, tid);
            return;
        }
        if (pt >= SEL_Q) return;
        fetch4(m.rx[k] + po, x + cb, nc, vec);
        fetch4(m.ry[k] + po, dy + cb, nc, vec);
        if (gated) fetch4(m.rz[k] + po, z + cb, nc, vec);
        if (a.dt_f32) fetch4(m.rd[k] + po, static_cast<const float *>(a.dt) + dt0 + cb, nc, vec);
        else fetch4(reinterpret_cast<T *>(m.rd[k]) + po, static_cast<const T *>(a.dt) + dt0 + cb, nc, vec);
    };
    auto put = [&](int cb, int k) {
        if (vec) return;
        const int nw = min(c_hi - cb, GC);
        lx.store(m.rx[k], n_tok, nw, tid);
        ly.store(m.ry[k], n_tok, nw, tid);
        if (gated) lz.store(m.rz[k], n_tok, nw, tid);
        if (!a.dt_f32) ld.store(reinterpret_cast<T *>(m.rd[k]), n_tok, nw, tid);
    };
    auto fetch_own = [&](int cb, int k) {                           // this thread's four of A and of what enters the chunk
        const int c = cb + tid * 4 / NP;
        if (c < c_hi) {
            fetch4(m.rA[k] + tid * 4, a.A + (int64_t)c * N + tid * 4 % NP, min(max(N - tid * 4 % NP, 0), 4), a.vecA);
            fetch4(m.rh[k] + tid * 4, a.states + e0 + (int64_t)cb * NP, 4, true);
            fetch4(m.ru[k] + tid * 4, a.adj + e0 + (int64_t)cb * NP, 4, true);
        }
        cp_async_commit();
    };
    auto put_pD = [&](int cb, int k) {                              // the warps' shares of dD and ddt_bias
        if (tid < GC && cb + tid < c_hi) {
            float2 v = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < GW; ++i) {
                v.x += m.red[k][i][tid].x;
                v.y += m.red[k][i][tid].y;
            }
            reinterpret_cast<float2 *>(a.pD)[(int64_t)slot * a.channels + cb + tid] = v;
        }
    };

    fetch(c_lo, 0);
    put(c_lo, 0);
    fetch_own(c_lo, 0);
    int k = 0;                                                      // the buffer of these channels' inputs
    for (int cb = c_lo; cb < c_hi; cb += GC, k ^= 1) {
        const int nc = pt < SEL_Q ? count(cb) : 0;
        const bool mine = cb + tid * 4 / NP < c_hi;                 // this thread's four of A exist
        cp_async_wait_all();                                        // (a thread uses what it fetched itself, or)
        if (!vec) __syncthreads();
        float Aq[4] = {0.f, 0.f, 0.f, 0.f};
        ulonglong2 hin = make_ulonglong2(0, 0), uin = hin;
        if (mine) {
#pragma unroll
            for (int e = 0; e < 4; ++e) Aq[e] = tid * 4 % NP + e < N ? sel_rate(m.rA[k][tid * 4 + e]) : 0.f;
            hin = *reinterpret_cast<const ulonglong2 *>(m.rh[k] + tid * 4);
            uin = *reinterpret_cast<const ulonglong2 *>(m.ru[k] + tid * 4);
        }
        put4(m.As + tid * 4, Aq);
        if (pt < SEL_Q) {
            float xv[4], yv[4], zv[4], r[4];
            Raw4<T> r1;
            r1.load(m.rx[k] + po, 4, true);
            r1.f(xv);
            r1.load(m.ry[k] + po, 4, true);
            r1.f(yv);
            if (gated) {
                r1.load(m.rz[k] + po, 4, true);
                r1.f(zv);
            }
            if (a.dt_f32) {
                Raw4<float> rd;
                rd.load(m.rd[k] + po, 4, true);
                rd.f(r);
            } else {
                r1.load(reinterpret_cast<const T *>(m.rd[k]) + po, 4, true);
                r1.f(r);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < nc) {
                    const float raw = r[i] + (a.bias ? a.bias[cb + pc + i] : 0.f);
                    v.x = sel_softplus(raw);
                    v.y = v.x * xv[i];
                    v.z = gated ? yv[i] * zv[i] * sigf(zv[i]) : yv[i];
                    v.w = sigf(raw);
                }
                m.sv[pt * GC + G::place(pc + i)] = v;
            }
        }
        __syncthreads();
        if (cb > c_lo) put_pD(cb - GC, k ^ 1);
        if (cb + GC < c_hi) {
            fetch(cb + GC, k ^ 1);
            fetch_own(cb + GC, k ^ 1);
        }
        // from zero
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int c = it * CPW + cw;
            const ulonglong2 av = *reinterpret_cast<const ulonglong2 *>(m.As + c * NP + q * 4);
            const float4 *vp = m.sv + w * GT * GC + G::place(c);
            f32x2 al[GT][2], h[2] = {0, 0}, u[2] = {0, 0};
            float sum = 0.f, yv[GT];
#pragma unroll
            for (int t = 0; t < GT; ++t) {
                const float4 v = vp[t * GC];
                const f32x2 dt2 = pk2(v.x, v.x), dx2 = pk2(v.y, v.y);
                yv[t] = v.z;
                sum += v.x;
                al[t][0] = ex2x2(mul2(dt2, av.x));
                al[t][1] = ex2x2(mul2(dt2, av.y));
                h[0] = fma2(al[t][0], h[0], mul2(dx2, Bv[t][0]));
                h[1] = fma2(al[t][1], h[1], mul2(dx2, Bv[t][1]));
            }
#pragma unroll
            for (int t = GT - 1; t >= 0; --t) {
                const f32x2 dy2 = pk2(yv[t], yv[t]);
                u[0] = mul2(al[t][0], fma2(Cv[t][0], dy2, u[0]));
                u[1] = mul2(al[t][1], fma2(Cv[t][1], dy2, u[1]));
            }
            *reinterpret_cast<ulonglong2 *>(&m.EX[0][it][w][lane * 4]) = make_ulonglong2(h[0], h[1]);
            *reinterpret_cast<ulonglong2 *>(&m.EX[1][it][w][lane * 4]) = make_ulonglong2(u[0], u[1]);
            if (q == 0) m.Sd[it][w][cw] = sum;
        }
        if (cb + GC < c_hi) put(cb + GC, k ^ 1);
        __syncthreads();
        {                                                           // warp w joins step w: the state onwards, the adjoint backwards
            ulonglong2 eh[GW], eu[GW];
            float sd[GW];
            const f32x2 A0 = pk2(Aq[0], Aq[1]), A1 = pk2(Aq[2], Aq[3]);
#pragma unroll
            for (int i = 0; i < GW; ++i) {
                eh[i] = *reinterpret_cast<const ulonglong2 *>(&m.EX[0][w][i][lane * 4]);
                eu[i] = *reinterpret_cast<const ulonglong2 *>(&m.EX[1][w][i][lane * 4]);
                sd[i] = m.Sd[w][i][cw];
            }
            f32x2 d0[GW], d1[GW];
#pragma unroll
            for (int i = 0; i < GW; ++i) {
                const f32x2 sd2 = pk2(sd[i], sd[i]);
                d0[i] = ex2x2(mul2(sd2, A0));
                d1[i] = ex2x2(mul2(sd2, A1));
            }
#pragma unroll
            for (int i = 0; i < GW; ++i) {
                const int l = GW - 1 - i;
                *reinterpret_cast<ulonglong2 *>(&m.EX[0][w][i][lane * 4]) = hin;
                *reinterpret_cast<ulonglong2 *>(&m.EX[1][w][l][lane * 4]) = uin;
                hin.x = fma2(d0[i], hin.x, eh[i].x);
                hin.y = fma2(d1[i], hin.y, eh[i].y);
                uin.x = fma2(d0[l], uin.x, eu[l].x);
                uin.y = fma2(d1[l], uin.y, eu[l].y);
            }
        }
        __syncthreads();
        // from what enters
#pragma unroll 1
        for (int it = 0; it < IT; ++it) {
            const int c = it * CPW + cw;
            const ulonglong2 av = *reinterpret_cast<const ulonglong2 *>(m.As + c * NP + q * 4);
            const ulonglong2 hv = *reinterpret_cast<const ulonglong2 *>(&m.EX[0][it][w][lane * 4]);
            const ulonglong2 uv = *reinterpret_cast<const ulonglong2 *>(&m.EX[1][it][w][lane * 4]);
            const float4 *vp = m.sv + w * GT * GC + G::place(c);
            f32x2 al[GT][2], h[GT + 1][2], u[2] = {uv.x, uv.y}, dA[2] = {0, 0};
            h[0][0] = hv.x;
            h[0][1] = hv.y;
            float ys[GT], es[GT], fs[GT];
            f32x2 dt2[GT], dx2[GT], dy2[GT];
#pragma unroll
            for (int t = 0; t < GT; ++t) {
                const float4 v = vp[t * GC];
                dt2[t] = pk2(v.x, v.x);
                dx2[t] = pk2(v.y, v.y);
                dy2[t] = pk2(v.z, v.z);
                al[t][0] = ex2x2(mul2(dt2[t], av.x));
                al[t][1] = ex2x2(mul2(dt2[t], av.y));
                h[t + 1][0] = fma2(al[t][0], h[t][0], mul2(dx2[t], Bv[t][0]));
                h[t + 1][1] = fma2(al[t][1], h[t][1], mul2(dx2[t], Bv[t][1]));
                ys[t] = sum2(fma2(h[t + 1][1], Cv[t][1], mul2(h[t + 1][0], Cv[t][0])));
                aC[t][0] = fma2(h[t + 1][0], dy2[t], aC[t][0]);
                aC[t][1] = fma2(h[t + 1][1], dy2[t], aC[t][1]);
            }
#pragma unroll
            for (int t = GT - 1; t >= 0; --t) {
                const f32x2 g0 = fma2(Cv[t][0], dy2[t], u[0]), g1 = fma2(Cv[t][1], dy2[t], u[1]);
                aB[t][0] = fma2(g0, dx2[t], aB[t][0]);
                aB[t][1] = fma2(g1, dx2[t], aB[t][1]);
                es[t] = sum2(fma2(g1, Bv[t][1], mul2(g0, Bv[t][0])));
                u[0] = mul2(al[t][0], g0);
                u[1] = mul2(al[t][1], g1);
                const f32x2 k0 = mul2(u[0], h[t][0]), k1 = mul2(u[1], h[t][1]);
                dA[0] = fma2(k0, dt2[t], dA[0]);
                dA[1] = fma2(k1, dt2[t], dA[1]);
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
                const int o = (w * GT + q) * OP + c;
                m.ov[0][o] = yq;
                m.ov[1][o] = eq;
                m.ov[2][o] = fq;
            }
            *reinterpret_cast<ulonglong2 *>(&m.DA[it][w][lane * 4]) = make_ulonglong2(dA[0], dA[1]);
        }
        __syncthreads();
        if (mine) {                                                 // warp w: step w's dA, over the warps' tokens
            f32x2 v0 = 0, v1 = 0;
#pragma unroll
            for (int i = 0; i < GW; ++i) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(&m.DA[w][i][lane * 4]);
                v0 = add2(v0, v.x);
                v1 = add2(v1, v.y);
            }
            *reinterpret_cast<ulonglong2 *>(a.pA + e0 + (int64_t)cb * NP) = make_ulonglong2(v0, v1);
        }
        float sD[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
        if (nc > 0) {
            float xv[4], yv[4], zv[4], ox[4], ot[4], oz[4], ya[4], ea[4], fa[4];
            const int o = pt * OP + pc;
            Raw4<T> r1;
            r1.load(m.rx[k] + po, 4, true);
            r1.f(xv);
            if (gated) {
                r1.load(m.ry[k] + po, 4, true);
                r1.f(yv);
                r1.load(m.rz[k] + po, 4, true);
                r1.f(zv);
            }
            Raw4<float> rv;
            rv.load(m.ov[0] + o, 4, true);
            rv.f(ya);
            rv.load(m.ov[1] + o, 4, true);
            rv.f(ea);
            rv.load(m.ov[2] + o, 4, true);
            rv.f(fa);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ox[i] = ot[i] = oz[i] = 0.f;
                if (i < nc) {
                    const float4 v = m.sv[pt * GC + G::place(pc + i)];
                    const float Dv = a.D ? a.D[cb + pc + i] : 0.f;
                    ox[i] = fmaf(ea[i], v.x, a.D ? Dv * v.z : 0.f);
                    ot[i] = fmaf(ea[i], xv[i], fa[i] * 0.6931471805599453f) * v.w;   // (f was summed with A log2(e))
                    if (gated) {
                        const float sg = sigf(zv[i]);
                        oz[i] = yv[i] * (a.D ? fmaf(Dv, xv[i], ya[i]) : ya[i]) * sg * fmaf(zv[i], 1.f - sg, 1.f);
                    }
                    sD[i] = v.z * xv[i];
                    sb[i] = ot[i];
                }
            }
            store4(dx + cb, ox, nc, a.vec_out);
            if (a.dt_f32) store4(static_cast<float *>(a.ddt) + ddt0 + cb, ot, nc, a.vec_out);
            else store4(static_cast<T *>(a.ddt) + ddt0 + cb, ot, nc, a.vec_out);
            if (gated) store4(dz + cb, oz, nc, a.vec_out);
        }
        // the chunk's share of dD and ddt_bias: over the warp's tokens (GC / 4 lanes each); the warps' below
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int o = GC / 4; o < 32; o <<= 1) {
                sD[i] += __shfl_xor_sync(0xffffffffu, sD[i], o);
                sb[i] += __shfl_xor_sync(0xffffffffu, sb[i], o);
            }
            if (lane < GC / 4) m.red[k][w][pc + i] = make_float2(sD[i], sb[i]);
        }
        __syncthreads();                                            // sv, ov and DA are free
    }
    put_pD(c_lo + (c_hi - c_lo - 1) / GC * GC, k ^ 1);
    // dB and dC of this channel set: over the warp's channels, then one row of NP values a token
    const int64_t rows = (int64_t)a.nbatch * a.seqlen * a.ngroups;
#pragma unroll
    for (int t = 0; t < GT; ++t) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int o = TPC; o < 32; o <<= 1) {
                aB[t][i] = add2(aB[t][i], __shfl_xor_sync(0xffffffffu, aB[t][i], o));
                aC[t][i] = add2(aC[t][i], __shfl_xor_sync(0xffffffffu, aC[t][i], o));
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

// The sums of the shares, each in a fixed order.  dA, dD and ddt_bias: a block takes 32 columns; warp w sums the
// chunk slots w, w + 8, ... in order, and the eight sums are added in order.  dB and dC (the blocks after
// them): a thread sums one value's channel sets in order.  86 MB of shares at 2 x 2048 tokens x 4096 channels in 19 us
// (4.5 TB/s); a launch for each kind took 2 us more in a call of 110.
template <typename T>
__global__ void __launch_bounds__(256) k_sel_sums(const SelArgs a, int64_t blocksA, int64_t blocksAD) {
    after_previous();
    __shared__ float red[8][32];
    if (blockIdx.x >= blocksAD) {
        const int64_t rows = (int64_t)a.nbatch * a.seqlen * a.ngroups, per = rows * a.NP;
        const int64_t i = (blockIdx.x - blocksAD) * 256 + threadIdx.x;
        if (i >= 2 * per) return;
        const int64_t row = i % per / a.NP;
        const int n = (int)(i % a.NP), which = i >= per;
        if (n >= a.N) return;
        float v = 0.f;
#pragma unroll 4
        for (int k = 0; k < a.nsets; ++k) v += a.pBC[k * 2 * per + i];
        const int g = (int)(row % a.ngroups);
        const int64_t tok = row / a.ngroups, b = tok / a.seqlen, t = tok % a.seqlen;
        if (which) static_cast<T *>(a.dC)[b * a.dCb + t * a.dCt + g * a.dCg + n] = from_f<T>(v);
        else static_cast<T *>(a.dB)[b * a.dBb + t * a.dBt + g * a.dBg + n] = from_f<T>(v);
        return;
    }
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

template <typename T, typename F, bool VEC>
cudaError_t launch_rev_rows(const SelArgs &a, cudaStream_t st) {
    static int attr[64] = {0};
    const size_t sm = F::template smem<T>(a.dt_f32);
    cudaError_t e = ensure_smem_attr(k_sel_rev<T, F, VEC>, (int)sm, attr);
    if (e != cudaSuccess) return e;
    const int cblocks = a.ngroups * ((a.dpg + F::CB - 1) / F::CB);
    return launch_early(k_sel_rev<T, F, VEC>, (unsigned)((int64_t)a.nseqs * a.nseg * cblocks), F::NT, sm, st, a, cblocks);
}
template <typename T, typename F>
cudaError_t launch_rev(const SelArgs &a, cudaStream_t st) {
    return a.vec && a.vecBC ? launch_rev_rows<T, F, true>(a, st) : launch_rev_rows<T, F, false>(a, st);
}
template <typename T, int NP, bool VEC>
cudaError_t launch_grad_rows(const SelArgs &a, cudaStream_t st) {
    static int attr[64] = {0};
    cudaError_t e = ensure_smem_attr(k_sel_grad<T, NP, VEC>, (int)sizeof(Grad<T, NP>), attr);
    if (e != cudaSuccess) return e;
    return launch_early(k_sel_grad<T, NP, VEC>, (unsigned)((int64_t)a.nslots * a.ngroups * a.nsets), GNT, sizeof(Grad<T, NP>), st, a);
}

template <typename T, int NP>
cudaError_t launch_grad(const SelArgs &a, cudaStream_t st) {
    return a.vec ? launch_grad_rows<T, NP, true>(a, st) : launch_grad_rows<T, NP, false>(a, st);
}

template <typename T>
cudaError_t rev(const SelArgs &a, cudaStream_t st) {
    switch (a.NP) {
        case 16: return launch_rev<T, RevCfg<4, 4, 1, 8, 16, 2>>(a, st);
        case 32: return launch_rev<T, RevCfg<8, 4, 1, 8, 16, 2>>(a, st);
        case 64: return launch_rev<T, RevCfg<8, 8, 1, 4, 16, 3>>(a, st);
        default: return launch_rev<T, RevCfg<8, 16, 1, 4, 16, 2>>(a, st);
    }
}
template <typename T>
cudaError_t run_bwd(const SelArgs &a, cudaStream_t st) {
    cudaError_t e;
    if (a.nseg > 1) {
        SelArgs b = a;
        b.ends = true;
        e = rev<T>(b, st);
        if (e != cudaSuccess) return e;
    }
    e = rev<T>(a, st);
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
    const int64_t bA = ((int64_t)a.channels * a.NP + 31) / 32, bD = ((int64_t)a.channels * 2 + 31) / 32;
    return launch_early(k_sel_sums<T>, (unsigned)(bA + bD + (n + 255) / 256), 256, 0, st, a, bA, bA + bD);
}

}  // namespace

// Channels per set: those for which the card's rounds of blocks (GOCC on each SM), each as long as its channels and
// a start worth 16 more (a block loads B and C and fills its pipeline), are over soonest.  At most 256: a set's own shares
// of dB and dC cost little by then.  Measured, training, dstate 16, bf16, by this rule / halving from 256 until
// eight blocks are there for each SM / until four are: 1 x 256 x 4096 59 / 73 / 65 us, 1 x 512 x 2048 63 / 73 / 67,
// 1 x 2048 x 1024 132 / 134 / 132, 4 x 1024 x 512 122 / 122 / 121, 2 x 2048 x 4096 704 with each.
void sel_bwd_sets(int channels, int ngroups, int64_t nslots, int *nsets, int *cps) {
    const int dpg = channels / ngroups;
    int64_t best = INT64_MAX;
    for (int c = 256; c >= 32; c -= 32) {
        const int n = (dpg + c - 1) / c;
        const int64_t rounds = (nslots * ngroups * n + kSMs * GOCC - 1) / (kSMs * GOCC), cost = rounds * (std::min(c, dpg) + 16);
        if (cost < best) {
            best = cost;
            *nsets = n;
            *cps = c;
        }
    }
}

cudaError_t sel_launch_bwd(SelArgs a, bool bf16, cudaStream_t st) {
    return bf16 ? run_bwd<__nv_bfloat16>(a, st) : run_bwd<float>(a, st);
}

}  // namespace ssd
