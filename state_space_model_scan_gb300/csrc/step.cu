// step.cu -- one token of the recurrence for each of a batch of requests, on a pool of states:
//
//   h <- exp(dt A) h + dt x B,   y = (C.h + D x) silu(z),   dt = softplus(dt_raw + dt_bias)
//
// with one A per head (ssd_step) or one per channel and state (ssd_selective_step).  Every state
// value is read once and written once and takes part in a handful of operations, so memory
// bounds it.  A row of dstate state values belongs to LPR lanes, each with NV pieces of V values (16
// bytes where rows allow it).  A thread issues the loads of RU pieces before it uses the first: of RU
// rows of one head, which share B, C, A and dt, or, in the selective form, of one row of RU requests,
// which share A.
//
// Measured: 256 requests x 80 heads x 64 x 128, bf16 states, 107 us for 676 MB (6.3 TB/s, 92% of a plain
// copy); 192 requests x 8192 channels x 16, fp32 states, 39.6 us for 215 MB (5.4 TB/s, 80%): an exponential for
// each value and a softplus for sixteen keep the issue slots 70% busy.  One request of 64 heads: 4 us, the launch.
#include <algorithm>

#include "selective.cuh"

namespace ssd {

namespace {

constexpr int ST_NT = 64;

struct StepArgs {
    void *state;
    const int32_t *idx;
    const void *x, *dt, *B, *C, *z;
    const float *A, *D, *bias;
    void *y;
    int nslots;                          // at most 2^31 - 1: slots are found by 32-bit indices
    int64_t slot_stride, xs, dts, zs, bs, cs, ys;
    int batch, segs, rows, spg, N;       // segments, rows of each, segments per B/C group
    int lpr, nrb;                        // lanes per row (a power of two), row blocks per segment
    bool dt_f32;
};

template <int V>
struct Piece {
    float v[V];
};
// A piece as it lies in memory: one value, or V = 4 or 8 of them in one or two accesses (bf16 stay packed
// until they are used, half the registers of the loads in flight).
template <typename U, int V>
struct Raw {
    uint32_t w[V * sizeof(U) / 4];
    __device__ __forceinline__ void load(const U *p) {
        if constexpr (V * sizeof(U) == 8) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x; w[1] = u.y;
        } else {
#pragma unroll
            for (int i = 0; i < (int)(V * sizeof(U) / 16); ++i) {
                const uint4 u = reinterpret_cast<const uint4 *>(p)[i];
                w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ float f(int e) const {
        if constexpr (sizeof(U) == 4) return __uint_as_float(w[e]);
        else return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
};
template <typename U>
struct Raw<U, 1> {
    U w;
    __device__ __forceinline__ void load(const U *p) { w = *p; }
    __device__ __forceinline__ float f(int) const { return to_f(w); }
};
template <int V>
__device__ __forceinline__ void stp(float *p, const Piece<V> &o) {
    if constexpr (V == 1) *p = o.v[0];
    else *reinterpret_cast<float4 *>(p) = make_float4(o.v[0], o.v[1], o.v[2], o.v[3]);
}
template <int V>
__device__ __forceinline__ void stp(__nv_bfloat16 *p, const Piece<V> &o) {
    if constexpr (V == 1) {
        *p = __float2bfloat16_rn(o.v[0]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(o.v[2 * i], o.v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

__device__ __forceinline__ int64_t slot_of(const StepArgs &a, int b) {
    const int s = a.idx ? a.idx[b] : b;
    return (unsigned)s < (unsigned)a.nslots ? s : -1;
}
template <typename T>
__device__ __forceinline__ float raw_dt(const StepArgs &a, int64_t at, int64_t par) {
    return (a.dt_f32 ? static_cast<const float *>(a.dt)[at] : to_f(static_cast<const T *>(a.dt)[at])) + (a.bias ? a.bias[par] : 0.f);
}

// One rate per head.  T: type of x, B, C, z, y.  ST: of the state.  Segments are heads.
template <typename T, typename ST, int V, int NV, int RU>
__global__ void __launch_bounds__(ST_NT) k_step_head(const StepArgs a) {
    after_previous();
    const int rb = blockIdx.x % a.nrb, bs = blockIdx.x / a.nrb, seg = bs % a.segs, b = bs / a.segs;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int l = lane & (a.lpr - 1), rpw = 32 / a.lpr;             // lane of the row, rows of a warp
    const int r0 = (rb * (ST_NT / 32) + w) * rpw * RU + lane / a.lpr;
    const int N = a.N;
    const int64_t first = (int64_t)seg * a.rows;                    // the head's first row
    T *y = static_cast<T *>(a.y) + b * a.ys + first;
    const int64_t slot = slot_of(a, b);
    if (slot < 0) {                                                 // padding
        for (int u = 0; u < RU; ++u)
            if (l == 0 && r0 + u * rpw < a.rows) y[r0 + u * rpw] = from_f<T>(0.f);
        return;
    }
    ST *st = static_cast<ST *>(a.state) + slot * a.slot_stride + first * N;
    const T *x = static_cast<const T *>(a.x) + b * a.xs + first;
    // every load first: the stores below would hold up later ones
    Raw<ST, V> h[RU][NV];
    Raw<T, V> Bv[NV], Cv[NV];
    float xv[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u)
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int n = (k * a.lpr + l) * V, r = r0 + u * rpw;
            if (r < a.rows && n < N) h[u][k].load(st + (int64_t)r * N + n);
        }
    const float raw = raw_dt<T>(a, b * a.dts + seg, seg), A = a.A[seg];
#pragma unroll
    for (int u = 0; u < RU; ++u) xv[u] = r0 + u * rpw < a.rows ? to_f(x[r0 + u * rpw]) : 0.f;
    const int64_t bc = (int64_t)(seg / a.spg) * N;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int n = (k * a.lpr + l) * V;
        if (n < N) {
            Bv[k].load(static_cast<const T *>(a.B) + b * a.bs + bc + n);
            Cv[k].load(static_cast<const T *>(a.C) + b * a.cs + bc + n);
        }
    }
    // where a row has at least RU lanes, lane u finishes row u; else its first lane every row
    const bool spread = a.lpr >= RU;
    const int ru = r0 + l * rpw;
    const bool fin = spread && l < RU && ru < a.rows;
    const float D = a.D ? a.D[seg] : 0.f;
    float zu = 0.f, xu = 0.f;
    if (fin) {
        xu = to_f(x[ru]);
        if (a.z) zu = to_f(static_cast<const T *>(a.z)[b * a.zs + first + ru]);
    }
    const float dt = sel_softplus(raw), decay = ex2f(dt * A * kLog2e);
    float acc[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
        const int r = r0 + u * rpw;
        const float dtx = dt * xv[u];
        acc[u] = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int n = (k * a.lpr + l) * V;
            if (r < a.rows && n < N) {
                Piece<V> o;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    o.v[e] = fmaf(decay, h[u][k].f(e), dtx * Bv[k].f(e));
                    acc[u] = fmaf(Cv[k].f(e), o.v[e], acc[u]);
                }
                stp<V>(st + (int64_t)r * N + n, o);
            }
        }
    }
    if (spread) {
        float v = reduce_scatter<RU>(acc, l & (RU - 1));
        for (int o = RU; o < a.lpr; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (fin) {
            if (a.D) v = fmaf(D, xu, v);
            y[ru] = from_f<T>(a.z ? sel_gate<T>(v, zu) : v);
        }
    } else {
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            for (int o = a.lpr >> 1; o > 0; o >>= 1) acc[u] += __shfl_xor_sync(0xffffffffu, acc[u], o);
            const int r = r0 + u * rpw;
            if (l == 0 && r < a.rows) {
                float v = a.D ? fmaf(D, xv[u], acc[u]) : acc[u];
                if (a.z) v = sel_gate<T>(v, to_f(static_cast<const T *>(a.z)[b * a.zs + first + r]));
                y[r] = from_f<T>(v);
            }
        }
    }
}

// One rate per channel and state.  Segments are B/C groups, rows channels; a thread takes one row of RU
// requests.  Lane u of a row that has RU lanes reads, softens and finishes request u for all of them.  (The gate's
// factor is taken after the sums: before them it waits for z, 47 us instead of 39.6 at the size above; and 88
// registers instead of 80, one block fewer on an SM, 42.)
template <typename T, typename ST, int V, int NV, int RU>
__global__ void __launch_bounds__(ST_NT, sizeof(T) == 2 && V * RU == 16 ? 12 : 1) k_step_channel(const StepArgs a) {
    after_previous();
    const int rb = blockIdx.x % a.nrb, bs = blockIdx.x / a.nrb, seg = bs % a.segs, b0 = bs / a.segs * RU;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int l = lane & (a.lpr - 1), rpw = 32 / a.lpr;
    const int r = (rb * (ST_NT / 32) + w) * rpw + lane / a.lpr;     // the row within its group
    const int N = a.N;
    const bool in = r < a.rows, spread = a.lpr >= RU;
    const int64_t c = (int64_t)seg * a.rows + min(r, a.rows - 1);   // the channel
    // Loads need no branch: what lies outside (rows, requests, slots, lanes past N) reads a place inside
    // instead, and is not stored.  (nslots is 1 at least: the launch sees to it.)
    ST *st[RU];
    bool live[RU];
    Raw<ST, V> h[RU][NV];
    Raw<float, V> Av[NV];
    Raw<T, V> Bv[RU][NV], Cv[RU][NV];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
        const int b = min(b0 + u, a.batch - 1), slot = a.idx ? a.idx[b] : b;
        live[u] = in && b0 + u < a.batch && (unsigned)slot < (unsigned)a.nslots;
        st[u] = static_cast<ST *>(a.state) + (live[u] ? slot : 0) * a.slot_stride + c * N;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int n0 = (k * a.lpr + l) * V, n = n0 < N ? n0 : 0;
#pragma unroll
        for (int u = 0; u < RU; ++u) h[u][k].load(st[u] + n);
        Av[k].load(a.A + c * N + n);
        const int64_t bc = (int64_t)seg * N + n;
        const T *Bp = static_cast<const T *>(a.B) + b0 * a.bs + bc, *Cp = static_cast<const T *>(a.C) + b0 * a.cs + bc;
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            Bv[u][k].load(Bp);
            Cv[u][k].load(Cp);
            Bp += b0 + u + 1 < a.batch ? a.bs : 0;
            Cp += b0 + u + 1 < a.batch ? a.cs : 0;
        }
    }
    // steps, inputs and gates: this lane's request (spread), or every request
    float dt[RU], xv[RU], gate[RU];
    const float D = a.D ? a.D[c] : 0.f;
#pragma unroll
    for (int u = 0; u < RU; ++u) {
        if (spread && u > 0) break;
        const int b = min(b0 + (spread ? l & (RU - 1) : u), a.batch - 1);
        const float raw = raw_dt<T>(a, b * a.dts + c, c);
        xv[u] = to_f(static_cast<const T *>(a.x)[b * a.xs + c]);
        gate[u] = a.z ? to_f(static_cast<const T *>(a.z)[b * a.zs + c]) : 0.f;
        dt[u] = sel_softplus(raw);
    }
    float acc[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
        const float du = spread ? __shfl_sync(0xffffffffu, dt[0], u, a.lpr) : dt[u];
        const float xu = spread ? __shfl_sync(0xffffffffu, xv[0], u, a.lpr) : xv[u];
        const float dtx = du * xu, dtl = du * kLog2e;
        acc[u] = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int n = (k * a.lpr + l) * V;
            if (n < N) {
                Piece<V> o;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    o.v[e] = fmaf(ex2f(dtl * Av[k].f(e)), h[u][k].f(e), dtx * Bv[u][k].f(e));
                    acc[u] = fmaf(Cv[u][k].f(e), o.v[e], acc[u]);
                }
                if (live[u]) stp<V>(st[u] + n, o);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < RU; ++u)
        if (!spread || u == 0) gate[u] = a.z ? sel_gate<T>(1.f, gate[u]) : 1.f;
    if (spread) {
        float v = reduce_scatter<RU>(acc, l & (RU - 1));
        for (int o = RU; o < a.lpr; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        bool lv = false;
#pragma unroll
        for (int u = 0; u < RU; ++u) lv = l == u ? live[u] : lv;
        if (in && l < RU && b0 + l < a.batch) {
            if (a.D) v = fmaf(D, xv[0], v);
            static_cast<T *>(a.y)[(b0 + l) * a.ys + c] = from_f<T>(lv ? v * gate[0] : 0.f);
        }
    } else {
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            for (int o = a.lpr >> 1; o > 0; o >>= 1) acc[u] += __shfl_xor_sync(0xffffffffu, acc[u], o);
            if (in && l == 0 && b0 + u < a.batch) {
                float v = a.D ? fmaf(D, xv[u], acc[u]) : acc[u];
                static_cast<T *>(a.y)[(b0 + u) * a.ys + c] = from_f<T>(live[u] ? v * gate[u] : 0.f);
            }
        }
    }
}

// ---- the gated delta rule, one token for each request:
//
//   h <- e^g h,  u = beta (v - h k),  h <- h + u k^T,  o = scale h q
//
// Both sums over the old state are taken in one pass (o = scale (e^g h q + u k.q)), so that a value is read and
// written once: bound by memory, and a thread has eight rows of the state on the way at once (four of more than 128 keys in fp32).
// 192 requests x 32 heads x 128 x 128, fp32 states, 810 MB: 1 / 2 / 4 / 8 rows 304 / 177 / 127 / 117 us (6.9 TB/s), 4 requests
// 9.4 / 7.3 / 5.9 / 5.9, one 4.8 / 4.6 / 4.5 / 4.7; 64 requests of 256 keys, 2 / 4 rows 86 / 81.  bf16 states 78 us (5.2 TB/s).
struct DeltaStepArgs {
    void *state;
    const int32_t *idx;
    const void *q, *k, *v, *g, *beta;
    void *o;
    int nslots;
    int64_t slot_stride, qs, ks, vs, gs, bs, os;
    int batch, H, V, K, hpg;             // heads, values, keys, heads per group of keys
    int lpr, nrb;                        // lanes per row of the state, row blocks per head
    float scale;
    bool g_f32, beta_f32;
};

template <typename T, typename ST, int V, int NV, int RU>
__global__ void __launch_bounds__(ST_NT) k_step_delta(const DeltaStepArgs a) {
    after_previous();
    const int rb = blockIdx.x % a.nrb, bh = blockIdx.x / a.nrb, head = bh % a.H, b = bh / a.H;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int l = lane & (a.lpr - 1), rpw = 32 / a.lpr;
    const int r0 = (rb * (ST_NT / 32) + w) * rpw * RU + lane / a.lpr;
    T *o = static_cast<T *>(a.o) + b * a.os + (int64_t)head * a.V;
    const int slot = a.idx ? a.idx[b] : b;
    if ((unsigned)slot >= (unsigned)a.nslots) {                      // padding
        for (int u = 0; u < RU; ++u)
            if (l == 0 && r0 + u * rpw < a.V) o[r0 + u * rpw] = from_f<T>(0.f);
        return;
    }
    ST *st = static_cast<ST *>(a.state) + slot * a.slot_stride + (int64_t)head * a.V * a.K;
    Raw<ST, V> h[RU][NV];
    Raw<T, V> kv[NV], qv[NV];
#pragma unroll
    for (int u = 0; u < RU; ++u)
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int n = (c * a.lpr + l) * V, r = r0 + u * rpw;
            if (r < a.V && n < a.K) h[u][c].load(st + (int64_t)r * a.K + n);
        }
    const int64_t row = (int64_t)(head / a.hpg) * a.K;
    const T *kp = static_cast<const T *>(a.k) + b * a.ks + row, *qp = static_cast<const T *>(a.q) + b * a.qs + row;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int n = (c * a.lpr + l) * V;
        if (n < a.K) {
            kv[c].load(kp + n);
            qv[c].load(qp + n);
        }
    }
    const int64_t gat = b * a.gs + head, bat = b * a.bs + head;
    const float g = a.g_f32 ? static_cast<const float *>(a.g)[gat] : to_f(static_cast<const __nv_bfloat16 *>(a.g)[gat]);
    const float beta = a.beta_f32 ? static_cast<const float *>(a.beta)[bat] : to_f(static_cast<const __nv_bfloat16 *>(a.beta)[bat]);
    const float decay = expf(g);
    const T *vp = static_cast<const T *>(a.v) + b * a.vs + (int64_t)head * a.V;
    // where a row has at least RU lanes, lane u finishes row u; else its first lane every row
    const bool spread = a.lpr >= RU;
    float vr[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
        if (spread && u > 0) break;
        const int r = r0 + (spread ? l & (RU - 1) : u) * rpw;
        vr[u] = r < a.V ? to_f(vp[r]) : 0.f;
    }
    float hk[RU], hq[RU], kq = 0.f;
#pragma unroll
    for (int u = 0; u < RU; ++u) {
        hk[u] = hq[u] = 0.f;
        const int r = r0 + u * rpw;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int n = (c * a.lpr + l) * V;
            if (r < a.V && n < a.K) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    hk[u] = fmaf(h[u][c].f(e), kv[c].f(e), hk[u]);
                    hq[u] = fmaf(h[u][c].f(e), qv[c].f(e), hq[u]);
                }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int n = (c * a.lpr + l) * V;
        if (n < a.K) {
#pragma unroll
            for (int e = 0; e < V; ++e) kq = fmaf(kv[c].f(e), qv[c].f(e), kq);
        }
    }
    for (int s = a.lpr >> 1; s > 0; s >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, s);
    float up[RU];
    if (spread) {
        float x = reduce_scatter<RU>(hk, l & (RU - 1)), y = reduce_scatter<RU>(hq, l & (RU - 1));
        for (int s = RU; s < a.lpr; s <<= 1) {
            x += __shfl_xor_sync(0xffffffffu, x, s);
            y += __shfl_xor_sync(0xffffffffu, y, s);
        }
        const float u = beta * (vr[0] - decay * x);
        const int r = r0 + l * rpw;
        if (l < RU && r < a.V) o[r] = from_f<T>(a.scale * fmaf(decay, y, u * kq));
#pragma unroll
        for (int i = 0; i < RU; ++i) up[i] = __shfl_sync(0xffffffffu, u, i, a.lpr);
    } else {
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            for (int s = a.lpr >> 1; s > 0; s >>= 1) {
                hk[u] += __shfl_xor_sync(0xffffffffu, hk[u], s);
                hq[u] += __shfl_xor_sync(0xffffffffu, hq[u], s);
            }
            up[u] = beta * (vr[u] - decay * hk[u]);
            const int r = r0 + u * rpw;
            if (l == 0 && r < a.V) o[r] = from_f<T>(a.scale * fmaf(decay, hq[u], up[u] * kq));
        }
    }
#pragma unroll
    for (int u = 0; u < RU; ++u) {
        const int r = r0 + u * rpw;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int n = (c * a.lpr + l) * V;
            if (r < a.V && n < a.K) {
                Piece<V> p;
#pragma unroll
                for (int e = 0; e < V; ++e) p.v[e] = fmaf(up[u], kv[c].f(e), decay * h[u][c].f(e));
                stp<V>(st + (int64_t)r * a.K + n, p);
            }
        }
    }
}

void lanes(StepArgs &a, int V) {
    a.lpr = 1;
    while (a.lpr < 32 && a.lpr * V < a.N) a.lpr <<= 1;
}
// (a grid has at most 2^31 - 1 blocks)
template <typename K>
cudaError_t launch_blocks(K kernel, int64_t blocks, cudaStream_t st, const StepArgs &a) {
    if (blocks > ((int64_t)1 << 31) - 1) return cudaErrorInvalidConfiguration;
    return launch_early(kernel, (unsigned)blocks, ST_NT, 0, st, a);
}
template <typename T, typename ST, int V, int NV, int RU>
cudaError_t launch_head(StepArgs a, cudaStream_t st) {
    lanes(a, V);
    const int per = (ST_NT / 32) * (32 / a.lpr) * RU;
    a.nrb = (a.rows + per - 1) / per;
    return launch_blocks(k_step_head<T, ST, V, NV, RU>, (int64_t)a.batch * a.segs * a.nrb, st, a);
}
template <typename T, typename ST, int V, int NV, int RU>
cudaError_t launch_channel(StepArgs a, cudaStream_t st) {
    lanes(a, V);
    const int per = (ST_NT / 32) * (32 / a.lpr), nb = (a.batch + RU - 1) / RU;
    a.nrb = (a.rows + per - 1) / per;
    return launch_blocks(k_step_channel<T, ST, V, NV, RU>, (int64_t)nb * a.segs * a.nrb, st, a);
}

// Rows or requests in flight per thread: measured at 256 requests x 80 heads x 64 x 128, bf16 states, 4 / 8 /
// 16 rows 116 / 110 / 170 us; at 192 requests x 8192 channels x 16, fp32 states, 1 / 2 / 4 / 8 requests 64 / 47 / 43 / 117 us.  A
// single request takes one each, for more blocks.
// Pieces of 16 bytes of state where every row of state, B, C (and A) allows them; else single values.
template <typename T, typename ST, bool CHANNEL>
cudaError_t pick(const StepArgs &a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(ST);
    constexpr uintptr_t bcs = V * sizeof(T) < 16 ? V * sizeof(T) : 16;
    const bool vec = a.N % V == 0 && (uintptr_t)a.state % 16 == 0 && a.slot_stride % V == 0 &&
                     (!CHANNEL || (uintptr_t)a.A % 16 == 0) && (uintptr_t)a.B % bcs == 0 && (uintptr_t)a.C % bcs == 0 &&
                     a.bs % V == 0 && a.cs % V == 0;
    if constexpr (CHANNEL) {
        if (!vec) return launch_channel<T, ST, 1, 8, 1>(a, st);
        if constexpr (V == 4) {
            if (a.N > 32 * V) return launch_channel<T, ST, V, 2, 1>(a, st);
        }
        return a.batch == 1 ? launch_channel<T, ST, V, 1, 1>(a, st) : launch_channel<T, ST, V, 1, 4>(a, st);
    } else {
        if (!vec) return launch_head<T, ST, 1, 8, 1>(a, st);
        if constexpr (V == 4) {
            if (a.N > 32 * V) return launch_head<T, ST, V, 2, 2>(a, st);
        }
        return a.batch < 8 ? launch_head<T, ST, V, 1, 2>(a, st) : launch_head<T, ST, V, 1, 8>(a, st);
    }
}
template <bool CHANNEL>
cudaError_t pick_types(const StepArgs &a, bool bf16, bool st_bf16, cudaStream_t st) {
    if (bf16)
        return st_bf16 ? pick<__nv_bfloat16, __nv_bfloat16, CHANNEL>(a, st) : pick<__nv_bfloat16, float, CHANNEL>(a, st);
    return st_bf16 ? pick<float, __nv_bfloat16, CHANNEL>(a, st) : pick<float, float, CHANNEL>(a, st);
}

bool type_ok(int t) { return t == SSD_F32 || t == SSD_BF16; }
bool al(const void *p, size_t n) { return (uintptr_t)p % n == 0; }

ssd_status step(const ssd_step_problem *p, bool selective, void *state, const int32_t *idx, const void *x, const void *dt,
                const float *A, const void *B, const void *C, const float *D, const void *z, const float *bias, void *y,
                cudaStream_t st) {
    if (p == nullptr || p->batch < 0 || p->nslots < 0 || p->nheads < 1 || p->headdim < 1 || p->ngroups < 1 ||
        p->dstate < 1 || p->nheads % p->ngroups != 0 || p->reserved != 0 || (selective && p->headdim != 1))
        return SSD_ERR_INVALID_ARGUMENT;
    if (!type_ok(p->dtype) || !type_ok(p->state_dtype) || !(p->dt_dtype == SSD_F32 || (selective && p->dt_dtype == p->dtype)))
        return SSD_ERR_INVALID_ARGUMENT;
    if (p->dstate > 256 || p->nheads > ((int64_t)1 << 24) || p->headdim > ((int64_t)1 << 16) ||
        p->nheads * p->headdim > ((int64_t)1 << 24) || p->batch > ((int64_t)1 << 20))
        return SSD_ERR_UNSUPPORTED;
    const int64_t rows = p->nheads * p->headdim, segs = selective ? p->ngroups : p->nheads, spr = rows / segs;
    if (p->batch == 0) return SSD_OK;
    if (!x || !dt || !A || !B || !C || !y || (p->nslots > 0 && !state)) return SSD_ERR_INVALID_ARGUMENT;
    const int64_t bc = p->ngroups * p->dstate, nd = selective ? rows : p->nheads;
    if (p->nslots > 1 && p->slot_stride < rows * p->dstate) return SSD_ERR_INVALID_ARGUMENT;
    if (p->batch > 1 && (p->x_stride < rows || p->y_stride < rows || (z && p->z_stride < rows) || p->dt_stride < nd ||
                         p->b_stride < bc || p->c_stride < bc))
        return SSD_ERR_INVALID_ARGUMENT;
    const size_t e = p->dtype == SSD_BF16 ? 2 : 4;
    if (!al(x, e) || !al(y, e) || !al(B, e) || !al(C, e) || !al(z, e) || !al(dt, p->dt_dtype == SSD_BF16 ? 2 : 4) ||
        !al(A, 4) || !al(D, 4) || !al(bias, 4) || !al(idx, 4) || !al(state, p->state_dtype == SSD_BF16 ? 2 : 4))
        return SSD_ERR_MISALIGNED;
    if (p->nslots == 0)                                             // every request is padding
        return cudaMemset2DAsync(y, p->y_stride * e, 0, rows * e, p->batch, st) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    StepArgs a{};
    a.state = state; a.idx = idx; a.x = x; a.dt = dt; a.A = A; a.B = B; a.C = C; a.D = D; a.z = z; a.bias = bias; a.y = y;
    a.nslots = (int)(p->nslots < 0x7fffffff ? p->nslots : 0x7fffffff); a.slot_stride = p->slot_stride;
    a.xs = p->x_stride; a.dts = p->dt_stride; a.zs = p->z_stride; a.bs = p->b_stride; a.cs = p->c_stride; a.ys = p->y_stride;
    a.batch = (int)p->batch; a.segs = (int)segs; a.rows = (int)spr; a.spg = (int)(segs / p->ngroups); a.N = (int)p->dstate;
    a.dt_f32 = p->dt_dtype == SSD_F32;
    const bool bf16 = p->dtype == SSD_BF16, sb = p->state_dtype == SSD_BF16;
    const cudaError_t err = selective ? pick_types<true>(a, bf16, sb, st) : pick_types<false>(a, bf16, sb, st);
    return err == cudaSuccess ? SSD_OK : err == cudaErrorInvalidConfiguration ? SSD_ERR_UNSUPPORTED : SSD_ERR_CUDA;
}

template <typename T, typename ST, int V, int NV, int RU>
cudaError_t launch_delta(DeltaStepArgs a, cudaStream_t st) {
    a.lpr = 1;
    while (a.lpr < 32 && a.lpr * V < a.K) a.lpr <<= 1;
    const int per = (ST_NT / 32) * (32 / a.lpr) * RU;
    a.nrb = (a.V + per - 1) / per;
    const int64_t blocks = (int64_t)a.batch * a.H * a.nrb;
    if (blocks > ((int64_t)1 << 31) - 1) return cudaErrorInvalidConfiguration;
    return launch_early(k_step_delta<T, ST, V, NV, RU>, (unsigned)blocks, ST_NT, 0, st, a);
}
template <typename T, typename ST>
cudaError_t pick_delta(const DeltaStepArgs &a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(ST);
    constexpr uintptr_t qk = V * sizeof(T) < 16 ? V * sizeof(T) : 16;
    const bool vec = a.K % V == 0 && (uintptr_t)a.state % 16 == 0 && a.slot_stride % V == 0 && (uintptr_t)a.q % qk == 0 &&
                     (uintptr_t)a.k % qk == 0 && a.qs % V == 0 && a.ks % V == 0;
    if (!vec) return launch_delta<T, ST, 1, 8, 1>(a, st);
    if constexpr (V == 4) {
        if (a.K > 32 * V) return launch_delta<T, ST, V, 2, 4>(a, st);
    }
    return launch_delta<T, ST, V, 1, 8>(a, st);
}

ssd_status delta_step(const ssd_delta_step_problem *p, void *state, const int32_t *idx, const void *q, const void *k, const void *v,
                      const void *g, const void *beta, void *o, cudaStream_t st) {
    if (p == nullptr || p->batch < 0 || p->nslots < 0 || p->nheads < 1 || p->headdim < 1 || p->ngroups < 1 || p->dstate < 1 ||
        p->nheads % p->ngroups != 0)
        return SSD_ERR_INVALID_ARGUMENT;
    if (!type_ok(p->dtype) || !type_ok(p->state_dtype) || !(p->g_dtype == SSD_F32 || p->g_dtype == p->dtype) ||
        !(p->beta_dtype == SSD_F32 || p->beta_dtype == p->dtype))
        return SSD_ERR_INVALID_ARGUMENT;
    if (p->dstate > 256 || p->nheads > ((int64_t)1 << 24) || p->headdim > ((int64_t)1 << 16) ||
        p->nheads * p->headdim > ((int64_t)1 << 24) || p->batch > ((int64_t)1 << 20))
        return SSD_ERR_UNSUPPORTED;
    if (p->batch == 0) return SSD_OK;
    if (!q || !k || !v || !g || !beta || !o || (p->nslots > 0 && !state)) return SSD_ERR_INVALID_ARGUMENT;
    const int64_t rows = p->nheads * p->headdim, qk = p->ngroups * p->dstate;
    if (p->nslots > 1 && p->slot_stride < rows * p->dstate) return SSD_ERR_INVALID_ARGUMENT;
    if (p->batch > 1 && (p->q_stride < qk || p->k_stride < qk || p->v_stride < rows || p->o_stride < rows ||
                         p->g_stride < p->nheads || p->beta_stride < p->nheads))
        return SSD_ERR_INVALID_ARGUMENT;
    const size_t e = p->dtype == SSD_BF16 ? 2 : 4;
    if (!al(q, e) || !al(k, e) || !al(v, e) || !al(o, e) || !al(g, p->g_dtype == SSD_BF16 ? 2 : 4) ||
        !al(beta, p->beta_dtype == SSD_BF16 ? 2 : 4) || !al(idx, 4) || !al(state, p->state_dtype == SSD_BF16 ? 2 : 4))
        return SSD_ERR_MISALIGNED;
    if (p->nslots == 0)
        return cudaMemset2DAsync(o, p->o_stride * e, 0, rows * e, p->batch, st) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    DeltaStepArgs a{};
    a.state = state; a.idx = idx; a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.o = o;
    a.nslots = (int)(p->nslots < 0x7fffffff ? p->nslots : 0x7fffffff); a.slot_stride = p->slot_stride;
    a.qs = p->q_stride; a.ks = p->k_stride; a.vs = p->v_stride; a.gs = p->g_stride; a.bs = p->beta_stride; a.os = p->o_stride;
    a.batch = (int)p->batch; a.H = (int)p->nheads; a.V = (int)p->headdim; a.K = (int)p->dstate; a.hpg = (int)(p->nheads / p->ngroups);
    a.scale = p->scale; a.g_f32 = p->g_dtype == SSD_F32; a.beta_f32 = p->beta_dtype == SSD_F32;
    const bool sb = p->state_dtype == SSD_BF16;
    cudaError_t err;
    if (p->dtype == SSD_BF16) err = sb ? pick_delta<__nv_bfloat16, __nv_bfloat16>(a, st) : pick_delta<__nv_bfloat16, float>(a, st);
    else err = sb ? pick_delta<float, __nv_bfloat16>(a, st) : pick_delta<float, float>(a, st);
    return err == cudaSuccess ? SSD_OK : err == cudaErrorInvalidConfiguration ? SSD_ERR_UNSUPPORTED : SSD_ERR_CUDA;
}

}  // namespace
}  // namespace ssd

extern "C" {

ssd_status ssd_step(const ssd_step_problem *p, void *state, const int32_t *idx, const void *x, const void *dt,
                    const float *A, const void *B, const void *C, const float *D, const void *z, const float *bias,
                    void *y, void *stream) {
    return ssd::step(p, false, state, idx, x, dt, A, B, C, D, z, bias, y, (cudaStream_t)stream);
}
ssd_status ssd_selective_step(const ssd_step_problem *p, void *state, const int32_t *idx, const void *x, const void *dt,
                              const float *A, const void *B, const void *C, const float *D, const void *z,
                              const float *bias, void *y, void *stream) {
    return ssd::step(p, true, state, idx, x, dt, A, B, C, D, z, bias, y, (cudaStream_t)stream);
}

ssd_status ssd_delta_step(const ssd_delta_step_problem *p, void *state, const int32_t *idx, const void *q, const void *k,
                          const void *v, const void *g, const void *beta, void *o, void *stream) {
    return ssd::delta_step(p, state, idx, q, k, v, g, beta, o, (cudaStream_t)stream);
}

}  // extern "C"
