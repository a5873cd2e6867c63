// step.cu -- one token of the recurrence for each of a batch of requests, on a pool of states:
//
//   h <- exp(dt A) h + dt x B,   y = (C.h + D x) silu(z),   dt = softplus(dt_raw + dt_bias)
//
// with one A per head (ssd_step) or one per channel and state (ssd_selective_step).  Every state
// value is read once and written once and takes part in a handful of operations, so memory
// bounds it.  The state is taken as segments of rows of dstate values: a segment is a head (its
// rows share A and dt) or a B/C group of the selective form (each row a channel with its own).  A row
// belongs to LPR lanes, each with NV pieces of V values (16 bytes where rows allow it); a
// warp issues the loads of RU rows per lane group before it uses the first, and sums their outputs
// over the lanes together.
#include <algorithm>

#include "selective.cuh"

namespace ssd {

namespace {

#ifndef STEP_NT
#define STEP_NT 128
#endif
constexpr int ST_NT = STEP_NT;

struct StepArgs {
    void *state;
    const int32_t *idx;
    const void *x, *dt, *B, *C, *z;
    const float *A, *D, *bias;
    void *y;
    int64_t nslots, slot_stride, xs, dts, zs, bs, cs, ys;
    int batch, segs, rows, spg, N;       // segments, rows of each, segments per B/C group
    int lpr, nrb;                        // lanes per row (a power of two), row blocks per segment
    bool dt_f32;
};

template <int V>
struct Piece {
    float v[V];
};
// A piece is one value, or 16 bytes of state: 4 fp32 or 8 bf16 (and as many values of A, B and C).
template <int V>
__device__ __forceinline__ void ldp(const float *p, Piece<V> &o) {
    if constexpr (V == 1) {
        o.v[0] = *p;
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 u = reinterpret_cast<const float4 *>(p)[i];
            o.v[4 * i] = u.x; o.v[4 * i + 1] = u.y; o.v[4 * i + 2] = u.z; o.v[4 * i + 3] = u.w;
        }
    }
}
template <int V>
__device__ __forceinline__ void ldp(const __nv_bfloat16 *p, Piece<V> &o) {
    if constexpr (V == 1) {
        o.v[0] = __bfloat162float(*p);
    } else if constexpr (V == 4) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        o.v[0] = __uint_as_float(u.x << 16); o.v[1] = __uint_as_float(u.x & 0xffff0000u);
        o.v[2] = __uint_as_float(u.y << 16); o.v[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o.v[2 * i] = __uint_as_float(w[i] << 16);
            o.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
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

// T: type of x, B, C, z, y.  ST: of the state.  V values a piece, NV pieces a lane; ROW_A: A and dt per row.
template <typename T, typename ST, int V, int NV, int RU, bool ROW_A>
__global__ void __launch_bounds__(ST_NT) k_step(const StepArgs a) {
    const int rb = blockIdx.x % a.nrb, bs = blockIdx.x / a.nrb, seg = bs % a.segs, b = bs / a.segs;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int l = lane & (a.lpr - 1), rpw = 32 / a.lpr;             // lane of the row, rows of a warp
    const int r0 = (rb * (ST_NT / 32) + w) * rpw * RU + lane / a.lpr;
    const int N = a.N;
    const int64_t first = (int64_t)seg * a.rows;                    // the segment's first row
    T *y = static_cast<T *>(a.y) + b * a.ys + first;
    const int64_t slot = a.idx ? a.idx[b] : b;
    if (slot < 0 || slot >= a.nslots) {                             // padding
        for (int u = 0; u < RU; ++u)
            if (l == 0 && r0 + u * rpw < a.rows) y[r0 + u * rpw] = from_f<T>(0.f);
        return;
    }
    ST *st = static_cast<ST *>(a.state) + slot * a.slot_stride + first * N;
    const T *x = static_cast<const T *>(a.x) + b * a.xs + first;
    // every load first: the stores below would hold up later ones
    Piece<V> h[RU][NV], Av[ROW_A ? RU : 1][NV], Bv[NV], Cv[NV];
    float xv[RU], dt[ROW_A ? RU : 1];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
        const int r = r0 + u * rpw;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int n = (k * a.lpr + l) * V;
            if (r < a.rows && n < N) {
                ldp<V>(st + (int64_t)r * N + n, h[u][k]);
                if (ROW_A) ldp<V>(a.A + (first + r) * N + n, Av[ROW_A ? u : 0][k]);
            }
        }
    }
    const T *B = static_cast<const T *>(a.B) + b * a.bs + (int64_t)(seg / a.spg) * N;
    const T *C = static_cast<const T *>(a.C) + b * a.cs + (int64_t)(seg / a.spg) * N;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int n = (k * a.lpr + l) * V;
        if (n < N) {
            ldp<V>(B + n, Bv[k]);
            ldp<V>(C + n, Cv[k]);
        }
    }
    auto load_dt = [&](int64_t at, int64_t par) {
        return (a.dt_f32 ? static_cast<const float *>(a.dt)[at] : to_f(static_cast<const T *>(a.dt)[at])) + (a.bias ? a.bias[par] : 0.f);
    };
#pragma unroll
    for (int u = 0; u < RU; ++u) {
        const int r = r0 + u * rpw;
        xv[u] = r < a.rows ? to_f(x[r]) : 0.f;
        if (ROW_A) dt[ROW_A ? u : 0] = r < a.rows ? load_dt(b * a.dts + first + r, first + r) : 0.f;
    }
    if (!ROW_A) dt[0] = load_dt(b * a.dts + seg, seg);
    // where a row has at least RU lanes, lane u finishes row u; else its first lane every row
    const bool spread = a.lpr >= RU;
    const int ru = r0 + (spread ? l : 0) * rpw;
    const bool fin = (spread ? l < RU : l == 0) && ru < a.rows;
    float zu = 0.f, xu = 0.f, Du = 0.f;
    if (spread && fin) {
        if (a.z) zu = to_f(static_cast<const T *>(a.z)[b * a.zs + first + ru]);
        if (a.D) {
            Du = a.D[ROW_A ? first + ru : seg];
            xu = to_f(x[ru]);
        }
    }
    float acc[RU];
    const float d0 = ROW_A ? 0.f : sel_softplus(dt[0]), decay = ROW_A ? 0.f : ex2f(d0 * a.A[seg] * kLog2e);
#pragma unroll
    for (int u = 0; u < RU; ++u) {
        const int r = r0 + u * rpw;
        acc[u] = 0.f;
        if (r < a.rows) {
            const float dv = ROW_A ? sel_softplus(dt[ROW_A ? u : 0]) : d0, dtx = dv * xv[u], dtl = dv * kLog2e;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int n = (k * a.lpr + l) * V;
                if (n < N) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float d = ROW_A ? ex2f(dtl * Av[ROW_A ? u : 0][k].v[e]) : decay;
                        h[u][k].v[e] = fmaf(d, h[u][k].v[e], dtx * Bv[k].v[e]);
                        acc[u] = fmaf(Cv[k].v[e], h[u][k].v[e], acc[u]);
                    }
                    stp<V>(st + (int64_t)r * N + n, h[u][k]);
                }
            }
        }
    }
    if (spread) {
        float v = reduce_scatter<RU>(acc, l & (RU - 1));
        for (int o = RU; o < a.lpr; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (fin) {
            v = fmaf(Du, xu, v);
            y[ru] = from_f<T>(a.z ? sel_gate<T>(v, zu) : v);
        }
    } else {
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            for (int o = a.lpr >> 1; o > 0; o >>= 1) acc[u] += __shfl_xor_sync(0xffffffffu, acc[u], o);
            const int r = r0 + u * rpw;
            if (l == 0 && r < a.rows) {
                float v = a.D ? fmaf(a.D[ROW_A ? first + r : seg], xv[u], acc[u]) : acc[u];
                if (a.z) v = sel_gate<T>(v, to_f(static_cast<const T *>(a.z)[b * a.zs + first + r]));
                y[r] = from_f<T>(v);
            }
        }
    }
}

template <typename T, typename ST, int V, int NV, int RU, bool ROW_A>
cudaError_t launch(StepArgs a, cudaStream_t st) {
    a.lpr = 1;
    while (a.lpr < 32 && a.lpr * V < a.N) a.lpr <<= 1;
    const int per = (ST_NT / 32) * (32 / a.lpr) * RU;
    a.nrb = (a.rows + per - 1) / per;
    k_step<T, ST, V, NV, RU, ROW_A><<<(unsigned)((int64_t)a.batch * a.segs * a.nrb), ST_NT, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T, typename ST, bool ROW_A>
cudaError_t pick(const StepArgs &a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(ST);
    const bool vec = a.N % V == 0 && (uintptr_t)a.state % 16 == 0 && a.slot_stride % V == 0 &&
                     (!ROW_A || (uintptr_t)a.A % 16 == 0) && (uintptr_t)a.B % (V * sizeof(T)) % 16 == 0 &&
                     (uintptr_t)a.C % (V * sizeof(T)) % 16 == 0 && a.bs % V == 0 && a.cs % V == 0;
    if (!vec) return launch<T, ST, 1, 8, 1, ROW_A>(a, st);
#ifndef STEP_RU
#define STEP_RU 4
#endif
    if constexpr (V == 4) {
        if (a.N > 32 * V) return launch<T, ST, V, 2, 2, ROW_A>(a, st);
    }
    return launch<T, ST, V, 1, STEP_RU, ROW_A>(a, st);
}
template <bool ROW_A>
cudaError_t pick_types(const StepArgs &a, bool bf16, bool st_bf16, cudaStream_t st) {
    if (bf16) return st_bf16 ? pick<__nv_bfloat16, __nv_bfloat16, ROW_A>(a, st) : pick<__nv_bfloat16, float, ROW_A>(a, st);
    return st_bf16 ? pick<float, __nv_bfloat16, ROW_A>(a, st) : pick<float, float, ROW_A>(a, st);
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
    if (p->batch * segs * ((spr + 3) / 4) > ((int64_t)1 << 31) - 1) return SSD_ERR_UNSUPPORTED;
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
    StepArgs a{};
    a.state = state; a.idx = idx; a.x = x; a.dt = dt; a.A = A; a.B = B; a.C = C; a.D = D; a.z = z; a.bias = bias; a.y = y;
    a.nslots = p->nslots; a.slot_stride = p->slot_stride;
    a.xs = p->x_stride; a.dts = p->dt_stride; a.zs = p->z_stride; a.bs = p->b_stride; a.cs = p->c_stride; a.ys = p->y_stride;
    a.batch = (int)p->batch; a.segs = (int)segs; a.rows = (int)spr; a.spg = (int)(segs / p->ngroups); a.N = (int)p->dstate;
    a.dt_f32 = p->dt_dtype == SSD_F32;
    const bool bf16 = p->dtype == SSD_BF16, sb = p->state_dtype == SSD_BF16;
    return (selective ? pick_types<true>(a, bf16, sb, st) : pick_types<false>(a, bf16, sb, st)) == cudaSuccess ? SSD_OK
                                                                                                            : SSD_ERR_CUDA;
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

}  // extern "C"
