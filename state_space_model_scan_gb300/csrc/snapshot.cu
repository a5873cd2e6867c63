// snapshot.cu -- states put aside in 8 bits and taken up again.  A row of dstate values h is kept as
// q = round_half_even(h 127 / m) and the scale m / 127, m = max |h|.  Bytes bound it: 4 or 2 read
// and 1 written per value, or the other way round.
//
// The maximum is taken over the values' bit patterns without the sign: as integers they are
// ordered like the magnitudes, with infinity and then every NaN above all finite ones, so that
// one comparison finds rows that cannot be kept.
#include <algorithm>

#include "common.cuh"

namespace ssd {

namespace {

#ifndef SNAP_RU
#define SNAP_RU 4
#endif
#ifndef SNAP_RL
#define SNAP_RL 4
#endif
constexpr int SN_NT = 256;   // threads

struct SnapArgs {
    void *states;
    const int32_t *sidx, *qidx;
    int8_t *q;
    float *scale;
    int64_t nslots, nsnaps, stride, rows;
    int N, lpr;
    int nrb;                             // row blocks per state
};

__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;
constexpr float kTiny = 1e-30f;          // below it 127 / m nears the end of fp32's range

// inverse step and scale of a row with largest magnitude bits m
__device__ __forceinline__ void row_scale(uint32_t m, float &inv, float &scale) {
    const float v = __uint_as_float(m);
    if (m >= kInfBits) {
        inv = 0.f;
        scale = __uint_as_float(0x7fc00000u);
    } else if (v < kTiny) {
        inv = scale = 0.f;
    } else {
        inv = __fdiv_rn(127.f, v);
        scale = __fdiv_rn(v, 127.f);
    }
}
__device__ __forceinline__ int quant(float h, float inv) { return inv == 0.f ? 0 : __float2int_rn(__fmul_rn(h, inv)); }

__device__ __forceinline__ void ld4s(const float *p, float (&v)[4]) {
    const float4 u = *reinterpret_cast<const float4 *>(p);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
}
__device__ __forceinline__ void ld4s(const __nv_bfloat16 *p, float (&v)[4]) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void st4s(float *p, const float (&v)[4]) { *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void st4s(__nv_bfloat16 *p, const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// Where this thread's rows are, RU of them rpw apart: false when either index of its pair is out of range.
template <int RU, typename ST>
__device__ __forceinline__ bool place(const SnapArgs &a, int64_t &r0, int &l, int &rpw, ST *&st, int8_t *&q, float *&sc) {
    const int i = blockIdx.x / a.nrb, rb = blockIdx.x % a.nrb;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    l = lane & (a.lpr - 1);
    rpw = 32 / a.lpr;
    r0 = ((int64_t)rb * (SN_NT / 32) + w) * rpw * RU + lane / a.lpr;
    const int64_t s = a.sidx ? a.sidx[i] : i, k = a.qidx ? a.qidx[i] : i;
    if (s < 0 || s >= a.nslots || k < 0 || k >= a.nsnaps) return false;
    st = static_cast<ST *>(a.states) + s * a.stride;
    q = a.q + k * a.rows * a.N;
    sc = a.scale + k * a.rows;
    return true;
}

// NV pieces of 4 values a lane in registers; NV = 0: single values, read twice.  The loads of RU rows
// are issued before the first is used.
template <typename ST, int NV, int RU>
__global__ void __launch_bounds__(SN_NT) k_snap_store(const SnapArgs a) {
    int64_t r0;
    int l, rpw;
    ST *st;
    int8_t *q;
    float *sc;
    if (!place<RU>(a, r0, l, rpw, st, q, sc)) return;
    const int N = a.N;
    float v[RU][NV > 0 ? NV : 1][4];
    if (NV > 0) {
#pragma unroll
        for (int u = 0; u < RU; ++u)
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int n = (k * a.lpr + l) * 4;
                const int64_t r = r0 + u * rpw;
                if (r < a.rows && n < N) ld4s(st + r * N + n, v[u][k]);
            }
    }
#pragma unroll
    for (int u = 0; u < RU; ++u) {
        const int64_t r = r0 + u * rpw;
        const bool in = r < a.rows;
        uint32_t m = 0;
        if (NV > 0) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (in && (k * a.lpr + l) * 4 < N) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) m = max(m, mag(v[u][k][e]));
                }
        } else if (in) {
            for (int n = l; n < N; n += a.lpr) m = max(m, mag(to_f(st[r * N + n])));
        }
        for (int o = a.lpr >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (!in) continue;
        float inv, scale;
        row_scale(m, inv, scale);
        if (l == 0) sc[r] = scale;
        if (NV > 0) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int n = (k * a.lpr + l) * 4;
                if (n < N) {
                    uint32_t p = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) p |= (uint32_t)(quant(v[u][k][e], inv) & 0xff) << (8 * e);
                    *reinterpret_cast<uint32_t *>(q + r * N + n) = p;
                }
            }
        } else {
            for (int n = l; n < N; n += a.lpr) q[r * N + n] = (int8_t)quant(to_f(st[r * N + n]), inv);
        }
    }
}

template <typename ST, bool VEC, int RU>
__global__ void __launch_bounds__(SN_NT) k_snap_load(const SnapArgs a) {
    int64_t r0;
    int l, rpw;
    ST *st;
    int8_t *q;
    float *sc;
    if (!place<RU>(a, r0, l, rpw, st, q, sc)) return;
    for (int n = l * (VEC ? 4 : 1); n < a.N; n += a.lpr * (VEC ? 4 : 1)) {
        char4 c[RU];
        float s[RU];
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            const int64_t r = r0 + u * rpw;
            if (r < a.rows) {
                s[u] = sc[r];
                if (VEC) c[u] = *reinterpret_cast<const char4 *>(q + r * a.N + n);
                else c[u].x = q[r * a.N + n];
            }
        }
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            const int64_t r = r0 + u * rpw;
            if (r < a.rows) {
                const float v[4] = {c[u].x * s[u], c[u].y * s[u], c[u].z * s[u], c[u].w * s[u]};
                if (VEC) st4s(st + r * a.N + n, v);
                else st[r * a.N + n] = from_f<ST>(v[0]);
            }
        }
    }
}

ssd_status make(const ssd_snapshot_problem *p, const void *states, const int32_t *sidx, const int8_t *q,
                const float *scales, const int32_t *slots, int ru, SnapArgs &a, bool &vec, unsigned &grid) {
    if (p == nullptr || p->count < 0 || p->rows < 1 || p->dstate < 1 || p->nslots < 0 || p->nsnapshots < 0 || p->reserved != 0)
        return SSD_ERR_INVALID_ARGUMENT;
    if (p->state_dtype != SSD_F32 && p->state_dtype != SSD_BF16) return SSD_ERR_INVALID_ARGUMENT;
    if (p->nslots > 1 && p->state_stride < p->rows * p->dstate) return SSD_ERR_INVALID_ARGUMENT;
    if (p->dstate > 1024 || p->rows > ((int64_t)1 << 31) || p->count > ((int64_t)1 << 24)) return SSD_ERR_UNSUPPORTED;
    grid = 0;
    if (p->count == 0 || p->nslots == 0 || p->nsnapshots == 0) return SSD_OK;
    if (!states || !q || !scales) return SSD_ERR_INVALID_ARGUMENT;
    const size_t es = p->state_dtype == SSD_BF16 ? 2 : 4;
    if ((uintptr_t)states % es || (uintptr_t)scales % 4 || (uintptr_t)sidx % 4 || (uintptr_t)slots % 4) return SSD_ERR_MISALIGNED;
    a.states = const_cast<void *>(states); a.sidx = sidx; a.qidx = slots; a.q = const_cast<int8_t *>(q);
    a.scale = const_cast<float *>(scales);
    a.nslots = p->nslots; a.nsnaps = p->nsnapshots; a.stride = p->state_stride; a.rows = p->rows; a.N = (int)p->dstate;
    vec = a.N % 4 == 0 && (uintptr_t)states % (4 * es) == 0 && (uintptr_t)q % 4 == 0 && (a.stride % 4 == 0 || a.nslots == 1);
    a.lpr = 1;
    while (a.lpr < 32 && a.lpr * (vec ? 4 : 1) < a.N) a.lpr <<= 1;
    const int64_t per = (int64_t)(SN_NT / 32) * (32 / a.lpr) * ru, nrb = (a.rows + per - 1) / per;
    if (nrb * p->count > ((int64_t)1 << 31) - 1) return SSD_ERR_UNSUPPORTED;
    a.nrb = (int)nrb;
    grid = (unsigned)(nrb * p->count);
    return SSD_OK;
}

constexpr int kStoreRows = SNAP_RU, kLoadRows = SNAP_RL;   // rows in flight per lane group

template <typename ST>
void store(const SnapArgs &a, bool vec, unsigned grid, cudaStream_t st) {
    const int nv = vec ? (a.N + 4 * a.lpr - 1) / (4 * a.lpr) : 0;
    if (nv == 0) k_snap_store<ST, 0, kStoreRows><<<grid, SN_NT, 0, st>>>(a);
    else if (nv == 1) k_snap_store<ST, 1, kStoreRows><<<grid, SN_NT, 0, st>>>(a);
    else if (nv == 2) k_snap_store<ST, 2, kStoreRows><<<grid, SN_NT, 0, st>>>(a);
    else if (nv <= 4) k_snap_store<ST, 4, kStoreRows><<<grid, SN_NT, 0, st>>>(a);
    else k_snap_store<ST, 8, kStoreRows><<<grid, SN_NT, 0, st>>>(a);
}
template <typename ST>
void load(const SnapArgs &a, bool vec, unsigned grid, cudaStream_t st) {
    if (vec) k_snap_load<ST, true, kLoadRows><<<grid, SN_NT, 0, st>>>(a);
    else k_snap_load<ST, false, kLoadRows><<<grid, SN_NT, 0, st>>>(a);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_snapshot_store(const ssd_snapshot_problem *p, const void *states, const int32_t *state_indices,
                              int8_t *snapshots, float *scales, const int32_t *slots, void *stream) {
    SnapArgs a{};
    bool vec = false;
    unsigned grid = 0;
    const ssd_status s = make(p, states, state_indices, snapshots, scales, slots, kStoreRows, a, vec, grid);
    if (s != SSD_OK || grid == 0) return s;
    if (p->state_dtype == SSD_BF16) store<__nv_bfloat16>(a, vec, grid, (cudaStream_t)stream);
    else store<float>(a, vec, grid, (cudaStream_t)stream);
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_snapshot_load(const ssd_snapshot_problem *p, const int8_t *snapshots, const float *scales,
                             const int32_t *slots, void *states, const int32_t *state_indices, void *stream) {
    SnapArgs a{};
    bool vec = false;
    unsigned grid = 0;
    const ssd_status s = make(p, states, state_indices, snapshots, scales, slots, kLoadRows, a, vec, grid);
    if (s != SSD_OK || grid == 0) return s;
    if (p->state_dtype == SSD_BF16) load<__nv_bfloat16>(a, vec, grid, (cudaStream_t)stream);
    else load<float>(a, vec, grid, (cudaStream_t)stream);
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
