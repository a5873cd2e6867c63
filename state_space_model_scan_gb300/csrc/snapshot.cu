// snapshot.cu -- states put aside in 8 bits and taken up again.  A row of dstate values h is kept as
// q = round_half_even(h ((1 / m) 127)) and the scale m / 127, m = max |h|, each step rounded to fp32.  Bytes bound
// it: 4 or 2 read and 1 written per value, or the other way round.  96 states of 4096 rows x 128, fp32, stored
// and loaded: 81 us for 506 MB (6.2 TB/s, 92% of a plain copy).
//
// A row belongs to LPR lanes, each with NV pieces of four values, so that one exchange of the maximum
// serves 16 values a lane.  The maximum lets a NaN through, so that one comparison finds rows that
// cannot be kept; q is rounded by adding 1.5 x 2^23, whose last byte then is the integer.
#include <algorithm>

#include "common.cuh"

namespace ssd {

namespace {

constexpr int SN_NT = 128;   // threads

struct SnapArgs {
    void *states;
    const int32_t *sidx, *qidx;
    int8_t *q;
    float *scale;
    int64_t nslots, nsnaps, stride, rows;
    int N, lpr;
    int nrb;                             // row blocks per state
};

__device__ __forceinline__ float max_nan(float a, float b) {   // a NaN wins
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
constexpr float kTiny = 1e-30f;          // below it 127 / m nears the end of fp32's range

// inverse step and scale of a row whose largest magnitude is m
__device__ __forceinline__ void row_scale(float m, float &inv, float &scale) {
    if (!(m < __int_as_float(0x7f800000))) {
        inv = 0.f;
        scale = __int_as_float(0x7fc00000);
    } else if (m < kTiny) {
        inv = scale = 0.f;
    } else {
        inv = __fmul_rn(__frcp_rn(m), 127.f);
        scale = __fdiv_rn(m, 127.f);
    }
}
// round_half_even(h inv) in the last byte; |h inv| <= 127 (1 + 2^-22)
__device__ __forceinline__ uint32_t quant(float h, float inv) {
    return __float_as_uint(__fadd_rn(__fmul_rn(h, inv), 12582912.f));
}

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

// The loads of RU rows of NV pieces a lane are issued before the first is used.
template <typename ST, int NV, int RU>
__global__ void __launch_bounds__(SN_NT) k_snap_store(const SnapArgs a) {
    after_previous();
    int64_t r0;
    int l, rpw;
    ST *st;
    int8_t *q;
    float *sc;
    if (!place<RU>(a, r0, l, rpw, st, q, sc)) return;
    const int N = a.N;
    float v[RU][NV][4];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
        const int64_t r = r0 + u * rpw;
        const ST *p = st + r * N + l * 4;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (r < a.rows && (k * a.lpr + l) * 4 < N) ld4s(p + k * a.lpr * 4, v[u][k]);
            else v[u][k][0] = v[u][k][1] = v[u][k][2] = v[u][k][3] = 0.f;
        }
    }
#pragma unroll
    for (int u = 0; u < RU; ++u) {
        const int64_t r = r0 + u * rpw;
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) m = max_nan(m, fabsf(v[u][k][e]));
        for (int o = a.lpr >> 1; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (r >= a.rows) continue;
        float inv, scale;
        row_scale(m, inv, scale);
        if (l == 0) sc[r] = scale;
        int8_t *o = q + r * N + l * 4;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if ((k * a.lpr + l) * 4 < N) {
                const uint32_t lo = __byte_perm(quant(v[u][k][0], inv), quant(v[u][k][1], inv), 0x0040);
                const uint32_t hi = __byte_perm(quant(v[u][k][2], inv), quant(v[u][k][3], inv), 0x0040);
                *reinterpret_cast<uint32_t *>(o + k * a.lpr * 4) = inv == 0.f ? 0u : __byte_perm(lo, hi, 0x5410);
            }
    }
}

template <typename ST, int NV, int RU>
__global__ void __launch_bounds__(SN_NT) k_snap_load(const SnapArgs a) {
    after_previous();
    int64_t r0;
    int l, rpw;
    ST *st;
    int8_t *q;
    float *sc;
    if (!place<RU>(a, r0, l, rpw, st, q, sc)) return;
    const int N = a.N;
    char4 c[RU][NV];
    float s[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
        const int64_t r = r0 + u * rpw;
        if (r < a.rows) {
            s[u] = sc[r];
            const int8_t *p = q + r * N + l * 4;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if ((k * a.lpr + l) * 4 < N) c[u][k] = *reinterpret_cast<const char4 *>(p + k * a.lpr * 4);
        }
    }
#pragma unroll
    for (int u = 0; u < RU; ++u) {
        const int64_t r = r0 + u * rpw;
        if (r < a.rows) {
            ST *p = st + r * N + l * 4;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if ((k * a.lpr + l) * 4 < N) {
                    const float v[4] = {c[u][k].x * s[u], c[u][k].y * s[u], c[u][k].z * s[u], c[u][k].w * s[u]};
                    st4s(p + k * a.lpr * 4, v);
                }
        }
    }
}

// Rows that do not allow four values an access: single ones, read twice.
template <typename ST>
__global__ void __launch_bounds__(SN_NT) k_snap_store1(const SnapArgs a) {
    after_previous();
    int64_t r;
    int l, rpw;
    ST *st;
    int8_t *q;
    float *sc;
    if (!place<1>(a, r, l, rpw, st, q, sc)) return;
    const bool in = r < a.rows;
    float m = 0.f;
    if (in)
        for (int n = l; n < a.N; n += a.lpr) m = max_nan(m, fabsf(to_f(st[r * a.N + n])));
    for (int o = a.lpr >> 1; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (!in) return;
    float inv, scale;
    row_scale(m, inv, scale);
    if (l == 0) sc[r] = scale;
    for (int n = l; n < a.N; n += a.lpr) q[r * a.N + n] = inv == 0.f ? 0 : (int8_t)(quant(to_f(st[r * a.N + n]), inv) & 0xff);
}
template <typename ST>
__global__ void __launch_bounds__(SN_NT) k_snap_load1(const SnapArgs a) {
    after_previous();
    int64_t r;
    int l, rpw;
    ST *st;
    int8_t *q;
    float *sc;
    if (!place<1>(a, r, l, rpw, st, q, sc) || r >= a.rows) return;
    const float s = sc[r];
    for (int n = l; n < a.N; n += a.lpr) st[r * a.N + n] = from_f<ST>(q[r * a.N + n] * s);
}

// How a row is cut: pieces a lane and rows in flight (0: single values).  At dstate 64 and above four pieces
// a lane, so that a row's lanes still read 64 bytes or more at once.  Round trip of 96 states of 4096 rows x 128,
// fp32: four pieces of one row 81 us, one piece of four rows to store and of eight to load 108 us.
struct Cut {
    int nv, ru;
};
Cut cut(bool vec, int N) {
    if (!vec) return {0, 1};
    if (N > 512) return {8, 1};
    if (N >= 64) return {4, 1};
    return {1, 4};
}

ssd_status make(const ssd_snapshot_problem *p, const void *states, const int32_t *sidx, const int8_t *q,
                const float *scales, const int32_t *slots, SnapArgs &a, Cut &how, unsigned &grid) {
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
    const bool vec = a.N % 4 == 0 && (uintptr_t)states % (4 * es) == 0 && (uintptr_t)q % 4 == 0 && (a.stride % 4 == 0 || a.nslots == 1);
    a.lpr = 1;
    how = cut(vec, a.N);
    while (a.lpr < 32 && a.lpr * (vec ? 4 * how.nv : 1) < a.N) a.lpr <<= 1;
    const int64_t per = (int64_t)(SN_NT / 32) * (32 / a.lpr) * how.ru, nrb = (a.rows + per - 1) / per;
    if (nrb * p->count > ((int64_t)1 << 31) - 1) return SSD_ERR_UNSUPPORTED;
    a.nrb = (int)nrb;
    grid = (unsigned)(nrb * p->count);
    return SSD_OK;
}

template <typename ST>
cudaError_t store(const SnapArgs &a, Cut how, unsigned grid, cudaStream_t st) {
    switch (how.nv) {
        case 0: return launch_early(k_snap_store1<ST>, grid, SN_NT, 0, st, a);
        case 1: return launch_early(k_snap_store<ST, 1, 4>, grid, SN_NT, 0, st, a);
        case 4: return launch_early(k_snap_store<ST, 4, 1>, grid, SN_NT, 0, st, a);
        default: return launch_early(k_snap_store<ST, 8, 1>, grid, SN_NT, 0, st, a);
    }
}
template <typename ST>
cudaError_t load(const SnapArgs &a, Cut how, unsigned grid, cudaStream_t st) {
    switch (how.nv) {
        case 0: return launch_early(k_snap_load1<ST>, grid, SN_NT, 0, st, a);
        case 1: return launch_early(k_snap_load<ST, 1, 4>, grid, SN_NT, 0, st, a);
        case 4: return launch_early(k_snap_load<ST, 4, 1>, grid, SN_NT, 0, st, a);
        default: return launch_early(k_snap_load<ST, 8, 1>, grid, SN_NT, 0, st, a);
    }
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_snapshot_store(const ssd_snapshot_problem *p, const void *states, const int32_t *state_indices,
                              int8_t *snapshots, float *scales, const int32_t *slots, void *stream) {
    SnapArgs a{};
    Cut how{};
    unsigned grid = 0;
    const ssd_status s = make(p, states, state_indices, snapshots, scales, slots, a, how, grid);
    if (s != SSD_OK || grid == 0) return s;
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = p->state_dtype == SSD_BF16 ? store<__nv_bfloat16>(a, how, grid, st) : store<float>(a, how, grid, st);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_snapshot_load(const ssd_snapshot_problem *p, const int8_t *snapshots, const float *scales,
                             const int32_t *slots, void *states, const int32_t *state_indices, void *stream) {
    SnapArgs a{};
    Cut how{};
    unsigned grid = 0;
    const ssd_status s = make(p, states, state_indices, snapshots, scales, slots, a, how, grid);
    if (s != SSD_OK || grid == 0) return s;
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = p->state_dtype == SSD_BF16 ? load<__nv_bfloat16>(a, how, grid, st) : load<float>(a, how, grid, st);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
