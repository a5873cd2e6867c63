// conv1d.cu -- causal depthwise convolution over the sequence axis with an optional SiLU,
// forward and backward: the step before the scan in a Mamba-2 block, run on the packed
// xBC = [x | B | C] channels (the Helion pull request for the Mamba-2 SSD path, "Summary":
// mamba_split_conv1d_scan_combined; "Testing": x, B and C are views of one packed buffer):
//
//   pre[t,c] = bias[c] + sum_{k<K} w[c,k] u[t-(K-1)+k, c]   (u := 0 before t's sequence start)
//   out[t,c] = silu(pre[t,c])  (or pre)
//
// The scan then reads x, B and C as strided views of `out` (no copy: the split is the view).
// A thread owns W consecutive channels and sweeps a run of tokens with its inputs' last K rows in
// registers, and, for the backward, also the K input-gradient rows still receiving contributions; the weight and bias gradients are per-tile partial sums added in a
// fixed order afterwards (bitwise reproducible).  Every access of a warp is one contiguous
// row piece: 4 channels a thread, 256 bytes in bf16 or 512 in fp32; in the single-token step 8, twice that.
#include <algorithm>

#include "f32x2.cuh"

namespace ssd {

namespace {

constexpr int TT = 64;        // tokens of a block of the backward
constexpr int KMAX = 8;

__device__ __forceinline__ void ld8(const __nv_bfloat16 *p, float *v) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const __nv_bfloat162 *e = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(e[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void ld8(const float *p, float *v) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void st8(__nv_bfloat16 *p, const float *v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void st8(float *p, const float *v) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

struct ConvArgs {
    int64_t B, L, Cn, S;          // batch rows, tokens per row, channels, sequences (packed) or 0
    int K;
    bool silu;
    const void *u, *dout;
    int64_t su_b, su_l, sd_b, sd_l;
    const float *w, *bias;        // w: [Cn][K]
    const int32_t *cu;            // packed sequences (B = 1) or NULL
    void *out, *du;
    int64_t so_b, so_l, sdu_b, sdu_l;
    float *partials;              // [tiles][Cn][K + 1]: dw shares, then the dbias share
    int64_t tiles_per_row;
    // carried windows: [nslots][K - 1][Cn] at slot stride sw, slot[s] of sequence s (or s), fresh where has[s] is 0
    void *win;
    int64_t nslots, sw;
    const int32_t *slot;
    const uint8_t *has;
};

// Sequence bookkeeping along a sweep: the start of the current token's sequence and the
// first token of the next one.
struct SeqCursor {
    int64_t start, next;
    int s;
    __device__ void init(const ConvArgs &a, int64_t t) {
        if (a.cu == nullptr) {
            start = 0;
            next = a.L;
            s = 0;
            return;
        }
        int lo = 0, hi = (int)a.S - 1;   // last s with cu[s] <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.cu[mid] <= t) lo = mid; else hi = mid - 1;
        }
        s = lo;
        start = max(a.cu[s], 0);   // clamped: a malformed cu_seqlens never moves a load off the row
        next = a.cu[s + 1];
    }
    // advances to token t (non-decreasing); true when t starts a new sequence
    __device__ bool advance(const ConvArgs &a, int64_t t) {
        if (a.cu == nullptr || t < next) return false;
        while (s + 1 < a.S && a.cu[s + 1] <= t) ++s;
        start = max(a.cu[s], 0);
        next = a.cu[s + 1];
        return true;
    }
};

// ---- backward: a staged sweep.  A block covers TT tokens x CB channels; its threads first copy the tile
// (plus the K-1 rows before and after it) into shared memory with cp.async -- a whole tile of loads in
// flight at once -- and then thread (piece j, token group g) sweeps its W channels over TGB = 16 tokens
// (W = 4, 256 threads, about 110 registers, two blocks per SM) from shared memory.
// (Measured: with W = 8 or 2 a tenth slower.)
constexpr int CB = 256;              // channels per block (32 pieces of 8)
constexpr int CTB = 128;             // backward: threads per block (two blocks per SM) ...
constexpr int TGB = TT / (CTB / 32); // ... and tokens per thread: 16
#define TAPS_BYTES(K) ((size_t)((K) + 1) * CB * sizeof(float))   // staged taps and bias
#ifndef CONV_BWD_W
#define CONV_BWD_W 4
#endif

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit_wait() {
    asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
}

// Copies rows [tb, tb + nrows) of a [L][channels] token matrix (row stride sl elements),
// channels [cbase, cbase + CB), into `dst` (row r at r * 32 pieces); rows outside [0, L) and
// channels past Cn are not copied (never read unmasked).
template <typename T>
__device__ __forceinline__ void stage_rows(const T *src, int64_t sl, int64_t tb, int nrows, int64_t L, int64_t cbase,
                                           int64_t Cn, T *dst) {
    for (int i = threadIdx.x; i < nrows * 32; i += blockDim.x) {
        const int r = i >> 5, j = i & 31;
        const int64_t t = tb + r, c = cbase + 8 * j;
        if (t >= 0 && t < L && c < Cn) {
            const T *g = src + t * sl + c;
            T *d = dst + (int64_t)r * (32 * 8) + 8 * j;
            if (sizeof(T) == 2) {
                cp_async16(d, g);
            } else {
                cp_async16(d, g);
                cp_async16(d + 4, g + 4);
            }
        }
    }
    cp_async_commit_wait();
}

// 4 channels: 8 bytes (bf16) or 16 bytes (fp32)
__device__ __forceinline__ void ld4(const __nv_bfloat16 *p, float *v) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}
__device__ __forceinline__ void ld4(const float *p, float *v) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void st4(__nv_bfloat16 *p, const float *v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    uint2 u;
    u.x = *reinterpret_cast<const uint32_t *>(&a);
    u.y = *reinterpret_cast<const uint32_t *>(&b);
    *reinterpret_cast<uint2 *>(p) = u;
}
__device__ __forceinline__ void st4(float *p, const float *v) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
// 2 channels: 4 bytes (bf16) or 8 bytes (fp32)
__device__ __forceinline__ void ld2(const __nv_bfloat16 *p, float *v) {
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(p));
    v[0] = a.x; v[1] = a.y;
}
__device__ __forceinline__ void ld2(const float *p, float *v) {
    const float2 a = *reinterpret_cast<const float2 *>(p);
    v[0] = a.x; v[1] = a.y;
}
__device__ __forceinline__ void st2(__nv_bfloat16 *p, const float *v) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v[0], v[1]);
}
__device__ __forceinline__ void st2(float *p, const float *v) { *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]); }
template <int W, typename T>
__device__ __forceinline__ void ldw(const T *p, float *v) {
    if (W == 8) ld8(p, v); else if (W == 4) ld4(p, v); else ld2(p, v);
}
template <int W, typename T>
__device__ __forceinline__ void stw(T *p, const float *v) {
    if (W == 8) st8(p, v); else if (W == 4) st4(p, v); else st2(p, v);
}

// logistic function with the fast exponential and divide (relative error ~1e-6; 1/inf = 0
// gives the right limit for very negative arguments)
__device__ __forceinline__ float sig_fast(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }
// the same for bf16 data, without the division's range checks.  Not (1 + tanh(v / 2)) / 2 with the approximate tanh, one
// operation of the multi-function unit instead of two: its error, 2^-12 of 1, is 1% of the result at v = -4 and all
// of it from v = -8 on.
__device__ __forceinline__ float sig_rcp(float v) { return rcpf(1.f + ex2f(-kLog2e * v)); }
template <typename T>
__device__ __forceinline__ float sig_t(float v) { return sizeof(T) == 2 ? sig_rcp(v) : sig_fast(v); }

// The block's taps and biases, staged once in shared memory as [k][channel] (then [K][c] =
// the bias): weight [Cn][K] holds channels cbase .. cbase+255 as 256K contiguous floats, read
// with consecutive threads on consecutive floats; a thread then reads its 8 channels of tap k
// as two 16-byte pieces.
template <int K>
__device__ __forceinline__ void stage_taps(const float *w, const float *bias, int64_t cbase, int64_t Cn, float *ws) {
    const int64_t nch = std::min<int64_t>(CB, Cn - cbase);
    for (int i = threadIdx.x; i < CB * K; i += blockDim.x) {
        const int c = i / K, k = i % K;
        ws[k * CB + c] = c < nch ? w[cbase * K + i] : 0.f;
    }
    for (int c = threadIdx.x; c < CB; c += blockDim.x)
        ws[K * CB + c] = (bias != nullptr && c < nch) ? bias[cbase + c] : 0.f;
}

// ---- forward.  A thread sweeps FT tokens of its W channels: it loads FB rows at a time straight from
// global memory (all in flight before the first is used; only the K - 1 rows before its run are read a
// second time), keeps the last K rows as fp32 pairs, and does the taps and the gate's products
// two channels to an instruction.
// Bytes bound it: at 8191 x 6144 bf16, width 4, 39 us for 201 MB (5.1 TB/s, 76% of a plain copy; instructions
// issue in 60% of the cycles), 41 in six packed pieces (40 with a single approximate tanh for the gate).  Before launches overlapped it took 46; W = 8 then at best 48, four rows in flight 47, 32
// tokens a run 50, 512-thread blocks 67, a staged tile in shared memory 56.
constexpr int kFwdW = 4, FG = 2, FT = 16, FB = 8;   // channels a thread; runs in a block; tokens of a run; rows in flight

// W neighbouring channels of one row, as they lie in memory
template <typename T, int W>
struct Row;
template <int W>
struct Row<float, W> {
    float4 v[W / 4];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ void store(float *p) const {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) reinterpret_cast<float4 *>(p)[i] = v[i];
    }
    __device__ __forceinline__ void load(const float *p) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) v[i] = reinterpret_cast<const float4 *>(p)[i];
    }
    __device__ __forceinline__ void pairs(f32x2 (&o)[W / 2]) const {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            o[2 * i] = pk2(v[i].x, v[i].y);
            o[2 * i + 1] = pk2(v[i].z, v[i].w);
        }
    }
};
template <int W>
struct Row<__nv_bfloat16, W> {
    uint32_t v[W / 2];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) v[i] = 0;
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
        if constexpr (W == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(v[0], v[1], v[2], v[3]);
        else *reinterpret_cast<uint2 *>(p) = make_uint2(v[0], v[1]);
    }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        if constexpr (W == 8) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            v[0] = u.x; v[1] = u.y;
        }
    }
    __device__ __forceinline__ void pairs(f32x2 (&o)[W / 2]) const {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) o[i] = pk2(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xffff0000u));
    }
};

// v (v silu's logistic function), in the arithmetic of sig_t<T>
template <typename T>
__device__ __forceinline__ f32x2 silu2(f32x2 v) {
    float lo, hi;
    if (sizeof(T) == 2) {
        up2(mul2(pk2(-kLog2e, -kLog2e), v), lo, hi);
        up2(add2(pk2(1.f, 1.f), pk2(ex2f(lo), ex2f(hi))), lo, hi);
        return mul2(v, pk2(rcpf(lo), rcpf(hi)));
    }
    up2(v, lo, hi);
    return pk2(lo * sig_fast(lo), hi * sig_fast(hi));
}
template <typename T, int W>
__device__ __forceinline__ void store_pairs(T *p, const f32x2 (&v)[W / 2]) {
    float o[W];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) up2(v[i], o[2 * i], o[2 * i + 1]);
    stw<W>(p, o);
}

// The carried window of sequence s (its rows are K - 1 back to 1 before the first token), or NULL for padding.
template <typename T>
__device__ __forceinline__ T *window(const ConvArgs &a, int64_t s, int K) {
    const int64_t k = a.slot ? a.slot[s] : s;
    if (K == 1 || k < 0 || k >= a.nslots) return nullptr;
    return static_cast<T *>(a.win) + k * a.sw;
}

// the taps over rows[0 .. K - 1] -> out
template <typename T, int K, int W>
__device__ __forceinline__ void one_row(const f32x2 (&w)[K][W / 2], const f32x2 (&bias)[W / 2], bool silu, T *out, const f32x2 (*rows)[W / 2]) {
    f32x2 acc[W / 2];
#pragma unroll
    for (int h = 0; h < W / 2; ++h) {
        acc[h] = bias[h];
#pragma unroll
        for (int k = 0; k < K; ++k) acc[h] = fma2(w[k][h], rows[k][h], acc[h]);
    }
    if (silu) {
#pragma unroll
        for (int h = 0; h < W / 2; ++h) acc[h] = silu2<T>(acc[h]);
    }
    store_pairs<T, W>(out, acc);
}

// With carried windows, a sequence's first K - 1 outputs and its new window come from the same
// thread, which reads the old window before it writes (other blocks never touch windows).  1025 tokens of 40
// sequences x 6144 take 10 us with all its loads at once, 12 with a token's after another's.
template <typename T, int K, int W>
__device__ void conv_edge(const ConvArgs &a, int64_t s, int64_t c0, const f32x2 (&w)[K][W / 2], const f32x2 (&bias)[W / 2]) {
    const int64_t b = a.cu ? 0 : s;
    const int64_t t0 = a.cu ? min(max((int64_t)a.cu[s], (int64_t)0), a.L) : 0;
    const int64_t t1 = a.cu ? min(max((int64_t)a.cu[s + 1], t0), a.L) : a.L;
    T *win = window<T>(a, s, K);
    const bool old = win != nullptr && (a.has == nullptr || a.has[s] != 0);
    const T *u = static_cast<const T *>(a.u) + b * a.su_b + c0;
    T *o = static_cast<T *>(a.out) + b * a.so_b + c0;
    const int n = (int)min(t1 - t0, (int64_t)(K - 1));
    if constexpr (K > 1) {
        Row<T, W> last[K - 1], first[K - 1], before[K - 1];   // everything is on its way before the first is used
        if (win) {
#pragma unroll
            for (int k = 0; k < K - 1; ++k) {   // new row k is K - 1 - k before the end: a token, or old row n + k
                const int64_t t = t1 - (K - 1) + k;
                last[k].zero();
                if (t >= t0) last[k].load(u + t * a.su_l);
                else if (old) last[k].load(win + (n + k) * a.Cn + c0);
            }
        }
        if (n > 0) {
#pragma unroll
            for (int k = 0; k < K - 1; ++k) {
                before[k].zero();
                if (old) before[k].load(win + k * a.Cn + c0);
                first[k].load(u + (t0 + min(k, n - 1)) * a.su_l);
            }
            f32x2 rows[2 * K - 2][W / 2];
#pragma unroll
            for (int k = 0; k < K - 1; ++k) {
                before[k].pairs(rows[k]);
                first[k].pairs(rows[K - 1 + k]);
            }
#pragma unroll
            for (int i = 0; i < K - 1; ++i)
                if (i < n) one_row<T, K, W>(w, bias, a.silu, o + (t0 + i) * a.so_l, rows + i);
        }
        if (win) {
#pragma unroll
            for (int k = 0; k < K - 1; ++k) last[k].store(win + k * a.Cn + c0);
        }
    }
}

// The tokens [s0, s1) of a run.  STARTS: sequences start there or less than K - 1 tokens before; a start clears the
// rows before it, and with CARRY the K - 1 outputs after it are conv_edge's.
template <typename T, int K, int W, bool CARRY, bool STARTS>
__device__ __forceinline__ void conv_run(const ConvArgs &a, SeqCursor &cur, int64_t s0, int64_t s1, const T *u, T *o,
                                         const f32x2 (&w)[K][W / 2], const f32x2 (&bias)[W / 2]) {
    f32x2 rows[K - 1 + FB][W / 2];
    const T *p = u + (s0 - (K - 1)) * a.su_l;
    T *q = o + s0 * a.so_l;
#pragma unroll
    for (int k = 0; k < K - 1; ++k, p += a.su_l) {
        Row<T, W> r;
        const bool in = !STARTS || s0 - (K - 1) + k >= cur.start;
        r.load(in ? p : u + s0 * a.su_l);
        r.pairs(rows[k]);
        if (!in) {
#pragma unroll
            for (int h = 0; h < W / 2; ++h) rows[k][h] = 0;
        }
    }
    const int n = (int)(s1 - s0);
    Row<T, W> raw[FB];
#pragma unroll
    for (int e = 0; e < FB; ++e, p += a.su_l)
        if (e < n) raw[e].load(p);
#pragma unroll 1
    for (int i = 0; i < n; i += FB) {
#pragma unroll
        for (int e = 0; e < FB; ++e, p += a.su_l) {
            raw[e].pairs(rows[K - 1 + e]);
            if (i + FB + e < n) raw[e].load(p);                 // FB rows are on their way all the time
            if (i + e < n) {
                bool put = true;
                if (STARTS) {
                    const int64_t t = s0 + i + e;
                    cur.advance(a, t);
                    const int fresh = (int)min(max(cur.start - (t - (K - 1)), (int64_t)0), (int64_t)K);   // rows before the start
                    if (fresh > 0) {
#pragma unroll
                        for (int k = 0; k < K; ++k)
#pragma unroll
                            for (int h = 0; h < W / 2; ++h) rows[e + k][h] = k < fresh ? 0 : rows[e + k][h];
                    }
                    put = !CARRY || fresh == 0;
                }
                if (put) one_row<T, K, W>(w, bias, a.silu, q, rows + e);
                q += a.so_l;
            }
        }
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
#pragma unroll
            for (int h = 0; h < W / 2; ++h) rows[k][h] = rows[FB + k][h];
    }
}

// CARRY: sequences go on from carried windows; the first blocks do their edges, which take longest.
template <typename T, int K, int W, bool CARRY>
__global__ void __launch_bounds__(FG * CB / W, K > 4 ? 1 : sizeof(T) == 2 ? 6 : 4) k_conv_fwd(const ConvArgs a, int cols) {
    after_previous();
    constexpr int NPC = CB / W;        // channel pieces of a block
    const int j = threadIdx.x % NPC, grp = threadIdx.x / NPC;
    int64_t bx = blockIdx.x / cols;
    const int64_t c0 = (int64_t)(blockIdx.x % cols) * CB + W * j;   // neighbouring blocks: one row's channels
    if (c0 >= a.Cn) return;
    f32x2 w[K][W / 2], bias[W / 2];
    {
        float wv[W * K];                // the W channels' taps are contiguous
        const float *wp = a.w + c0 * K;
        if ((uintptr_t)a.w % 16 == 0) {
#pragma unroll
            for (int i = 0; i < W * K / 4; ++i) {
                const float4 v = reinterpret_cast<const float4 *>(wp)[i];
                wv[4 * i] = v.x; wv[4 * i + 1] = v.y; wv[4 * i + 2] = v.z; wv[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < W * K; ++i) wv[i] = wp[i];
        }
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
#pragma unroll
            for (int k = 0; k < K; ++k) w[k][i] = pk2(wv[2 * i * K + k], wv[(2 * i + 1) * K + k]);
            bias[i] = a.bias ? pk2(a.bias[c0 + 2 * i], a.bias[c0 + 2 * i + 1]) : pk2(0.f, 0.f);
        }
    }
    const int64_t runs = (a.L + FT * FG - 1) / (FT * FG);       // blocks per row
    if (CARRY) {
        const int64_t ns = a.cu ? a.S : a.B, edges = (ns + FG - 1) / FG;
        if (bx < edges) {
            if (bx * FG + grp < ns) conv_edge<T, K, W>(a, bx * FG + grp, c0, w, bias);
            return;
        }
        bx -= edges;
    }
    const int64_t b = bx / runs, s0 = (bx % runs * FG + grp) * FT, s1 = std::min(a.L, s0 + FT);   // this thread's tokens
    if (s0 >= s1) return;
    const T *u = static_cast<const T *>(a.u) + b * a.su_b + c0;
    T *o = static_cast<T *>(a.out) + b * a.so_b + c0;
    SeqCursor cur;
    cur.init(a, s0);
    if (s0 - (K - 1) < cur.start || s1 > cur.next)              // a sequence starts within the run, or less than K - 1 tokens before it
        conv_run<T, K, W, CARRY, true>(a, cur, s0, s1, u, o, w, bias);
    else
        conv_run<T, K, W, CARRY, false>(a, cur, s0, s1, u, o, w, bias);
}

// Backward over the thread's tokens [s0, s1): the sweep runs t from s0 to s1 + K - 2 computing
// g[t] = dout[t] act'(pre[t]); g[t] reaches du[t - (K-1) + k] (same sequence) for every k;
// du[t'] is complete once t passes t' + K - 1 and leaves then.  dw and dbias take the thread's
// tokens t in [s0, s1); the eight token groups' shares are summed in order in shared memory.
template <typename T, int K, int W>   // W channels per thread (8: 128 threads, 4: 256 threads)
__global__ void __launch_bounds__(CTB * 8 / W)
k_conv_bwd(const ConvArgs a) {
    constexpr int NPC = CB / W;        // channel pieces per row
    constexpr int NT = NPC * (TT / TGB);
    extern __shared__ __align__(16) uint8_t conv_sm[];
    constexpr int RU = TT + 2 * (K - 1), RD = TT + K - 1;
    float *ws = reinterpret_cast<float *>(conv_sm);                    // taps [K][CB], bias [CB]
    T *tu = reinterpret_cast<T *>(conv_sm + TAPS_BYTES(K));            // u rows t0-(K-1) .. t0+TT+K-2
    T *td = tu + RU * 256;                                             // dout rows t0 .. t0+TT+K-2
    float *red = reinterpret_cast<float *>(conv_sm + TAPS_BYTES(K));   // after the sweep: [group][K+1][256]
    const int j = threadIdx.x % NPC, grp = threadIdx.x / NPC;
    const int64_t cbase = (int64_t)blockIdx.y * CB, c0 = cbase + W * j;
    const int64_t b = blockIdx.x / a.tiles_per_row, t0 = (blockIdx.x % a.tiles_per_row) * TT;
    const int64_t tb = t0 - (K - 1);
    stage_taps<K>(a.w, a.bias, cbase, a.Cn, ws);
    stage_rows(static_cast<const T *>(a.u) + b * a.su_b, a.su_l, tb, RU, a.L, cbase, a.Cn, tu);
    stage_rows(static_cast<const T *>(a.dout) + b * a.sd_b, a.sd_l, t0, RD, a.L, cbase, a.Cn, td);
    __syncthreads();
    const bool live = c0 < a.Cn;
    const int64_t s0 = t0 + (int64_t)grp * TGB, s1 = std::min(a.L, s0 + TGB);
    float w[K][W], bias[W], dw[K][W], db[W];
#pragma unroll
    for (int k = 0; k <= K; ++k) {   // the thread's W channels of tap k (k = K: the bias)
        float *dst = k < K ? w[k < K ? k : 0] : bias;
#pragma unroll
        for (int e = 0; e < W; ++e) dst[e] = ws[k * CB + W * j + e];
    }
#pragma unroll
    for (int e = 0; e < W; ++e) {
        db[e] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k][e] = 0.f;
    }
    if (live && s0 < s1) {
        T *du = static_cast<T *>(a.du) + b * a.sdu_b + c0;
        const T *ucol = tu + W * j, *dcol = td + W * j;
        SeqCursor cur;
        cur.init(a, s0);
        float ring[K][W];   // inputs u[t - (K-1) + k]
        float acc[K][W];    // du[t - (K-1) + k] being summed
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < W; ++e) acc[k][e] = 0.f;
        const int64_t tend_all = std::min(a.L, s1 + K - 1);
        if (s0 - (K - 1) >= cur.start && tend_all <= cur.next) {
            // The thread's whole window (its tokens, the K-1 before and after) lies in one
            // sequence: no sequence starts to test, 32-bit counters, pointers that step a row.
            const T *up = ucol + (int)(s0 - t0) * 256, *dp = dcol + (int)(s0 - t0) * 256;
#pragma unroll
            for (int k = 0; k < K - 1; ++k) ldw<W>(up + k * 256, ring[k]);
            up += (K - 1) * 256;
            T *dup = du + (s0 - (K - 1)) * a.sdu_l;   // du[t - (K-1)] of the current t
            const int nown = (int)(s1 - s0), ntot = (int)(tend_all - s0);
#pragma unroll 4   // the ring and accumulator rotation becomes register renaming
            for (int i = 0; i < ntot; ++i) {
                ldw<W>(up, ring[K - 1]);
                up += 256;
                float dv[W];
                ldw<W>(dp, dv);
                dp += 256;
                float g[W];
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    float pre = bias[e];
#pragma unroll
                    for (int k = 0; k < K; ++k) pre = fmaf(w[k][e], ring[k][e], pre);
                    if (a.silu) {
                        const float sg = sig_t<T>(pre);
                        g[e] = dv[e] * sg * (1.f + pre * (1.f - sg));
                    } else {
                        g[e] = dv[e];
                    }
                }
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int e = 0; e < W; ++e) acc[k][e] = fmaf(w[k][e], g[e], acc[k][e]);
                if (i < nown) {   // this thread's token: its dw / dbias shares
#pragma unroll
                    for (int e = 0; e < W; ++e) {
#pragma unroll
                        for (int k = 0; k < K; ++k) dw[k][e] = fmaf(g[e], ring[k][e], dw[k][e]);
                        db[e] += g[e];
                    }
                }
                if (i >= K - 1) stw<W>(dup, acc[0]);   // du[s0 + i - (K-1)] is complete
                dup += a.sdu_l;
#pragma unroll
                for (int k = 0; k < K - 1; ++k)
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        ring[k][e] = ring[k + 1][e];
                        acc[k][e] = acc[k + 1][e];
                    }
#pragma unroll
                for (int e = 0; e < W; ++e) acc[K - 1][e] = 0.f;
            }
            // rows whose windows would run past the end of the row (tend_all clamped to L)
            for (int64_t tdone = tend_all - (K - 1); tdone < s1; ++tdone) {
                if (tdone >= s0) stw<W>(du + tdone * a.sdu_l, acc[0]);
#pragma unroll
                for (int k = 0; k < K - 1; ++k)
#pragma unroll
                    for (int e = 0; e < W; ++e) acc[k][e] = acc[k + 1][e];
#pragma unroll
                for (int e = 0; e < W; ++e) acc[K - 1][e] = 0.f;
            }
        } else {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            const int64_t tp = s0 - (K - 1) + k;
            if (tp >= cur.start) ldw<W>(ucol + (int)(tp - tb) * 256, ring[k]);
            else {
#pragma unroll
                for (int e = 0; e < W; ++e) ring[k][e] = 0.f;
            }
        }
        const int64_t tend = std::min(a.L, s1 + K - 1);
        for (int64_t t = s0; t < tend; ++t) {
            if (cur.advance(a, t)) {
#pragma unroll
                for (int k = 0; k < K - 1; ++k)
#pragma unroll
                    for (int e = 0; e < W; ++e) ring[k][e] = 0.f;
            }
            ldw<W>(ucol + (int)(t - tb) * 256, ring[K - 1]);
            float dv[W];
            ldw<W>(dcol + (int)(t - t0) * 256, dv);
            float g[W];
#pragma unroll
            for (int e = 0; e < W; ++e) {
                float pre = bias[e];
#pragma unroll
                for (int k = 0; k < K; ++k) pre = fmaf(w[k][e], ring[k][e], pre);
                if (a.silu) {
                    const float sg = sig_t<T>(pre);
                    g[e] = dv[e] * sg * (1.f + pre * (1.f - sg));
                } else {
                    g[e] = dv[e];
                }
            }
            const bool own = t < s1;   // this thread's token: its dw / dbias shares
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int64_t tp = t - (K - 1) + k;
                if (tp >= cur.start) {   // u[tp] fed pre[t] (same sequence)
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        acc[k][e] = fmaf(w[k][e], g[e], acc[k][e]);
                        if (own) dw[k][e] = fmaf(g[e], ring[k][e], dw[k][e]);
                    }
                }
            }
            if (own) {
#pragma unroll
                for (int e = 0; e < W; ++e) db[e] += g[e];
            }
            const int64_t tdone = t - (K - 1);   // du[tdone] has all its contributions now
            if (tdone >= s0 && tdone < s1) stw<W>(du + tdone * a.sdu_l, acc[0]);
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    ring[k][e] = ring[k + 1][e];
                    acc[k][e] = acc[k + 1][e];
                }
#pragma unroll
            for (int e = 0; e < W; ++e) acc[K - 1][e] = 0.f;
        }
        // the last rows, whose windows would run past the end of the row: acc[0] now holds
        // du[tend - (K-1)]; rows before s0 are skipped over
        for (int64_t tdone = tend - (K - 1); tdone < s1; ++tdone) {
            if (tdone >= s0) stw<W>(du + tdone * a.sdu_l, acc[0]);
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
#pragma unroll
                for (int e = 0; e < W; ++e) acc[k][e] = acc[k + 1][e];
#pragma unroll
            for (int e = 0; e < W; ++e) acc[K - 1][e] = 0.f;
        }
        }   // general path
    }
    __syncthreads();   // the staged tiles are no longer read: reuse them for the group sums
#pragma unroll
    for (int e = 0; e < W; ++e) {
#pragma unroll
        for (int k = 0; k < K; ++k) red[((grp * (K + 1)) + k) * 256 + W * j + e] = dw[k][e];
        red[((grp * (K + 1)) + K) * 256 + W * j + e] = db[e];
    }
    __syncthreads();
    float *pp = a.partials + (int64_t)blockIdx.x * a.Cn * (K + 1);
    for (int i = threadIdx.x; i < 256 * (K + 1); i += NT) {
        const int c = i / (K + 1), k = i % (K + 1);   // channel within the block, tap (K: bias)
        if (cbase + c >= a.Cn) continue;
        float sum = 0.f;
        for (int q = 0; q < TT / TGB; ++q) sum += red[(q * (K + 1) + k) * 256 + c];
        pp[(cbase + c) * (K + 1) + k] = sum;
    }
}

// dw / dbias: the column sums of the per-tile shares [tiles][Cn (K+1)] in a fixed order.  A
// block takes 32 columns; warp w sums tiles w, w + 8, ... in ascending order (four loads in
// flight), and the eight warp sums are added in warp order.
__global__ void __launch_bounds__(256) k_conv_dw(const float *partials, int64_t tiles, int64_t Cn, int K, float *dw,
                                                 float *db) {
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t n = Cn * (K + 1), i = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (i < n) {
        const float *col = partials + i;
        int64_t t = w;
        for (; t + 24 < tiles; t += 32) {
            const float a0 = col[t * n], a1 = col[(t + 8) * n], a2 = col[(t + 16) * n], a3 = col[(t + 24) * n];
            s += a0;
            s += a1;
            s += a2;
            s += a3;
        }
        for (; t < tiles; t += 8) s += col[t * n];
    }
    red[w][lane] = s;
    __syncthreads();
    if (w == 0 && i < n) {
        float tot = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) tot += red[q][lane];
        const int64_t c = i / (K + 1);
        const int k = (int)(i - c * (K + 1));
        if (k < K) dw[c * K + k] = tot;
        else if (db) db[c] = tot;
    }
}

// One token for each of a batch of requests: thread (request, 8 channels) reads the window's K - 1
// rows and the new one, and writes the window one row on.  64 requests x 6144, bf16: 4 us, the launch (6.4 MB).
template <typename T, int K>
__global__ void __launch_bounds__(128) k_conv_step(const ConvArgs a, int cols) {
    after_previous();
    const int64_t c0 = ((int64_t)(blockIdx.x % cols) * 128 + threadIdx.x) * 8, b = blockIdx.x / cols;
    if (c0 >= a.Cn) return;
    T *win = window<T>(a, b, K);
    float rows[K][8], w[8 * K];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
        if (win) ld8(win + k * a.Cn + c0, rows[k]);
        else {
#pragma unroll
            for (int e = 0; e < 8; ++e) rows[k][e] = 0.f;
        }
    }
    ld8(static_cast<const T *>(a.u) + b * a.su_b + c0, rows[K - 1]);
    const float *wp = a.w + c0 * K;   // the 8 channels' taps are contiguous
    if ((uintptr_t)a.w % 16 == 0) {
#pragma unroll
        for (int i = 0; i < 2 * K; ++i) {
            const float4 v = reinterpret_cast<const float4 *>(wp)[i];
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8 * K; ++i) w[i] = wp[i];
    }
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        acc[e] = a.bias ? a.bias[c0 + e] : 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) acc[e] = fmaf(w[e * K + k], rows[k][e], acc[e]);
        if (a.silu) acc[e] *= sig_t<T>(acc[e]);
    }
    st8(static_cast<T *>(a.out) + b * a.so_b + c0, acc);
    if (win) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) st8(win + k * a.Cn + c0, rows[k + 1]);
    }
}

template <typename T, int K>
size_t bwd_smem() {
    const size_t stage = (size_t)(2 * TT + 3 * (K - 1)) * 256 * sizeof(T);
    const size_t red = (size_t)(TT / TGB) * (K + 1) * 256 * sizeof(float);
    return TAPS_BYTES(K) + (stage > red ? stage : red);
}
template <typename T, int K, bool CARRY>
cudaError_t launch_fwd_k(const ConvArgs &a, cudaStream_t st) {
    const int64_t ns = a.cu ? a.S : a.B;
    const int64_t blocks = a.B * ((a.L + FT * FG - 1) / (FT * FG)) + (CARRY ? (ns + FG - 1) / FG : 0);
    const int64_t cols = (a.Cn + CB - 1) / CB;
    if (blocks * cols > ((int64_t)1 << 31) - 1) return cudaErrorInvalidConfiguration;
    return launch_early(k_conv_fwd<T, K, kFwdW, CARRY>, (unsigned)(blocks * cols), FG * CB / kFwdW, 0, st, a, (int)cols);
}
constexpr int kBwdW = CONV_BWD_W;   // channels per thread of the backward sweep
template <typename T, int K>
cudaError_t launch_bwd_k(const ConvArgs &a, dim3 grid, cudaStream_t st) {
    static int attr[64] = {0};
    const size_t sm = bwd_smem<T, K>();
    cudaError_t e = ensure_smem_attr(k_conv_bwd<T, K, kBwdW>, (int)sm, attr);
    if (e != cudaSuccess) return e;
    k_conv_bwd<T, K, kBwdW><<<grid, CTB * 8 / kBwdW, sm, st>>>(a);
    return cudaGetLastError();
}

template <typename T, bool CARRY>
cudaError_t launch_fwd(const ConvArgs &a, cudaStream_t st) {
    switch (a.K) {
        case 1: return launch_fwd_k<T, 1, CARRY>(a, st);
        case 2: return launch_fwd_k<T, 2, CARRY>(a, st);
        case 3: return launch_fwd_k<T, 3, CARRY>(a, st);
        case 4: return launch_fwd_k<T, 4, CARRY>(a, st);
        case 5: return launch_fwd_k<T, 5, CARRY>(a, st);
        case 6: return launch_fwd_k<T, 6, CARRY>(a, st);
        case 7: return launch_fwd_k<T, 7, CARRY>(a, st);
        default: return launch_fwd_k<T, 8, CARRY>(a, st);
    }
}
template <typename T>
cudaError_t launch_bwd(const ConvArgs &a, dim3 grid, cudaStream_t st) {
    switch (a.K) {
        case 1: return launch_bwd_k<T, 1>(a, grid, st);
        case 2: return launch_bwd_k<T, 2>(a, grid, st);
        case 3: return launch_bwd_k<T, 3>(a, grid, st);
        case 4: return launch_bwd_k<T, 4>(a, grid, st);
        case 5: return launch_bwd_k<T, 5>(a, grid, st);
        case 6: return launch_bwd_k<T, 6>(a, grid, st);
        case 7: return launch_bwd_k<T, 7>(a, grid, st);
        default: return launch_bwd_k<T, 8>(a, grid, st);
    }
}

template <typename T>
cudaError_t launch_step(const ConvArgs &a, cudaStream_t st) {
    const int cols = (int)((a.Cn / 8 + 127) / 128);
    const unsigned grid = (unsigned)(cols * a.B);
    switch (a.K) {
        case 1: return launch_early(k_conv_step<T, 1>, grid, 128, 0, st, a, cols);
        case 2: return launch_early(k_conv_step<T, 2>, grid, 128, 0, st, a, cols);
        case 3: return launch_early(k_conv_step<T, 3>, grid, 128, 0, st, a, cols);
        case 4: return launch_early(k_conv_step<T, 4>, grid, 128, 0, st, a, cols);
        case 5: return launch_early(k_conv_step<T, 5>, grid, 128, 0, st, a, cols);
        case 6: return launch_early(k_conv_step<T, 6>, grid, 128, 0, st, a, cols);
        case 7: return launch_early(k_conv_step<T, 7>, grid, 128, 0, st, a, cols);
        default: return launch_early(k_conv_step<T, 8>, grid, 128, 0, st, a, cols);
    }
}

bool al16(const void *p) { return ((uintptr_t)p) % 16 == 0; }

// Host checks shared by both directions.  Token tensors: [batch, seqlen, channels] at element
// strides (row, token); channels contiguous.
ssd_status check_conv(const ssd_conv_problem *p, bool varlen) {
    if (p == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    if (p->batch < 1 || p->seqlen < 0 || p->channels < 1 || p->width < 1 || p->reserved != 0)
        return SSD_ERR_INVALID_ARGUMENT;
    if (p->dtype < SSD_F32 || p->dtype > SSD_BF16 || p->activation < 0 || p->activation > 1)
        return SSD_ERR_INVALID_ARGUMENT;
    if (varlen && (p->batch != 1 || p->nseqs < 1)) return SSD_ERR_INVALID_ARGUMENT;
    if (!varlen && p->nseqs != 0) return SSD_ERR_INVALID_ARGUMENT;
    if (p->width > KMAX || p->channels % 8 != 0 || p->seqlen > ((int64_t)1 << 31) || p->nseqs > ((int64_t)1 << 24))
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}
ssd_status check_tok(const ssd_conv_problem *p, const void *t, int64_t sb, int64_t sl) {
    if (p->seqlen == 0) return SSD_OK;
    if (t == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    if (sl < p->channels || (p->batch > 1 && sb < sl * p->seqlen)) return SSD_ERR_INVALID_ARGUMENT;
    if (!al16(t) || sl % 8 != 0 || sb % 8 != 0) return SSD_ERR_MISALIGNED;
    return SSD_OK;
}

ssd_status check_win(const ssd_conv_problem *p, const void *win, int64_t nslots, int64_t stride, const int32_t *slot) {
    if (nslots < 0) return SSD_ERR_INVALID_ARGUMENT;
    if ((uintptr_t)slot % 4 != 0) return SSD_ERR_MISALIGNED;
    if (nslots == 0 || p->width == 1) return SSD_OK;
    if (win == nullptr || (nslots > 1 && stride < (p->width - 1) * p->channels)) return SSD_ERR_INVALID_ARGUMENT;
    return al16(win) && (nslots == 1 || stride % 8 == 0) ? SSD_OK : SSD_ERR_MISALIGNED;
}

#define CONV_TRY(expr)                 \
    do {                               \
        ssd_status _s = (expr);        \
        if (_s != SSD_OK) return _s;   \
    } while (0)

ConvArgs make_args(const ssd_conv_problem *p, const float *w, const float *bias, const int32_t *cu) {
    ConvArgs a{};
    a.B = p->batch; a.L = p->seqlen; a.Cn = p->channels; a.S = cu ? p->nseqs : 0; a.K = (int)p->width;
    a.silu = p->activation == 1;
    a.w = w; a.bias = bias; a.cu = cu;
    a.tiles_per_row = (p->seqlen + TT - 1) / TT;
    return a;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_conv1d_fwd(const ssd_conv_problem *p, const void *x, int64_t x_sb, int64_t x_sl, const float *weight,
                          const float *bias, const int32_t *cu_seqlens, void *out, int64_t out_sb, int64_t out_sl,
                          void *stream) {
    CONV_TRY(check_conv(p, cu_seqlens != nullptr));
    CONV_TRY(check_tok(p, x, x_sb, x_sl));
    CONV_TRY(check_tok(p, out, out_sb, out_sl));
    if (weight == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    if (p->seqlen == 0) return SSD_OK;
    ConvArgs a = make_args(p, weight, bias, cu_seqlens);
    a.u = x; a.su_b = x_sb; a.su_l = x_sl; a.out = out; a.so_b = out_sb; a.so_l = out_sl;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = p->dtype == SSD_BF16 ? launch_fwd<__nv_bfloat16, false>(a, st) : launch_fwd<float, false>(a, st);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_conv1d_prompt(const ssd_conv_problem *p, const void *x, int64_t x_sb, int64_t x_sl, const float *weight,
                             const float *bias, const int32_t *cu_seqlens, void *conv_states, int64_t nslots,
                             int64_t slot_stride, const int32_t *state_indices, const uint8_t *has_initial, void *out,
                             int64_t out_sb, int64_t out_sl, void *stream) {
    CONV_TRY(check_conv(p, cu_seqlens != nullptr));
    CONV_TRY(check_tok(p, x, x_sb, x_sl));
    CONV_TRY(check_tok(p, out, out_sb, out_sl));
    if (weight == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    CONV_TRY(check_win(p, conv_states, nslots, slot_stride, state_indices));
    ConvArgs a = make_args(p, weight, bias, cu_seqlens);
    a.u = x; a.su_b = x_sb; a.su_l = x_sl; a.out = out; a.so_b = out_sb; a.so_l = out_sl;
    a.win = conv_states; a.nslots = nslots; a.sw = slot_stride; a.slot = state_indices; a.has = has_initial;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = p->dtype == SSD_BF16 ? launch_fwd<__nv_bfloat16, true>(a, st) : launch_fwd<float, true>(a, st);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_conv1d_step(const ssd_conv_problem *p, const void *x, int64_t x_stride, const float *weight,
                           const float *bias, void *conv_states, int64_t nslots, int64_t slot_stride,
                           const int32_t *state_indices, void *out, int64_t out_stride, void *stream) {
    CONV_TRY(check_conv(p, false));
    if (p->seqlen != 1) return SSD_ERR_INVALID_ARGUMENT;
    if (p->batch * ((p->channels + 1023) / 1024) > ((int64_t)1 << 31) - 1) return SSD_ERR_UNSUPPORTED;
    CONV_TRY(check_tok(p, x, x_stride, p->channels));
    CONV_TRY(check_tok(p, out, out_stride, p->channels));
    if (weight == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    CONV_TRY(check_win(p, conv_states, nslots, slot_stride, state_indices));
    ConvArgs a = make_args(p, weight, bias, nullptr);
    a.u = x; a.su_b = x_stride; a.out = out; a.so_b = out_stride;
    a.win = conv_states; a.nslots = nslots; a.sw = slot_stride; a.slot = state_indices;
    const cudaError_t e = p->dtype == SSD_BF16 ? launch_step<__nv_bfloat16>(a, (cudaStream_t)stream)
                                               : launch_step<float>(a, (cudaStream_t)stream);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_conv1d_bwd_workspace_size(const ssd_conv_problem *p, size_t *bytes) {
    if (bytes == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    CONV_TRY(check_conv(p, p != nullptr && p->nseqs != 0));
    const int64_t tiles = p->batch * ((p->seqlen + TT - 1) / TT);
    *bytes = (size_t)std::max<int64_t>(tiles, 1) * (size_t)p->channels * (size_t)(p->width + 1) * sizeof(float);
    return SSD_OK;
}

ssd_status ssd_conv1d_bwd(const ssd_conv_problem *p, const void *x, int64_t x_sb, int64_t x_sl, const float *weight,
                          const float *bias, const int32_t *cu_seqlens, const void *dout, int64_t dout_sb,
                          int64_t dout_sl, void *dx, int64_t dx_sb, int64_t dx_sl, float *dweight, float *dbias,
                          void *workspace, size_t workspace_bytes, void *stream) {
    CONV_TRY(check_conv(p, cu_seqlens != nullptr));
    CONV_TRY(check_tok(p, x, x_sb, x_sl));
    CONV_TRY(check_tok(p, dout, dout_sb, dout_sl));
    CONV_TRY(check_tok(p, dx, dx_sb, dx_sl));
    if (weight == nullptr || dweight == nullptr || (bias != nullptr && dbias == nullptr)) return SSD_ERR_INVALID_ARGUMENT;
    const int64_t tiles = p->batch * ((p->seqlen + TT - 1) / TT);
    const size_t need = (size_t)std::max<int64_t>(tiles, 1) * (size_t)p->channels * (size_t)(p->width + 1) * sizeof(float);
    if (workspace == nullptr || workspace_bytes < need) return SSD_ERR_WORKSPACE_TOO_SMALL;
    if (!al16(workspace)) return SSD_ERR_MISALIGNED;
    cudaStream_t st = (cudaStream_t)stream;
    ConvArgs a = make_args(p, weight, bias, cu_seqlens);
    a.u = x; a.su_b = x_sb; a.su_l = x_sl; a.dout = dout; a.sd_b = dout_sb; a.sd_l = dout_sl;
    a.du = dx; a.sdu_b = dx_sb; a.sdu_l = dx_sl; a.partials = static_cast<float *>(workspace);
    if (tiles > 0) {
        const dim3 grid((unsigned)tiles, (unsigned)((a.Cn + CB - 1) / CB));
        const cudaError_t e =
            p->dtype == SSD_BF16 ? launch_bwd<__nv_bfloat16>(a, grid, st) : launch_bwd<float>(a, grid, st);
        if (e != cudaSuccess) return SSD_ERR_CUDA;
    } else {
        if (cudaMemsetAsync(workspace, 0, need, st) != cudaSuccess) return SSD_ERR_CUDA;
    }
    const int64_t n = p->channels * (p->width + 1);
    k_conv_dw<<<(unsigned)((n + 31) / 32), 256, 0, st>>>(
        a.partials, std::max<int64_t>(tiles, 1), p->channels, (int)p->width, dweight, dbias);
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
