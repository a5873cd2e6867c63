// qk_norm.cu -- queries and keys normalised per head, weighted and rotated by position, in one pass, and its backward:
//
//   n = x rstd w,  rstd = 1 / sqrt(mean x^2 + eps) or 1 / sqrt(sum x^2 + eps)
//   (y_a, y_b) = (n_a c - n_b s, n_a s + n_b c)
//   dn = w o (rotation backwards of dy),  dx = rstd (dn - x rstd <dn, x rstd> / (dim or 1)),  dw = sum of (rotated back dy) o x rstd
//
// A few operations a value, each value read once (backwards x and dy) and written once: bound by memory.  A head's vector
// belongs to 32 lanes or a power of two fewer, V neighbouring features each, so that a load is 16 bytes
// and the partner of a rotated feature lies in another lane's registers (a shuffle) or, interleaved, in
// the lane's own.  A group of lanes takes several heads of one token: their loads are all on the way
// before the first is used, and the token's cosines and sines are loaded once for them.  What the shapes or addresses keep
// from that goes feature by feature through shared memory.  The weights' gradients are summed in registers over a
// block's tokens, then over its groups, then by a second launch over the blocks, each in a fixed order.
// 8192 tokens x 40 heads of 128, bf16: 32.2 us for 172 MB (5.3 TB/s, 79% of a plain copy); backwards 4096 tokens 32 us for 129 MB and 5 for the weights' sums.
#include "selective.cuh"

namespace ssd {

namespace {

// Threads of a forward block: 7 blocks of 128 leave 72 registers a thread and start anew more evenly: 32.2 us where 3 of 256 took 35.8
// (8192 tokens x 40 heads of 128; 6 of 128 34.0, 8 of 128, 64 registers, 36.8).
constexpr int QK_FWD_NT = 128;
constexpr int QK_NT = 256, QK_HB_MIN = 2, QK_MAXD = 512;
constexpr int QK_BLOCKS = 3 * kSMs;     // of the backward: each leaves its share of the weights' gradients

struct QkSide {                         // queries, or keys
    const void *x, *dy;
    void *y;                            // the output, or dx
    int64_t xs[3], dys[3], ys[3];       // element strides: batch row, token, head
    const float *w;
    int heads, per;                     // heads, items of a token
    uint32_t items;                     // tokens x per
    float *share;                       // [blocks of this side][dim], or NULL
    float *dw;
};
struct QkArgs {
    QkSide side[2];
    int blocks0, blocks1;               // blocks of either side
    const float *cos, *sin;
    const int32_t *pos;
    int64_t pos_stride;
    int seqlen, dim, half, rows;        // half: rotary / 2; rows: of the table
    int lpr;
    float eps, inv;                     // inv: 1 / dim, or 1
    bool interleaved;
};

// An item's place: token, first head; and the token's position, -1 for padding.
struct QkAt {
    int64_t b;
    int t, h0, pos;
};
__device__ __forceinline__ QkAt qk_at(const QkArgs &a, const QkSide &s, uint32_t item, int hb) {
    QkAt q;
    const uint32_t tok = item / (uint32_t)s.per, b = tok / (uint32_t)a.seqlen;
    q.h0 = (int)(item - tok * s.per) * hb;
    q.b = b;
    q.t = (int)(tok - b * a.seqlen);
    q.pos = 0;
    if (a.half > 0) {
        q.pos = a.pos ? a.pos[q.b * a.pos_stride + q.t] : q.t;
        if ((unsigned)q.pos >= (unsigned)a.rows) q.pos = -1;
    }
    return q;
}

// V features at a place divisible by V, as they lie in memory (two bf16 to a register)
template <typename T, int V>
struct QkRaw {
    uint32_t w[V * sizeof(T) / 4];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int c = 0; c < (int)(V * sizeof(T) / 16); ++c) {
            const uint4 u = reinterpret_cast<const uint4 *>(p)[c];
            w[4 * c] = u.x; w[4 * c + 1] = u.y; w[4 * c + 2] = u.z; w[4 * c + 3] = u.w;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < (int)(V * sizeof(T) / 4); ++e) w[e] = 0u;
    }
    __device__ __forceinline__ void to(f32x2 (&f)[V / 2]) const {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            if constexpr (sizeof(T) == 4) f[e] = pk2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
            else f[e] = pk2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
        }
    }
};
template <typename T, int V>
__device__ __forceinline__ void qk_store(T *p, const f32x2 (&f)[V / 2]) {
    float x[V];
#pragma unroll
    for (int e = 0; e < V / 2; ++e) up2(f[e], x[2 * e], x[2 * e + 1]);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int c = 0; c < V / 8; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[8 * c + 2 * e], x[8 * c + 2 * e + 1]);
                w[e] = *reinterpret_cast<const uint32_t *>(&h);
            }
            reinterpret_cast<uint4 *>(p)[c] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll
        for (int c = 0; c < V / 4; ++c) reinterpret_cast<float4 *>(p)[c] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
    }
}

// The token's rotation of a lane's features: feature e becomes c x_e + s x_partner (backwards, by the opposite angle, c x_e - s x_partner),
// the sign of the sine with the feature.  The partner lies in another lane (its loaded registers are exchanged, before they are
// unpacked) or, interleaved, is the neighbour.
template <typename T, int V, bool INTER>
struct QkTurn {
    f32x2 c[V / 2], s[V / 2];
    int from, pl;                       // lane of the partners, and its place in the group
    __device__ __forceinline__ void load(const QkArgs &a, int pos, int l, int lane, bool back) {
        const int e0 = l * V;
        const bool on = e0 < 2 * a.half && pos >= 0;         // (a padding token's outputs are set to zero, and the table may be empty)
        const int64_t row = (int64_t)pos * a.half;
        from = lane;
        pl = l;
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            c[e] = pk2(1.f, 1.f);
            s[e] = 0;
        }
        if (!on) return;
        if constexpr (INTER) {
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                const float x = a.cos[row + e0 / 2 + e], y = a.sin[row + e0 / 2 + e];
                c[e] = pk2(x, x);
                s[e] = back ? pk2(y, -y) : pk2(-y, y);
            }
        } else {
            const bool second = e0 >= a.half;
            const int i = second ? e0 - a.half : e0;
            pl = second ? l - a.half / V : l + a.half / V;
            from = lane + pl - l;
            const float sign = second != back ? 1.f : -1.f;
#pragma unroll
            for (int e = 0; e < V; e += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(a.cos + row + i + e), y = *reinterpret_cast<const float4 *>(a.sin + row + i + e);
                c[e / 2] = pk2(x.x, x.y);
                c[e / 2 + 1] = pk2(x.z, x.w);
                s[e / 2] = mul2(pk2(sign, sign), pk2(y.x, y.y));
                s[e / 2 + 1] = mul2(pk2(sign, sign), pk2(y.z, y.w));
            }
        }
    }
    // the partners of a row's features
    __device__ __forceinline__ void partners(const QkRaw<T, V> &x, const f32x2 (&f)[V / 2], f32x2 (&p)[V / 2]) const {
        if constexpr (INTER) {
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                float u, v;
                up2(f[e], u, v);
                p[e] = pk2(v, u);
            }
        } else {
            QkRaw<T, V> y;
#pragma unroll
            for (int e = 0; e < (int)(V * sizeof(T) / 4); ++e) y.w[e] = __shfl_sync(0xffffffffu, x.w[e], from);
            y.to(p);
        }
    }
};

__device__ __forceinline__ float qk_group(float v, int lpr) {
    for (int o = lpr >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int V>
__device__ __forceinline__ void qk_weight(f32x2 (&w)[V / 2], const float *p, bool in) {
#pragma unroll
    for (int e = 0; e < V / 2; ++e) w[e] = pk2(1.f, 1.f);
    if (p && in)
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            const float4 u = *reinterpret_cast<const float4 *>(p + e);
            w[e / 2] = pk2(u.x, u.y);
            w[e / 2 + 1] = pk2(u.z, u.w);
        }
}

// y = rstd (c w x + s w' x'), x' and w' the partners': their factors are the token's
template <typename T, int V, bool INTER, int HB>
__global__ void __launch_bounds__(QK_FWD_NT, V <= 8 ? 7 : 4) k_qk_fwd(const QkArgs a) {
    after_previous();
    const bool keys = blockIdx.x >= a.blocks0;
    const QkSide &s = a.side[keys];
    const int lane = threadIdx.x & 31, l = lane & (a.lpr - 1), gpb = QK_FWD_NT / a.lpr;
    const uint32_t item = (uint32_t)(blockIdx.x - (keys ? a.blocks0 : 0)) * gpb + threadIdx.x / a.lpr;
    const bool live = item < s.items;                        // (idle groups stay for the shuffles)
    const QkAt q = qk_at(a, s, live ? item : s.items - 1, HB);
    const bool in = l * V < a.dim;
    const T *x = static_cast<const T *>(s.x) + q.b * s.xs[0] + q.t * s.xs[1] + q.h0 * s.xs[2] + l * V;
    T *y = static_cast<T *>(s.y) + q.b * s.ys[0] + q.t * s.ys[1] + q.h0 * s.ys[2] + l * V;
    QkRaw<T, V> v[HB];
    QkTurn<T, V, INTER> r;
#pragma unroll
    for (int u = 0; u < HB; ++u) {
        if (in && q.h0 + u < s.heads) v[u].load(x + u * s.xs[2]);
        else v[u].zero();
    }
    if (a.half > 0) r.load(a, q.pos, l, lane, false);
    f32x2 w[V / 2];
    qk_weight<V>(w, s.w ? s.w + l * V : nullptr, in);
    if (a.half > 0) {
        f32x2 wp[V / 2];
        if constexpr (INTER) {
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                float u, t;
                up2(w[e], u, t);
                wp[e] = pk2(t, u);
            }
        } else {
            qk_weight<V>(wp, s.w ? s.w + r.pl * V : nullptr, in);
        }
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            w[e] = mul2(w[e], r.c[e]);
            r.s[e] = mul2(wp[e], r.s[e]);
        }
    }
#pragma unroll
    for (int u = 0; u < HB; ++u) {
        f32x2 f[V / 2], m = 0;
        v[u].to(f);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) m = fma2(f[e], f[e], m);
        float rstd = rsqrtf(fmaf(qk_group(sum2(m), a.lpr), a.inv, a.eps));
        if (a.half > 0) {
            f32x2 p[V / 2];
            r.partners(v[u], f, p);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) f[e] = fma2(r.s[e], p[e], mul2(w[e], f[e]));
        } else {
#pragma unroll
            for (int e = 0; e < V / 2; ++e) f[e] = mul2(w[e], f[e]);
        }
        const f32x2 rr = pk2(rstd, rstd);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) f[e] = q.pos < 0 ? 0 : mul2(rr, f[e]);
        if (live && in && q.h0 + u < s.heads) qk_store<T, V>(y + u * s.ys[2], f);
    }
}

template <typename T, int V, bool INTER, int HB>
__global__ void __launch_bounds__(QK_NT, V <= 8 ? 3 : 2) k_qk_bwd(const QkArgs a) {
    after_previous();
    __shared__ float sum[QK_NT * V];
    const bool keys = blockIdx.x >= a.blocks0;
    const QkSide &s = a.side[keys];
    const int lane = threadIdx.x & 31, l = lane & (a.lpr - 1), gpb = QK_NT / a.lpr, grp = threadIdx.x / a.lpr;
    const int nb = keys ? a.blocks1 : a.blocks0, bi = blockIdx.x - (keys ? a.blocks0 : 0);
    const bool in = l * V < a.dim;
    f32x2 w[V / 2], acc[V / 2];
    qk_weight<V>(w, s.w ? s.w + l * V : nullptr, in);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) acc[e] = 0;
    for (uint32_t first = (uint32_t)bi * gpb; first < s.items; first += (uint32_t)nb * gpb) {
        const bool live = first + grp < s.items;
        const QkAt q = qk_at(a, s, live ? first + grp : s.items - 1, HB);
        const T *x = static_cast<const T *>(s.x) + q.b * s.xs[0] + q.t * s.xs[1] + q.h0 * s.xs[2] + l * V;
        const T *dy = static_cast<const T *>(s.dy) + q.b * s.dys[0] + q.t * s.dys[1] + q.h0 * s.dys[2] + l * V;
        T *dx = static_cast<T *>(s.y) + q.b * s.ys[0] + q.t * s.ys[1] + q.h0 * s.ys[2] + l * V;
        QkRaw<T, V> xr[HB], dr[HB];
        QkTurn<T, V, INTER> r;
#pragma unroll
        for (int u = 0; u < HB; ++u) {
            if (live && in && q.pos >= 0 && q.h0 + u < s.heads) {
                xr[u].load(x + u * s.xs[2]);
                dr[u].load(dy + u * s.dys[2]);
            } else {
                xr[u].zero();
                dr[u].zero();
            }
        }
        if (a.half > 0) r.load(a, q.pos, l, lane, true);
#pragma unroll
        for (int u = 0; u < HB; ++u) {
            f32x2 xv[V / 2], dv[V / 2], m = 0, d2 = 0;
            xr[u].to(xv);
            dr[u].to(dv);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) m = fma2(xv[e], xv[e], m);
            // (a vector that is not there: rstd could be infinite with eps 0)
            const float power = fmaf(qk_group(sum2(m), a.lpr), a.inv, a.eps), rstd = live && q.pos >= 0 && q.h0 + u < s.heads ? rsqrtf(power) : 0.f;
            if (a.half > 0) {
                f32x2 p[V / 2];
                r.partners(dr[u], dv, p);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) dv[e] = fma2(r.s[e], p[e], mul2(r.c[e], dv[e]));
            }
            const f32x2 rr = pk2(rstd, rstd);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                xv[e] = mul2(rr, xv[e]);
                acc[e] = fma2(dv[e], xv[e], acc[e]);
                dv[e] = mul2(w[e], dv[e]);
                d2 = fma2(dv[e], xv[e], d2);
            }
            const float d = -qk_group(sum2(d2), a.lpr) * a.inv;
            const f32x2 dd = pk2(d, d);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) dv[e] = mul2(rr, fma2(dd, xv[e], dv[e]));
            if (live && in && q.h0 + u < s.heads) qk_store<T, V>(dx + u * s.ys[2], dv);
        }
    }
    if (!s.share) return;
#pragma unroll
    for (int e = 0; e < V / 2; ++e) up2(acc[e], sum[(grp * a.lpr + l) * V + 2 * e], sum[(grp * a.lpr + l) * V + 2 * e + 1]);
    __syncthreads();
    for (int e = threadIdx.x; e < a.dim; e += QK_NT) {
        float t = 0.f;
        for (int g = 0; g < gpb; ++g) t += sum[g * a.lpr * V + e];
        s.share[(int64_t)bi * a.dim + e] = t;
    }
}

// ---- any shape and address: a warp a head's vector, features 32 apart, the rotation through shared memory.
template <typename T, bool BACK>
__global__ void __launch_bounds__(QK_NT) k_qk_any(const QkArgs a) {
    after_previous();
    __shared__ float rows[QK_NT / 32][QK_MAXD], grads[BACK ? QK_NT / 32 : 1][QK_MAXD];
    const bool keys = blockIdx.x >= a.blocks0;
    const QkSide &s = a.side[keys];
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, D = a.dim;
    const int nb = keys ? a.blocks1 : a.blocks0, bi = blockIdx.x - (keys ? a.blocks0 : 0);
    float *row = rows[wp];
    if (BACK)
        for (int e = lane; e < D; e += 32) grads[wp][e] = 0.f;
    for (uint32_t item = (uint32_t)bi * (QK_NT / 32) + wp; item < s.items; item += (uint32_t)nb * (QK_NT / 32)) {
        const QkAt q = qk_at(a, s, item, QK_HB_MIN);
        for (int u = 0; u < QK_HB_MIN && q.h0 + u < s.heads; ++u) {
            const T *x = static_cast<const T *>(s.x) + q.b * s.xs[0] + q.t * s.xs[1] + (q.h0 + u) * s.xs[2];
            T *y = static_cast<T *>(s.y) + q.b * s.ys[0] + q.t * s.ys[1] + (q.h0 + u) * s.ys[2];
            if (q.pos < 0) {
                for (int e = lane; e < D; e += 32) y[e] = from_f<T>(0.f);
                continue;
            }
            float m = 0.f;
            for (int e = lane; e < D; e += 32) m = fmaf(to_f(x[e]), to_f(x[e]), m);
            const float rstd = rsqrtf(fmaf(warp_sum(m), a.inv, a.eps));
            __syncwarp();
            const T *dy = BACK ? static_cast<const T *>(s.dy) + q.b * s.dys[0] + q.t * s.dys[1] + (q.h0 + u) * s.dys[2] : nullptr;
            for (int e = lane; e < D; e += 32) row[e] = BACK ? to_f(dy[e]) : to_f(x[e]) * rstd * (s.w ? s.w[e] : 1.f);
            __syncwarp();
            float d = 0.f;
            for (int e = lane; e < D; e += 32) {
                float v = row[e];
                if (e < 2 * a.half) {
                    const bool second = a.interleaved ? e & 1 : e >= a.half;
                    const int i = a.interleaved ? e / 2 : second ? e - a.half : e;
                    const float p = row[a.interleaved ? e ^ 1 : second ? e - a.half : e + a.half];
                    const float c = a.cos[(int64_t)q.pos * a.half + i], sn = a.sin[(int64_t)q.pos * a.half + i];
                    v = v * c + p * (second != BACK ? sn : -sn);
                }
                if (BACK) {
                    const float n = to_f(x[e]) * rstd;
                    grads[wp][e] = fmaf(v, n, grads[wp][e]);
                    d = fmaf(v * (s.w ? s.w[e] : 1.f), n, d);
                } else {
                    y[e] = from_f<T>(v);
                }
            }
            if (BACK) {
                d = warp_sum(d) * a.inv;
                for (int e = lane; e < D; e += 32) {             // the rotation again: nothing holds 16 features a lane
                    float v = row[e];
                    if (e < 2 * a.half) {
                        const bool second = a.interleaved ? e & 1 : e >= a.half;
                        const int i = a.interleaved ? e / 2 : second ? e - a.half : e;
                        const float p = row[a.interleaved ? e ^ 1 : second ? e - a.half : e + a.half];
                        const float c = a.cos[(int64_t)q.pos * a.half + i], sn = a.sin[(int64_t)q.pos * a.half + i];
                        v = v * c + p * (second ? -sn : sn);
                    }
                    y[e] = from_f<T>(rstd * fmaf(-d, to_f(x[e]) * rstd, v * (s.w ? s.w[e] : 1.f)));
                }
            }
        }
    }
    if (BACK && s.share) {
        __syncthreads();
        for (int e = threadIdx.x; e < D; e += QK_NT) {
            float t = 0.f;
            for (int g = 0; g < QK_NT / 32; ++g) t += grads[g][e];
            s.share[(int64_t)bi * D + e] = t;
        }
    }
}

// sum of the blocks' shares: 32 features a block, 32 threads a feature
__global__ void __launch_bounds__(1024) k_qk_dw(const QkArgs a) {
    after_previous();
    __shared__ float part[32][33];
    const int per = (a.dim + 31) / 32, side = blockIdx.x / per, e = blockIdx.x % per * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    const QkSide &s = a.side[side];
    if (!s.share) return;
    const int n = side ? a.blocks1 : a.blocks0;
    float t = 0.f;
    if (e < a.dim)
#pragma unroll 4
        for (int b = g; b < n; b += 32) t += s.share[(int64_t)b * a.dim + e];
    part[g][threadIdx.x & 31] = t;
    __syncthreads();
    const float v = warp_sum(part[threadIdx.x & 31][g]);     // warp g: feature g
    if ((threadIdx.x & 31) == 0 && blockIdx.x % per * 32 + g < a.dim) s.dw[blockIdx.x % per * 32 + g] = v;
}

bool al(const void *p, size_t n) { return (uintptr_t)p % n == 0; }

// strides and address of a tensor whose heads are read or written in pieces of 16 bytes
bool pieces(const void *p, const int64_t *s, const ssd_qk_problem *q, int heads) {
    const int64_t n = q->dtype == SSD_BF16 ? 8 : 4;
    return al(p, 16) && (q->batch == 1 || s[0] % n == 0) && (q->seqlen == 1 || s[1] % n == 0) && (heads == 1 || s[2] % n == 0);
}

ssd_status check_tensor(const ssd_qk_problem *p, const ssd_tensor &t, int64_t heads, bool written) {
    if (heads == 0) return SSD_OK;
    if (t.ptr == nullptr || t.dtype != p->dtype || (p->dim > 1 && t.stride[3] != 1)) return SSD_ERR_INVALID_ARGUMENT;
    const int64_t n[3] = {p->batch, p->seqlen, heads};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && t.stride[i] < (written ? p->dim : 0)) return SSD_ERR_INVALID_ARGUMENT;
    return al(t.ptr, p->dtype == SSD_BF16 ? 2 : 4) ? SSD_OK : SSD_ERR_MISALIGNED;
}

ssd_status check(const ssd_qk_problem *p, const ssd_qk_args *f) {
    if (p == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    if (p->batch < 0 || p->seqlen < 0 || p->q_heads < 1 || p->k_heads < 0 || p->dim < 1 || p->rotary < 0 || p->rotary % 2 != 0 ||
        p->rotary > p->dim || p->table_rows < 0 || !(p->eps >= 0.f) || (p->mode != SSD_QK_RMS && p->mode != SSD_QK_L2) ||
        (p->interleaved != 0 && p->interleaved != 1) || (p->dtype != SSD_F32 && p->dtype != SSD_BF16))
        return SSD_ERR_INVALID_ARGUMENT;
    const int64_t tokens = p->batch * p->seqlen;
    if (p->dim > QK_MAXD || p->batch > ((int64_t)1 << 30) || p->seqlen > ((int64_t)1 << 30) || p->q_heads > ((int64_t)1 << 16) || p->k_heads > ((int64_t)1 << 16) ||
        tokens > ((int64_t)1 << 30) || p->table_rows > ((int64_t)1 << 30) || tokens * ((p->q_heads + 1) / QK_HB_MIN + (p->k_heads + 1) / QK_HB_MIN) > ((int64_t)1 << 30))
        return SSD_ERR_UNSUPPORTED;
    if (f == nullptr) return SSD_OK;
    if (tokens == 0) return SSD_OK;
    ssd_status s = check_tensor(p, f->q, p->q_heads, false);
    if (s == SSD_OK) s = check_tensor(p, f->k, p->k_heads, false);
    if (s != SSD_OK) return s;
    if (p->rotary > 0 && p->table_rows > 0 && (!f->cos || !f->sin)) return SSD_ERR_INVALID_ARGUMENT;
    if (!al(f->q_weight, 4) || !al(f->k_weight, 4) || !al(f->cos, 4) || !al(f->sin, 4) || !al(f->positions, 4)) return SSD_ERR_MISALIGNED;
    return SSD_OK;
}

void set3(int64_t *to, const ssd_tensor &t) {
    for (int i = 0; i < 3; ++i) to[i] = t.stride[i];
}

// V: features of a lane in the kernels by pieces, 0 where the shapes or addresses do not allow them
QkArgs make(const ssd_qk_problem *p, const ssd_qk_args *f, const ssd_tensor &yq, const ssd_tensor &yk, const ssd_tensor *dyq, const ssd_tensor *dyk, int *V, int *HB) {
    QkArgs a{};
    const ssd_tensor *x[2] = {&f->q, &f->k}, *y[2] = {&yq, &yk}, *dy[2] = {dyq, dyk};
    const int64_t heads[2] = {p->q_heads, p->k_heads};
    const int64_t tokens = p->batch * p->seqlen;
    const int least = p->dtype == SSD_BF16 ? 8 : 4;
    *V = p->dim <= 32 * least ? least : 2 * least;
    if (p->dim > 32 * *V) *V = 16;
    bool vec = p->dim % *V == 0 && (p->interleaved ? p->rotary : p->rotary / 2) % *V == 0 && (p->rotary == 0 || (al(f->cos, 16) && al(f->sin, 16)));
    for (int i = 0; i < 2; ++i) {
        QkSide &s = a.side[i];
        s.x = x[i]->ptr; s.y = y[i]->ptr; set3(s.xs, *x[i]); set3(s.ys, *y[i]);
        s.heads = (int)heads[i];
        s.w = i ? f->k_weight : f->q_weight;
        if (heads[i] == 0) continue;
        vec = vec && al(s.w, 16) && pieces(s.x, s.xs, p, s.heads) && pieces(s.y, s.ys, p, s.heads);
        if (dy[i]) {
            s.dy = dy[i]->ptr;
            set3(s.dys, *dy[i]);
            vec = vec && pieces(s.dy, s.dys, p, s.heads);
        }
    }
    if (!vec) *V = 0;
    // Heads of an item: 128 bytes of them on the way to a lane (backwards 64 of x and of dy each) where that still fills the card, two where
    // few tokens come.  8192 tokens x 40 heads of 128: 4 / 8 heads 39 / 32 us; backwards 4096 tokens 32.7 / 48.6.
    const int64_t lanes = tokens * (p->q_heads + p->k_heads) * p->dim / (*V ? *V : 16);
    const int many = (dyq != nullptr ? 64 : 128) / ((*V ? *V : 16) * (p->dtype == SSD_BF16 ? 2 : 4));
    *HB = *V && many > QK_HB_MIN && lanes / many >= 2 * kSMs * QK_NT ? many : QK_HB_MIN;
    for (int i = 0; i < 2; ++i) {
        a.side[i].per = (int)((heads[i] + *HB - 1) / *HB);
        a.side[i].items = (uint32_t)(tokens * a.side[i].per);
    }
    a.cos = f->cos; a.sin = f->sin; a.pos = f->positions; a.pos_stride = p->pos_stride;
    a.seqlen = (int)p->seqlen; a.dim = (int)p->dim; a.half = (int)(p->rotary / 2); a.rows = (int)p->table_rows;
    a.eps = p->eps;
    a.inv = p->mode == SSD_QK_RMS ? 1.f / (float)p->dim : 1.f;
    a.interleaved = p->interleaved != 0;
    a.lpr = 1;
    while (a.lpr < 32 && a.lpr * *V < p->dim) a.lpr <<= 1;
    if (*V == 0) a.lpr = 32;
    return a;
}
int blocks_for(const QkArgs &a, int side, int64_t most) {
    const int64_t gpb = (most == 0 ? QK_FWD_NT : QK_NT) / a.lpr, n = (a.side[side].items + gpb - 1) / gpb;   // most 0: forwards, a group an item
    if (most == 0) return (int)n;
    const uint64_t all = (uint64_t)a.side[0].items + a.side[1].items;   // blocks in proportion to the items
    const int64_t share = std::max<int64_t>(1, (int64_t)((uint64_t)most * a.side[side].items / all));
    return (int)(a.side[side].items == 0 ? 0 : std::min(n, share));
}

template <typename T, int V, bool INTER, int HB>
cudaError_t launch(const QkArgs &a, bool back, cudaStream_t st) {
    const unsigned grid = (unsigned)(a.blocks0 + a.blocks1);
    if (!back) return launch_early(k_qk_fwd<T, V, INTER, HB>, grid, QK_FWD_NT, 0, st, a);
    return launch_early(k_qk_bwd<T, V, INTER, HB>, grid, QK_NT, 0, st, a);
}
template <typename T, int V>
cudaError_t pick_hb(const QkArgs &a, int HB, bool back, cudaStream_t st) {
    constexpr int fwd = 128 / (V * sizeof(T)), bwd = 64 / (V * sizeof(T));
    if constexpr (fwd > QK_HB_MIN) {
        if (!back && HB == fwd) return a.interleaved ? launch<T, V, true, fwd>(a, back, st) : launch<T, V, false, fwd>(a, back, st);
    }
    if constexpr (bwd > QK_HB_MIN) {
        if (back && HB == bwd) return a.interleaved ? launch<T, V, true, bwd>(a, back, st) : launch<T, V, false, bwd>(a, back, st);
    }
    return a.interleaved ? launch<T, V, true, QK_HB_MIN>(a, back, st) : launch<T, V, false, QK_HB_MIN>(a, back, st);
}
template <typename T>
cudaError_t pick(const QkArgs &a, int V, int HB, bool back, cudaStream_t st) {
    constexpr int least = 16 / sizeof(T);
    if (V == 0) {
        const unsigned grid = (unsigned)(a.blocks0 + a.blocks1);
        return back ? launch_early(k_qk_any<T, true>, grid, QK_NT, 0, st, a) : launch_early(k_qk_any<T, false>, grid, QK_NT, 0, st, a);
    }
    if (V == least) return pick_hb<T, least>(a, HB, back, st);
    if constexpr (least == 4) {
        if (V == 8) return pick_hb<T, 8>(a, HB, back, st);
    }
    return pick_hb<T, 16>(a, HB, back, st);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_qk_norm_fwd(const ssd_qk_problem *p, const ssd_qk_args *f, void *stream) {
    if (f == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    if (ssd_status s = check(p, f); s != SSD_OK) return s;
    if (p->batch * p->seqlen == 0) return SSD_OK;
    if (ssd_status s = check_tensor(p, f->q_out, p->q_heads, true); s != SSD_OK) return s;
    if (ssd_status s = check_tensor(p, f->k_out, p->k_heads, true); s != SSD_OK) return s;
    int V, HB;
    QkArgs a = make(p, f, f->q_out, f->k_out, nullptr, nullptr, &V, &HB);
    a.blocks0 = blocks_for(a, 0, V ? 0 : 16 * kSMs);
    a.blocks1 = blocks_for(a, 1, V ? 0 : 16 * kSMs);
    const cudaError_t e = p->dtype == SSD_BF16 ? pick<__nv_bfloat16>(a, V, HB, false, (cudaStream_t)stream) : pick<float>(a, V, HB, false, (cudaStream_t)stream);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_qk_norm_bwd_workspace_size(const ssd_qk_problem *p, size_t *bytes) {
    if (bytes == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    if (ssd_status s = check(p, nullptr); s != SSD_OK) return s;
    *bytes = (size_t)2 * QK_BLOCKS * (size_t)p->dim * sizeof(float);
    return SSD_OK;
}

ssd_status ssd_qk_norm_bwd(const ssd_qk_problem *p, const ssd_qk_bwd_args *b, void *workspace, size_t workspace_bytes, void *stream) {
    if (b == nullptr) return SSD_ERR_INVALID_ARGUMENT;
    const ssd_qk_args *f = &b->fwd;
    if (ssd_status s = check(p, f); s != SSD_OK) return s;
    float *dw[2] = {f->q_weight ? b->dq_weight : nullptr, f->k_weight ? b->dk_weight : nullptr};   // (without heads of keys theirs is zero)
    if ((f->q_weight && !dw[0]) || (f->k_weight && p->k_heads > 0 && !dw[1])) return SSD_ERR_INVALID_ARGUMENT;
    if (!al(dw[0], 4) || !al(dw[1], 4)) return SSD_ERR_MISALIGNED;
    cudaStream_t st = (cudaStream_t)stream;
    if (p->batch * p->seqlen == 0) {
        for (float *d : dw)
            if (d && cudaMemsetAsync(d, 0, (size_t)p->dim * sizeof(float), st) != cudaSuccess) return SSD_ERR_CUDA;
        return SSD_OK;
    }
    for (const ssd_tensor *t : {&b->dq_out, &b->dq})
        if (ssd_status s = check_tensor(p, *t, p->q_heads, t == &b->dq); s != SSD_OK) return s;
    for (const ssd_tensor *t : {&b->dk_out, &b->dk})
        if (ssd_status s = check_tensor(p, *t, p->k_heads, t == &b->dk); s != SSD_OK) return s;
    if (dw[0] || dw[1]) {
        if (workspace == nullptr || workspace_bytes < (size_t)2 * QK_BLOCKS * (size_t)p->dim * sizeof(float)) return SSD_ERR_WORKSPACE_TOO_SMALL;
        if (!al(workspace, 256)) return SSD_ERR_MISALIGNED;
    }
    int V, HB;
    QkArgs a = make(p, f, b->dq, b->dk, &b->dq_out, &b->dk_out, &V, &HB);
    a.blocks0 = blocks_for(a, 0, QK_BLOCKS);
    a.blocks1 = blocks_for(a, 1, QK_BLOCKS);
    for (int i = 0; i < 2; ++i) {
        a.side[i].dw = dw[i];
        a.side[i].share = dw[i] ? static_cast<float *>(workspace) + (size_t)i * QK_BLOCKS * p->dim : nullptr;
    }
    cudaError_t e = p->dtype == SSD_BF16 ? pick<__nv_bfloat16>(a, V, HB, true, st) : pick<float>(a, V, HB, true, st);
    if (e == cudaSuccess && (dw[0] || dw[1])) {
        e = launch_early(k_qk_dw, (unsigned)(2 * ((a.dim + 31) / 32)), 1024, 0, st, a);
    }
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
