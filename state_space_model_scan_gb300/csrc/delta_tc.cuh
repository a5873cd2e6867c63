// delta_tc.cuh -- what the gated delta rule's tensor-core kernels share: operand tiles, their loads, two-term bf16.
//
// Tiles are 128-byte-swizzled images: rows of 64 bf16 (128 bytes), 16-byte piece q of row r at piece q ^ (r & 7).  A tile of
// 64 tokens x 128 features is two such images of 64 rows, 8 KB each (features 0..63, 64..127).
#pragma once

#include <algorithm>

#include "delta.cuh"
#include "tc_common.cuh"

namespace ssd {
namespace dtc {

using namespace tc;

constexpr uint32_t HALF = DQ * 128;              // 64 rows of 128 bytes
constexpr uint32_t TOK_BYTES = 2 * HALF;         // 64 tokens x 128 features
constexpr uint32_t MAT_BYTES = HALF;             // 64 x 64
constexpr uint32_t GATE_BYTES = DGATES * 4;
// per chunk and head, one after the other as they are loaded: the inverse's two terms, att, gates; for a backward also the two terms of
// the transposed inverse with beta on the other side
constexpr uint32_t SYS_HI = 0, SYS_LO = MAT_BYTES, ATT = 2 * MAT_BYTES, GATES = 3 * MAT_BYTES, OPS_BYTES = GATES + GATE_BYTES;
constexpr uint32_t SYS_T = OPS_BYTES, OPS_BOTH = OPS_BYTES + 2 * MAT_BYTES;
constexpr uint32_t STATE_BYTES = 128 * 128 * 2;  // kept state: two images (keys 0..63, 64..127) of 128 rows (values)
constexpr uint32_t VAL_BYTES = DQ * 128 * 2;     // kept U, and mu: [64][128], plain

constexpr uint32_t SEG_BYTES = 128 * 128 * 4;    // of a segment: its end in fp32; its matrix as two states' images

// Segments of the chains of nseqs x H sequences and heads, at most `chunks` long: one of `first` chunks, nseg - 2 of `len`, one of the
// rest.  Two launches: the first takes the first segment as it is and, of each one between, its end from a zero state and its
// matrix; the second, which knows the state that every segment starts from, those and the last.  So the first segment
// lasts as long as what goes on beside it on the other SMs, and the last one too; the blocks for those between come in
// waves.  A block costs one step more than its chunks, joining the ends before a segment 0.8 each, the second launch eight.
// (8192 tokens of 32 heads: 184 us of chains instead of 340 in one launch, or 260 in three equal segments; 2 x 2048 of 32 was 104 cut and
// 102 in one, so it stays whole.)
inline void delta_segments(int64_t nseqs, int64_t H, int64_t chunks, int *nseg, int *first, int *len) {
    const int64_t sms = kDeltaSMs, U = nseqs * H;
    *nseg = 1;
    *first = *len = 0;
    double best = (double)chunks;
    if (U >= sms) return;
    for (int64_t k = 1; k <= 30; ++k) {
        const int64_t w1 = (2 * k * U + sms - U - 1) / (sms - U), w2 = (k * U + sms - U - 1) / (sms - U), n = w1 + k + w2, s = (chunks + n - 1) / n;
        const int64_t last = chunks - (w1 + k) * s;
        if (w1 > 3) break;                                   // (ends and matrices are memory: 128 KB each)
        if (s < 4 || last < 1) continue;
        const double t = (double)w1 * (s + 1) + std::max<int64_t>(last, w2 * (s + 1)) + 0.8 * k + 8;
        if (t < best) {
            best = t;
            *nseg = (int)k + 2;
            *first = (int)(w1 * s);
            *len = (int)s;
        }
    }
}

// K-major operand at K step k (16 elements), images of `half` bytes; MN-major operand at K step k (16 rows)
__device__ __forceinline__ uint64_t kmaj(uint32_t base, int k, uint32_t half) {
    return sdesc(base + (uint32_t)(k >> 2) * half + (uint32_t)(k & 3) * 32u, 16u, 1024u);
}
__device__ __forceinline__ uint64_t mnmaj(uint32_t base, int k, uint32_t half) { return sdesc(base + (uint32_t)k * 2048u, half, 1024u); }

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// a and b as the sum of two bf16 each: off by 2^-17 of the value at most
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(a, b);
    lo = pack_bf16(a - bf_lo(hi), b - bf_hi(hi));
}

// Rows [0, 64) of a token tensor (row r at p + r step, n features, `len` rows exist) into a tile at `dst`, whose images lie `half`
// bytes apart, by NT threads, element by element; zeros elsewhere.  For rows that no tensor map describes.
template <int NT>
__device__ __forceinline__ void load_rows(uint8_t *dst, uint32_t half, const __nv_bfloat16 *p, int64_t step, int len, int n, int t) {
    const int q = t & 15;
    for (int r = t >> 4; r < 64; r += NT / 16) {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (r < len) {
            const unsigned short *s = reinterpret_cast<const unsigned short *>(p) + r * step;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (q * 8 + e < n) w[e >> 1] |= (uint32_t)s[q * 8 + e] << (16 * (e & 1));
        }
        *reinterpret_cast<uint4 *>(dst + (q >> 3) * half + r * 128 + (((q & 7) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
// zeros in rows [len, 64)
template <int NT>
__device__ __forceinline__ void zero_rows(uint8_t *dst, uint32_t half, int len, int t) {
    for (int e = len * 16 + t; e < 64 * 16; e += NT)
        *reinterpret_cast<uint4 *>(dst + ((e >> 3) & 1) * half + (e >> 4) * 128 + ((e & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
}
// a tile by TMA (one thread): features past the tensor's are zeros, and so are tokens past its last
__device__ __forceinline__ void tma_rows(uint8_t *dst, uint32_t half, const CUtensorMap *m, uint64_t *bar, const DeltaChunk &c, int h) {
    tma_load_4d(dst, m, bar, 0, h, c.t0, c.b);
    tma_load_4d(dst + half, m, bar, 64, h, c.t0, c.b);
}
__device__ __forceinline__ const __nv_bfloat16 *tok_rows(const void *p, const int64_t *s, const DeltaChunk &c, int h) {
    return static_cast<const __nv_bfloat16 *>(p) + c.b * s[0] + c.t0 * s[1] + h * s[2];
}

}  // namespace dtc

// Tensor maps of the token tensors [feature][head][token][batch row], a box 64 features of 64 tokens; has*: the tensor has one.
// out: o, backwards dv, without a swizzle, a box 128 features of 64 tokens.  U, mu: [chunk and head][64][128] in the workspace or
// kept, read as swizzled tiles.
struct DeltaMaps {
    CUtensorMap q, k, v, dO, out, U, mu, dq, dk;
    bool has_q, has_k, has_v, has_dO, has_out, has_vals, has_dqk;
};
// delta_tc.cu: bf16 data, headdim and dstate up to 128
cudaError_t delta_tc_fwd(const DeltaArgs &a, const DeltaMaps &m, cudaStream_t st);
// whether the tensor has a map (16-byte rows, strides of 16-byte multiples)
bool delta_map(CUtensorMap *m, const void *p, int64_t inner, int64_t heads, int64_t tokens, int64_t batch, const int64_t *strides, bool out = false);
cudaError_t delta_tc_bwd(const DeltaArgs &a, const DeltaMaps &m, cudaStream_t st);

}  // namespace ssd
