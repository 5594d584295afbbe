// hqq_kv_attn.cuh -- attention over a quantised key/value cache: what its kernels share.
#pragma once

#include "hqq_kv.cuh"

namespace hqq_kv {

struct __align__(16) Cut {  // a pair that is cut between CTAs c0 .. c1; b = -1: none
    int b, pair, c0, c1;
};

// One attention call.  Rows are (sequence b, query i of nq, query head h); the `share` = heads /
// kv_heads query heads of one key head, and the nq queries, read the same keys and values.  A pair
// is a block of such rows of one sequence and key head, and the tokens that it reads.
struct Attn {
    Cache c;
    const uint16_t *q;
    int64_t q_batch, q_token, q_head;  // strides, in values
    bool q_wide;                       // q can be read 8 bytes at a time
    int batch, nq, heads, share;
    const int32_t *pages;              // a row of pages_stride for each sequence
    int64_t pages_stride;
    const int32_t *lens;               // [batch]
    int64_t max_len;
    int64_t window;                    // 0: none; below max_len
    const int32_t *prefix_pages;       // of the prefix that every sequence shares
    int64_t prefix_len;
    float scale_log2;                  // softmax scale * log2(e)
    int row_blocks;                    // of one sequence's rows
    int ctas;                          // that share the sequences' own tokens evenly; 0: one to a pair
    int64_t prefix_chunk;              // tokens of the prefix that a CTA reads
    int prefix_splits;
    uint16_t *out;                     // [batch][nq][heads][D]
    float *lse;                        // [batch][nq][heads], null: not wanted
    // Partial results, each normalised by itself, with their log-sum-exp in powers of two:
    float *part_o, *part_lse;          // [prefix_splits + 1][rows][D]: the prefix's chunks, then whole
                                       // pairs; null without a prefix
    float *slot_o, *slot_lse;          // [2 ctas][rows of a pair][D]: pairs cut between CTAs
    Cut *cuts;                         // [ctas]: the pair that begins in a CTA's share and ends in another's
    bool bf;
};

// how a call is divided, and its workspace
struct AttnPlan {
    int64_t prefix_chunk;
    int ctas, pair_rows, row_blocks, prefix_splits, prefix_row_blocks;
    bool prefix_tc;  // the prefix by hqq_kv_prefix_tc_kernel
    int64_t window;  // 0 where it hides nothing
    size_t part_floats, slot_floats, bytes;
};

// A query row that the products can take: below 2^100, so that one power of two brings it into fp16,
// and, in units of the scores, below 2^84: D (255 + |zero|) scale of a key is below 2^40, so that
// every score lies above kLowest.  Any other row is made NaN.  big: the bits of its largest magnitude.
constexpr float kLowest = -0x1p126f;  // a maximum before any score
__device__ __forceinline__ bool row_in_range(uint32_t big, float scale_log2) {
    return big < (227u << 23) && __uint_as_float(big) * scale_log2 < 0x1p84f;
}

// The largest score of a block, in powers of two, that can be answered: the roundings of m = max(s)
// unit and of the bound (m + kLag) / unit, 2^-24 of the score each, go to the exponent s unit - m, 0.6
// in all at 2^22, where w is still below 2^15.7.  Beyond, the row is made NaN.
constexpr float kScoreLimit = 0x1p22f;
__device__ __forceinline__ bool score_in_range(float top) { return fabsf(top) < kScoreLimit || top == kLowest; }

// What a row's raw scores, of q * up and codes * 2^-24, are multiplied by.  Not 0, by which a hidden
// token's -infinity would become NaN.
__device__ __forceinline__ float row_unit(float up, float scale_log2) { return fmaxf(0x1p24f / up * scale_log2, 0x1p-126f); }

// The running maximum may lag behind by this many powers of two before the sums are rescaled:
// weights stay below 2^8 of what they are relative to.  w is kept within fp16 by 2^7 * 2^8 < 65504.
constexpr float kLag = 8.0f;
constexpr float kWeightUnit = 128.0f;

// A 32-bit word holds codes in two halves that an operand register takes side by side.  Code u of
// byte h of the halves is brought to bit up(u): as high as it can be below the fp16 exponent at
// one shift for two codes, because the tensor cores align a subnormal number as if its leading
// bit were at the top, and what they drop is relative to that.  (Relative error of the log-sum-exp,
// D = 128, largest of g = 32, 64, 128 and 2 to 20000 tokens: with the codes where they lie 5.6e-6 at
// 2 bits and 1.3e-6 at 4, like this 7e-8 and 2e-7; 3e-7 at 8 bits, which have no room above.)
template <int NB>
__host__ __device__ constexpr int code_up(int u) {
    return NB == 2 ? 6 + 2 * (u & 1) : NB == 4 ? 2 + 4 * (u & 1) : 0;
}

// a shift that stays one instruction for all the fields that are masked out of its result (left to
// itself, the compiler masks first and then shifts each field)
template <int BY>
__device__ __forceinline__ uint32_t shifted(uint32_t v) {
    uint32_t y = v;
    if constexpr (BY > 0) asm("shl.b32 %0, %1, %2;" : "=r"(y) : "r"(v), "n"(BY));
    if constexpr (BY < 0) asm("shr.u32 %0, %1, %2;" : "=r"(y) : "r"(v), "n"(-BY));
    return y;
}

template <int NB>
__device__ __forceinline__ uint32_t code_pair(uint32_t v, int h, int u) {
    const uint32_t mask = (((1u << NB) - 1u) * 0x00010001u) << code_up<NB>(u);
    if constexpr (NB == 2) {  // codes 0, 1 of a byte to bits 6, 8; codes 2, 3 too
        const int shift = 6 - 8 * h - 4 * (u >> 1);
        return (shift == 6 ? shifted<6>(v) : shift == 2 ? shifted<2>(v) : shift == -2 ? shifted<-2>(v) : shifted<-6>(v)) & mask;
    } else if constexpr (NB == 4) {
        return (h == 0 ? shifted<2>(v) : shifted<-6>(v)) & mask;
    } else {
        return (h == 0 ? v : shifted<-8>(v)) & mask;
    }
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a sequence's own tokens that count
__device__ __forceinline__ int64_t own_len(const Attn &a, int b) {
    const int64_t n = __ldg(a.lens + b);
    return n < 0 ? 0 : n > a.max_len ? a.max_len : n;
}

// tokens [lo, hi) of the sequence (or of the prefix) that query i of sequence b sees
template <bool PREFIX>
__device__ __forceinline__ void visible(const Attn &a, int64_t len, int i, int64_t &lo, int64_t &hi) {
    const int64_t end = len - a.nq + 1 + i;  // among the sequence's own tokens
    lo = 0;
    if constexpr (PREFIX) {
        hi = end < 0 ? a.prefix_len + end : a.prefix_len;
    } else {
        hi = end;
        if (a.window > 0 && end > a.window) lo = end - a.window;
    }
    if (hi < 0) hi = 0;
}

// the tensor-core prefix (hqq_kv_prefix.cu): its layouts, the rows of a CTA, tokens of a tile
constexpr int kTcRows = 128, kTcTokens = 64;
inline bool prefix_tc_layout(const hqq_kv_cache_t &c) { return c.head_dim <= 128 && c.group_size >= 64; }
cudaError_t launch_prefix_tc(const hqq_kv_cache_t &cache, const Attn &a, int row_tiles, cudaStream_t st);

}  // namespace hqq_kv
