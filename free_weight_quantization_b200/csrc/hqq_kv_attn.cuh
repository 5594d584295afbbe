// hqq_kv_attn.cuh -- attention over a quantised key/value cache: what its kernels share.
#pragma once

#include "hqq_kv.cuh"

namespace hqq_kv {

// One attention call.  Rows are (sequence b, query i of nq, query head h); the `share` = heads /
// kv_heads query heads of one key head, and the nq queries, read the same keys and values.
struct Attn {
    Cache c;
    const uint16_t *q;
    int64_t q_batch, q_token, q_head;  // strides, in values
    int batch, nq, heads, share;
    const int32_t *pages;              // a row of pages_stride for each sequence
    int64_t pages_stride;
    const int32_t *lens;               // [batch]
    int64_t max_len;
    int64_t window;                    // 0: none
    const int32_t *prefix_pages;       // [..] of the prefix that every sequence shares
    int64_t prefix_len;
    float scale_log2;                  // softmax scale * log2(e)
    int64_t chunk;                     // tokens of one split
    int splits, prefix_splits;         // of each sequence's own tokens; of the prefix
    uint16_t *out;                     // [batch][nq][heads][D]
    float *lse;                        // [batch][nq][heads], null: not wanted
    float *part_o;                     // [prefix_splits + splits][batch * nq * heads][D], null: one split
    float *part_lse;                   // [prefix_splits + splits][batch * nq * heads], in powers of two
    bool bf;
};

// splits of the work and workspace of a call
struct AttnPlan {
    int64_t chunk, prefix_chunk;
    int splits, prefix_splits, row_blocks, prefix_row_blocks;
    size_t bytes;
};

}  // namespace hqq_kv
