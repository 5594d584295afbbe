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
    int64_t window;                    // 0: none
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
    size_t part_floats, slot_floats, bytes;
};

}  // namespace hqq_kv
