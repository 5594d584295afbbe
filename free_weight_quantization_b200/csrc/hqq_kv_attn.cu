// hqq_kv_attn.cu -- attention of few query rows over a quantised, paged key/value cache
// (hqq_kv_attention), and over a prefix that a batch shares (hqq_kv_prefix_attention).
//
//   o_r = sum_t p_rt v_t / sum_t p_rt,   p_rt = exp(scale q_r . k_t),
//   k_t[d] = (a_td - kz_tg) ks_tg,       v_t[d] = (c_td - vz_tg) vs_tg     (g: the group of d)
//
// The codes go into the matrix instructions as they are, and the metadata stay outside:
//   q_r . k_t = sum_g ks_tg ( sum_{d in g} q_rd a_td  -  kz_tg sum_{d in g} q_rd )
//   sum_t p_rt v_td = sum_t w_rtg c_td - sum_t w_rtg vz_tg,               w_rtg = p_rt vs_tg
// so no value is rounded to 16 bits on the key side (a code is a whole number below 256, and q a
// 16-bit number; each product is exact in binary32), and on the value side only w is, to fp16,
// once for both sums, relative to a power of two of its group.
//
// A code needs no conversion either: a field of up to 8 low bits in a 16-bit half is the fp16
// subnormal code * 2^-24, and one that sits s bits higher code * 2^(s - 24), which the tensor
// cores take as any other number.  So one AND of a word of codes gives two operands; the factors
// 2^-s are put into q (keys: a code's place is fixed for each d) and into the result (values).
//
// Both products are taken transposed, with the tokens (then the value's elements) along the 16
// rows of mma.m16n8k16 and 8 query rows along its columns:
//   S^T = K Q^T:  lane 4r + j holds run j of token r's key (D / 4 codes, one wide load) and of
//                 token r + 8's;
//   O^T = V^T W^T: lane 4r + j holds run r of the values of tokens 2j, 2j+1, 2j+8, 2j+9; pairs of
//                 tokens are put side by side with one byte permute; W^T is S^T's layout, turned
//                 by movmatrix.
// Each warp brings its blocks of 16 tokens into a ring of its own in shared memory with 16-byte
// asynchronous copies, several blocks ahead, and reads them from there as operands: no barriers
// between warps in the loop.  It keeps a running maximum and sum in binary32; the warps of a CTA
// meet in shared memory at the end.
//
// The tokens of all sequences and key heads are laid end to end in units of 64 and divided evenly
// among as many CTAs as the GPU holds at once, whatever the lengths are; the lengths are read on
// the device.  A pair of a sequence and a key head that is cut between CTAs leaves its parts in
// the workspace, and hqq_kv_join_kernel joins them in the order of the tokens.
//
// What bounds it: per block of 16 tokens a warp has 296 instructions at 4 bits and D = 128 (290 at 2
// bits), and the integer units issue every other cycle.  Between 8192 and 16384 tokens of 64
// sequences x 8 key heads a token more costs 1.19 of what its bytes cost at the card's copy rate
// (6.55 TB/s); a call of 64 x 4096 takes 76 us (46 for its bytes), of which some 20 are the way in
// (lengths, page table, first codes: three trips to memory), the change from one pair to the next,
// and the join.  2-bit codes take the same instructions for half the bytes (74 us, 26 for the bytes);
// 16 rows a CTA 118 us for twice the products; 32 rows, a second pass over the codes, 207.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "hqq_common.cuh"
#include "hqq_kv_attn.cuh"

namespace {

using namespace hqq_kv;

constexpr int kAttnWarps = 4, kAttnThreads = 32 * kAttnWarps;
constexpr int kBlock = 16;                      // tokens of one step of a warp
constexpr int kUnit = kBlock * kAttnWarps;       // of one step of a CTA
constexpr int kSms = 148;

template <int N>
struct Words {
    uint32_t w[N];
};

// the 4 or fewer, 8 or 16 bytes of a piece of a lane's run, from shared memory (2 bytes: low half)
template <int NBYTES>
__device__ __forceinline__ void lds_piece(uint32_t *w, uint32_t at) {
    if constexpr (NBYTES == 2) asm volatile("{.reg .u16 t; ld.shared.u16 t, [%1]; cvt.u32.u16 %0, t;}" : "=r"(w[0]) : "r"(at));
    else if constexpr (NBYTES == 4) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at));
    else if constexpr (NBYTES == 8) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
    else asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
}

__device__ __forceinline__ void copy16(bool wanted, uint32_t to, const void *from) {
    asm volatile(
        "{.reg .pred p; setp.ne.b32 p, %2, 0; @p cp.async.cg.shared.global [%0], [%1], 16;}" ::"r"(to), "l"(from),
        "r"((int)wanted) : "memory");
}

// How the D / 4 codes of a lane's run of a key become D / 8 operand registers of two codes each:
// register x holds codes lo(x) and hi(x) of the run, scaled by 2^(up(x) - 24).
template <int D, int NB, int NG>
struct KeyRegs {
    // a word whose halves belong to different groups is spread out first (2-bit codes, g = 32)
    static constexpr bool kSpread = D / NG / kKeyPieces < 32 / NB;
    static constexpr int kU = 8 / NB;
    static constexpr int kSpan = kSpread ? kU : 2 * kU;  // registers of one 16- or 32-bit unit
    __host__ __device__ static constexpr int lo(int x) { return x / kSpan * 2 * kSpan + x % kSpan; }
    __host__ __device__ static constexpr int hi(int x) { return lo(x) + kSpan; }
    __host__ __device__ static constexpr int up(int x) { return code_up<NB>(x % kU); }
    template <int N>
    __device__ static __forceinline__ uint32_t reg(const Words<N> &run, int x) {
        if constexpr (kSpread) {
            const int unit = x / kSpan;
            return code_pair<NB>(__byte_perm(run.w[unit / 2], 0, unit & 1 ? 0x4342 : 0x4140), 0, x % kU);
        } else {
            return code_pair<NB>(run.w[x / kSpan], x % kSpan / kU, x % kU);
        }
    }
};

// Code x of a lane's run of the values (D / 8 codes) of two tokens, side by side, scaled by
// 2^(up(x) - 24).  The run of the first token is `a` or `b`: sel_lo and sel_hi say which (the byte
// permutes for the words' low and high halves).
template <int NB>
struct ValueRegs {
    static constexpr int kU = 8 / NB, kSpan = 2 * kU;
    __host__ __device__ static constexpr int up(int x) { return code_up<NB>(x % kU); }
    template <int N>
    __device__ static __forceinline__ uint32_t reg(const Words<N> &a, const Words<N> &b, int x, uint32_t sel_lo,
                                                   uint32_t sel_hi) {
        const int unit = x / kSpan;
        return code_pair<NB>(__byte_perm(a.w[unit / 2], b.w[unit / 2], unit & 1 ? sel_hi : sel_lo), x % kSpan / kU, x % kU);
    }
};

// Where 16-byte chunk c of token t's row lies among the chunks of a block of 16 rows of n chunks,
// so that a warp's reads of keys (lanes 4r + j: run j of token r) and of values (run r of token 2j
// or 2j + 1, the odd lanes' two in the other order) meet in no bank.  The 8 chunks of a 128-byte
// line are the banks of a 16-byte access.  Token t + 8 always lies 8 rows behind t.
__host__ __device__ constexpr int key_chunk(int n, int t, int c) {
    const int f = n == 8 ? (t & 1) : n == 16 ? (c >> 3) ^ 2 * (t & 1) : 0;
    return t * n + (c ^ f);
}

__host__ __device__ constexpr int value_chunk(int n, int t, int c) {
    const int p = (t >> 1) & 3;
    if (n == 16) return t * n + (c ^ ((p & 1) | (p & 2) << 1));
    if (n == 8) return t * n + (c ^ 2 * p);
    if (n == 4) return t * n + (c ^ 2 * ((t >> 2) & 1));
    if (n == 2) return (t * n + c) ^ 4 * ((t >> 2) & 1);
    return t * n + c;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the transpose of an 8 x 8 matrix of 16-bit values that the warp holds a row to four lanes
__device__ __forceinline__ uint32_t turn(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// v, from here on a value of its own: what is derived from the lane's number stays in a register
// instead of being derived again in every step (23 LOP3 and some 20 other instructions a block)
__device__ __forceinline__ uint32_t pinned(uint32_t v) { return __shfl_sync(0xffffffffu, v, threadIdx.x & 31); }

template <typename T>
__device__ __forceinline__ const T *pinned(const T *p) {
    const uint64_t v = (uint64_t)p;
    return (const T *)((uint64_t)pinned((uint32_t)(v >> 32)) << 32 | pinned((uint32_t)v));
}

// What a kernel of this layout keeps in shared memory and how many of its CTAs an SM holds.
template <int D, int NB, int NG, int RB>
struct Shape {
    static constexpr int kRowBytes = D * NB / 8, kChunks = kRowBytes / 16;
    static constexpr int kCodeBytes = kBlock * kRowBytes, kMetaBytes = kBlock * NG * 4;
    static constexpr int kStage = 2 * (kCodeBytes + kMetaBytes);  // keys, values, their metadata
    // blocks in flight: some 8 KB for each warp
    static constexpr int kStages = kStage >= 6144 ? 2 : kStage > 2560 ? 3 : kStage >= 1536 ? 4 : 6;
    static constexpr int kRow = D + 4;  // floats of a row of results: 16-byte stores, two to a bank
    static constexpr int kRing = kAttnWarps * kStages * kStage;
    static constexpr int kResult = kAttnWarps * 8 * RB * (kRow + 2) * 4;
    static constexpr int kRows = kRing > kResult ? kRing : kResult;  // the query rows lie behind
    static constexpr int kSmem = kRows + 8 * RB * (D * 2 + NG * 4 + 12);
    static constexpr int kCtas = D == 256 || RB == 2 ? 2 : 4;
};

// What a pair costs beside its tokens (its queries, the filling of the rings, its results), in units:
// pairs of short sequences would otherwise make a CTA's share longer than the others.
// (16 sequences of 1 to 2048 tokens x 32 heads: 43 us without, 34 with.)
constexpr uint32_t kFixed = 3;

// units of one pair of sequence b: kFixed that stand for no tokens, and at least one of tokens, so
// that each pair has a CTA that writes its rows
__device__ __forceinline__ uint32_t units_of(const Attn &a, int b) {
    int64_t span = own_len(a, b);
    if (a.window > 0) span = min(span, a.window + a.nq + kBlock);
    return kFixed + max((uint32_t)((span + kUnit - 1) / kUnit), 1u);
}

// CTA c's share of `total` units: the first total % ctas have one more
struct Shares {
    uint32_t each, more;
    __device__ Shares(uint32_t total, uint32_t ctas) : each(total / ctas), more(total % ctas) {}
    __device__ uint32_t begin(uint32_t c) const { return c * each + min(c, more); }
    __device__ uint32_t owner(uint32_t x) const {  // of unit x
        const uint32_t longer = more * (each + 1);
        return x < longer ? x / (each + 1) : more + (x - longer) / each;
    }
};

// Where a CTA's share begins, and what the sequences' units add up to; for all threads.
struct Start {
    uint32_t total, begin;  // units of all pairs; of those, the first of this CTA
    uint32_t before;        // units of the sequences before b
    int b;                  // the sequence that unit `begin` belongs to
};

__device__ __forceinline__ Start find_start(const Attn &a, Start *shared) {
    __shared__ uint32_t sums[kAttnWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t per = a.row_blocks * a.c.heads;
    const int chunk = (a.batch + kAttnThreads - 1) / kAttnThreads;  // sequences of a thread
    const int b0 = min((int)threadIdx.x * chunk, a.batch), b1 = min(b0 + chunk, a.batch);
    uint32_t sum = 0;
    for (int b = b0; b < b1; ++b) sum += units_of(a, b) * per;
    uint32_t upto = sum;
#pragma unroll
    for (int x = 1; x < 32; x *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, x);
        if (lane >= x) upto += y;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    uint32_t total = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
        if (w < warp) upto += sums[w];
        total += sums[w];
    }
    const uint32_t begin = Shares(total, a.ctas).begin(blockIdx.x);
    if (begin < upto && begin >= upto - sum) {  // one thread, if the share is not empty
        uint32_t before = upto - sum;
        int b = b0;
        for (;;) {
            const uint32_t u = units_of(a, b) * per;
            if (begin < before + u) break;
            before += u;
            ++b;
        }
        *shared = Start{total, begin, before, b};
    }
    __syncthreads();
    return begin < total ? *shared : Start{total, begin, total, a.batch};
}

// One segment: units [unit0, unit1) of a pair's tokens, by all warps of the CTA.  The result goes to
// part_o and part_lse, by the row of the pair (by_slot) or of the output, or to the outputs themselves
// where there are none.
template <int D, int NB, int NG, int RB, bool PREFIX>
__device__ __forceinline__ void attend_segment(const Attn &a, int b0, int row0, int head, uint32_t unit0, uint32_t unit1,
                                               float *part_o, float *part_lse, bool by_slot, unsigned char *smem) {
    using S = Shape<D, NB, NG, RB>;
    using KRegs = KeyRegs<D, NB, NG>;
    using VRegs = ValueRegs<NB>;
    constexpr int g = D / NG, KR = D / 8, VR = D / 8, RU = 8 * RB, n = S::kChunks;
    constexpr int kKeyBytes = S::kRowBytes / 4, kValueBytes = S::kRowBytes / 8;
    constexpr int kKeyPiece = kKeyBytes < 16 ? kKeyBytes : 16, kValuePiece = kValueBytes < 16 ? kValueBytes : 16;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, j = lane & 3;
    const int unit_rows = a.nq * a.share;                       // rows of one sequence and key head
    const int total_rows = PREFIX ? a.batch * unit_rows : unit_rows;

    // rows of one key head are numbered l = (b - b0) * nq * share + i * share + (h - head * share);
    // the output's row of that
    auto out_row = [&](int l) -> int64_t {
        const int b = b0 + l / unit_rows, i = l % unit_rows / a.share, h = l % a.share;
        return ((int64_t)b * a.nq + i) * a.heads + head * a.share + h;
    };

    // ---- the tokens of this segment that some row of the block may see
    const int last_row = min(row0 + RU, total_rows) - 1;
    int64_t first = 0, last;
    if constexpr (PREFIX) {
        last = a.prefix_len;
    } else {
        const int64_t len = own_len(a, b0);
        int64_t lo, hi;
        visible<PREFIX>(a, len, row0 / a.share, first, hi);
        visible<PREFIX>(a, len, last_row / a.share, lo, last);
        last = min(last, len);
    }
    const int64_t from = (first & ~(int64_t)(kBlock - 1)) + (int64_t)unit0 * kUnit;
    const int64_t to = max(min(from + (int64_t)(unit1 - unit0) * kUnit, last), from);

    // ---- this thread's share of the query rows: on its way while the page table is
    constexpr int T = kAttnThreads / RU, E = D / T;  // threads of a row, elements of a thread
    const int rr = threadIdx.x / T, d0 = threadIdx.x % T * E, lrow = row0 + rr;
    const bool live = lrow < total_rows;
    const int lc = live ? lrow : row0;
    const int b = b0 + lc / unit_rows, i = lc % unit_rows / a.share, h = head * a.share + lc % a.share;
    const uint16_t *q = a.q + b * a.q_batch + i * a.q_token + h * a.q_head + d0;
    uint32_t raw[E / 2];
    if (a.q_wide) {
#pragma unroll
        for (int e = 0; e < E / 4; ++e) *reinterpret_cast<uint2 *>(raw + 2 * e) = __ldg((const uint2 *)q + e);
    } else {
#pragma unroll
        for (int e = 0; e < E / 2; ++e) raw[e] = __ldg(q + 2 * e) | (uint32_t)__ldg(q + 2 * e + 1) << 16;
    }

    // ---- copies: this warp's block number `it` of the segment into stage it % kStages
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (S::kStages * S::kStage);
    const int steps = (int)((to - from + kBlock - 1) / kBlock - warp + kAttnWarps - 1) / kAttnWarps;
    constexpr int mc = S::kMetaBytes / 16;  // chunks of metadata of each side
    const uint8_t *k_from = pinned(a.c.codes[0] + 16 * lane), *v_from = pinned(a.c.codes[1] + 16 * lane);
    static_assert(mc <= 32 && 2 * mc % 8 == 0, "NG is 1, 2, 4 or 8");
    const uint8_t *m_from = pinned((const uint8_t *)a.c.meta[lane >= mc ? 1 : 0] + 16 * (lane % mc));
    const uint8_t *m2_from = (const uint8_t *)a.c.meta[1] + 16 * lane;  // where a side has 32 chunks
    const uint32_t k_place = pinned(16 * key_chunk(n, lane / n, lane % n));
    const uint32_t v_place = pinned(S::kCodeBytes + 16 * value_chunk(n, lane / n, lane % n));
    const uint32_t m_place = pinned(2 * S::kCodeBytes + 16 * lane);
    int block_of_lane = 0;    // where block number it - it % 32 + lane lies, in blocks; -1: nowhere
    uint32_t there = 0;       // bit i: the block copied i steps ago lies in the pool
    auto copy = [&](int it, uint32_t to_stage) {  // past the last block: nothing
        if ((it & 31) == 0) {
            const int64_t t = from + (int64_t)(warp + (it + lane) * kAttnWarps) * kBlock;
            block_of_lane = -1;
            if (t < to) {
                const int32_t *table = PREFIX ? a.prefix_pages : a.pages + b0 * a.pages_stride;
                const int page = __ldg(table + (t >> a.c.page_shift));
                if (page >= 0 && page < a.c.pages)
                    block_of_lane = (int)(row_of(a.c, page, head, (int)t & ((1 << a.c.page_shift) - 1)) / kBlock);
            }
        }
        const int block = __shfl_sync(0xffffffffu, block_of_lane, it & 31);
        const bool in = block >= 0;
        there = 2 * there + (in ? 1u : 0u);
        const uint8_t *k = k_from + (int64_t)block * S::kCodeBytes, *v = v_from + (int64_t)block * S::kCodeBytes;
        const uint8_t *m = m_from + (int64_t)block * S::kMetaBytes;
        const uint32_t k_to = to_stage + k_place, v_to = to_stage + v_place;
        if constexpr (n >= 2) {
#pragma unroll
            for (int i = 0; i < n / 2; ++i) {
                // 32 chunks on, a value's chunk has another place in its row (value_chunk)
                constexpr int p_step = n == 8 ? 2 : n == 16 ? 1 : 0;
                const int p = i * p_step & 3, turned = n == 8 ? 2 * p : n == 16 ? (p & 1) | (p & 2) << 1 : 0;
                copy16(in, k_to + 512 * i, k + 512 * i);
                copy16(in, turned ? to_stage + (v_place ^ (16 * turned)) + 512 * i : v_to + 512 * i, v + 512 * i);
            }
        } else {
            copy16(in && lane < kBlock, k_to, k);
            copy16(in && lane < kBlock, v_to, v);
        }
        // the metadata's 2 mc chunks, keys first: by the first lanes, or two by each lane
        const uint32_t m_to = to_stage + m_place;
        copy16(in && m_place < 2 * S::kCodeBytes + 32 * mc, m_to, m);
        if constexpr (2 * mc > 32) copy16(in, m_to + 512, m2_from + (int64_t)block * S::kMetaBytes);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) copy(i, ring + i * S::kStage);

    // ---- the rows: scaled by a power of two that takes a row's largest magnitude to [2^14, 2^15)
    // (exact, but for values 2^-20 below the largest; it makes bf16 fit fp16), into shared memory
    // in the order of the keys' registers: lane 4r + j holds row r's share of run j
    uint32_t *rows_q = reinterpret_cast<uint32_t *>(smem + S::kRows);          // [RB][KR / 4][32 lanes][4]
    float *rows_sum = reinterpret_cast<float *>(rows_q + RB * 32 * KR);        // [RU][NG]: sums of q
    float *rows_unit = rows_sum + RU * NG;                                     // [RU]
    int *rows_lo = reinterpret_cast<int *>(rows_unit + RU), *rows_hi = rows_lo + RU;  // visible tokens from `from`
    {
        float x[E];
        uint32_t big = 0;  // the bits of the largest magnitude; a NaN's are above any number's
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t w = live ? raw[e / 2] : 0u;
            x[e] = a.bf ? __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16) : to_f32<false>((uint16_t)(e & 1 ? w >> 16 : w));
            big = max(big, __float_as_uint(fabsf(x[e])));
        }
#pragma unroll
        for (int y = 1; y < T; y *= 2) big = max(big, __shfl_xor_sync(0xffffffffu, big, y));
        // 2^(14 - floor(log2 big)); both it and its inverse stay normal
        const int ex = big > 0 ? min(max((int)(big >> 23) - 127, -100), 100) : 0;
        const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
        // a row with an infinity, a NaN or numbers out of range becomes NaN in every product: its score of
        // each token that it sees is NaN, and its result (an infinite score would look like a hidden token)
        const float by = row_in_range(big, a.scale_log2) ? up : __uint_as_float(0x7fc00000u);
        float sum = 0.0f;
        __half *to_q = reinterpret_cast<__half *>(rows_q);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] *= by;
            sum += x[e];
            const int d = d0 + e, run = d % g / (g / 4), code = d / g * (g / 4) + d % (g / 4);
            const int reg = code / (2 * KRegs::kSpan) * KRegs::kSpan + code % KRegs::kSpan;
            const float down = __uint_as_float((uint32_t)(127 - code_up<NB>(reg % KRegs::kU)) << 23);
            // in 16-byte pieces that the 32 lanes of a row block read side by side
            const int at = (rr / 8 * (KR / 4) + reg / 4) * 128 + (rr % 8 * 4 + run) * 4 + reg % 4;
            to_q[at * 2 + code / KRegs::kSpan % 2] = __float2half_rn(x[e] * down);
        }
#pragma unroll
        for (int y = 1; y < g / E; y *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, y);
        if (d0 % g == 0) rows_sum[rr * NG + d0 / g] = sum * 0x1p-24f;
        if (d0 == 0) {
            int64_t lo, hi;
            visible<PREFIX>(a, own_len(a, b), i, lo, hi);
            // a row that is not there (q = 0) may see everything: its result is not written
            const int64_t cap = to - from;
            rows_hi[rr] = live ? (int)min(max(hi - from, (int64_t)0), cap) : (int)cap;
            rows_lo[rr] = live ? (int)min(max(lo - from, (int64_t)0), cap) : 0;
            rows_unit[rr] = row_unit(up, a.scale_log2);
        }
    }
    __syncthreads();
    // of this lane, as result columns 2j and 2j + 1
    float qs[RB][2][NG];
    float unit[RB][2];           // what a result is to be multiplied by: powers of two out
    const int there_lo = (int)max(first - from, (int64_t)0), there_hi = (int)(to - from);  // tokens, from `from`
    int all_lo = there_lo, all_hi = there_hi;  // those that every row of the block sees
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int rr = 8 * rb + 2 * j + y;
#pragma unroll
            for (int x = 0; x < NG; ++x) qs[rb][y][x] = rows_sum[rr * NG + x];
            unit[rb][y] = rows_unit[rr];
            all_hi = min(all_hi, rows_hi[rr]);
            all_lo = max(all_lo, rows_lo[rr]);
        }
    }
    all_hi = __reduce_min_sync(0xffffffffu, all_hi);
    all_lo = __reduce_max_sync(0xffffffffu, all_lo);

    // O^T: row r of an MMA's 16 is element 2mb of run r, row r + 8 element 2mb + 1; columns are rows
    // 2j, 2j + 1.  oz: the same for the zero points, sum of w vz (each row of the 16 alike)
    float o[RB][VR / 2][4], oz[RB][NG][4];
    float m[RB][2], l[RB][2], bound[RB][2];  // bound: a raw score above it asks for a new maximum
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
#pragma unroll
            for (int x = 0; x < VR / 2; ++x) o[rb][x][y] = 0.0f;
#pragma unroll
            for (int x = 0; x < NG; ++x) oz[rb][x][y] = 0.0f;
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            m[rb][y] = kLowest;
            bound[rb][y] = -INFINITY;
            l[rb][y] = 0.0f;
        }
    }
    // what a group's value scales are multiplied by: kWeightUnit over a power of two that is at least
    // every scale of the group so far, so that its weights lie within fp16 whatever the others' scales are
    float vin[NG];
#pragma unroll
    for (int x = 0; x < NG; ++x) vin[x] = kWeightUnit * 0x1p24f;

    const uint32_t k_at = pinned(16 * key_chunk(n, r, j * kKeyBytes / 16) + j * kKeyBytes % 16);
    // the odd lanes read the second token of a pair first
    const int va = 2 * j + (j & 1), vb = 2 * j + 1 - (j & 1);
    const uint32_t v_at[2] = {pinned(S::kCodeBytes + 16 * value_chunk(n, va, r * kValueBytes / 16) + r * kValueBytes % 16),
                              pinned(S::kCodeBytes + 16 * value_chunk(n, vb, r * kValueBytes / 16) + r * kValueBytes % 16)};
    const uint32_t sel_lo = pinned(j & 1 ? 0x1054u : 0x5410u), sel_hi = pinned(j & 1 ? 0x3276u : 0x7632u);
    const uint32_t q_at = (uint32_t)__cvta_generic_to_shared(rows_q) + 16 * lane;
    const uint32_t m_at = pinned(2 * S::kCodeBytes + r * NG * 4);

    uint32_t w[RB][NG][2], z[NG][2];  // a block's weights and its value zero points, as operands
    // O^T += V^T W^T of the block whose stage is at `at`
    auto values = [&](uint32_t at) {
        Words<(kValueBytes + 3) / 4> v[4];
#pragma unroll
        for (int i = 0; i < (kValueBytes + kValuePiece - 1) / kValuePiece; ++i)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const uint32_t from_at = at + (kValueBytes > 16 ? v_at[y & 1] ^ (uint32_t)(16 * i) : v_at[y & 1]);
                lds_piece<kValuePiece>(v[y].w + 4 * i, from_at + (y >> 1) * 8 * S::kRowBytes);
            }
#pragma unroll
        for (int x = 0; x < NG; ++x) {
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) mma_16816(oz[rb][x], z[x][0], z[x][0], z[x][1], z[x][1], w[rb][x][0], w[rb][x][1]);
#pragma unroll
            for (int mb = x * (g / 16); mb < (x + 1) * (g / 16); ++mb) {
                const uint32_t a0 = VRegs::reg(v[0], v[1], 2 * mb, sel_lo, sel_hi);
                const uint32_t a1 = VRegs::reg(v[0], v[1], 2 * mb + 1, sel_lo, sel_hi);
                const uint32_t a2 = VRegs::reg(v[2], v[3], 2 * mb, sel_lo, sel_hi);
                const uint32_t a3 = VRegs::reg(v[2], v[3], 2 * mb + 1, sel_lo, sel_hi);
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) mma_16816(o[rb][mb], a0, a1, a2, a3, w[rb][x][0], w[rb][x][1]);
            }
        }
    };

    uint32_t s_at = ring;  // block it's stage
    const uint32_t ring_last = ring + (S::kStages - 1) * S::kStage;
    for (int it = 0, t0 = warp * kBlock; it < steps; ++it, t0 += kUnit) {
        // block `it` has arrived for every lane, and every lane is done with block it - 1, whose
        // stage the next copy takes
        asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 2) : "memory");
        __syncwarp();
        copy(it + S::kStages - 1, s_at == ring ? ring_last : s_at - S::kStage);
        Words<(kKeyBytes + 3) / 4> k0, k1;
#pragma unroll
        for (int i = 0; i < kKeyBytes / kKeyPiece; ++i) {
            // the chunks of a run lie together, or exchanged as the swizzle says
            const uint32_t at = s_at + (kKeyBytes > 16 ? k_at ^ (uint32_t)(16 * i) : k_at);
            lds_piece<kKeyPiece>(k0.w + 4 * i, at);
            lds_piece<kKeyPiece>(k1.w + 4 * i, at + 8 * S::kRowBytes);
        }
        uint32_t km[2][NG], vm[2][NG];  // (scale, zero)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            constexpr int piece = NG >= 4 ? 16 : NG * 4;
#pragma unroll
            for (int x = 0; x < NG * 4 / piece; ++x) {
                const uint32_t at = s_at + m_at + y * 8 * NG * 4 + x * 16;
                lds_piece<piece>(km[y] + 4 * x, at);
                lds_piece<piece>(vm[y] + 4 * x, at + S::kMetaBytes);
            }
        }
        auto meta = [](uint32_t m2) { return __half22float2(*reinterpret_cast<const __half2 *>(&m2)); };

        uint32_t qb[RB][KR];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int x = 0; x < KR; x += 4) lds_piece<16>(qb[rb] + x, q_at + (rb * (KR / 4) + x / 4) * 512);
        // ---- S^T: raw scores
        float s[RB][4];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int y = 0; y < 4; ++y) s[rb][y] = 0.0f;
#pragma unroll
        for (int x = 0; x < NG; ++x) {
            float c[RB][4];
#pragma unroll
            for (int rb = 0; rb < RB; ++rb)
#pragma unroll
                for (int y = 0; y < 4; ++y) c[rb][y] = 0.0f;
#pragma unroll
            for (int st = x * (g / 16); st < (x + 1) * (g / 16); ++st) {
                const uint32_t a0 = KRegs::reg(k0, 2 * st), a1 = KRegs::reg(k1, 2 * st);
                const uint32_t a2 = KRegs::reg(k0, 2 * st + 1), a3 = KRegs::reg(k1, 2 * st + 1);
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) mma_16816(c[rb], a0, a1, a2, a3, qb[rb][2 * st], qb[rb][2 * st + 1]);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float2 kz = meta(km[y >> 1][x]);
#pragma unroll
                for (int rb = 0; rb < RB; ++rb)
                    s[rb][y] = __fmaf_rn(kz.x, __fmaf_rn(-kz.y, qs[rb][y & 1][x], c[rb][y]), s[rb][y]);
            }
        }
        // ---- where some row does not see all 16 tokens, or their page is not there.  Rows that hold
        // no token of this sequence hold anything: their codes are finite numbers, their scores are
        // replaced, and the values' metadata too
        const bool in = there >> (S::kStages - 1) & 1u;
        if (!in || t0 < all_lo || t0 + kBlock > all_hi) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int t = t0 + r + 8 * y;
                const bool live = in && t >= there_lo && t < there_hi;
#pragma unroll
                for (int x = 0; x < NG; ++x) vm[y][x] = live ? vm[y][x] : 0u;
#pragma unroll
                for (int rb = 0; rb < RB; ++rb)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int rr = 8 * rb + 2 * j + c;
                        if (!live || t >= rows_hi[rr] || t < rows_lo[rr]) s[rb][2 * y + c] = -INFINITY;
                    }
            }
        }
        // ---- a new maximum, or a larger value scale than any before: rescale
        float vw[NG][2], most = 0.0f;
#pragma unroll
        for (int x = 0; x < NG; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                vw[x][y] = __low2float(*reinterpret_cast<const __half2 *>(&vm[y][x])) * vin[x];
                most = fmaxf(most, vw[x][y]);
            }
        bool more = most > kWeightUnit;
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int y = 0; y < 2; ++y) more |= fmaxf(s[rb][y], s[rb][y + 2]) > bound[rb][y];
        if (__any_sync(0xffffffffu, more)) {
            float fv[NG];
#pragma unroll
            for (int x = 0; x < NG; ++x) {
                // a new unit has room for scales four times as large, so that few blocks ask for one
                const uint32_t big = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(vw[x][0], vw[x][1])));
                // kWeightUnit / 4 over the power of two at or above big
                const uint32_t less = __float_as_uint(kWeightUnit / 4.0f) + (127u << 23) - ((big + 0x007fffffu) & 0x7f800000u);
                fv[x] = big > __float_as_uint(kWeightUnit) ? __uint_as_float(less) : 1.0f;
                vin[x] *= fv[x];
#pragma unroll
                for (int y = 0; y < 2; ++y) vw[x][y] *= fv[x];
            }
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                float f[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float top = fmaxf(s[rb][y], s[rb][y + 2]);
#pragma unroll
                    for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    top = fmaxf(top * unit[rb][y], m[rb][y]);
                    f[y] = exp2_fast(m[rb][y] - top);
                    m[rb][y] = top;
                    bound[rb][y] = top == kLowest ? -INFINITY : (top + kLag) / unit[rb][y];
                    l[rb][y] *= score_in_range(top) ? f[y] : __uint_as_float(0x7fc00000u);
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
#pragma unroll
                    for (int x = 0; x < VR / 2; ++x) o[rb][x][y] *= f[y & 1] * fv[x / (g / 16)];
#pragma unroll
                    for (int x = 0; x < NG; ++x) oz[rb][x][y] *= f[y & 1] * fv[x];
                }
            }
        }
        // ---- weights
        float p[RB][4];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                p[rb][y] = exp2_fast(__fmaf_rn(s[rb][y], unit[rb][y & 1], -m[rb][y & 1]));
                l[rb][y & 1] += p[rb][y];
            }
#pragma unroll
        for (int x = 0; x < NG; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                // a column of the tokens' zero points, alike for all 16 rows of an operand
                z[x][y] = turn(__byte_perm(vm[y][x], 0, 0x3232));
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) {
                    const __half2 h = __floats2half2_rn(p[rb][2 * y] * vw[x][y], p[rb][2 * y + 1] * vw[x][y]);
                    w[rb][x][y] = turn(*reinterpret_cast<const uint32_t *>(&h));
                }
            }
        values(s_at);
        s_at = s_at == ring_last ? ring : s_at + S::kStage;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the rings are free: the results take their place

    // ---- the warps' results meet in shared memory, in units of the values
    float *res = reinterpret_cast<float *>(smem), *res_m = res + kAttnWarps * RU * S::kRow, *res_l = res_m + kAttnWarps * RU;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
#pragma unroll
            for (int x = 4; x < 32; x *= 2) l[rb][y] += __shfl_xor_sync(0xffffffffu, l[rb][y], x);
            if (r == 0) {
                res_m[warp * RU + 8 * rb + 2 * j + y] = m[rb][y];
                res_l[warp * RU + 8 * rb + 2 * j + y] = l[rb][y];
            }
        }
        constexpr int s8 = g / 8;
#pragma unroll
        for (int x = 0; x < VR; x += 4) {  // s8 is 4 or more: four elements in a row
            const int d = x / s8 * g + r * s8 + x % s8;
            const float vu = __uint_as_float(0x7f000000u - __float_as_uint(vin[x / s8]));  // 1 over a power of two
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    e[i] = __fmaf_rn(o[rb][(x + i) / 2][2 * (i & 1) + y], 0x1p24f / (float)(1 << VRegs::up(x + i)),
                                     -oz[rb][x / s8][y]) * vu;
                *reinterpret_cast<float4 *>(res + (warp * RU + 8 * rb + 2 * j + y) * S::kRow + d) = make_float4(e[0], e[1], e[2], e[3]);
            }
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < RU * (D / 4); e += kAttnThreads) {
        const int rr = e / (D / 4), d = e % (D / 4) * 4;
        if (row0 + rr > last_row) break;
        float top = kLowest;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, res_m[w * RU + rr]);
        float sum = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
            const float f = exp2_fast(res_m[w * RU + rr] - top);
            sum = __fmaf_rn(res_l[w * RU + rr], f, sum);
            const float4 v = *reinterpret_cast<const float4 *>(res + (w * RU + rr) * S::kRow + d);
            acc[0] = __fmaf_rn(v.x, f, acc[0]);
            acc[1] = __fmaf_rn(v.y, f, acc[1]);
            acc[2] = __fmaf_rn(v.z, f, acc[2]);
            acc[3] = __fmaf_rn(v.w, f, acc[3]);
        }
        // a sum of zero is a row that sees nothing; a NaN stays
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const float lse = sum == 0.0f ? -INFINITY : top + log2f(sum);
        const int64_t orow = out_row(row0 + rr);
        if (part_o) {
            const int64_t at = by_slot ? rr : orow;
            *reinterpret_cast<float4 *>(part_o + at * D + d) = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
            if (d == 0) part_lse[at] = lse;
        } else {
            uint16_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = a.bf ? from_f32<true>(acc[i] * inv) : from_f32<false>(acc[i] * inv);
            *reinterpret_cast<uint2 *>(a.out + orow * D + d) =
                make_uint2(y[0] | (uint32_t)y[1] << 16, y[2] | (uint32_t)y[3] << 16);
            if (d == 0 && a.lse) a.lse[orow] = lse * 0.6931471805599453f;
        }
    }
}

// The sequences' own tokens.  a.ctas = 0: CTA x has pair x.  Otherwise CTA x has its share of all
// pairs' units, in order: the end of one pair, whole pairs, the beginning of another.
template <int D, int NB, int NG, int RB>
__global__ void __launch_bounds__(kAttnThreads, (Shape<D, NB, NG, RB>::kCtas)) hqq_kv_attn_kernel(const Attn a) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Start start_s;
    constexpr int RU = 8 * RB;
    const int per = a.row_blocks * a.c.heads;  // pairs of a sequence
    const int64_t rows = (int64_t)a.batch * a.nq * a.heads;
    float *whole_o = a.part_o ? a.part_o + a.prefix_splits * rows * D : nullptr;
    float *whole_lse = a.part_o ? a.part_lse + a.prefix_splits * rows : nullptr;
    int b, pair;             // pair: of the sequence, row block * heads + head
    uint32_t at, left;       // the next unit of the pair; units left of this CTA's share
    uint32_t total = 0, begin = 0;
    Cut cut{-1, 0, 0, 0};
    if (a.ctas == 0) {
        b = (int)blockIdx.x / per;
        pair = (int)blockIdx.x % per;
        at = 0;
        left = units_of(a, b);
    } else {
        const Start start = find_start(a, &start_s);
        total = start.total;
        begin = start.begin;
        left = Shares(total, a.ctas).begin(blockIdx.x + 1) - begin;
        b = start.b;
        if (left > 0) {
            const uint32_t units = units_of(a, b);
            pair = (int)((begin - start.before) / units);
            at = begin - start.before - pair * units;
        }
    }
    while (left > 0) {
        const uint32_t units = units_of(a, b), take = min(units - at, left), end = at + take;
        if (end > kFixed) {
            const bool top = at <= kFixed, whole = top && end == units;  // top: the pair's first tokens
            float *po = whole_o, *pl = whole_lse;
            if (!whole) {  // the first part of a pair goes to the CTA's second slot
                const int64_t slot = (2 * (int64_t)blockIdx.x + (top ? 1 : 0)) * RU;
                po = a.slot_o + slot * D;
                pl = a.slot_lse + slot;
                if (top)
                    cut = Cut{b, pair, (int)blockIdx.x, (int)Shares(total, a.ctas).owner(begin + units - at - 1)};
            }
            attend_segment<D, NB, NG, RB, false>(a, b, pair / a.c.heads * RU, pair % a.c.heads, top ? 0 : at - kFixed,
                                                 end - kFixed, po, pl, !whole, smem);
            __syncthreads();  // the results have been read: the rings may take their place again
        }
        left -= take;
        begin += take;
        at = 0;
        if (++pair == per) {
            pair = 0;
            ++b;
        }
    }
    if (a.ctas > 0 && threadIdx.x == 0) a.cuts[blockIdx.x] = cut;
    // the join waits for this kernel only, and may read what the prefix's wrote: that one first
    if (a.prefix_splits > 0) wait_prerequisite();
}

// The prefix: CTA (x, y, z) has chunk x for block y of the batch's rows and key head z.
template <int D, int NB, int NG, int RB>
__global__ void __launch_bounds__(kAttnThreads, (Shape<D, NB, NG, RB>::kCtas)) hqq_kv_prefix_kernel(const Attn a) {
    extern __shared__ __align__(16) unsigned char smem[];
    allow_dependents();  // the sequences' own tokens need nothing of this
    const int64_t rows = (int64_t)a.batch * a.nq * a.heads;
    const uint32_t units = (uint32_t)(a.prefix_chunk / kUnit);
    attend_segment<D, NB, NG, RB, true>(a, 0, (int)blockIdx.y * 8 * RB, (int)blockIdx.z, blockIdx.x * units,
                                        (blockIdx.x + 1) * units, a.part_o + blockIdx.x * rows * D,
                                        a.part_lse + blockIdx.x * rows, false, smem);
}

// Joins the parts of one row, a warp to every kJoinWarps-th part, in the order of the tokens (the
// prefix's chunks first).  Without a prefix CTA (x, y) has row y of the pair that begins in CTA x's
// share and ends in another's; with one, row y of pair x.
constexpr int kJoinWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) hqq_kv_join_kernel(const Attn a, int pair_rows) {
    __shared__ float acc_s[kJoinWarps][D], sum_s[kJoinWarps];
    constexpr int E = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    wait_prerequisite();
    Cut cut = {(int)blockIdx.x / (a.row_blocks * a.c.heads), (int)blockIdx.x % (a.row_blocks * a.c.heads), 0, 0};
    if (a.prefix_splits == 0) {
        {
            const int4 w = __ldcg((const int4 *)(a.cuts + blockIdx.x));
            cut = Cut{w.x, w.y, w.z, w.w};
        }
        if (cut.b < 0) return;
    } else {
        // the CTAs that wrote this pair's parts, if it was cut
        __shared__ int2 found;
        if (threadIdx.x == 0) found = make_int2(0, 0);
        __syncthreads();
        for (int c = threadIdx.x; c < a.ctas; c += 32 * kJoinWarps) {
            const int4 w = __ldcg((const int4 *)(a.cuts + c));
            if (w.x == cut.b && w.y == cut.pair) found = make_int2(w.z, w.w);
        }
        __syncthreads();
        cut.c0 = found.x;
        cut.c1 = found.y;
    }
    const int head = cut.pair % a.c.heads, l = cut.pair / a.c.heads * pair_rows + (int)blockIdx.y;
    if (l >= a.nq * a.share) return;  // no such row
    const int64_t rows = (int64_t)a.batch * a.nq * a.heads;
    const int64_t row = ((int64_t)cut.b * a.nq + l / a.share) * a.heads + head * a.share + l % a.share;
    const int c0 = cut.c0, c1 = cut.c1, parts = a.prefix_splits + c1 - c0 + 1;
    auto find = [&](int p, const float *&o, const float *&lse) {
        if (p < a.prefix_splits || c0 == c1) {
            o = a.part_o + (p * rows + row) * D;
            lse = a.part_lse + p * rows + row;
        } else {
            const int c = c0 + p - a.prefix_splits;
            const int64_t at = (2 * (int64_t)c + (c == c0 ? 1 : 0)) * pair_rows + blockIdx.y;
            o = a.slot_o + at * D;
            lse = a.slot_lse + at;
        }
    };
    const float *o, *e;
    float top = kLowest;
    for (int p = lane; p < parts; p += 32) {
        find(p, o, e);
        top = fmaxf(top, __ldcg(e));
    }
#pragma unroll
    for (int x = 16; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    // four parts at a time, all their loads on the way before the first is used
    constexpr int kAtOnce = 4, kVec = E < 4 ? E : 4;
    float acc[E], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.0f;
    for (int p = warp; p < parts; p += kJoinWarps * kAtOnce) {
        float x[kAtOnce][E], at[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            at[u] = -INFINITY;
#pragma unroll
            for (int i = 0; i < E; ++i) x[u][i] = 0.0f;
            if (p + u * kJoinWarps >= parts) continue;
            find(p + u * kJoinWarps, o, e);
            at[u] = __ldcg(e);
#pragma unroll
            for (int i = 0; i < E; i += kVec) {
                if constexpr (kVec == 4) *reinterpret_cast<float4 *>(x[u] + i) = __ldcg((const float4 *)(o + lane * E + i));
                else *reinterpret_cast<float2 *>(x[u] + i) = __ldcg((const float2 *)(o + lane * E + i));
            }
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const float f = exp2_fast(at[u] - top);  // a part that saw nothing holds zeros
            sum += f;
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] = __fmaf_rn(x[u][i], f, acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) acc_s[warp][lane * E + i] = acc[i];
    if (lane == 0) sum_s[warp] = sum;
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 32 * kJoinWarps) {
        float y = 0.0f, z = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            y += acc_s[w][d];
            z += sum_s[w];
        }
        y = z == 0.0f ? 0.0f : y / z;  // zero: the row sees nothing; a NaN, of a part too, stays
        a.out[row * D + d] = a.bf ? from_f32<true>(y) : from_f32<false>(y);
        if (d == 0 && a.lse) a.lse[row] = z == 0.0f ? -INFINITY : (top + log2f(z)) * 0.6931471805599453f;
    }
}

// Rows of a key head over the whole batch above which the prefix goes to the tcgen05 kernel, which
// takes 128 at a time.  Whole calls in us, that kernel / the one above, 4 bits, D = 128, g = 64:
//   8 key heads   4096 tokens 32 rows 22 / 18, 64 rows 23 / 20, 128 rows 25 / 31;
//                 32768 tokens 32 rows 56 / 38, 64 rows 57 / 60, 128 rows 60 / 115
//   2 key heads   128 rows, 4096 tokens 23 / 19, 32768 tokens 37 / 39
//   1 key head    128 rows, 1000 tokens 21 / 12, 4096 tokens 22 / 13, 32768 tokens 28 / 29
// 2 and 8 bits and D = 64 lie alike (8 key heads, 128 rows x 32768: 58 / 110, 68 / 113, 41 / 74).  So
// the rule is right where the prefix's work fills the GPU, and costs up to 9 us where one or two key
// heads have a short one.
constexpr int kTcMinRows = 64;

constexpr float kLog2e = 1.4426950408889634f;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// rows that a CTA takes: 8, or 16 where a key head has more (and the accumulators fit)
int rows_per_cta(int head_dim, int64_t rows) { return rows > 8 && head_dim <= 128 ? 16 : 8; }

int make_attn_plan(const hqq_kv_cache_t *cache, int64_t batch, int64_t nq, int64_t heads, int64_t max_len,
                   int64_t window, int64_t prefix_len, AttnPlan *pl) {
    Cache c;
    const int rc = check_cache(cache, &c);
    if (rc != HQQ_OK) return rc;
    if (batch < 0 || nq < 0 || heads <= 0 || max_len < 0 || window < 0 || prefix_len < 0 || heads % c.heads)
        return HQQ_ERR_ARG;
    // rows and pairs are counted in 31 bits, blocks of a grid's second and third dimension in 16
    if (max_len > INT32_MAX || prefix_len > INT32_MAX || batch > 65535 || nq > 65535 ||
        batch * nq > INT32_MAX / heads)
        return HQQ_ERR_UNSUPPORTED;
    *pl = AttnPlan{};
    // a window of max_len tokens hides none; below it, sums with nq stay far within 64 bits
    if (window >= max_len) window = 0;
    pl->window = window;
    if (batch * nq == 0) return HQQ_OK;  // no rows: nothing is launched
    const int64_t rows = nq * (heads / c.heads);
    const int ru = pl->pair_rows = rows_per_cta(cache->head_dim, rows);
    pl->row_blocks = (int)ceil_div(rows, ru);
    const int per_sm = cache->head_dim == 256 || ru == 16 ? 2 : 4;
    int64_t span = max_len;
    if (window > 0) span = std::min<int64_t>(span, window + nq + kBlock);
    const int64_t units = kFixed + std::max<int64_t>(1, ceil_div(span, kUnit)), pairs = batch * c.heads * pl->row_blocks;
    // Pairs of at most 1024 tokens have a CTA each, and no join: one launch, and about as many steps in
    // a row as the join costs.  Longer ones are shared among all SMs; a share is at least 4 units.
    // In us, a CTA each / shared, 4 bits, g = 64:
    //   32 heads on 8, D = 128   1 x 500 tokens 8.1 / 9.9, 1 x 1000 11.7 / 10.0, 16 x 1000 12.3 / 16.1,
    //                            64 x 1000 23.8 / 31.7, 1 x 2000 18.2 / 10.3, 16 x 2000 19.7 / 20.4
    //   the same, D = 64         1 x 1000 9.2 / 9.1, 16 x 1000 9.6 / 13.0; D = 256: 15.8 / 11.9, 17.0 / 21.5
    //   8 heads on 1, D = 128    1 x 500 8.3 / 9.9, 1 x 1000 11.9 / 10.0, 16 x 1000 12.3 / 10.7, 64 x 1000 12.5 / 14.0
    // So a call of few pairs near 1024 tokens loses up to 2 us (D = 256: 4) to the rule, one of many
    // gains up to 8.
    if (units > kFixed + 16)
        pl->ctas = (int)std::min<int64_t>(kSms * per_sm, std::max<int64_t>(pairs, ceil_div(pairs * units, 4)));
    if (pairs > INT32_MAX / units) return HQQ_ERR_UNSUPPORTED;  // units are counted in 31 bits
    pl->slot_floats = (size_t)2 * pl->ctas * ru;
    pl->prefix_tc = prefix_len > 0 && rows * batch > kTcMinRows && prefix_tc_layout(*cache);
    if (pl->prefix_tc) {
        pl->prefix_row_blocks = (int)ceil_div(rows * batch, kTcRows);
        if (pl->prefix_row_blocks > 65535 || c.heads > 65535) return HQQ_ERR_UNSUPPORTED;
        const int64_t want = std::max<int64_t>(1, 2 * kSms / ((int64_t)c.heads * pl->prefix_row_blocks));
        pl->prefix_chunk = std::max<int64_t>(4 * kTcTokens, ceil_div(ceil_div(prefix_len, want), kTcTokens) * kTcTokens);
    } else if (prefix_len > 0) {
        const int pru = rows_per_cta(cache->head_dim, rows * batch);
        pl->prefix_row_blocks = (int)ceil_div(rows * batch, pru);
        if (pl->prefix_row_blocks > 65535 || c.heads > 65535) return HQQ_ERR_UNSUPPORTED;
        const int64_t want = std::max<int64_t>(1, kSms * (cache->head_dim == 256 || pru == 16 ? 2 : 4) /
                                                      ((int64_t)c.heads * pl->prefix_row_blocks));
        pl->prefix_chunk = std::max<int64_t>(4 * kUnit, ceil_div(ceil_div(prefix_len, want), kUnit) * kUnit);
    }
    if (prefix_len > 0) {
        pl->prefix_splits = (int)ceil_div(prefix_len, pl->prefix_chunk);
        pl->part_floats = (size_t)(pl->prefix_splits + 1) * (size_t)(batch * nq * heads);
    }
    pl->bytes = (pl->slot_floats + pl->part_floats) * (cache->head_dim + 1) * sizeof(float) + pl->ctas * sizeof(Cut);
    return HQQ_OK;
}

// `beside`: may start before the kernel in front of it has ended
template <typename K, typename... Args>
cudaError_t launch_attn(K kernel, dim3 grid, int threads, int smem, bool beside, cudaStream_t st, Args... args) {
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = beside ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int run_attention(const hqq_kv_cache_t *cache, const Attn &a, const AttnPlan &pl, cudaStream_t st) {
    if ((int64_t)a.batch * a.nq == 0) return HQQ_OK;
    const int64_t pairs = (int64_t)a.batch * a.row_blocks * a.c.heads;
    return with_layout(*cache, [&](auto dim, auto bits, auto groups) {
        constexpr int D = dim, NB = bits, NG = groups;
        constexpr int kWide = D <= 128 ? 2 : 1;
        cudaError_t e = cudaSuccess;
        if (pl.prefix_splits > 0) {
            const dim3 grid(pl.prefix_splits, pl.prefix_row_blocks, a.c.heads);
            if (pl.prefix_tc)
                e = launch_prefix_tc(*cache, a, pl.prefix_row_blocks, st);
            else if (rows_per_cta(D, (int64_t)a.nq * a.share * a.batch) == 16)
                e = launch_attn(hqq_kv_prefix_kernel<D, NB, NG, kWide>, grid, kAttnThreads, Shape<D, NB, NG, kWide>::kSmem, false, st, a);
            else
                e = launch_attn(hqq_kv_prefix_kernel<D, NB, NG, 1>, grid, kAttnThreads, Shape<D, NB, NG, 1>::kSmem, false, st, a);
            if (e != cudaSuccess) return HQQ_ERR_CUDA;
        }
        const dim3 grid(a.ctas ? a.ctas : (unsigned)pairs);
        const bool beside = pl.prefix_splits > 0;
        if (pl.pair_rows == 16)
            e = launch_attn(hqq_kv_attn_kernel<D, NB, NG, kWide>, grid, kAttnThreads, Shape<D, NB, NG, kWide>::kSmem, beside, st, a);
        else
            e = launch_attn(hqq_kv_attn_kernel<D, NB, NG, 1>, grid, kAttnThreads, Shape<D, NB, NG, 1>::kSmem, beside, st, a);
        if (e != cudaSuccess) return HQQ_ERR_CUDA;
        if (a.ctas || pl.prefix_splits)
            e = launch_attn(hqq_kv_join_kernel<D>, dim3(pl.prefix_splits ? (unsigned)pairs : (unsigned)a.ctas, std::min(pl.pair_rows, a.nq * a.share)),
                            32 * kJoinWarps, 0, true, st, a, pl.pair_rows);
        return e == cudaSuccess ? HQQ_OK : HQQ_ERR_CUDA;
    });
}

int check_attention(const hqq_kv_cache_t *cache, const void *q, int dtype, int64_t batch, int64_t nq, int64_t heads,
                    const int32_t *pages, int64_t max_pages, const int32_t *lens, int64_t max_len, float scale,
                    void *out, float *lse, void *workspace, size_t workspace_bytes, const AttnPlan &pl) {
    if (dtype != HQQ_FP16 && dtype != HQQ_BF16) return HQQ_ERR_ARG;
    if (max_pages < 0 || ceil_div(max_len, cache->page_size) > max_pages || !(scale > 0.0f) || !std::isfinite(scale * kLog2e))
        return HQQ_ERR_ARG;
    if (batch == 0 || nq == 0) return HQQ_OK;
    if (!q || !lens || !out || (max_pages > 0 && !pages)) return HQQ_ERR_ARG;
    if (!aligned_to(q, 2) || !aligned_to(pages, 4) || !aligned_to(lens, 4) || !aligned_to(out, 16) || !aligned_to(lse, 4))
        return HQQ_ERR_ALIGN;
    if (pl.bytes) {
        if (!workspace || workspace_bytes < pl.bytes) return HQQ_ERR_WORKSPACE;
        if (!aligned_to(workspace, 16)) return HQQ_ERR_ALIGN;
    }
    return HQQ_OK;
}

void fill_parts(Attn *a, const AttnPlan &pl, int head_dim, void *workspace) {
    a->row_blocks = pl.row_blocks;
    a->ctas = pl.ctas;
    a->prefix_chunk = pl.prefix_chunk;
    a->prefix_splits = pl.prefix_splits;
    float *w = (float *)workspace;
    if (pl.ctas) {
        a->cuts = (Cut *)w;
        w += pl.ctas * sizeof(Cut) / sizeof(float);
    }
    if (pl.slot_floats) {
        a->slot_o = w;
        w += pl.slot_floats * head_dim;
    }
    if (pl.part_floats) {
        a->part_o = w;
        w += pl.part_floats * head_dim;
    }
    a->slot_lse = w;
    a->part_lse = w + pl.slot_floats;
}

}  // namespace

extern "C" size_t hqq_kv_attention_workspace_bytes(const hqq_kv_cache_t *cache, int64_t batch, int64_t nq,
                                                   int64_t heads, int64_t max_len, int64_t window,
                                                   int64_t prefix_len) {
    AttnPlan pl;
    return make_attn_plan(cache, batch, nq, heads, max_len, window, prefix_len, &pl) == HQQ_OK ? pl.bytes : 0;
}

extern "C" int hqq_kv_attention(const hqq_kv_cache_t *cache, const void *q, int dtype, int64_t batch, int64_t nq,
                                int64_t heads, int64_t q_batch_stride, int64_t q_token_stride, int64_t q_head_stride,
                                const int32_t *pages, int64_t pages_stride, int64_t max_pages, const int32_t *lens, int64_t max_len,
                                int64_t window, float scale, void *out, float *lse, void *workspace,
                                size_t workspace_bytes, void *stream) {
    AttnPlan pl;
    int rc = make_attn_plan(cache, batch, nq, heads, max_len, window, 0, &pl);
    if (rc == HQQ_OK)
        rc = check_attention(cache, q, dtype, batch, nq, heads, pages, max_pages, lens, max_len, scale, out, lse,
                             workspace, workspace_bytes, pl);
    if (rc != HQQ_OK) return rc;
    Attn a = {};
    check_cache(cache, &a.c);
    a.q = (const uint16_t *)q;
    a.q_batch = q_batch_stride;
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.q_wide = aligned_to(q, 8) && (q_batch_stride | q_token_stride | q_head_stride) % 4 == 0;
    a.batch = (int)batch;
    a.nq = (int)nq;
    a.heads = (int)heads;
    a.share = (int)heads / a.c.heads;
    a.pages = pages;
    a.pages_stride = pages_stride;
    a.lens = lens;
    a.max_len = max_len;
    a.window = pl.window;
    a.scale_log2 = scale * kLog2e;
    a.out = (uint16_t *)out;
    a.lse = lse;
    a.bf = dtype == HQQ_BF16;
    fill_parts(&a, pl, cache->head_dim, workspace);
    return run_attention(cache, a, pl, (cudaStream_t)stream);
}

extern "C" int hqq_kv_prefix_attention(const hqq_kv_cache_t *cache, const void *q, int dtype, int64_t batch, int64_t nq,
                                       int64_t heads, int64_t q_batch_stride, int64_t q_token_stride,
                                       int64_t q_head_stride, const int32_t *prefix_pages, int64_t prefix_len,
                                       const int32_t *pages, int64_t pages_stride, int64_t max_pages, const int32_t *lens, int64_t max_len,
                                       float scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
                                       void *stream) {
    AttnPlan pl;
    int rc = make_attn_plan(cache, batch, nq, heads, max_len, 0, prefix_len, &pl);
    if (rc == HQQ_OK)
        rc = check_attention(cache, q, dtype, batch, nq, heads, pages, max_pages, lens, max_len, scale, out, lse,
                             workspace, workspace_bytes, pl);
    if (rc != HQQ_OK) return rc;
    if (prefix_len > 0 && !prefix_pages) return HQQ_ERR_ARG;
    if (!aligned_to(prefix_pages, 4)) return HQQ_ERR_ALIGN;
    Attn a = {};
    check_cache(cache, &a.c);
    a.q = (const uint16_t *)q;
    a.q_batch = q_batch_stride;
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.q_wide = aligned_to(q, 8) && (q_batch_stride | q_token_stride | q_head_stride) % 4 == 0;
    a.batch = (int)batch;
    a.nq = (int)nq;
    a.heads = (int)heads;
    a.share = (int)heads / a.c.heads;
    a.pages = pages;
    a.pages_stride = pages_stride;
    a.lens = lens;
    a.max_len = max_len;
    a.prefix_pages = prefix_pages;
    a.prefix_len = prefix_len;
    a.scale_log2 = scale * kLog2e;
    a.out = (uint16_t *)out;
    a.lse = lse;
    a.bf = dtype == HQQ_BF16;
    fill_parts(&a, pl, cache->head_dim, workspace);
    return run_attention(cache, a, pl, (cudaStream_t)stream);
}
