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
// once for both sums.
//
// A code needs no conversion either: a field of up to 8 low bits in a 16-bit half is the fp16
// subnormal code * 2^-24, and one that sits s bits higher code * 2^(s - 24), which the tensor
// cores take as any other number.  So one AND of a word of codes gives two operands; the factors
// 2^-s are put into q (keys: a code's place is fixed for each d) and into the result (values).
//
// Both products are taken transposed, with the tokens (then the value's elements) along the 16
// rows of mma.m16n8k16 and 8 query rows along its columns:
//   S^T = K Q^T:  lane 4r + j holds run j of token r's key (D / 4 codes, one wide load from
//                 memory: a warp's loads cover 16 whole rows) and of token r + 8's;
//   O^T = V^T W^T: lane 4r + j holds run r of the values of tokens 2j, 2j+1, 2j+8, 2j+9; pairs of
//                 tokens are put side by side with one byte permute; W^T is S^T's layout, turned
//                 by movmatrix.
// The operands thus go from memory to registers and into the tensor cores: no shared memory, no
// barriers in the loop.  Each warp takes every kWarps-th block of 16 tokens of its CTA's chunk and
// keeps a running maximum and sum in binary32; they meet in shared memory at the end, and the
// chunks of a long sequence in a second kernel, both in a fixed order.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "hqq_common.cuh"
#include "hqq_kv_attn.cuh"

namespace {

using namespace hqq_kv;

constexpr int kAttnWarps = 4, kAttnThreads = 32 * kAttnWarps;
constexpr int kBlock = 16;          // tokens of one step of a warp
constexpr float kNegInf = -INFINITY;
// The running maximum may lag behind by this many powers of two before the sums are rescaled:
// weights stay below 2^8 of what they are relative to.  w is kept within fp16 by 2^6 * 2^8 < 65504.
constexpr float kLag = 8.0f;
constexpr float kWeightUnit = 64.0f;

template <int N>
struct Words {
    uint32_t w[N];
};

// the NBYTES of a lane's run, as 32-bit words (a run of 2 bytes: in the low half)
template <int NBYTES>
__device__ __forceinline__ Words<(NBYTES + 3) / 4> load_run(const uint8_t *p) {
    Words<(NBYTES + 3) / 4> r;
    if constexpr (NBYTES == 2) {
        r.w[0] = __ldg((const uint16_t *)p);
    } else if constexpr (NBYTES == 4) {
        r.w[0] = __ldg((const uint32_t *)p);
    } else if constexpr (NBYTES == 8) {
        const uint2 v = __ldg((const uint2 *)p);
        r.w[0] = v.x;
        r.w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < NBYTES / 16; ++i) {
            const uint4 v = __ldg((const uint4 *)p + i);
            r.w[4 * i] = v.x;
            r.w[4 * i + 1] = v.y;
            r.w[4 * i + 2] = v.z;
            r.w[4 * i + 3] = v.w;
        }
    }
    return r;
}

// How the D / 4 codes of a lane's run of a key become D / 8 operand registers of two codes each:
// register x holds codes lo(x) and hi(x) of the run, scaled by 2^(up(x) - 24).
template <int D, int NB, int NG>
struct KeyRegs {
    // a word whose halves belong to different groups is spread out first (2-bit codes, g = 32)
    static constexpr bool kSpread = D / NG / kKeyPieces < 32 / NB;
    static constexpr int kSpan = kSpread ? 8 / NB : 16 / NB;  // registers of one 16- or 32-bit unit
    static constexpr int kU = 8 / NB;
    __host__ __device__ static constexpr int lo(int x) {
        return kSpread ? x / kSpan * 2 * kSpan + x % kSpan : x / kSpan * 2 * kSpan + x % kSpan;
    }
    __host__ __device__ static constexpr int hi(int x) { return lo(x) + kSpan; }
    __host__ __device__ static constexpr int up(int x) { return NB * (x % kU); }
    template <int N>
    __device__ static __forceinline__ uint32_t reg(const Words<N> &run, int x) {
        constexpr uint32_t mask = ((1u << NB) - 1u) * 0x00010001u;
        if constexpr (kSpread) {
            const int unit = x / kSpan;
            const uint32_t v = __byte_perm(run.w[unit / 2], 0, unit & 1 ? 0x4342 : 0x4140);
            return v & (mask << up(x));
        } else {
            const int y = x % kSpan;
            return (run.w[x / kSpan] >> (y / kU * 8)) & (mask << up(x));
        }
    }
};

// Code x of a lane's run of the values (D / 8 codes) of two tokens, side by side, scaled by
// 2^(up(x) - 24).
template <int NB>
struct ValueRegs {
    static constexpr int kU = 8 / NB, kSpan = 16 / NB;
    __host__ __device__ static constexpr int up(int x) { return NB * (x % kU); }
    template <int N>
    __device__ static __forceinline__ uint32_t reg(const Words<N> &a, const Words<N> &b, int x) {
        constexpr uint32_t mask = ((1u << NB) - 1u) * 0x00010001u;
        const int unit = x / kSpan, y = x % kSpan;
        const uint32_t v = __byte_perm(a.w[unit / 2], b.w[unit / 2], unit & 1 ? 0x7632 : 0x5410);
        return (v >> (y / kU * 8)) & (mask << up(x));
    }
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the transpose of an 8 x 8 matrix of 16-bit values that the warp holds a row to four lanes
__device__ __forceinline__ uint32_t turn(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Rows of one key head are numbered l = (b - b0) * nq * share + i * share + (h - head * share).

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

template <int D, int NB, int NG, int RB>
struct Smem {
    float o[kAttnWarps][8 * RB][D];
    float m[kAttnWarps][8 * RB], l[kAttnWarps][8 * RB];
};

template <int D, int NB, int NG, int RB, bool PREFIX>
__global__ void __launch_bounds__(kAttnThreads) hqq_kv_attn_kernel(const Attn a) {
    constexpr int g = D / NG, KR = D / 8, VR = D / 8, RU = 8 * RB;
    constexpr int kKeyBytes = D * NB / 32, kValueBytes = D * NB / 64, kRowBytes = D * NB / 8;
    using KRegs = KeyRegs<D, NB, NG>;
    using VRegs = ValueRegs<NB>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    auto &sm = *reinterpret_cast<Smem<D, NB, NG, RB> *>(smem_raw);

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, j = lane & 3;
    const int split = blockIdx.x, b0 = PREFIX ? 0 : (int)blockIdx.z / a.c.heads, head = (int)blockIdx.z % a.c.heads;
    const int unit_rows = a.nq * a.share;                       // rows of one sequence and key head
    const int total_rows = PREFIX ? a.batch * unit_rows : unit_rows;
    const int row0 = (int)blockIdx.y * RU;
    const int part = PREFIX ? split : a.prefix_splits + split;  // where the partial result goes
    const int64_t all_rows = (int64_t)a.batch * a.nq * a.heads;

    // output row of local row l
    auto out_row = [&](int l) -> int64_t {
        const int b = b0 + l / unit_rows, i = l % unit_rows / a.share, h = l % a.share;
        return ((int64_t)b * a.nq + i) * a.heads + head * a.share + h;
    };

    // ---- the tokens of this chunk that some row of the block may see
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
    const int64_t from = (first & ~(int64_t)(kBlock - 1)) + (int64_t)split * a.chunk;
    const int64_t to = min(from + a.chunk, last);
    if (from >= to) {  // nothing here: the chunk's weight is zero
        if (a.part_lse) {
            for (int l = row0 + (int)threadIdx.x; l <= last_row; l += kAttnThreads)
                a.part_lse[part * all_rows + out_row(l)] = kNegInf;
        } else {
            for (int l = row0; l <= last_row; ++l) {
                const int64_t o = out_row(l);
                for (int d = threadIdx.x; d < D; d += kAttnThreads) a.out[o * D + d] = 0;
                if (a.lse && threadIdx.x == 0) a.lse[o] = kNegInf;
            }
        }
        return;
    }

    // ---- the rows of this lane: as operand column r, and as result columns 2j and 2j + 1
    uint32_t qb[RB][KR];      // q, paired as the keys' registers are
    float qs[RB][2][NG];      // sum of q over each group, for result columns
    float unit[RB][2];        // what a result is to be multiplied by: powers of two out
    int hi_[RB][2], lo_[RB][2];  // visible tokens, relative to `from`
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int l = row0 + 8 * rb + r;
        const bool live = l < total_rows;
        const int lc = live ? l : row0;
        const int b = b0 + lc / unit_rows, i = lc % unit_rows / a.share, h = head * a.share + lc % a.share;
        const uint16_t *q = a.q + b * a.q_batch + i * a.q_token + h * a.q_head;
        // each row is scaled by a power of two that takes its largest magnitude to [2^14, 2^15):
        // exact, but for values 2^-22 below the largest, and it makes bf16 fit fp16
        float big = 0.0f;
#pragma unroll
        for (int x = 0; x < KR; ++x) {
            const int e[2] = {KRegs::lo(x), KRegs::hi(x)};
            float v[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int d = e[y] / (g / 4) * g + j * (g / 4) + e[y] % (g / 4);
                const uint16_t raw = live ? __ldg(q + d) : (uint16_t)0;
                v[y] = a.bf ? to_f32<true>(raw) : to_f32<false>(raw);
                big = fmaxf(big, fabsf(v[y]));
            }
            qb[rb][x] = a.bf ? (__float_as_uint(v[0]) >> 16) | (__float_as_uint(v[1]) & 0xffff0000u)
                             : (uint32_t)from_f32<false>(v[0]) | (uint32_t)from_f32<false>(v[1]) << 16;
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // 2^(14 - floor(log2 big)); both it and its inverse stay normal
        const int ex = big > 0.0f ? min(max((int)(__float_as_uint(big) >> 23) - 127, -100), 100) : 0;
        const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
        float sum[NG];
#pragma unroll
        for (int x = 0; x < NG; ++x) sum[x] = 0.0f;
#pragma unroll
        for (int x = 0; x < KR; ++x) {
            const uint32_t w = qb[rb][x];
            float v0 = a.bf ? __uint_as_float(w << 16) : to_f32<false>((uint16_t)w);
            float v1 = a.bf ? __uint_as_float(w & 0xffff0000u) : to_f32<false>((uint16_t)(w >> 16));
            v0 *= up;
            v1 *= up;
            sum[x * NG / KR] += v0 + v1;
            const float down = 1.0f / (float)(1 << KRegs::up(x));
            const __half2 p = __floats2half2_rn(v0 * down, v1 * down);
            qb[rb][x] = *reinterpret_cast<const uint32_t *>(&p);
        }
#pragma unroll
        for (int x = 0; x < NG; ++x) {
            sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
            sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
            sum[x] *= 0x1p-24f;
        }
        const float un = 0x1p24f / up * a.scale_log2;
        int64_t lo, hi;
        visible<PREFIX>(a, own_len(a, b), i, lo, hi);
        const int64_t cap = to - from;
        const int rel_hi = live ? (int)min(max(hi - from, (int64_t)0), cap) : 0;
        const int rel_lo = (int)min(max(lo - from, (int64_t)0), cap);
#pragma unroll
        for (int y = 0; y < 2; ++y) {  // lane 4 (2j + y) holds row 2j + y
            const int src = 4 * (2 * j + y);
#pragma unroll
            for (int x = 0; x < NG; ++x) qs[rb][y][x] = __shfl_sync(0xffffffffu, sum[x], src);
            unit[rb][y] = __shfl_sync(0xffffffffu, un, src);
            hi_[rb][y] = __shfl_sync(0xffffffffu, rel_hi, src);
            lo_[rb][y] = __shfl_sync(0xffffffffu, rel_lo, src);
        }
    }

    float o[RB][VR / 2][4];   // O^T: rows are elements 2mb, 2mb + 1 of run r, columns rows 2j, 2j + 1
    float oz[RB][2][NG];      // sum of w vz
    float m[RB][2], l[RB][2];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
#pragma unroll
        for (int x = 0; x < VR / 2; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) o[rb][x][y] = 0.0f;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            m[rb][y] = kNegInf;
            l[rb][y] = 0.0f;
#pragma unroll
            for (int x = 0; x < NG; ++x) oz[rb][y][x] = 0.0f;
        }
    }
    float vref = 0x1p-24f;    // a power of two, at least every value scale so far

    const int span = (int)(to - from);
    const int blocks = (span + kBlock - 1) / kBlock;
    const int32_t *table = PREFIX ? a.prefix_pages : a.pages + b0 * a.pages_stride;
    int page_of_lane = 0;     // the page of this warp's block number it + lane - it % 32
    for (int it = 0, blk = warp; blk < blocks; ++it, blk += kAttnWarps) {
        if ((it & 31) == 0) {
            const int64_t t = from + (int64_t)(blk + lane * kAttnWarps) * kBlock;
            page_of_lane = t < to ? __ldg(table + (t >> a.c.page_shift)) : -1;
        }
        const int page = __shfl_sync(0xffffffffu, page_of_lane, it & 31);
        if (page < 0 || page >= a.c.pages) continue;  // a page that is not there is not seen
        const int t0 = blk * kBlock;                   // relative to `from`
        const int64_t row = row_of(a.c, page, head, (int)((from + t0) & ((1 << a.c.page_shift) - 1)));

        // ---- loads.  Rows of the page behind the last token hold anything: their codes are
        // finite numbers, and their metadata are replaced by zeros
        Words<(kKeyBytes + 3) / 4> k0, k1;
        Words<(kValueBytes + 3) / 4> v0, v1, v2, v3;
        k0 = load_run<kKeyBytes>(a.c.codes[0] + (row + r) * kRowBytes + j * kKeyBytes);
        k1 = load_run<kKeyBytes>(a.c.codes[0] + (row + r + 8) * kRowBytes + j * kKeyBytes);
        v0 = load_run<kValueBytes>(a.c.codes[1] + (row + 2 * j) * kRowBytes + r * kValueBytes);
        v1 = load_run<kValueBytes>(a.c.codes[1] + (row + 2 * j + 1) * kRowBytes + r * kValueBytes);
        v2 = load_run<kValueBytes>(a.c.codes[1] + (row + 2 * j + 8) * kRowBytes + r * kValueBytes);
        v3 = load_run<kValueBytes>(a.c.codes[1] + (row + 2 * j + 9) * kRowBytes + r * kValueBytes);
        float2 km[2][NG], vm[2][NG];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int64_t t = from + t0 + r + 8 * y;
            const bool there = t >= first && t < to;
#pragma unroll
            for (int x = 0; x < NG; ++x) {
                km[y][x] = vm[y][x] = make_float2(0.0f, 0.0f);
                if (there) {
                    km[y][x] = __half22float2(__ldg(a.c.meta[0] + (row + r + 8 * y) * NG + x));
                    vm[y][x] = __half22float2(__ldg(a.c.meta[1] + (row + r + 8 * y) * NG + x));
                }
            }
        }

        // ---- S^T and its scores, in powers of two
        float s[RB][4];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
#pragma unroll
            for (int y = 0; y < 4; ++y) s[rb][y] = 0.0f;
#pragma unroll
            for (int x = 0; x < NG; ++x) {
                float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int st = x * (g / 16); st < (x + 1) * (g / 16); ++st)
                    mma_16816(c, KRegs::reg(k0, 2 * st), KRegs::reg(k1, 2 * st), KRegs::reg(k0, 2 * st + 1),
                              KRegs::reg(k1, 2 * st + 1), qb[rb][2 * st], qb[rb][2 * st + 1]);
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    s[rb][y] = __fmaf_rn(km[y >> 1][x].x, __fmaf_rn(-km[y >> 1][x].y, qs[rb][y & 1][x], c[y]), s[rb][y]);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int t = t0 + r + 8 * (y >> 1);
                const bool seen = t < hi_[rb][y & 1] && t >= lo_[rb][y & 1];
                s[rb][y] = seen ? s[rb][y] * unit[rb][y & 1] : kNegInf;
            }
        }
        // ---- a new maximum, or a larger value scale than any before: rescale
        float vs = 0.0f;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int x = 0; x < NG; ++x) vs = fmaxf(vs, vm[y][x].x);
        bool more = vs > vref;
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int y = 0; y < 2; ++y) more |= fmaxf(s[rb][y], s[rb][y + 2]) > m[rb][y] + kLag;
        if (__any_sync(0xffffffffu, more)) {
            float big = vs;
#pragma unroll
            for (int x = 16; x > 0; x /= 2) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, x));
            // the power of two at or above it
            const float up = fmaxf(vref, __uint_as_float((__float_as_uint(big) + 0x007fffffu) & 0x7f800000u));
            const float fv = vref / up;
            vref = up;
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                float f[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float top = fmaxf(s[rb][y], s[rb][y + 2]);
#pragma unroll
                    for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    top = fmaxf(top, m[rb][y]);
                    f[y] = m[rb][y] == kNegInf ? 1.0f : exp2_fast(m[rb][y] - top);  // nothing to rescale yet
                    m[rb][y] = top;
                    l[rb][y] *= f[y];
                    f[y] *= fv;
#pragma unroll
                    for (int x = 0; x < NG; ++x) oz[rb][y][x] *= f[y];
                }
#pragma unroll
                for (int x = 0; x < VR / 2; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) o[rb][x][y] *= f[y & 1];
            }
        }
        // ---- weights
        float p[RB][4];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                p[rb][y] = m[rb][y & 1] == kNegInf ? 0.0f : exp2_fast(s[rb][y] - m[rb][y & 1]);
                l[rb][y & 1] += p[rb][y];
            }
        const float vin = kWeightUnit / vref;
#pragma unroll
        for (int x = 0; x < NG; ++x) {
            const float v_a = vm[0][x].x * vin, v_b = vm[1][x].x * vin;
            uint32_t w0[RB], w1[RB];
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                const __half2 h0 = __floats2half2_rn(p[rb][0] * v_a, p[rb][1] * v_a);
                const __half2 h1 = __floats2half2_rn(p[rb][2] * v_b, p[rb][3] * v_b);
                const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
                oz[rb][0][x] = __fmaf_rn(f1.x, vm[1][x].y, __fmaf_rn(f0.x, vm[0][x].y, oz[rb][0][x]));
                oz[rb][1][x] = __fmaf_rn(f1.y, vm[1][x].y, __fmaf_rn(f0.y, vm[0][x].y, oz[rb][1][x]));
                w0[rb] = turn(*reinterpret_cast<const uint32_t *>(&h0));
                w1[rb] = turn(*reinterpret_cast<const uint32_t *>(&h1));
            }
            // ---- O^T of this group's elements
#pragma unroll
            for (int mb = x * (g / 16); mb < (x + 1) * (g / 16); ++mb) {
                const uint32_t a0 = VRegs::reg(v0, v1, 2 * mb), a1 = VRegs::reg(v0, v1, 2 * mb + 1);
                const uint32_t a2 = VRegs::reg(v2, v3, 2 * mb), a3 = VRegs::reg(v2, v3, 2 * mb + 1);
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) mma_16816(o[rb][mb], a0, a1, a2, a3, w0[rb], w1[rb]);
            }
        }
    }

    // ---- the warps' results meet in shared memory, in units of the values
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
#pragma unroll
            for (int x = 4; x < 32; x *= 2) {
                l[rb][y] += __shfl_xor_sync(0xffffffffu, l[rb][y], x);
#pragma unroll
                for (int z = 0; z < NG; ++z) oz[rb][y][z] += __shfl_xor_sync(0xffffffffu, oz[rb][y][z], x);
            }
            if (r == 0) {
                sm.m[warp][8 * rb + 2 * j + y] = m[rb][y];
                sm.l[warp][8 * rb + 2 * j + y] = l[rb][y];
            }
        }
        const float vu = vref / kWeightUnit;
#pragma unroll
        for (int x = 0; x < VR; ++x) {
            constexpr int s8 = g / 8;
            const int d = x / s8 * g + r * s8 + x % s8;
            const float out_unit = 0x1p24f / (float)(1 << VRegs::up(x));
#pragma unroll
            for (int y = 0; y < 2; ++y)
                sm.o[warp][8 * rb + 2 * j + y][d] =
                    __fmaf_rn(o[rb][x / 2][2 * (x & 1) + y], out_unit, -oz[rb][y][x / s8]) * vu;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < RU * D; e += kAttnThreads) {
        const int rr = e / D, d = e % D, lrow = row0 + rr;
        if (lrow >= total_rows) break;
        float top = kNegInf;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, sm.m[w][rr]);
        float sum = 0.0f, acc = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
            const float f = sm.m[w][rr] == kNegInf ? 0.0f : exp2_fast(sm.m[w][rr] - top);
            sum = __fmaf_rn(sm.l[w][rr], f, sum);
            if (f > 0.0f) acc = __fmaf_rn(sm.o[w][rr][d], f, acc);
        }
        const float y = sum > 0.0f ? acc / sum : 0.0f;
        const int64_t orow = out_row(lrow);
        if (a.part_o) {
            a.part_o[(part * all_rows + orow) * D + d] = y;
            if (d == 0) a.part_lse[part * all_rows + orow] = sum > 0.0f ? top + log2f(sum) : kNegInf;
        } else {
            a.out[orow * D + d] = a.bf ? from_f32<true>(y) : from_f32<false>(y);
            if (d == 0 && a.lse) a.lse[orow] = sum > 0.0f ? (top + log2f(sum)) * 0.6931471805599453f : kNegInf;
        }
    }
}

// The chunks of one row, joined: a warp to a row, in the order of the chunks.
template <int D>
__global__ void __launch_bounds__(128) hqq_kv_join_kernel(const Attn a) {
    wait_prerequisite();
    const int64_t rows = (int64_t)a.batch * a.nq * a.heads;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, parts = a.prefix_splits + a.splits;
    if (row >= rows) return;
    float top = kNegInf;
    for (int p = lane; p < parts; p += 32) top = fmaxf(top, a.part_lse[p * rows + row]);
#pragma unroll
    for (int x = 16; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    float acc[D / 32], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = 0.0f;
    if (top > kNegInf)
        for (int p = 0; p < parts; ++p) {
            const float e = a.part_lse[p * rows + row];
            if (e == kNegInf) continue;  // what lies there for this row was never written
            const float f = exp2_fast(e - top);
            sum += f;
            const float *o = a.part_o + (p * rows + row) * D;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) acc[i] = __fmaf_rn(o[lane + 32 * i], f, acc[i]);
        }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const float y = sum > 0.0f ? acc[i] / sum : 0.0f;
        a.out[row * D + lane + 32 * i] = a.bf ? from_f32<true>(y) : from_f32<false>(y);
    }
    if (a.lse && lane == 0) a.lse[row] = sum > 0.0f ? (top + log2f(sum)) * 0.6931471805599453f : kNegInf;
}

constexpr int64_t kSms = 148;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// rows that a CTA takes: 8, or 16 where a key head has more (and the accumulators fit)
int rows_per_cta(int head_dim, int64_t rows) { return rows > 8 && head_dim <= 128 ? 16 : 8; }

// Splits `len` tokens among about 148 * 4 CTAs for `others` independent ones: chunks of whole
// steps of a CTA, not so short that joining costs more than it gives.
void split_tokens(int64_t len, int64_t others, int64_t *chunk, int *splits) {
    const int64_t step = kBlock * kAttnWarps;
    const int64_t want = std::max<int64_t>(1, 4 * kSms / std::max<int64_t>(1, others));
    int64_t c = ceil_div(ceil_div(std::max<int64_t>(len, 1), want), step) * step;
    c = std::max<int64_t>(c, 2 * step);
    *chunk = c;
    *splits = (int)std::max<int64_t>(1, ceil_div(len, c));
}

int make_attn_plan(const hqq_kv_cache_t *cache, int64_t batch, int64_t nq, int64_t heads, int64_t max_len,
                   int64_t window, int64_t prefix_len, AttnPlan *pl) {
    Cache c;
    const int rc = check_cache(cache, &c);
    if (rc != HQQ_OK) return rc;
    if (batch < 0 || nq < 0 || heads <= 0 || max_len < 0 || window < 0 || prefix_len < 0 || heads % c.heads)
        return HQQ_ERR_ARG;
    // rows are counted in 31 bits, blocks of a grid's second and third dimension in 16
    if (max_len > INT32_MAX || prefix_len > INT32_MAX || batch > 65535 / c.heads || nq > 65535 ||
        batch * nq > INT32_MAX / heads)
        return HQQ_ERR_UNSUPPORTED;
    const int64_t rows = nq * (heads / c.heads);
    const int ru = rows_per_cta(cache->head_dim, rows);
    pl->row_blocks = (int)ceil_div(rows, ru);
    if (pl->row_blocks > 65535) return HQQ_ERR_UNSUPPORTED;
    int64_t span = max_len;
    // a block of rows sees at most the window of each of its queries, and its first block's head
    if (window > 0) span = std::min<int64_t>(span, window + nq + kBlock);
    split_tokens(span, batch * c.heads * pl->row_blocks, &pl->chunk, &pl->splits);
    pl->prefix_splits = 0;
    pl->prefix_chunk = 0;
    pl->prefix_row_blocks = 0;
    if (prefix_len > 0) {
        const int pru = rows_per_cta(cache->head_dim, rows * batch);
        pl->prefix_row_blocks = (int)ceil_div(rows * batch, pru);
        if (pl->prefix_row_blocks > 65535) return HQQ_ERR_UNSUPPORTED;
        split_tokens(prefix_len, (int64_t)c.heads * pl->prefix_row_blocks, &pl->prefix_chunk, &pl->prefix_splits);
    }
    const int parts = pl->splits + pl->prefix_splits;
    pl->bytes = 0;
    if (parts > 1) pl->bytes = (size_t)parts * (size_t)(batch * nq * heads) * (cache->head_dim + 1) * sizeof(float) + 16;
    return HQQ_OK;
}

template <int D, int NB, int NG, int RB, bool PREFIX>
cudaError_t launch_attn(const Attn &a, int row_blocks, cudaStream_t st) {
    auto k = hqq_kv_attn_kernel<D, NB, NG, RB, PREFIX>;
    constexpr int smem = (int)sizeof(Smem<D, NB, NG, RB>);
    if constexpr (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid(PREFIX ? a.prefix_splits : a.splits, row_blocks, PREFIX ? a.c.heads : a.batch * a.c.heads);
    k<<<grid, kAttnThreads, smem, st>>>(a);
    return cudaGetLastError();
}

int run_attention(const hqq_kv_cache_t *cache, Attn a, const AttnPlan &pl, cudaStream_t st) {
    if ((int64_t)a.batch * a.nq == 0) return HQQ_OK;
    const int rows = a.nq * a.share;
    const int rc = with_layout(*cache, [&](auto dim, auto bits, auto groups) {
        constexpr int D = dim, NB = bits, NG = groups;
        constexpr int kWide = D <= 128 ? 2 : 1;
        cudaError_t e = cudaSuccess;
        if (pl.prefix_splits > 0) {
            Attn p = a;
            p.chunk = pl.prefix_chunk;
            if (rows_per_cta(D, (int64_t)rows * a.batch) == 16) e = launch_attn<D, NB, NG, kWide, true>(p, pl.prefix_row_blocks, st);
            else e = launch_attn<D, NB, NG, 1, true>(p, pl.prefix_row_blocks, st);
            if (e != cudaSuccess) return HQQ_ERR_CUDA;
        }
        if (rows_per_cta(D, rows) == 16) e = launch_attn<D, NB, NG, kWide, false>(a, pl.row_blocks, st);
        else e = launch_attn<D, NB, NG, 1, false>(a, pl.row_blocks, st);
        if (e != cudaSuccess) return HQQ_ERR_CUDA;
        if (a.part_o) {
            const int64_t all = (int64_t)a.batch * a.nq * a.heads;
            e = launch_pdl(hqq_kv_join_kernel<D>, (unsigned)ceil_div(all, 4), 128u, 0, st, a);
        }
        return e == cudaSuccess ? HQQ_OK : HQQ_ERR_CUDA;
    });
    return rc;
}

int check_attention(const hqq_kv_cache_t *cache, const void *q, int dtype, int64_t batch, int64_t nq, int64_t heads,
                    const int32_t *pages, int64_t max_pages, const int32_t *lens, int64_t max_len, float scale,
                    void *out, float *lse, void *workspace, size_t workspace_bytes, const AttnPlan &pl) {
    if (dtype != HQQ_FP16 && dtype != HQQ_BF16) return HQQ_ERR_ARG;
    if (max_pages < 0 || max_len > max_pages * (int64_t)cache->page_size || !(scale > 0.0f) || !std::isfinite(scale))
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
    a->chunk = pl.chunk;
    a->splits = pl.splits;
    a->prefix_splits = pl.prefix_splits;
    if (!pl.bytes) return;
    const size_t rows = (size_t)(pl.splits + pl.prefix_splits) * a->batch * a->nq * a->heads;
    a->part_o = (float *)workspace;
    a->part_lse = a->part_o + rows * head_dim;
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
    a.batch = (int)batch;
    a.nq = (int)nq;
    a.heads = (int)heads;
    a.share = (int)heads / a.c.heads;
    a.pages = pages;
    a.pages_stride = pages_stride;
    a.lens = lens;
    a.max_len = max_len;
    a.window = window;
    a.scale_log2 = scale * 1.4426950408889634f;
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
    a.scale_log2 = scale * 1.4426950408889634f;
    a.out = (uint16_t *)out;
    a.lse = lse;
    a.bf = dtype == HQQ_BF16;
    fill_parts(&a, pl, cache->head_dim, workspace);
    return run_attention(cache, a, pl, (cudaStream_t)stream);
}
