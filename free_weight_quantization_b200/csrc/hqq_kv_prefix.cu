// hqq_kv_prefix.cu -- the shared prefix of hqq_kv_prefix_attention on the tcgen05 tensor cores, for
// batches that put many query rows on one key head.
//
// A CTA has 128 query rows of one key head (of any sequences) and a chunk of the prefix, which it
// takes in tiles of 64 tokens:
//     S_g = Q_g (A_g - kz_g)^T   for each group g of the keys' elements; A: the codes as they are
//     s   = sum_g ks_g S_g,   p = exp2(s - m),   O += p V
// As in hqq_kv_attn.cu the keys' codes are exact (fp16 subnormals, their power of two in Q) and
// their scales stay in binary32 outside the product; the zero points are one more step of it, 16
// wide: the row's -sum Q_g in two fp16 parts against (kz, kz).  The values are computed in binary32,
// (c - vz) vs, relative to a power of two at the group's largest scale so far, and rounded to fp16
// once, as the weights p are.
// What a row needs of each token is thus NG floats; all of it (ks, kz, vs of each group) would be
// read by 128 rows 24 bytes a token, and shared memory gives 128 bytes a cycle: 1500 cycles for a
// tile whose products take 600.
//
// Sixteen warps, two CTAs on an SM:
//   * four producer warps turn the codes of a tile into operands in shared memory (128-byte
//     swizzle; keys K-major, values with the elements along the rows), two stages;
//   * one lane issues the tcgen05.mma: S_g (128 x 64, binary32, tensor memory), then O with the
//     weights as the A operand in tensor memory, where they take the place of S;
//   * eight softmax warps: two threads have a row, 32 tokens of a tile each; they read their
//     scores from tensor memory, keep a common running maximum and a sum each, and write the
//     weights.  O is rescaled in tensor memory only when the maximum has grown by more than 2^8, or
//     a larger value scale appears.  (Four warps with a thread to a row: 114 us a call where this took 104.)
// The two CTAs of an SM cover each other's turns: while one's scores are in its softmax warps the
// other's products run.
//
// What bounds it: the turn of a tile, scores - weights - products, which tensor memory leaves no room
// to overlap within a CTA (S of two groups and O fill its 256 columns).  64 sequences x 32 heads
// behind 32768 tokens, 8 key heads, 4 bits, g = 64: 91 us, half of the issue slots, 380 TFLOP/s; the
// products alone would take 21.
//
// Waits on mbarriers are bounded: one that runs out (none should) makes the CTA write NaN, which the
// join passes on; the other roles' waits run out in their turn, and the CTA ends once its products have.
#include <type_traits>

#include "hqq_kv_attn.cuh"
#include "hqq_umma.cuh"

namespace {

using namespace hqq_kv;

constexpr int kTcThreads = 512, kSoftmaxThreads = 256;
// registers of a thread: 64 at launch (two CTAs of 512), divided so that the sum is the same
constexpr int kTcLaunchRegs = 64, kSoftmaxRegs = 80, kProducerRegs = 64, kIssueRegs = 32;
static_assert(2 * kSoftmaxRegs + kProducerRegs + kIssueRegs <= 4 * kTcLaunchRegs, "setmaxnreg draws on the launch's registers");
static_assert(kSoftmaxRegs > kTcLaunchRegs && kProducerRegs == kTcLaunchRegs && kIssueRegs < kTcLaunchRegs,
              "an increase to fewer registers, or a decrease to more, is an illegal instruction");

template <int D, int NG>
struct TcShape {
    static constexpr int kBlocks = D / 64;  // of 64 elements: 128 bytes, a row of the swizzle
    static constexpr int kQ = kBlocks * kTcRows * 128, kTile = kBlocks * kTcTokens * 128;
    // the zero points' step: of its 16 columns 8 are held, two of them not zero, and 8 lie in one piece
    // of zeros for all
    static constexpr int kZqG = kTcRows * 16, kZkG = kTcTokens * 16, kZero = kZqG;
    static constexpr int kMeta = NG * kTcTokens * 4 + 16;  // ks; valid[2], the values' unit of each group
    static constexpr int kZq0 = kQ, kStage0 = kZq0 + NG * kZqG, kZk0 = kStage0 + 4 * kTile, kZero0 = kZk0 + 2 * NG * kZkG;
    static constexpr int kMeta0 = kZero0 + kZero;
    static constexpr int kTops0 = kMeta0 + 2 * kMeta;      // [2 stages][4 warps][NG]: largest value scales
    static constexpr int kBars = kTops0 + 32 * NG;
    static constexpr int kRow0 = kBars + 64;                   // [2][128] floats: what a row's two threads exchange
    static constexpr int kSmem = kRow0 + 8 * kTcRows + 1024;   // + alignment slack
    static constexpr int kOCol = NG * kTcTokens;               // O behind S in tensor memory
    static constexpr int kCols = kOCol + D <= 128 ? 128 : 256;
};

// Codes e = 0 .. 7 of a stored run of 8 lie at place(e) of 8 fp16 values in a row of an operand.
template <int NB>
__host__ __device__ constexpr int place(int e) {
    return NB == 8 ? e / 4 * 4 + e % 2 * 2 + e / 2 % 2 : 2 * (e % 4) + e / 4;
}

// by what power of two the keys' code e is scaled, beside 2^-24
template <int NB>
__host__ __device__ constexpr int place_up(int e) { return NB == 8 ? 0 : code_up<NB>(NB == 4 ? e % 4 % 2 : e % 4); }

// 8 codes as stored (NB bytes in w[0], w[1]) to 8 fp16: code * 2^(place_up - 24)
template <int NB>
__device__ __forceinline__ uint4 key_chunk8(const uint32_t *w) {
    if constexpr (NB == 8)
        return make_uint4(code_pair<8>(w[0], 0, 0), code_pair<8>(w[0], 1, 0), code_pair<8>(w[1], 0, 0), code_pair<8>(w[1], 1, 0));
    else if constexpr (NB == 4)
        return make_uint4(code_pair<4>(w[0], 0, 0), code_pair<4>(w[0], 0, 1), code_pair<4>(w[0], 1, 0), code_pair<4>(w[0], 1, 1));
    else {
        const uint32_t v = __byte_perm(w[0], 0, 0x4140);
        return make_uint4(code_pair<2>(v, 0, 0), code_pair<2>(v, 0, 1), code_pair<2>(v, 0, 2), code_pair<2>(v, 0, 3));
    }
}

// The same 8 codes in the same places as values: (code - zero) * scale, rounded once.  A code
// becomes a binary32 number by one byte permute: under the exponent of 128 (2^15 for 8-bit codes)
// its byte counts whole numbers, and the same number is added to the zero point beforehand, which
// moves it by at most 2^-17 (2^-9 of 255) of a step.
template <int NB>
__host__ __device__ constexpr float code_base() { return NB == 8 ? 32768.0f : 128.0f; }

template <int NB>
__device__ __forceinline__ float code_float(uint32_t bytes, int i) {
    if constexpr (NB == 8) return __uint_as_float(__byte_perm(bytes, 0x47000000u, 0x7404u + (uint32_t)(i << 4)));
    else return __uint_as_float(__byte_perm(bytes, 0x43000000u, 0x7044u + (uint32_t)(i << 8)));
}

template <int NB>
__device__ __forceinline__ uint4 value_chunk8(const uint32_t *w, float less, float scale) {
    uint32_t lo[4], hi[4], y[4];  // the words whose bytes are a pair's codes, and which bytes
    int il[4], ih[4];
    if constexpr (NB == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) lo[i] = hi[i] = w[i / 2], il[i] = i & 1, ih[i] = 2 + (i & 1);
    } else if constexpr (NB == 4) {
        const uint32_t ev = w[0] & 0x0F0F0F0Fu, od = (w[0] >> 4) & 0x0F0F0F0Fu;
#pragma unroll
        for (int i = 0; i < 4; ++i) lo[i] = hi[i] = i & 1 ? od : ev, il[i] = i / 2, ih[i] = 2 + i / 2;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) lo[i] = hi[i] = (w[0] >> (2 * i)) & 0x03030303u, il[i] = 0, ih[i] = 1;
    }
    const float2 l2 = make_float2(-less, -less), s2 = make_float2(scale, scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __fmul2_rn(__fadd2_rn(make_float2(code_float<NB>(lo[i], il[i]), code_float<NB>(hi[i], ih[i])), l2), s2);
        const __half2 h = __floats2half2_rn(v.x, v.y);
        y[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(y[0], y[1], y[2], y[3]);
}

__device__ __forceinline__ void sts16(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ float4 lds_f4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
    return v;
}

__device__ __forceinline__ void sts_f(uint32_t at, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory"); }
__device__ __forceinline__ void sts_u(uint32_t at, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory"); }

// 16 columns of this thread's lane of tensor memory (its warp's 32 lanes)
__device__ __forceinline__ void tmem_ld16(uint32_t at, float (&v)[16]) {
    uint32_t *u = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(at));
}

__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t *u) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(at), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]),
          "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// mbar_wait, in line (a call would hold registers that the register split does not have) and
// without naps, which cost a tile's turn some hundred cycles each; a test itself waits a while
__device__ __forceinline__ bool wait_for(uint32_t addr, uint32_t parity) {
    for (uint32_t i = 0; i < kMbarWaitLimit; ++i)
        if (mbar_try(addr, parity)) return true;
    return false;
}

// whether p holds for any of the 64 threads that meet at named barrier `id`
__device__ __forceinline__ bool any_of_pair(int id, bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\tbarrier.cta.red.or.pred q, %1, 64, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(id), "r"((uint32_t)p) : "memory");
    return r != 0;
}

__device__ __forceinline__ void meet_pair(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }

// one lane of a converged warp.  The products' descriptors live in uniform registers: behind this
// the compiler knows that a single lane issues them, behind `lane == 0` it does not, and moves
// each operand over on its own
__device__ __forceinline__ bool elected() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred P1;\n\telect.sync _|P1, 0xffffffff;\n\tselp.b32 %0, 1, 0, P1;\n\t}" : "=r"(p));
    return p != 0;
}

// D binary32, A and B fp16, M = 128; `along_n`: B's elements lie along N
__host__ __device__ constexpr uint32_t tc_idesc(int n, bool along_n) {
    return (1u << 4) | (along_n ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTcRows >> 4) << 24);
}

// A descriptor's low word has the address and the leading offset, the high word the rest; in 16-byte
// units the address carries nowhere, so that a step along an operand is one 32-bit addition.
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo, uint32_t layout) { return (sbo >> 4) | 1u << 14 | layout << 29; }

__device__ __forceinline__ uint32_t desc_lo(uint32_t at, uint32_t lbo) { return (at >> 4) | (lbo >> 4) << 16; }

// D (+)= A B, both in shared memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}"
        ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(add ? 1u : 0u) : "memory");
}

// the same with A in tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 y, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}"
        ::"r"(d), "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(add ? 1u : 0u) : "memory");
}

template <int D, int NB, int NG>
__global__ void __launch_bounds__(kTcThreads, 2) hqq_kv_prefix_tc_kernel(const Attn a) {
    using S = TcShape<D, NG>;
    constexpr int g = D / NG, CH = D / 8;  // 8-code chunks of a row
    extern __shared__ unsigned char smem_raw[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the sequences' own tokens need nothing of this
    __shared__ uint32_t tmem_slot;
    __shared__ volatile uint32_t failed;  // a wait ran out somewhere
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), role = warp >> 2;  // 0, 1 softmax, 2 producers, 3 issue
    const int split = blockIdx.x, row0 = (int)blockIdx.y * kTcRows, head = blockIdx.z;
    const uint32_t base = ((uint32_t)__cvta_generic_to_shared(smem_raw) + 1023u) & ~1023u;
    const uint32_t bars = base + S::kBars;
    const uint32_t kv_full = bars, kv_free = bars + 16, s_full = bars + 32, p_full = bars + 40, done = bars + 48;
    const int64_t from = (int64_t)split * a.prefix_chunk, to = min(from + a.prefix_chunk, a.prefix_len);
    const int tiles = (int)((to - from + kTcTokens - 1) / kTcTokens);
    const int unit_rows = a.nq * a.share, total_rows = a.batch * unit_rows;
    const int64_t rows = (int64_t)a.batch * a.nq * a.heads;

    // the zero points' step: all but two of its 16 columns stay zero
    for (int i = tid; i < NG * S::kZqG / 16; i += kTcThreads) sts16(base + S::kZq0 + 16 * i, make_uint4(0, 0, 0, 0));
    for (int i = tid; i < (2 * NG * S::kZkG + S::kZero) / 16; i += kTcThreads) sts16(base + S::kZk0 + 16 * i, make_uint4(0, 0, 0, 0));
    if (tid == 0) {
        failed = 0;
        for (int s = 0; s < 2; ++s) {
            mbar_init(kv_full + 8 * s, 128);  // every producer thread has stored
            mbar_init(kv_free + 8 * s, 1);    // the products that read the stage have completed
        }
        mbar_init(s_full, 1);    // scores are complete
        mbar_init(p_full, kSoftmaxThreads);  // every softmax thread has stored its weights
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"((uint32_t)__cvta_generic_to_shared(&tmem_slot)), "n"(S::kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::);
    }

    __syncthreads();  // the zeros are in place
    // ---- the rows, 8 elements to a thread: each row scaled by a power of two that takes its largest
    // magnitude to [2^14, 2^15), into shared memory in the order of the keys' operands
    {
        constexpr int T = D / 8;  // threads of a row: neighbours in a warp
        for (int at = tid; at < kTcRows * T; at += kTcThreads) {  // whole warps: 128 T is a multiple of 32
            const int rr = at / T, d = at % T * 8, l = row0 + rr;
            const bool there = l < total_rows;
            const int lc = there ? l : row0;
            const int b = lc / unit_rows, i = lc % unit_rows / a.share, h = head * a.share + lc % a.share;
            const uint16_t *q = a.q + b * a.q_batch + i * a.q_token + h * a.q_head + d;
            uint32_t raw[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (a.q_wide) {
                    *reinterpret_cast<uint2 *>(raw + 2 * e) = __ldg((const uint2 *)(q + 4 * e));
                } else {
                    raw[2 * e] = __ldg(q + 4 * e) | (uint32_t)__ldg(q + 4 * e + 1) << 16;
                    raw[2 * e + 1] = __ldg(q + 4 * e + 2) | (uint32_t)__ldg(q + 4 * e + 3) << 16;
                }
            }
            float v[8], sum = 0.0f;
            uint32_t big = 0;  // the bits of the largest magnitude
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t w = there ? raw[e / 2] : 0u;
                v[e] = a.bf ? __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16) : to_f32<false>((uint16_t)(e & 1 ? w >> 16 : w));
                big = max(big, __float_as_uint(fabsf(v[e])));
            }
#pragma unroll
            for (int x = 1; x < T; x *= 2) big = max(big, __shfl_xor_sync(0xffffffffu, big, x));
            const int ex = big > 0 ? min(max((int)(big >> 23) - 127, -100), 100) : 0;
            const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
            const float by = row_in_range(big, a.scale_log2) ? up : __uint_as_float(0x7fc00000u);  // out of range: a row of NaN
            __half y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] *= by;
                sum += v[e];
                y[place<NB>(e)] = __float2half_rn(v[e] * (1.0f / (float)(1 << place_up<NB>(e))));
            }
            const int o = d % g, c = d / g * (g / 8) + o / (g / 4) * (g / 32) + o % (g / 4) / 8;
            sts16(base + c / 8 * (kTcRows * 128) + rr * 128 + ((c % 8) ^ (rr & 7)) * 16, *reinterpret_cast<const uint4 *>(y));
#pragma unroll
            for (int x = 1; x < g / 8; x *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            if (d % g == 0) {
                // the zero points' step: the negative sum, times the 2^6 that they are divided by, in two parts
                const float z = -64.0f * 0x1p-24f * sum;
                const __half top = __float2half_rn(z), rest = __float2half_rn(z - __half2float(top));
                const __half2 two = __halves2half2(top, rest);
                sts_u(base + S::kZq0 + d / g * S::kZqG + rr * 16, *reinterpret_cast<const uint32_t *>(&two));
            }
            if (d == 0) sts_f(base + S::kMeta0 + rr * 4, row_unit(up, a.scale_log2));  // until the tiles come
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    // a softmax thread's row
    float unit = 0.0f;
    int64_t orow = 0, limit = 0;
    bool live = false;
    const int lrow = tid & (kTcRows - 1), hf = (tid >> 7) & 1;  // two threads to a row, 32 tokens of a tile each
    if (role < 2) {
        const int l = row0 + lrow;
        live = l < total_rows;
        const int lc = live ? l : row0;
        const int b = lc / unit_rows, i = lc % unit_rows / a.share, h = head * a.share + lc % a.share;
        orow = ((int64_t)b * a.nq + i) * a.heads + h;
        int64_t lo;
        visible<true>(a, own_len(a, b), i, lo, limit);
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(unit) : "r"(base + S::kMeta0 + lrow * 4));
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;

    bool ok = true;
    float m = kLowest, vref[NG];
#pragma unroll
    for (int x = 0; x < NG; ++x) vref[x] = 0x1p-24f;
    float2 l2 = make_float2(0.0f, 0.0f);
    if (role == 2) {
        // ---- producers: thread (t, h) has half h of token t's key and value
        constexpr int kVecs = D * NB / 256 + (D * NB % 256 != 0);   // 16-byte pieces of half a row (8 bytes: one)
        constexpr int kHalf = D * NB / 16;                          // bytes of half a row
        const int t = tid & 63, h = (tid >> 6) & 1;
        auto page_of = [&](int tile) -> int {
            const int64_t tok = from + (int64_t)tile * kTcTokens + t;
            return tok < to ? __ldg(a.prefix_pages + (tok >> a.c.page_shift)) : -1;
        };
        struct Held {
            uint32_t k[kVecs * 4], v[kVecs * 4], km[NG], vm[NG];
            bool in;
        };
        auto load = [&](int tile, int page, Held &x) {
            x.in = page >= 0 && page < a.c.pages;
            const int64_t tok = from + (int64_t)tile * kTcTokens + t;
            const int64_t row = x.in ? row_of(a.c, page, head, (int)tok & ((1 << a.c.page_shift) - 1)) : 0;
            const uint8_t *k = a.c.codes[0] + row * (2 * kHalf) + h * kHalf, *v = a.c.codes[1] + row * (2 * kHalf) + h * kHalf;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                uint4 kk = make_uint4(0, 0, 0, 0), vv = kk;
                if (x.in) {
                    if constexpr (kHalf >= 16) {
                        kk = __ldg((const uint4 *)k + i);
                        vv = __ldg((const uint4 *)v + i);
                    } else {
                        const uint2 k2 = __ldg((const uint2 *)k), v2 = __ldg((const uint2 *)v);
                        kk = make_uint4(k2.x, k2.y, 0, 0);
                        vv = make_uint4(v2.x, v2.y, 0, 0);
                    }
                }
                *reinterpret_cast<uint4 *>(x.k + 4 * i) = kk;
                *reinterpret_cast<uint4 *>(x.v + 4 * i) = vv;
            }
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                x.km[i] = x.in ? __ldg((const uint32_t *)(a.c.meta[0] + row * NG + i)) : 0u;
                x.vm[i] = x.in ? __ldg((const uint32_t *)(a.c.meta[1] + row * NG + i)) : 0u;
            }
        };
        // 2- and 4-bit codes are fetched a tile ahead; of 8-bit codes two tiles do not fit the registers
        constexpr bool kAhead = NB < 8;
        Held cur, next;
        load(0, page_of(0), cur);
        int page = page_of(1);
        float unit_v[NG];  // a power of two, at least the group's every value scale so far
#pragma unroll
        for (int x = 0; x < NG; ++x) unit_v[x] = 0x1p-24f;
        for (int i = 0; i < tiles; ++i) {
            const int st = i & 1;
            if constexpr (kAhead) {
                load(i + 1, page, next);
                page = page_of(i + 2);
            }
            float less[NG], scale[NG];
            // the tile's largest value scale of each group: two warps hold the 64 tokens, twice.  Two
            // buffers: a warp that is ahead writes tile i + 1's while another still reads tile i's, and
            // it writes tile i + 2's only after all have met in tile i + 1, their reads of tile i's done
            const uint32_t tops = base + S::kTops0 + st * (16 * NG);
#pragma unroll
            for (int x = 0; x < NG; ++x) {
                const float2 vm = __half22float2(*reinterpret_cast<const __half2 *>(&cur.vm[x]));
                less[x] = vm.y + code_base<NB>();
                scale[x] = vm.x;
                const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(vm.x));
                if (lane == 0) sts_u(tops + ((warp & 3) * NG + x) * 4, top);
            }
            asm volatile("barrier.cta.sync 5, 128;" ::: "memory");
#pragma unroll
            for (int x = 0; x < NG; ++x) {
                uint32_t t0, t1;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(t0) : "r"(tops + x * 4));
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(t1) : "r"(tops + (NG + x) * 4));
                unit_v[x] = fmaxf(unit_v[x], __uint_as_float((max(t0, t1) + 0x007fffffu) & 0x7f800000u));
                scale[x] *= 1.0f / unit_v[x];
            }
            if (i >= 2 && ok) {
                ok = wait_for(kv_free + 8 * st, (uint32_t)((i >> 1) - 1) & 1u);
                if (!ok) failed = 1;  // before this tile is handed over: who sees its products sees it
            }
            const uint32_t kt = base + S::kStage0 + st * 2 * S::kTile, vt = kt + S::kTile, mt = base + S::kMeta0 + st * S::kMeta;
#pragma unroll
            for (int x = 0; x < CH / 2; ++x) {
                // stored chunk number h * CH / 2 + x of the row; of a 2-bit word's two chunks one half
                uint32_t kw[2], vw[2];
                if constexpr (NB == 8) {
                    kw[0] = cur.k[2 * x], kw[1] = cur.k[2 * x + 1];
                    vw[0] = cur.v[2 * x], vw[1] = cur.v[2 * x + 1];
                } else if constexpr (NB == 4) {
                    kw[0] = cur.k[x], vw[0] = cur.v[x];
                } else {
                    kw[0] = cur.k[x / 2] >> (16 * (x & 1)), vw[0] = cur.v[x / 2] >> (16 * (x & 1));
                }
                // where its codes belong: keys in 4 runs, values in 8, each with a share of every group
                const int cx = h * (CH / 2) + x;
                const int kr = x % (D / 32), kg = kr / (g / 32), kc = kg * (g / 8) + cx / (D / 32) * (g / 32) + kr % (g / 32);
                const int vr = x % (D / 64), vg = vr / (g / 64), vc = vg * (g / 8) + cx / (D / 64) * (g / 64) + vr % (g / 64);
                sts16(kt + kc / 8 * (kTcTokens * 128) + t * 128 + ((kc % 8) ^ (t & 7)) * 16, key_chunk8<NB>(kw));
                sts16(vt + vc / 8 * (kTcTokens * 128) + t * 128 + ((vc % 8) ^ (t & 7)) * 16,
                      value_chunk8<NB>(vw, less[vg], scale[vg]));
            }
            if (h == 0) {
#pragma unroll
                for (int x = 0; x < NG; ++x) {
                    const float2 km = __half22float2(*reinterpret_cast<const __half2 *>(&cur.km[x]));
                    const __half2 z = __float2half2_rn(km.y * 0x1p-6f);
                    sts_f(mt + (x * kTcTokens + t) * 4, km.x);
                    sts_u(base + S::kZk0 + (st * NG + x) * S::kZkG + t * 16, *reinterpret_cast<const uint32_t *>(&z));
                }
                const uint32_t in = __ballot_sync(0xffffffffu, cur.in);
                if (lane == 0) sts_u(mt + NG * kTcTokens * 4 + (t >> 5) * 4, in);
            } else if (t == 0) {
#pragma unroll
                for (int x = 0; x < NG; ++x) sts_f(mt + NG * kTcTokens * 4 + 8 + x * 4, unit_v[x]);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(kv_full + 8 * st);
            if constexpr (kAhead) {
                cur = next;
            } else {
                load(i + 1, page, cur);
                page = page_of(i + 2);
            }
        }
    } else if (role == 3) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == 12 && elected()) {
            constexpr uint32_t s_idesc = tc_idesc(kTcTokens, false), o_idesc = tc_idesc(D, true);
            constexpr uint32_t hi = desc_hi(1024, 2), z_hi = desc_hi(128, 0);
            const uint32_t tm = tmem;
            const uint32_t q_lo = desc_lo(base, 16), k_lo = desc_lo(base + S::kStage0, 16);
            // 16 tokens of values: two groups of 8 rows; blocks of 64 elements lie a tile's rows apart
            const uint32_t v_lo = desc_lo(base + S::kStage0 + S::kTile, kTcTokens * 128);
            // the zero points: pieces of 8 rows of 16 bytes without a swizzle, 128 bytes apart; the second 8
            // of 16 columns are the zeros behind them
            const uint32_t z0 = base >> 4;
            auto scores = [&](auto stage) {
                constexpr int st = decltype(stage)::value;
#pragma unroll
                for (int x = 0; x < NG; ++x) {
                    constexpr uint32_t q0 = S::kZq0, k0 = S::kZk0 + st * NG * S::kZkG;
                    const uint32_t zq = q0 + x * S::kZqG, zk = k0 + x * S::kZkG;
                    mma_ss(tm + x * kTcTokens, z0 + (zq / 16 | (S::kZero0 - zq) / 16 << 16), z0 + (zk / 16 | (S::kZero0 - zk) / 16 << 16),
                           z_hi, s_idesc, false);
#pragma unroll
                    for (int k = 0; k < g / 16; ++k) {
                        const int e = x * g + k * 16;  // 16 elements: 32 bytes along a swizzled row
                        mma_ss(tm + x * kTcTokens, q_lo + (e / 64 * (kTcRows * 128) + e % 64 * 2) / 16,
                               k_lo + (st * 2 * S::kTile + e / 64 * (kTcTokens * 128) + e % 64 * 2) / 16, hi, s_idesc, true);
                    }
                }
            };
            auto outputs = [&](auto stage, bool add) {
                constexpr int st = decltype(stage)::value;
                // a half's weights lie over its own scores of group 0
#pragma unroll
                for (int k = 0; k < kTcTokens / 16; ++k)
                    mma_ts(tm + S::kOCol, tm + k / 2 * 32 + k % 2 * 8, v_lo + (st * 2 * S::kTile + k * 2048) / 16, hi, o_idesc, add || k > 0);
            };
            auto tile = [&](int i, auto stage) {
                constexpr int st = decltype(stage)::value;
                fence_after();
                if (ok) scores(stage);
                umma_commit(s_full);
                // the next tile, so that its scores follow this one's values at once
                if (ok && i + 1 < tiles) ok = wait_for(kv_full + 8 * (st ^ 1), (uint32_t)((i + 1) >> 1) & 1u);
                if (ok) ok = wait_for(p_full, (uint32_t)i & 1u);
                fence_after();
                if (ok) outputs(stage, i > 0);
                umma_commit(kv_free + 8 * st);
            };
            if (ok) ok = wait_for(kv_full, 0u);
            for (int i = 0; i < tiles; i += 2) {
                tile(i, std::integral_constant<int, 0>{});
                if (i + 1 < tiles) tile(i + 1, std::integral_constant<int, 1>{});
            }
            if (!ok) failed = 1;
            umma_commit(done);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        constexpr int N = kTcTokens / 2;  // tokens of a thread
        constexpr float kUp = 6.0f;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16), mine = lanes + 32 * hf;
        const int pair = 1 + (warp & 3);  // the named barrier of the two warps that share rows
        const uint32_t row_at = base + S::kRow0 + lrow * 4;
        float bound = -INFINITY;
        const int span = (int)(to - from);
        const int lim = live ? (int)min(max(limit - from, (int64_t)0), (int64_t)span) : span;  // a row that is not there sees all
        const int all = __reduce_min_sync(0xffffffffu, lim);
        for (int i = 0; i < tiles; ++i) {
            const int st = i & 1, t0 = i * kTcTokens + N * hf;
            const uint32_t mt = base + S::kMeta0 + st * S::kMeta;
            if (ok) ok = wait_for(kv_full + 8 * st, (uint32_t)(i >> 1) & 1u);
            if (ok) ok = wait_for(s_full, (uint32_t)i & 1u);
            fence_after();
            float2 s[N / 2];
#pragma unroll
            for (int c = 0; c < N / 16; ++c) {
                float x[NG][16];
#pragma unroll
                for (int y = 0; y < NG; ++y) tmem_ld16(mine + y * kTcTokens + 16 * c, x[y]);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    float2 r[2];
#pragma unroll
                    for (int y = 0; y < NG; ++y) {
                        const float4 ks = lds_f4(mt + (y * kTcTokens + N * hf + 16 * c + e) * 4);
                        const float2 a0 = make_float2(x[y][e], x[y][e + 1]), a1 = make_float2(x[y][e + 2], x[y][e + 3]);
                        r[0] = y == 0 ? __fmul2_rn(make_float2(ks.x, ks.y), a0) : __ffma2_rn(make_float2(ks.x, ks.y), a0, r[0]);
                        r[1] = y == 0 ? __fmul2_rn(make_float2(ks.z, ks.w), a1) : __ffma2_rn(make_float2(ks.z, ks.w), a1, r[1]);
                    }
                    s[8 * c + e / 2] = r[0];
                    s[8 * c + e / 2 + 1] = r[1];
                }
            }
            const float4 said = lds_f4(mt + NG * kTcTokens * 4);  // valid[2], the values' units
            const uint32_t valid = __float_as_uint(hf ? said.y : said.x);
            const float to_v[2] = {said.z, said.w};
            if (t0 + N > all || valid != 0xffffffffu) {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const bool seen = (valid >> e & 1u) && t0 + e < lim;
                    float &v = e & 1 ? s[e / 2].y : s[e / 2].x;
                    v = seen ? v : -INFINITY;
                }
            }
            float tops[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) tops[e] = fmaxf(s[e].x, s[e].y);
#pragma unroll
            for (int e = 4; e < N / 2; ++e) tops[e & 3] = fmaxf(tops[e & 3], fmaxf(s[e].x, s[e].y));
            float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
            bool more = top > bound;
#pragma unroll
            for (int x = 0; x < NG; ++x) more |= to_v[x] > vref[x];
            if (any_of_pair(pair, more)) {
                sts_f(row_at + hf * kTcRows * 4, top);
                meet_pair(pair);
                float other;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(other) : "r"(row_at + (hf ^ 1) * kTcRows * 4));
                top = fmaxf(fmaxf(top, other) * unit, m);
                const float f = exp2_fast(m - top);
                float fo[NG];
#pragma unroll
                for (int x = 0; x < NG; ++x) {
                    fo[x] = f * (vref[x] / to_v[x]);
                    vref[x] = to_v[x];
                }
                m = top;
                bound = top == kLowest ? -INFINITY : (top + kLag) / unit;
                const float fl = score_in_range(top) ? f : __uint_as_float(0x7fc00000u);
                l2.x *= fl;
                l2.y *= fl;
                if (i > 0) {  // the products up to tile i - 1 have completed: S of tile i came after them
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        float x[16];
                        tmem_ld16(lanes + S::kOCol + hf * (D / 2) + 16 * c, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) x[e] *= fo[NG == 1 ? 0 : hf];  // a half of two groups is one
                        tmem_st16(lanes + S::kOCol + hf * (D / 2) + 16 * c, reinterpret_cast<const uint32_t *>(x));
                    }
                }
            }
            // weights: p times 2^6, to keep small ones normal in fp16
            const float2 u2 = make_float2(unit, unit), m2 = make_float2(kUp - m, kUp - m);
            uint32_t w[N / 2];
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
                const float2 y = __ffma2_rn(s[e], u2, m2);
                const float2 p = make_float2(exp2_fast(y.x), exp2_fast(y.y));
                l2 = __fadd2_rn(l2, p);
                const __half2 h = __floats2half2_rn(p.x, p.y);
                w[e] = *reinterpret_cast<const uint32_t *>(&h);
            }
            tmem_st16(mine, w);
            tmem_wait_st();
            fence_before();
            mbar_arrive(p_full);
        }
        // ---- the chunk's result, normalised by itself: half of the elements each
        // (also where a wait ran out: the products in flight read shared memory and write tensor memory)
        if (!wait_for(done, 0u)) ok = false;
        ok = ok && !failed;
        fence_after();
        meet_pair(pair);  // the other's maximum has been read
        sts_f(row_at + hf * kTcRows * 4, ok ? l2.x + l2.y : -1.0f);
        meet_pair(pair);
        float other;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(other) : "r"(row_at + (hf ^ 1) * kTcRows * 4));
        ok = ok && !(other < 0.0f);
        const float sum = l2.x + l2.y + other;
        const float f = !ok ? __int_as_float(0x7fc00000) : sum == 0.0f ? 0.0f : vref[NG == 1 ? 0 : hf] / sum;
        // by way of shared memory (everything there has been read), so that a row goes out in one piece:
        // rows 16 bytes more than D floats apart, which meet in no bank
        constexpr uint32_t kRow = D * 4 + 16;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            float x[16];
            tmem_ld16(lanes + S::kOCol + hf * (D / 2) + 16 * c, x);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                // operand chunk x8: of a group, run p, 8 elements from d on
                const int x8 = hf * (D / 16) + 2 * c + k, grp = x8 / (g / 8), in_g = x8 % (g / 8);
                const int d = grp * g + in_g / (g / 64) * (g / 8) + in_g % (g / 64) * 8;
                uint32_t y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = sum != 0.0f || !ok ? __float_as_uint(x[8 * k + place<NB>(e)] * f) : 0u;
                sts16(base + (uint32_t)lrow * kRow + d * 4, make_uint4(y[0], y[1], y[2], y[3]));
                sts16(base + (uint32_t)lrow * kRow + d * 4 + 16, make_uint4(y[4], y[5], y[6], y[7]));
            }
        }
        meet_pair(pair);
        for (int r = 16 * hf; r < 16 * hf + 16; ++r) {  // half of the pair's 32 rows each
            const int64_t to_row = __shfl_sync(0xffffffffu, orow, r);
            const int rr = 32 * (warp & 3) + r;
            if (row0 + rr >= total_rows) break;
            if (lane < D / 4)
                *reinterpret_cast<float4 *>(a.part_o + (split * rows + to_row) * D + 4 * lane) = lds_f4(base + (uint32_t)rr * kRow + 16 * lane);
        }
        if (live && hf == 0) a.part_lse[split * rows + orow] = !ok ? f : sum == 0.0f ? -INFINITY : m - kUp + log2f(sum);
    }
    fence_before();
    __syncthreads();
    if (warp == 12) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kCols));
    }
}

static_assert(TcShape<128, 1>::kBars >= kTcRows * (128 * 4 + 16) && TcShape<64, 1>::kBars >= kTcRows * (64 * 4 + 16),
              "room for the results");
static_assert(2 * (TcShape<128, 2>::kSmem + 1024) <= 228 * 1024, "two CTAs on an SM");

template <int D, int NB, int NG>
cudaError_t launch(const Attn &a, int row_tiles, cudaStream_t st) {
    auto k = hqq_kv_prefix_tc_kernel<D, NB, NG>;
    constexpr int smem = TcShape<D, NG>::kSmem;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    k<<<dim3(a.prefix_splits, row_tiles, a.c.heads), kTcThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <int D, int NG>
cudaError_t launch_bits(int nbits, const Attn &a, int row_tiles, cudaStream_t st) {
    return nbits == 2 ? launch<D, 2, NG>(a, row_tiles, st) : nbits == 4 ? launch<D, 4, NG>(a, row_tiles, st) : launch<D, 8, NG>(a, row_tiles, st);
}

}  // namespace

namespace hqq_kv {

cudaError_t launch_prefix_tc(const hqq_kv_cache_t &c, const Attn &a, int row_tiles, cudaStream_t st) {
    if (c.head_dim == 64) return launch_bits<64, 1>(c.nbits, a, row_tiles, st);
    return c.group_size == 64 ? launch_bits<128, 2>(c.nbits, a, row_tiles, st) : launch_bits<128, 1>(c.nbits, a, row_tiles, st);
}

}  // namespace hqq_kv
