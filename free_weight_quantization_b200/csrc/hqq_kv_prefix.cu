// hqq_kv_prefix.cu -- the shared prefix of hqq_kv_prefix_attention on the tcgen05 tensor cores, for
// batches that put many query rows on one key head.
//
// A CTA has 128 query rows of one key head (of any sequences) and a chunk of the prefix, which it
// takes in tiles of 64 tokens:
//     S_g = Q_g A_g^T            for each group g of the keys' elements; A: the codes as they are
//     s   = sum_g ks_g (S_g - kz_g sum Q_g),   p = exp2(s - m)
//     O_g += (p vs_g) (C_g - vz_g)
// As in hqq_kv_attn.cu the keys' codes are exact (fp16 subnormals, their power of two in Q), scales
// stay in binary32 outside the products, and p vs is rounded to fp16 once; C - vz is rounded to
// fp16 (exact where the zero point has few bits), which saves the zero points' sum over tokens.
//
// Twelve warps, two CTAs on an SM:
//   * four producer warps turn the codes of a tile into operands in shared memory (128-byte
//     swizzle; keys K-major, values with the elements along the rows), two stages, and the
//     metadata into binary32 arrays;
//   * one lane issues the tcgen05.mma: S_g (128 x 64, binary32, tensor memory), then O_g with the
//     weights as the A operand in tensor memory, where they take the place of S;
//   * four softmax warps: a thread has one row, reads its scores from tensor memory, keeps the
//     running maximum and sum, and writes the weights.  O is rescaled in tensor memory only when
//     the maximum has grown by more than 2^8, or a larger value scale appears.
// The two CTAs of an SM cover each other's turns: while one's scores are in its softmax warps the
// other's products run.
//
// Waits on mbarriers are bounded: one that runs out (none should) makes the CTA write NaN; the other
// roles' waits run out in their turn, and the CTA ends.
#include <type_traits>

#include "hqq_kv_attn.cuh"
#include "hqq_umma.cuh"

namespace {

using namespace hqq_kv;

constexpr int kTcThreads = 384;
// registers of a thread: 80 at launch (two CTAs of 384), divided so that the sum is the same
constexpr int kTcLaunchRegs = 80, kSoftmaxRegs = 144, kProducerRegs = 72, kIssueRegs = 24;
static_assert(kSoftmaxRegs + kProducerRegs + kIssueRegs <= 3 * kTcLaunchRegs, "setmaxnreg draws on the launch's registers");

template <int D, int NG>
struct TcShape {
    static constexpr int kBlocks = D / 64;  // of 64 elements: 128 bytes, a row of the swizzle
    static constexpr int kQ = kBlocks * kTcRows * 128, kTile = kBlocks * kTcTokens * 128;
    static constexpr int kMeta = 3 * NG * kTcTokens * 4 + 16;  // ks, -kz, vs; valid[2], largest vs[2]
    static constexpr int kStage0 = kQ, kMeta0 = kQ + 4 * kTile, kBars = kMeta0 + 2 * kMeta;
    static constexpr int kSmem = kBars + 64 + 1024;            // + alignment slack
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

// the field of NB bits at bit `at` of both halves of v, less z: with the exponent of 1024 put
// above it a field is 1024 + code * 2^at, and the code is exact after one multiply-add
template <int NB>
__device__ __forceinline__ uint32_t field_less(uint32_t v, int at, __half2 z) {
    const uint32_t x = (v & ((((1u << NB) - 1u) * 0x00010001u) << at)) | 0x64006400u;
    const float unit = 1.0f / (float)(1 << at);
    const __half2 c = at == 0 ? __hadd2(*reinterpret_cast<const __half2 *>(&x), __float2half2_rn(-1024.0f))
                              : __hfma2(*reinterpret_cast<const __half2 *>(&x), __float2half2_rn(unit), __float2half2_rn(-1024.0f * unit));
    const __half2 y = __hsub2(c, z);
    return *reinterpret_cast<const uint32_t *>(&y);
}

// the same 8 codes in the same places, less their zero point
template <int NB>
__device__ __forceinline__ uint4 value_chunk8(const uint32_t *w, __half2 z) {
    if constexpr (NB == 8)
        return make_uint4(field_less<8>(w[0], 0, z), field_less<8>(w[0] >> 8, 0, z), field_less<8>(w[1], 0, z), field_less<8>(w[1] >> 8, 0, z));
    else if constexpr (NB == 4)
        return make_uint4(field_less<4>(w[0], 0, z), field_less<4>(w[0], 4, z), field_less<4>(w[0] >> 8, 0, z), field_less<4>(w[0] >> 8, 4, z));
    else {
        const uint32_t v = __byte_perm(w[0], 0, 0x4140);
        return make_uint4(field_less<2>(v, 0, z), field_less<2>(v, 2, z), field_less<2>(v, 4, z), field_less<2>(v, 6, z));
    }
}

__device__ __forceinline__ void sts16(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ float4 lds_f4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
    return v;
}

__device__ __forceinline__ uint2 lds_u2(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
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

// mbar_wait, in line: a call would hold registers that the register split does not have
__device__ __forceinline__ bool wait_for(uint32_t addr, uint32_t parity) {
    for (uint32_t i = 0; i < kMbarWaitLimit; ++i) {
        if (mbar_try(addr, parity)) return true;
        if (i >= 4) __nanosleep(32);
    }
    return false;
}

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

template <int D, int NB, int NG>
__global__ void __launch_bounds__(kTcThreads, 2) hqq_kv_prefix_tc_kernel(const Attn a) {
    using S = TcShape<D, NG>;
    constexpr int g = D / NG, CH = D / 8;  // 8-code chunks of a row
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile uint32_t failed;  // a wait ran out somewhere
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), role = warp >> 2;  // 0 softmax, 1 producers, 2 issue
    const int split = blockIdx.x, row0 = (int)blockIdx.y * kTcRows, head = blockIdx.z;
    const uint32_t base = ((uint32_t)__cvta_generic_to_shared(smem_raw) + 1023u) & ~1023u;
    const uint32_t bars = base + S::kBars;
    const uint32_t kv_full = bars, kv_free = bars + 16, s_full = bars + 32, p_full = bars + 40, done = bars + 48;
    const int64_t from = (int64_t)split * a.prefix_chunk, to = min(from + a.prefix_chunk, a.prefix_len);
    const int tiles = (int)((to - from + kTcTokens - 1) / kTcTokens);
    const int unit_rows = a.nq * a.share, total_rows = a.batch * unit_rows;
    const int64_t rows = (int64_t)a.batch * a.nq * a.heads;

    if (tid == 0) {
        failed = 0;
        for (int s = 0; s < 2; ++s) {
            mbar_init(kv_full + 8 * s, 128);  // every producer thread has stored
            mbar_init(kv_free + 8 * s, 1);    // the products that read the stage have completed
        }
        mbar_init(s_full, 1);    // scores are complete
        mbar_init(p_full, 128);  // every softmax thread has stored its weights
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"((uint32_t)__cvta_generic_to_shared(&tmem_slot)), "n"(S::kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::);
    }

    // ---- a softmax thread's row: scaled by a power of two that takes its largest magnitude to
    // [2^14, 2^15), into shared memory in the order of the keys' operands
    float qs[NG], unit = 0.0f;
    int64_t orow = 0, limit = 0;
    bool live = false;
    if (role == 0) {
        const int l = row0 + tid;
        live = l < total_rows;
        const int lc = live ? l : row0;
        const int b = lc / unit_rows, i = lc % unit_rows / a.share, h = head * a.share + lc % a.share;
        orow = ((int64_t)b * a.nq + i) * a.heads + h;
        int64_t lo;
        visible<true>(a, own_len(a, b), i, lo, limit);
        const uint16_t *q = a.q + b * a.q_batch + i * a.q_token + h * a.q_head;
        uint32_t raw[D / 2];
        float big = 0.0f;
#pragma unroll
        for (int e = 0; e < D / 2; e += 2) {
            if (a.q_wide) *reinterpret_cast<uint2 *>(raw + e) = __ldg((const uint2 *)(q + 2 * e));
            else {
                raw[e] = __ldg(q + 2 * e) | (uint32_t)__ldg(q + 2 * e + 1) << 16;
                raw[e + 1] = __ldg(q + 2 * e + 2) | (uint32_t)__ldg(q + 2 * e + 3) << 16;
            }
        }
        auto at = [&](int e) {
            const uint32_t w = raw[e / 2];
            return a.bf ? __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16) : to_f32<false>((uint16_t)(e & 1 ? w >> 16 : w));
        };
#pragma unroll
        for (int e = 0; e < D; ++e) big = fmaxf(big, fabsf(at(e)));
        const int ex = big > 0.0f ? min(max((int)(__float_as_uint(big) >> 23) - 127, -100), 100) : 0;
        const float up = live ? __uint_as_float((uint32_t)(127 + 14 - ex) << 23) : 0.0f;
        unit = 0x1p24f / __uint_as_float((uint32_t)(127 + 14 - ex) << 23) * a.scale_log2;
#pragma unroll
        for (int x = 0; x < NG; ++x) {
            float sum = 0.0f;
#pragma unroll
            for (int o = 0; o < g; o += 8) {  // 8 elements: one stored chunk
                __half y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = at(x * g + o + e) * up;
                    sum += v;
                    y[place<NB>(e)] = __float2half_rn(v * (1.0f / (float)(1 << place_up<NB>(e))));
                }
                const int c = x * (g / 8) + o / (g / 4) * (g / 32) + o % (g / 4) / 8;
                sts16(base + c / 8 * (kTcRows * 128) + tid * 128 + ((c % 8) ^ (tid & 7)) * 16, *reinterpret_cast<const uint4 *>(y));
            }
            qs[x] = sum * 0x1p-24f;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;

    bool ok = true;
    if (role == 1) {
        // ---- producers: thread (t, h) has half h of token t's key and value
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
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
        Held cur, next;
        load(0, page_of(0), cur);
        int page = page_of(1);
        for (int i = 0; i < tiles; ++i) {
            const int st = i & 1;
            load(i + 1, page, next);
            page = page_of(i + 2);
            if (i >= 2 && ok) ok = wait_for(kv_free + 8 * st, (uint32_t)((i >> 1) - 1) & 1u);
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
                const uint32_t z = __byte_perm(cur.vm[vg], 0, 0x3232);
                sts16(kt + kc / 8 * (kTcTokens * 128) + t * 128 + ((kc % 8) ^ (t & 7)) * 16, key_chunk8<NB>(kw));
                sts16(vt + vc / 8 * (kTcTokens * 128) + t * 128 + ((vc % 8) ^ (t & 7)) * 16,
                      value_chunk8<NB>(vw, *reinterpret_cast<const __half2 *>(&z)));
            }
            uint32_t top = 0;
#pragma unroll
            for (int x = 0; x < NG; ++x) {
                const float2 km = __half22float2(*reinterpret_cast<const __half2 *>(&cur.km[x]));
                const float vs = __low2float(*reinterpret_cast<const __half2 *>(&cur.vm[x]));
                if (h == 0) {
                    sts_f(mt + (x * kTcTokens + t) * 4, km.x);
                    sts_f(mt + ((NG + x) * kTcTokens + t) * 4, -km.y);
                } else {
                    sts_f(mt + ((2 * NG + x) * kTcTokens + t) * 4, vs);
                    top = max(top, __float_as_uint(vs));
                }
            }
            const uint32_t in = __ballot_sync(0xffffffffu, cur.in), most = __reduce_max_sync(0xffffffffu, top);
            if (lane == 0) sts_u(mt + 3 * NG * kTcTokens * 4 + (h == 0 ? 0 : 8) + (t >> 5) * 4, h == 0 ? in : most);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(kv_full + 8 * st);
            cur = next;
        }
        if (!ok) failed = 1;
    } else if (role == 2) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == 8 && elected()) {
            constexpr uint32_t s_idesc = tc_idesc(kTcTokens, false), o_idesc = tc_idesc(g, true);
            for (int i = 0; i < tiles; ++i) {
                const int st = i & 1;
                const uint32_t kt = base + S::kStage0 + st * 2 * S::kTile, vt = kt + S::kTile;
                if (ok) ok = wait_for(kv_full + 8 * st, (uint32_t)(i >> 1) & 1u);
                fence_after();
                if (ok) {
#pragma unroll
                    for (int x = 0; x < NG; ++x)
#pragma unroll
                        for (int k = 0; k < g / 16; ++k) {
                            const int e = x * g + k * 16;  // 16 elements: 32 bytes along a swizzled row
                            const uint64_t da = umma_desc(base + e / 64 * (kTcRows * 128) + e % 64 * 2, 16, 1024, 2);
                            const uint64_t db = umma_desc(kt + e / 64 * (kTcTokens * 128) + e % 64 * 2, 16, 1024, 2);
                            asm volatile(
                                "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                                "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                                ::"r"(tmem + x * kTcTokens), "l"(da), "l"(db), "r"(s_idesc), "r"(k > 0 ? 1u : 0u) : "memory");
                        }
                }
                umma_commit(s_full);
                if (ok) ok = wait_for(p_full, (uint32_t)i & 1u);
                fence_after();
                if (ok) {
#pragma unroll
                    for (int x = 0; x < NG; ++x)
#pragma unroll
                        for (int k = 0; k < kTcTokens / 16; ++k) {
                            // 16 tokens: two groups of 8 rows; blocks of 64 elements lie a tile's rows apart
                            const uint64_t db = umma_desc(vt + x * g / 64 * (kTcTokens * 128) + k * 2048, kTcTokens * 128, 1024, 2);
                            asm volatile(
                                "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                                "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                                ::"r"(tmem + S::kOCol + x * g), "r"(tmem + x * (kTcTokens / 2) + 8 * k), "l"(db), "r"(o_idesc),
                                  "r"(i > 0 || k > 0 ? 1u : 0u) : "memory");
                        }
                }
                umma_commit(kv_free + 8 * st);
            }
            if (!ok) failed = 1;
            umma_commit(done);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
        float m = kLowest, bound = -INFINITY, vref = 0x1p-24f, vin = kWeightUnit * 0x1p24f;
        float2 l2 = make_float2(0.0f, 0.0f);
        const int span = (int)(to - from);
        const int lim = live ? (int)min(max(limit - from, (int64_t)0), (int64_t)span) : span;  // a row that is not there sees all
        const int all = __reduce_min_sync(0xffffffffu, lim);
        for (int i = 0; i < tiles; ++i) {
            const int st = i & 1, t0 = i * kTcTokens;
            const uint32_t mt = base + S::kMeta0 + st * S::kMeta;
            if (ok) ok = wait_for(kv_full + 8 * st, (uint32_t)(i >> 1) & 1u);
            if (ok) ok = wait_for(s_full, (uint32_t)i & 1u);
            fence_after();
            float2 s[kTcTokens / 2];
#pragma unroll
            for (int c = 0; c < kTcTokens / 16; ++c) {
                float x[NG][16];
#pragma unroll
                for (int y = 0; y < NG; ++y) tmem_ld16(lanes + y * kTcTokens + 16 * c, x[y]);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    float2 r[2];
#pragma unroll
                    for (int y = 0; y < NG; ++y) {
                        const float4 ks = lds_f4(mt + (y * kTcTokens + 16 * c + e) * 4);
                        const float4 kz = lds_f4(mt + ((NG + y) * kTcTokens + 16 * c + e) * 4);
                        const float2 q2 = make_float2(qs[y], qs[y]);
                        const float2 a0 = __ffma2_rn(make_float2(kz.x, kz.y), q2, make_float2(x[y][e], x[y][e + 1]));
                        const float2 a1 = __ffma2_rn(make_float2(kz.z, kz.w), q2, make_float2(x[y][e + 2], x[y][e + 3]));
                        r[0] = y == 0 ? __fmul2_rn(make_float2(ks.x, ks.y), a0) : __ffma2_rn(make_float2(ks.x, ks.y), a0, r[0]);
                        r[1] = y == 0 ? __fmul2_rn(make_float2(ks.z, ks.w), a1) : __ffma2_rn(make_float2(ks.z, ks.w), a1, r[1]);
                    }
                    s[8 * c + e / 2] = r[0];
                    s[8 * c + e / 2 + 1] = r[1];
                }
            }
            const uint2 valid = lds_u2(mt + 3 * NG * kTcTokens * 4), most = lds_u2(mt + 3 * NG * kTcTokens * 4 + 8);
            if (t0 + kTcTokens > all || (valid.x & valid.y) != 0xffffffffu) {
#pragma unroll
                for (int e = 0; e < kTcTokens; ++e) {
                    const bool seen = ((e < 32 ? valid.x : valid.y) >> (e & 31) & 1u) && t0 + e < lim;
                    float &v = e & 1 ? s[e / 2].y : s[e / 2].x;
                    v = seen ? v : -INFINITY;
                }
            }
            float top = fmaxf(s[0].x, s[0].y);
#pragma unroll
            for (int e = 1; e < kTcTokens / 2; ++e) top = fmaxf(top, fmaxf(s[e].x, s[e].y));
            const float vs = __uint_as_float(max(most.x, most.y));
            if (__any_sync(0xffffffffu, top > bound || vs > vref)) {
                const float up = fmaxf(vref, __uint_as_float((__float_as_uint(vs) + 0x007fffffu) & 0x7f800000u));
                top = fmaxf(top * unit, m);
                const float f = exp2_fast(m - top);
                const float fo = f * (vref / up);
                vref = up;
                vin = kWeightUnit / up;
                m = top;
                bound = top == kLowest ? -INFINITY : (top + kLag) / unit;
                l2.x *= f;
                l2.y *= f;
                if (i > 0) {  // the products up to tile i - 1 have completed: S of tile i came after them
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        float x[16];
                        tmem_ld16(lanes + S::kOCol + 16 * c, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) x[e] *= fo;
                        tmem_st16(lanes + S::kOCol + 16 * c, reinterpret_cast<const uint32_t *>(x));
                    }
                }
            }
            const float2 u2 = make_float2(unit, unit), m2 = make_float2(-m, -m), v2 = make_float2(vin, vin);
#pragma unroll
            for (int e = 0; e < kTcTokens / 2; ++e) {
                const float2 y = __ffma2_rn(s[e], u2, m2);
                s[e] = make_float2(exp2_fast(y.x), exp2_fast(y.y));
                l2 = __fadd2_rn(l2, s[e]);
                s[e] = __fmul2_rn(s[e], v2);
            }
#pragma unroll
            for (int y = 0; y < NG; ++y)
#pragma unroll
                for (int c = 0; c < kTcTokens / 32; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float4 v = lds_f4(mt + ((2 * NG + y) * kTcTokens + 32 * c + 2 * e) * 4);
                        const float2 w0 = __fmul2_rn(s[16 * c + e], make_float2(v.x, v.y));
                        const float2 w1 = __fmul2_rn(s[16 * c + e + 1], make_float2(v.z, v.w));
                        const __half2 h0 = __floats2half2_rn(w0.x, w0.y), h1 = __floats2half2_rn(w1.x, w1.y);
                        w[e] = *reinterpret_cast<const uint32_t *>(&h0);
                        w[e + 1] = *reinterpret_cast<const uint32_t *>(&h1);
                    }
                    tmem_st16(lanes + y * (kTcTokens / 2) + 16 * c, w);
                }
            tmem_wait_st();
            fence_before();
            mbar_arrive(p_full);
        }
        // ---- the chunk's result, normalised by itself
        if (ok) ok = wait_for(done, 0u);
        ok = __all_sync(0xffffffffu, ok && !failed);
        fence_after();
        const float sum = l2.x + l2.y;
        const float f = !ok ? __int_as_float(0x7fc00000) : sum > 0.0f ? vref / kWeightUnit / sum : 0.0f;
        float *out = a.part_o + (split * rows + orow) * D;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            float x[16];
            tmem_ld16(lanes + S::kOCol + 16 * c, x);
            tmem_wait_ld();
            if (live) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    // operand chunk 2c + k: of group x8, run p, 8 elements from d on
                    const int x8 = 2 * c + k, grp = x8 / (g / 8), in_g = x8 % (g / 8);
                    const int d = grp * g + in_g / (g / 64) * (g / 8) + in_g % (g / 64) * 8;
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = sum > 0.0f || !ok ? x[8 * k + place<NB>(e)] * f : 0.0f;
                    *reinterpret_cast<float4 *>(out + d) = make_float4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<float4 *>(out + d + 4) = make_float4(y[4], y[5], y[6], y[7]);
                }
            }
        }
        if (live) a.part_lse[split * rows + orow] = !ok ? f : sum > 0.0f ? m + log2f(sum) : -INFINITY;
    }
    fence_before();
    __syncthreads();
    if (warp == 8) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kCols));
    }
}

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
