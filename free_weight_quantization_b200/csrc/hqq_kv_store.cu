// hqq_kv_store.cu -- the key/value cache: the check of its description, quantising rows as they
// are written (hqq_kv_append) and reading them back (hqq_kv_read).
//
// Each group of a row starts from its least and largest value as a weight's group does, and its
// codes are rounded against the scale and zero point as they are stored:
//     scale = fp16(max(fl(fl(hi - lo) / (2^b - 1)), fl(max(|lo|, |hi|) 2^-10), 2^-24))
//     zero  = fp16(fl(-lo inv)),  inv = fl(1 / scale)
//     code  = clip(rint(fl(fl(x inv) + zero)), 0, 2^b - 1)
// with fl() binary32 round to nearest even, one rounding for each operation, so that any program
// that follows the same steps gets the same bits.  The second bound keeps the zero point of a
// group of nearly equal values within +-1024 steps, where fp16 holds it to half a step; the last
// is the least fp16.  Inputs are clamped to the fp16 range (a NaN becomes its lower end), so the
// stored metadata are finite whatever is written.
#include <algorithm>
#include <type_traits>

#include "hqq_kv.cuh"

namespace hqq_kv {

int check_cache(const hqq_kv_cache_t *cache, Cache *c) {
    if (!cache) return HQQ_ERR_ARG;
    if (cache->num_pages < 0 || cache->kv_heads <= 0 || cache->page_size <= 0) return HQQ_ERR_ARG;
    if (cache->nbits < 1 || cache->nbits > 8 || cache->group_size <= 0 || cache->head_dim <= 0 ||
        cache->head_dim % cache->group_size)
        return HQQ_ERR_ARG;
    if (cache->nbits != 2 && cache->nbits != 4 && cache->nbits != 8) return HQQ_ERR_UNSUPPORTED;
    if (cache->head_dim != 64 && cache->head_dim != 128 && cache->head_dim != 256) return HQQ_ERR_UNSUPPORTED;
    if (cache->group_size != 32 && cache->group_size != 64 && cache->group_size != 128) return HQQ_ERR_UNSUPPORTED;
    int shift = 0;
    while ((1 << shift) < cache->page_size && shift < 12) ++shift;
    if ((1 << shift) != cache->page_size || shift < 4 || shift > 10) return HQQ_ERR_UNSUPPORTED;
    // blocks of 16 rows are counted in 31 bits (of the smallest rows, 320 GB for keys and values)
    if (cache->kv_heads > 65535 || cache->num_pages > (int64_t(1) << 34) / cache->page_size / cache->kv_heads)
        return HQQ_ERR_UNSUPPORTED;
    const void *p[4] = {cache->k_codes, cache->v_codes, cache->k_meta, cache->v_meta};
    for (const void *q : p) {
        if (cache->num_pages > 0 && !q) return HQQ_ERR_ARG;
        if (!aligned_to(q, 16)) return HQQ_ERR_ALIGN;
    }
    c->codes[0] = (uint8_t *)cache->k_codes;
    c->codes[1] = (uint8_t *)cache->v_codes;
    c->meta[0] = (__half2 *)cache->k_meta;
    c->meta[1] = (__half2 *)cache->v_meta;
    c->pages = cache->num_pages;
    c->page_shift = shift;
    c->heads = cache->kv_heads;
    return HQQ_OK;
}

}  // namespace hqq_kv

namespace {

using namespace hqq_kv;

constexpr int kStoreThreads = 256;
constexpr int kPerThread = 8;  // values of a row that one thread holds: 16 bytes

struct StoreArgs {
    Cache c;
    const uint16_t *x[2];       // append: keys and values, strided
    int64_t token_stride[2], head_stride[2];
    uint16_t *y[2];             // values as read back, [tokens][heads][D]; null: not wanted
    const int64_t *slots;
    int64_t tokens;
    bool wide;                  // x can be read 16 bytes at a time
};

// bytes [0, N) of v to p, aligned to N
template <int N>
__device__ __forceinline__ void put(uint8_t *p, uint64_t v) {
    if constexpr (N == 1) *p = (uint8_t)v;
    else if constexpr (N == 2) *(uint16_t *)p = (uint16_t)v;
    else if constexpr (N == 4) *(uint32_t *)p = (uint32_t)v;
    else *(uint64_t *)p = v;
}

template <int N>
__device__ __forceinline__ uint64_t take(const uint8_t *p) {
    if constexpr (N == 1) return __ldg(p);
    else if constexpr (N == 2) return __ldg((const uint16_t *)p);
    else if constexpr (N == 4) return __ldg((const uint32_t *)p);
    else return __ldg((const unsigned long long *)p);
}

// byte offset within a row's codes of element d
template <int D, int NB, int NG, int P>
__device__ __forceinline__ int code_byte(int d) {
    constexpr int g = D / NG, s = g / P;
    return ((d % g) / s * (D / P) + d / g * s + d % s) * NB / 8;
}

// The 8 codes of elements d .. d+7 (lowest in the lowest bits) to or from a row.  A run of g / P
// elements is stored together: 8 codes lie in one place, or in two where a run has 4.
template <int D, int NB, int NG, int P>
__device__ __forceinline__ void put_codes(uint8_t *row, int d, uint64_t codes) {
    if constexpr (D / NG / P >= 8) {
        put<NB>(row + code_byte<D, NB, NG, P>(d), codes);
    } else {
        put<NB / 2>(row + code_byte<D, NB, NG, P>(d), codes);
        put<NB / 2>(row + code_byte<D, NB, NG, P>(d + 4), codes >> (4 * NB));
    }
}

template <int D, int NB, int NG, int P>
__device__ __forceinline__ uint64_t take_codes(const uint8_t *row, int d) {
    if constexpr (D / NG / P >= 8) {
        return take<NB>(row + code_byte<D, NB, NG, P>(d));
    } else {
        return take<NB / 2>(row + code_byte<D, NB, NG, P>(d)) |
               take<NB / 2>(row + code_byte<D, NB, NG, P>(d + 4)) << (4 * NB);
    }
}

// 8 codes as four pairs (e, e + 4) of 16-bit whole numbers, the order in which a word of codes falls
// apart into halves
struct Codes8 {
    uint32_t pair[4];
};

template <int NB>
__device__ __forceinline__ uint64_t join_codes(const Codes8 &c) {
    if constexpr (NB == 8) {
        const uint32_t a = c.pair[0] | c.pair[1] << 8, b = c.pair[2] | c.pair[3] << 8;
        return (uint64_t)__byte_perm(a, b, 0x7632) << 32 | __byte_perm(a, b, 0x5410);
    } else {
        const uint32_t w = c.pair[0] | c.pair[1] << NB | c.pair[2] << (2 * NB) | c.pair[3] << (3 * NB);
        return NB == 4 ? w : __byte_perm(w, 0, 0x4420);
    }
}

template <int NB>
__device__ __forceinline__ Codes8 split_codes(uint64_t codes) {
    Codes8 c;
    if constexpr (NB == 8) {
        const uint32_t lo = (uint32_t)codes, hi = (uint32_t)(codes >> 32);
#pragma unroll
        for (int i = 0; i < 4; ++i) c.pair[i] = __byte_perm(lo, hi, 0x0400u + 0x0101u * i) & 0x00FF00FFu;
    } else {
        const uint32_t w = NB == 4 ? (uint32_t)codes : __byte_perm((uint32_t)codes, 0, 0x4140);
#pragma unroll
        for (int i = 0; i < 4; ++i) c.pair[i] = (w >> (NB * i)) & (((1u << NB) - 1u) * 0x00010001u);
    }
    return c;
}

// (code - zero) * scale of 8 codes, rounded once more to 16 bits
template <bool BF>
__device__ __forceinline__ uint4 values_of(const Codes8 &c, float scale, float zero) {
    float2 v[4];  // elements i and i + 4
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // 2^23 + c and back: c, exactly
        const float2 q = make_float2(__uint_as_float(__byte_perm(c.pair[i], 0x4B000000u, 0x7610)),
                                     __uint_as_float(__byte_perm(c.pair[i], 0x4B000000u, 0x7632)));
        v[i] = __fmul2_rn(__fadd2_rn(__fadd2_rn(q, make_float2(-8388608.0f, -8388608.0f)), make_float2(-zero, -zero)),
                          make_float2(scale, scale));
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = i < 2 ? v[2 * i].x : v[2 * i - 4].y, b = i < 2 ? v[2 * i + 1].x : v[2 * i - 3].y;
        if constexpr (BF) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __half2 h = __floats2half2_rn(a, b);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// max(a, b) of pairs of 16-bit values; a NaN stays
template <bool BF>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (BF) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Quantises 8 values of one row; the D/NG/8 threads of its group are neighbours in a warp.
template <int D, int NB, int NG, int P, bool BF>
__device__ __forceinline__ void append_part(const StoreArgs &a, int side, uint32_t r, int d,
                                            int64_t row, bool inside, bool live, const uint4 raw) {
    constexpr int g = D / NG;
    constexpr float top = (float)((1 << NB) - 1);
    uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    // the largest value and the largest negated one, in 16 bits: exact, and half the work
    uint32_t most = max2<BF>(max2<BF>(w[0], w[1]), max2<BF>(w[2], w[3]));
    uint32_t less = max2<BF>(max2<BF>(w[0] ^ 0x80008000u, w[1] ^ 0x80008000u), max2<BF>(w[2] ^ 0x80008000u, w[3] ^ 0x80008000u));
    uint32_t ends = max2<BF>(__byte_perm(most, less, 0x5410), __byte_perm(most, less, 0x7632));  // (largest, -least)
#pragma unroll
    for (int m = 1; m < g / 8; m *= 2) ends = max2<BF>(ends, __shfl_xor_sync(0xffffffffu, ends, m));
    float hi = to_f32<BF>((uint16_t)ends), lo = -to_f32<BF>((uint16_t)(ends >> 16));
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = BF ? __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16) : to_f32<BF>((uint16_t)(w[i / 2] >> (16 * (i & 1))));
    // a NaN, an infinity or a value that fp16 has not: clamped, all threads of the warp in step
    if (__any_sync(0xffffffffu, !(hi <= 65504.0f && lo >= -65504.0f))) {
        hi = -65504.0f;
        lo = 65504.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = fminf(fmaxf(x[i], -65504.0f), 65504.0f);
            lo = fminf(lo, x[i]);
            hi = fmaxf(hi, x[i]);
        }
#pragma unroll
        for (int m = 1; m < g / 8; m *= 2) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
        }
    }
    const float step = __fdiv_rn(__fsub_rn(hi, lo), top);
    const float least = __fmul_rn(fmaxf(fabsf(lo), fabsf(hi)), 0x1p-10f);
    const __half scale_h = __float2half_rn(fmaxf(fmaxf(step, least), 0x1p-24f));
    const float scale = __half2float(scale_h), inv = __frcp_rn(scale);
    const __half zero_h = __float2half_rn(__fmul_rn(-lo, inv));
    const float zero = __half2float(zero_h);
    Codes8 c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // one by one: the packed product and sum were seen merged into one operation with one rounding
        const float2 t = make_float2(__fadd_rn(__fmul_rn(x[i], inv), zero), __fadd_rn(__fmul_rn(x[i + 4], inv), zero));
        // rint, ties to even, into the low bits; the scale and zero point are rounded, so that it can
        // lie a little outside 0 .. 2^b - 1
        const float2 u = __fadd2_rn(t, make_float2(12582912.0f, 12582912.0f));
        const uint32_t p = __byte_perm(__float_as_uint(u.x), __float_as_uint(u.y), 0x5410);
        c.pair[i] = __vmins2(__vmaxs2(p, 0u), (uint32_t)((1 << NB) - 1) * 0x00010001u);
    }
    if (live) {
        put_codes<D, NB, NG, P>(a.c.codes[side] + row * (D * NB / 8), d, join_codes<NB>(c));
        if (d % g == 0) a.c.meta[side][row * NG + d / g] = __halves2half2(scale_h, zero_h);
    }
    if (inside && a.y[side]) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live) v = values_of<BF>(c, scale, zero);
        *(uint4 *)(a.y[side] + (int64_t)r * D + d) = v;
    }
}

// 8 values that need not be aligned: a call, or its 8 loads go along as predicated-off ones
__device__ __noinline__ uint4 load8_singly(const uint16_t *p) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)__ldg(p + 2 * i) | (uint32_t)__ldg(p + 2 * i + 1) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 load8(const uint16_t *p, bool wide) { return wide ? __ldg((const uint4 *)p) : load8_singly(p); }

// One thread for 8 values of a key and the same 8 of its value: D / 8 threads a row, every load and
// store of a warp covers whole 32-byte sectors, two 16-byte loads are in flight for each thread.
// 8192 tokens x 32 heads x 128, with the values returned: 67 us where its bytes take 47; 440
// instructions a warp keep the issue slots 80 % busy.
template <int D, int NB, int NG, bool BF>
__global__ void __launch_bounds__(kStoreThreads) hqq_kv_append_kernel(const StoreArgs a) {
    constexpr int kRows = kStoreThreads / (D / kPerThread);
    const uint32_t rows = (uint32_t)a.tokens * a.c.heads;  // below 2^31
    const uint32_t r0 = blockIdx.x * kRows + threadIdx.x / (D / kPerThread);
    const uint32_t r = min(r0, rows - 1);  // whole warps take part in the exchanges below
    const int d = (int)(threadIdx.x % (D / kPerThread)) * kPerThread;
    const uint32_t token = r / (uint32_t)a.c.heads;
    const int head = (int)(r - token * a.c.heads);
    const uint4 k = load8(a.x[0] + token * a.token_stride[0] + head * a.head_stride[0] + d, a.wide);
    const uint4 v = load8(a.x[1] + token * a.token_stride[1] + head * a.head_stride[1] + d, a.wide);
    const int64_t slot = __ldg(a.slots + token);
    const int64_t page = slot >> a.c.page_shift;
    const bool inside = r0 < rows, live = inside && slot >= 0 && page < a.c.pages;
    const int64_t row = live ? row_of(a.c, page, head, (int)(slot & ((1 << a.c.page_shift) - 1))) : 0;
    append_part<D, NB, NG, kKeyPieces, BF>(a, 0, r, d, row, inside, live, k);
    append_part<D, NB, NG, kValuePieces, BF>(a, 1, r, d, row, inside, live, v);
}

// The same threads with kReadRows rows each, a block's rows apart: a slot's number, then its codes
// and metadata, are two trips to memory, on which several rows go together (one row a thread: 41 us
// for 32768 tokens x 8 heads x 128, bound by the wait; four 34, its bytes take 26).
constexpr int kReadRows = 4;

template <int D, int NB, int NG, bool BF>
__global__ void __launch_bounds__(kStoreThreads) hqq_kv_read_kernel(const StoreArgs a) {
    constexpr int kRows = kStoreThreads / (D / kPerThread), g = D / NG;
    const uint32_t rows = (uint32_t)a.tokens * a.c.heads, r0 = blockIdx.x * (kRows * kReadRows) + threadIdx.x / (D / kPerThread);
    const int d = (int)(threadIdx.x % (D / kPerThread)) * kPerThread;
    int64_t row[kReadRows];  // -1: nothing there
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        const uint32_t r = r0 + i * kRows;
        const uint32_t token = min(r, rows - 1) / (uint32_t)a.c.heads;
        const int head = (int)(r - token * a.c.heads);
        const int64_t slot = __ldg(a.slots + token), page = slot >> a.c.page_shift;
        row[i] = r < rows && slot >= 0 && page < a.c.pages ? row_of(a.c, page, head, (int)(slot & ((1 << a.c.page_shift) - 1))) : -1;
    }
    uint64_t kc[kReadRows], vc[kReadRows];
    __half2 km[kReadRows], vm[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        if (row[i] >= 0) {
            kc[i] = take_codes<D, NB, NG, kKeyPieces>(a.c.codes[0] + row[i] * (D * NB / 8), d);
            vc[i] = take_codes<D, NB, NG, kValuePieces>(a.c.codes[1] + row[i] * (D * NB / 8), d);
            km[i] = __ldg(a.c.meta[0] + row[i] * NG + d / g);
            vm[i] = __ldg(a.c.meta[1] + row[i] * NG + d / g);
        }
    }
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        const uint32_t r = r0 + i * kRows;
        uint4 k = make_uint4(0, 0, 0, 0), v = k;
        if (row[i] >= 0) {
            const float2 kz = __half22float2(km[i]), vz = __half22float2(vm[i]);
            k = values_of<BF>(split_codes<NB>(kc[i]), kz.x, kz.y);
            v = values_of<BF>(split_codes<NB>(vc[i]), vz.x, vz.y);
        }
        if (r < rows) {
            if (a.y[0]) *(uint4 *)(a.y[0] + (int64_t)r * D + d) = k;
            if (a.y[1]) *(uint4 *)(a.y[1] + (int64_t)r * D + d) = v;
        }
    }
}

template <bool APPEND>
int launch_store(const hqq_kv_cache_t &cache, const StoreArgs &a, bool bf, cudaStream_t st) {
    return with_layout(cache, [&](auto dim, auto bits, auto groups) {
        constexpr int D = dim, NB = bits, NG = groups;
        constexpr int kRows = kStoreThreads / (D / kPerThread) * (APPEND ? 1 : kReadRows);
        const unsigned blocks = (unsigned)((a.tokens * a.c.heads + kRows - 1) / kRows);
        if constexpr (APPEND) {
            if (bf) hqq_kv_append_kernel<D, NB, NG, true><<<blocks, kStoreThreads, 0, st>>>(a);
            else hqq_kv_append_kernel<D, NB, NG, false><<<blocks, kStoreThreads, 0, st>>>(a);
        } else {
            if (bf) hqq_kv_read_kernel<D, NB, NG, true><<<blocks, kStoreThreads, 0, st>>>(a);
            else hqq_kv_read_kernel<D, NB, NG, false><<<blocks, kStoreThreads, 0, st>>>(a);
        }
        return cudaGetLastError() == cudaSuccess ? HQQ_OK : HQQ_ERR_CUDA;
    });
}

int check_tokens(const Cache &c, int64_t tokens, int dtype) {
    if (tokens < 0 || (dtype != HQQ_FP16 && dtype != HQQ_BF16)) return HQQ_ERR_ARG;
    if (tokens > INT32_MAX / c.heads) return HQQ_ERR_UNSUPPORTED;
    return HQQ_OK;
}

}  // namespace

extern "C" int hqq_kv_append(const hqq_kv_cache_t *cache, const void *k, const void *v, int dtype,
                             int64_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                             int64_t v_token_stride, int64_t v_head_stride, const int64_t *slots,
                             void *k_values, void *v_values, void *stream) {
    StoreArgs a = {};
    int rc = check_cache(cache, &a.c);
    if (rc == HQQ_OK) rc = check_tokens(a.c, tokens, dtype);
    if (rc != HQQ_OK) return rc;
    if (tokens == 0) return HQQ_OK;
    if (!k || !v || !slots) return HQQ_ERR_ARG;
    if (!aligned_to(k, 2) || !aligned_to(v, 2) || !aligned_to(slots, 8) || !aligned_to(k_values, 16) ||
        !aligned_to(v_values, 16))
        return HQQ_ERR_ALIGN;
    a.x[0] = (const uint16_t *)k;
    a.x[1] = (const uint16_t *)v;
    a.token_stride[0] = k_token_stride;
    a.token_stride[1] = v_token_stride;
    a.head_stride[0] = k_head_stride;
    a.head_stride[1] = v_head_stride;
    a.y[0] = (uint16_t *)k_values;
    a.y[1] = (uint16_t *)v_values;
    a.slots = slots;
    a.tokens = tokens;
    a.wide = aligned_to(k, 16) && aligned_to(v, 16) &&
             (k_token_stride | k_head_stride | v_token_stride | v_head_stride) % 8 == 0;
    return launch_store<true>(*cache, a, dtype == HQQ_BF16, (cudaStream_t)stream);
}

extern "C" int hqq_kv_read(const hqq_kv_cache_t *cache, const int64_t *slots, int64_t tokens, int dtype,
                           void *k_out, void *v_out, void *stream) {
    StoreArgs a = {};
    int rc = check_cache(cache, &a.c);
    if (rc == HQQ_OK) rc = check_tokens(a.c, tokens, dtype);
    if (rc != HQQ_OK) return rc;
    if (tokens == 0) return HQQ_OK;
    if (!slots || (!k_out && !v_out)) return HQQ_ERR_ARG;
    if (!aligned_to(slots, 8) || !aligned_to(k_out, 16) || !aligned_to(v_out, 16)) return HQQ_ERR_ALIGN;
    a.y[0] = (uint16_t *)k_out;
    a.y[1] = (uint16_t *)v_out;
    a.slots = slots;
    a.tokens = tokens;
    return launch_store<false>(*cache, a, dtype == HQQ_BF16, (cudaStream_t)stream);
}
