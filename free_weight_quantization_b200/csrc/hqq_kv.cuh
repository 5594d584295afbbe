// hqq_kv.cuh -- what the key/value cache's translation units share: the cache as the kernels see
// it, the element types, and the order in which a row's codes are stored.
//
// A row (one token's key or value of one head) is D values in groups of g.  Its codes are stored
// as kPieces runs, each holding the same share of every group: element d = gamma*g + p*(g/P) + i
// (0 <= i < g/P) is code p*(D/P) + gamma*(g/P) + i of the row, with P = 4 for keys and 8 for
// values.  P is the number of lanes of a warp that hold one token's key (value) as an operand of
// an mma.sync: lane p reads run p with one wide load and finds its share of every group there.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "hqq_b200.h"

namespace hqq_kv {

constexpr int kKeyPieces = 4, kValuePieces = 8;

struct Cache {
    uint8_t *codes[2];  // keys, values: [pages][heads][page][D * nbits / 8]
    __half2 *meta[2];   // [pages][heads][page][D / g] (scale, zero)
    int64_t pages;
    int page_shift;     // log2(page_size)
    int heads;
};

// the row of (page, head, offset within the page); the caller has checked the page
__host__ __device__ __forceinline__ int64_t row_of(const Cache &c, int64_t page, int head, int at) {
    return ((page * c.heads + head) << c.page_shift) + at;
}

// Checks the description of a cache and fills `c`; HQQ_OK or an HQQ_ERR_* code.
int check_cache(const hqq_kv_cache_t *cache, Cache *c);

inline bool aligned_to(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// calls f with the constants (head_dim, nbits, groups a row) of a checked cache
template <typename F>
auto with_layout(const hqq_kv_cache_t &c, F f) {
    auto by_groups = [&](auto dim, auto bits) {
        constexpr int D = decltype(dim)::value;
        switch (c.group_size) {
        case 32: return f(dim, bits, std::integral_constant<int, D / 32>{});
        case 64: return f(dim, bits, std::integral_constant<int, D / 64>{});
        default:
            if constexpr (D >= 128) return f(dim, bits, std::integral_constant<int, D / 128>{});
            else return f(dim, bits, std::integral_constant<int, 1>{});
        }
    };
    auto by_bits = [&](auto dim) {
        switch (c.nbits) {
        case 2: return by_groups(dim, std::integral_constant<int, 2>{});
        case 4: return by_groups(dim, std::integral_constant<int, 4>{});
        default: return by_groups(dim, std::integral_constant<int, 8>{});
        }
    };
    switch (c.head_dim) {
    case 64: return by_bits(std::integral_constant<int, 64>{});
    case 128: return by_bits(std::integral_constant<int, 128>{});
    default: return by_bits(std::integral_constant<int, 256>{});
    }
}

// 16-bit values: BF selects bf16 over fp16
template <bool BF>
__device__ __forceinline__ float to_f32(uint16_t x) {
    if constexpr (BF) return __uint_as_float((uint32_t)x << 16);
    else return __half2float(__ushort_as_half(x));
}

template <bool BF>
__device__ __forceinline__ uint16_t from_f32(float x) {
    if constexpr (BF) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
    else return __half_as_ushort(__float2half_rn(x));
}

}  // namespace hqq_kv
