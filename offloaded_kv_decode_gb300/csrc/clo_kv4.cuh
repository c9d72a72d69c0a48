// clo_kv4.cuh -- the 4-bit paged cache's record and 16-bit element types,
// shared by the append, gather and attention kernels (layout: clo_kv4.h).
#pragma once

#include <cuda_bf16.h>

#include "clo_device.cuh"
#include "clo_kv4.h"

namespace clo {

constexpr int KV4_D = 128;
constexpr int KV4_BLOCK = 16;
constexpr int KV4_ROW = KV4_D / 2;                 // bytes of codes of one token's K (or V)
constexpr int KV4_CODES = KV4_BLOCK * KV4_ROW;     // bytes of codes of K (or V) in a record
constexpr int KV4_PARAMS = 2 * KV4_CODES;          // where the (scale, zero) pairs start
constexpr int KV4_MAX_B = 4096;

// Bytes of a record with NG groups of channels.
__host__ __device__ constexpr int kv4_record(int ng) { return KV4_PARAMS + KV4_BLOCK * 2 * ng * 4; }

// Groups a row is cut into, or 0 if this build does not have the size.
inline int kv4_groups(int group) { return group == 32 || group == 64 || group == 128 ? KV4_D / group : 0; }

inline bool kv4_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Where the 32-bit code word of channels 8i .. 8i + 7 (i < 16) of token t
// lies in a record.
__device__ __forceinline__ int kv4_k_word(int t, int i) { return t * KV4_ROW + ((i & 3) * 4 + (i >> 2)) * 4; }
__device__ __forceinline__ int kv4_v_word(int t, int i) {
    return KV4_CODES + t * KV4_ROW + (((i >> 2) ^ ((t >> 1) & 3)) * 4 + (i & 3)) * 4;
}

// Where the (scale, zero) pair of group g of token t's K (kv = 0) or V (1) lies.
__device__ __forceinline__ int kv4_param(int t, int kv, int ng, int g) {
    return KV4_PARAMS + ((t * 2 + kv) * ng + g) * 4;
}

template <bool BF16>
__device__ __forceinline__ float2 kv4_unpack2(uint32_t w) {
    if constexpr (BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <bool BF16>
__device__ __forceinline__ uint32_t kv4_pack2(float lo, float hi) {
    if constexpr (BF16) {
        __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t*>(&b);
    } else {
        return pack_half2(lo, hi);
    }
}

// The same, but fp16 has its largest value where the rounding would pass it: a
// scale is rounded up, so code 15 of a group that reaches 65504 may lie up to 64
// above.  A NaN stays one.
template <bool BF16>
__device__ __forceinline__ uint32_t kv4_pack2_finite(float lo, float hi) {
    if constexpr (BF16) {
        return kv4_pack2<true>(lo, hi);
    } else {
        uint32_t d;
        asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
        return d;
    }
}

}  // namespace clo
