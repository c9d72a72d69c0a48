// clo_paged.cuh -- what the kernels of the 16-bit paged cache share: its shape
// and the conversion of 16-bit elements.
#pragma once

#include "clo_kv4.cuh"
#include "clo_paged.h"

namespace clo {

constexpr int PG_D = 128;
constexpr int PG_BLOCK = 16;
constexpr int PG_ROW = PG_D * 2;               // bytes of a row
constexpr int PG_BLOCK_BYTES = PG_BLOCK * PG_ROW;
constexpr int PG_RECORD = 272;                 // bytes of a record of bounds
constexpr int PG_MAX_B = 4096;
constexpr int PG_MAX_G = 8;

inline bool pg_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool pg_dtype_ok(clo_dtype t) { return t == CLO_F16 || t == CLO_BF16; }

// A pair of 16-bit values as fp32, and back (rounded to the nearest).
template <bool BF16>
__device__ __forceinline__ float2 pg_unpack(uint32_t w) {
    return kv4_unpack2<BF16>(w);
}
template <bool BF16>
__device__ __forceinline__ uint32_t pg_pack(float lo, float hi) {
    return kv4_pack2<BF16>(lo, hi);
}

__device__ __forceinline__ bool pg_finite(float x) { return fabsf(x) <= 3.402823466e38f; }

}  // namespace clo
