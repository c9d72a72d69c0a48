// clo_kv4_cache.cu -- clo_kv4_append and clo_kv4_gather: 16-bit K and V rows
// into the 4-bit paged cache and back (format: clo_kv4.h).
//
// A warp takes one (token, KV head): lanes 0-15 its K row, lanes 16-31 its V
// row, 8 channels (16 bytes of the 16-bit tensor, one 32-bit word of codes) a
// lane.  A group of channels is then 4, 8 or 16 neighbouring lanes, and its
// minimum and maximum take 2, 3 or 4 shuffles.
#include "clo_kv4.cuh"

namespace clo {

constexpr int CACHE_THREADS = 256;
constexpr int CACHE_CTAS_PER_SM = 8;

struct CacheArgs {
    const void* k;
    const void* v;
    long long k_stride, v_stride;  // elements between tokens
    uint8_t* pool;
    const int32_t* slots;
    int32_t* err_flag;
    int N, Hkv, num_blocks;
};

// A slot in the cache, or -1 for one to skip.
__device__ __forceinline__ int checked_slot(int slot, int num_blocks, bool& bad) {
    if (slot >= 0 && slot / KV4_BLOCK < num_blocks) return slot;
    bad |= slot != -1;
    return -1;
}

// The codes and the (scale, zero) pair of this lane's 8 channels; `lanes`
// neighbouring lanes share a group.
template <bool BF16>
__device__ __forceinline__ void quantise(const uint4 raw, int lanes, uint32_t& codes, __half2& pair) {
    float x[8];
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = kv4_unpack2<BF16>(w[j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
    }
    float lo = x[0], hi = x[0], sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        lo = fminf(lo, x[j]);
        hi = fmaxf(hi, x[j]);
        sum += x[j] * 0.f;  // NaN if any element is NaN or infinite
    }
    for (int o = 1; o < lanes; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(FULL_MASK, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(FULL_MASK, hi, o));
        sum += __shfl_xor_sync(FULL_MASK, sum, o);
    }
    const bool finite = sum == 0.f;
    if (BF16) {
        lo = fminf(fmaxf(lo, -65504.f), 65504.f);
        hi = fminf(fmaxf(hi, -65504.f), 65504.f);
    }
    const __half zero_h = __float2half_rd(lo);
    const float zero = __half2float(zero_h);
    // Rounded up, so that below, where 15 times an fp16 value (exact in fp32)
    // is compared with it, the answer is the exact difference's.
    const float reach = __fsub_ru(hi, zero);
    // The fp16 value next to reach / 15, moved up if it is below it.
    __half scale_h = __float2half_rn(reach * (1.f / 15.f));
    if (15.f * __half2float(scale_h) < reach)
        scale_h = __ushort_as_half(static_cast<unsigned short>(__half_as_ushort(scale_h) + 1));
    const float scale = __half2float(scale_h);
    codes = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float f = x[j];
        if (BF16) f = fminf(fmaxf(f, -65504.f), 65504.f);
        const float c = scale > 0.f ? rintf((f - zero) / scale) : 0.f;
        codes |= static_cast<uint32_t>(c) << (4 * j);
    }
    pair = __halves2half2(scale_h, zero_h);
    if (!finite) {
        codes = 0;
        pair = __halves2half2(__ushort_as_half(0x7fff), __ushort_as_half(0x7fff));
    }
}

template <bool BF16, int NG>
__global__ void __launch_bounds__(CACHE_THREADS) kv4_append_kernel(const CacheArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, kv = lane >> 4, i = lane & 15;
    const unsigned warps = gridDim.x * (CACHE_THREADS / 32);
    const unsigned units = static_cast<unsigned>(a.N) * a.Hkv;
    const uint8_t* src = static_cast<const uint8_t*>(kv ? a.v : a.k);
    const long long stride = kv ? a.v_stride : a.k_stride;
    bool bad = false;
    for (unsigned u = blockIdx.x * (CACHE_THREADS / 32) + (threadIdx.x >> 5); u < units; u += warps) {
        const int n = u / a.Hkv, h = u - n * static_cast<unsigned>(a.Hkv);
        const int slot = checked_slot(a.slots[n], a.num_blocks, bad);
        if (slot < 0) continue;
        const uint4 raw = *reinterpret_cast<const uint4*>(src + 2 * (n * stride + h * KV4_D + i * 8));
        uint32_t codes;
        __half2 pair;
        quantise<BF16>(raw, 16 / NG, codes, pair);
        const int t = slot % KV4_BLOCK;
        uint8_t* rec = a.pool + (static_cast<long long>(slot / KV4_BLOCK) * a.Hkv + h) * kv4_record(NG);
        *reinterpret_cast<uint32_t*>(rec + (kv ? kv4_v_word(t, i) : kv4_k_word(t, i))) = codes;
        if (i % (16 / NG) == 0)
            *reinterpret_cast<__half2*>(rec + kv4_param(t, kv, NG, i / (16 / NG))) = pair;
    }
    if (bad) report_error(a.err_flag, CLO_FLAG_BAD_INDEX);
}

template <bool BF16, int NG>
__global__ void __launch_bounds__(CACHE_THREADS) kv4_gather_kernel(const CacheArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, kv = lane >> 4, i = lane & 15;
    const unsigned warps = gridDim.x * (CACHE_THREADS / 32);
    const unsigned units = static_cast<unsigned>(a.N) * a.Hkv;
    uint4* dst = static_cast<uint4*>(const_cast<void*>(kv ? a.v : a.k));
    bool bad = false;
    for (unsigned u = blockIdx.x * (CACHE_THREADS / 32) + (threadIdx.x >> 5); u < units; u += warps) {
        const int n = u / a.Hkv, h = u - n * static_cast<unsigned>(a.Hkv);
        const int slot = checked_slot(a.slots[n], a.num_blocks, bad);
        uint4 o = make_uint4(0u, 0u, 0u, 0u);
        if (slot >= 0) {
            const int t = slot % KV4_BLOCK;
            const uint8_t* rec = a.pool + (static_cast<long long>(slot / KV4_BLOCK) * a.Hkv + h) * kv4_record(NG);
            const uint32_t codes = *reinterpret_cast<const uint32_t*>(rec + (kv ? kv4_v_word(t, i) : kv4_k_word(t, i)));
            const float2 p = __half22float2(
                *reinterpret_cast<const __half2*>(rec + kv4_param(t, kv, NG, i / (16 / NG))));
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = fmaf(static_cast<float>((codes >> (4 * j)) & 15u), p.x, p.y);
            o.x = kv4_pack2<BF16>(x[0], x[1]);
            o.y = kv4_pack2<BF16>(x[2], x[3]);
            o.z = kv4_pack2<BF16>(x[4], x[5]);
            o.w = kv4_pack2<BF16>(x[6], x[7]);
        }
        dst[static_cast<long long>(u) * 16 + i] = o;
    }
    if (bad) report_error(a.err_flag, CLO_FLAG_BAD_INDEX);
}

using CacheKernel = void (*)(const CacheArgs);

static clo_status launch_cache(CacheKernel kernel, const CacheArgs& a, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0 || !prepare_kernel(reinterpret_cast<const void*>(kernel), 0)) return CLO_ERR_CUDA;
    const long long units = static_cast<long long>(a.N) * a.Hkv;
    long long grid = (units + CACHE_THREADS / 32 - 1) / (CACHE_THREADS / 32);
    const long long most = static_cast<long long>(sms) * CACHE_CTAS_PER_SM;
    if (grid > most) grid = most;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(CACHE_THREADS), 0, stream, a) == cudaSuccess
               ? CLO_OK
               : CLO_ERR_CUDA;
}

// What both calls check; nothing is set where there is nothing to do.
static clo_status check_cache(const void* k, const void* v, clo_dtype dtype, const int32_t* slots, int N,
                              int Hkv, int d, const uint8_t* pool, int num_blocks, int block_size,
                              int group, const int32_t* err_flag) {
    if (N < 0 || Hkv < 1 || num_blocks < 1) return CLO_ERR_INVALID_ARG;
    if (dtype != CLO_F16 && dtype != CLO_BF16) return CLO_ERR_INVALID_ARG;
    if (N > 0 && (k == nullptr || v == nullptr || slots == nullptr || pool == nullptr)) return CLO_ERR_INVALID_ARG;
    if (!kv4_aligned(k, 16) || !kv4_aligned(v, 16) || !kv4_aligned(pool, 16) || !kv4_aligned(slots, 4) ||
        !kv4_aligned(err_flag, 4))
        return CLO_ERR_INVALID_ARG;
    if (d != KV4_D || block_size != KV4_BLOCK || kv4_groups(group) == 0) return CLO_ERR_UNSUPPORTED;
    // Slots and (token, head) counts are 32-bit.
    if (static_cast<long long>(N) * Hkv >= (1ll << 31) || num_blocks > (1 << 27)) return CLO_ERR_UNSUPPORTED;
    return CLO_OK;
}

template <bool BF16>
static CacheKernel append_kernel(int ng) {
    return ng == 1 ? kv4_append_kernel<BF16, 1> : ng == 2 ? kv4_append_kernel<BF16, 2> : kv4_append_kernel<BF16, 4>;
}
template <bool BF16>
static CacheKernel gather_kernel(int ng) {
    return ng == 1 ? kv4_gather_kernel<BF16, 1> : ng == 2 ? kv4_gather_kernel<BF16, 2> : kv4_gather_kernel<BF16, 4>;
}

}  // namespace clo

using namespace clo;

extern "C" size_t clo_kv4_block_bytes(int block_size, int d, int group) {
    const int ng = kv4_groups(group);
    return block_size == KV4_BLOCK && d == KV4_D && ng > 0 ? static_cast<size_t>(kv4_record(ng)) : 0;
}

extern "C" clo_status clo_kv4_append(const void* k, const void* v, long long k_stride, long long v_stride,
                                     clo_dtype dtype, const int32_t* slot_map, int N, int Hkv, int d,
                                     uint8_t* pool, int num_blocks, int block_size, int group,
                                     int32_t* err_flag, cudaStream_t stream) {
    const clo_status st = check_cache(k, v, dtype, slot_map, N, Hkv, d, pool, num_blocks, block_size, group, err_flag);
    if (st != CLO_OK) return st;
    const long long row = static_cast<long long>(Hkv) * d;
    if (N > 1 && (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0 ||
                  k_stride > (1ll << 40) || v_stride > (1ll << 40)))
        return CLO_ERR_INVALID_ARG;
    if (N == 0) return CLO_OK;
    CacheArgs a{k, v, k_stride, v_stride, pool, slot_map, err_flag, N, Hkv, num_blocks};
    const int ng = kv4_groups(group);
    return launch_cache(dtype == CLO_BF16 ? append_kernel<true>(ng) : append_kernel<false>(ng), a, stream);
}

extern "C" clo_status clo_kv4_gather(const uint8_t* pool, int num_blocks, int block_size, int group,
                                     const int32_t* slot_map, int N, int Hkv, int d, void* k, void* v,
                                     clo_dtype dtype, int32_t* err_flag, cudaStream_t stream) {
    const clo_status st = check_cache(k, v, dtype, slot_map, N, Hkv, d, pool, num_blocks, block_size, group, err_flag);
    if (st != CLO_OK) return st;
    if (N == 0) return CLO_OK;
    CacheArgs a{k, v, 0, 0, const_cast<uint8_t*>(pool), slot_map, err_flag, N, Hkv, num_blocks};
    const int ng = kv4_groups(group);
    return launch_cache(dtype == CLO_BF16 ? gather_kernel<true>(ng) : gather_kernel<false>(ng), a, stream);
}
