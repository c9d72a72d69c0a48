// clo_kv4_cache.cu -- clo_kv4_append and clo_kv4_gather: 16-bit K and V rows
// into the 4-bit paged cache and back (format: clo_kv4.h).
//
// A warp takes a (token, KV head) at a time: lanes 0-15 its K row, lanes 16-31
// its V row, 8 channels (16 bytes of the 16-bit tensor, one 32-bit word of
// codes) a lane.  A group of channels is then 4, 8 or 16 neighbouring lanes,
// and its minimum and maximum take 2, 3 or 4 shuffles of one register, (min,
// -max) as a pair of 16-bit values under a pairwise minimum.
//
// Both are streams: HBM bounds them, and next the issue slots (at HBM's rate an
// SM has 110 warp instructions for a row pair of the append).  So a warp has the
// rows of 4 (token, head)s in flight, the rows are loaded without waiting for
// their slots, and fp32 work is done on pairs (the f32x2 instructions).
#include "clo_kv4.cuh"

namespace clo {

constexpr int CACHE_THREADS = 256;
constexpr int CACHE_CTAS_PER_SM = 8;
constexpr int CACHE_UNROLL = 4;  // (token, head) pairs a warp has in flight

struct CacheArgs {
    const void* k;
    const void* v;
    long long k_stride, v_stride;  // elements between tokens
    uint8_t* pool;
    const int32_t* slots;
    int32_t* err_flag;
    int N, Hkv, num_blocks;
};

// 16 bytes that are read once.
__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
    return __ldcs(reinterpret_cast<const uint4*>(p));
}

// A slot in the cache, or -1 for one to skip.
__device__ __forceinline__ int checked_slot(int slot, int num_blocks, bool& bad) {
    if (slot >= 0 && slot / KV4_BLOCK < num_blocks) return slot;
    bad |= slot != -1;
    return -1;
}

// Pairs of fp32 values in one register pair.
__device__ __forceinline__ uint64_t pair2(float x, float y) {
    return static_cast<uint64_t>(__float_as_uint(x)) | (static_cast<uint64_t>(__float_as_uint(y)) << 32);
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// (min, -max) of this lane's 8 elements, as 16-bit values of the input's type;
// NaN where there is a NaN.
template <bool BF16>
__device__ __forceinline__ uint32_t least2(uint32_t a, uint32_t b) {
    if constexpr (BF16) {
        const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                             *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    } else {
        const __half2 r = __hmin2_nan(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
}

constexpr uint32_t SIGNS = 0x80008000u;  // of a pair of 16-bit values

// The codes and the (scale, zero) pair of this lane's 8 channels; 16 / NG
// neighbouring lanes share a group.
template <bool BF16, int NG>
__device__ __forceinline__ void quantise(const uint4 raw, uint32_t& codes, uint32_t& pair) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    const uint32_t lo = least2<BF16>(least2<BF16>(w[0], w[1]), least2<BF16>(w[2], w[3]));
    const uint32_t up = least2<BF16>(least2<BF16>(w[0] ^ SIGNS, w[1] ^ SIGNS),
                                     least2<BF16>(w[2] ^ SIGNS, w[3] ^ SIGNS));
    uint32_t ends = least2<BF16>(__byte_perm(lo, up, 0x5410), __byte_perm(lo, up, 0x7632));
#pragma unroll
    for (int o = 1; o < 16 / NG; o <<= 1) ends = least2<BF16>(ends, __shfl_xor_sync(FULL_MASK, ends, o));
    const float2 e = kv4_unpack2<BF16>(ends);
    float least = e.x, most = -e.y;
    const bool finite = fabsf(least) < INFINITY && fabsf(most) < INFINITY;
    bool clamp = false;
    if (BF16) {
        clamp = least < -65504.f || most > 65504.f;
        least = fminf(fmaxf(least, -65504.f), 65504.f);
        most = fminf(fmaxf(most, -65504.f), 65504.f);
    }
    const __half zero_h = __float2half_rd(least);
    const float zero = __half2float(zero_h);
    // Rounded up, so that below, where 15 times an fp16 value (exact in fp32)
    // is compared with it, the answer is the exact difference's.
    const float reach = __fsub_ru(most, zero);
    // The fp16 value next to reach / 15, moved up if it is below it.
    __half scale_h = __float2half_rn(reach * (1.f / 15.f));
    if (15.f * __half2float(scale_h) < reach)
        scale_h = __ushort_as_half(static_cast<unsigned short>(__half_as_ushort(scale_h) + 1));
    const float scale = __half2float(scale_h);
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
    inv = scale > 0.f ? inv : 0.f;
    // Quotients by the reciprocal, put right by their remainder (Markstein's
    // correction): a quotient half way between two codes comes out exact, so
    // it is rounded to the even one.  Adding 1.5 * 2^23 leaves the code in the
    // low bits; the eight constants are taken off together.
    constexpr float MAGIC = 12582912.f;
    constexpr uint32_t MAGICS = 0x4B400000u * 0x11111111u;
    const uint64_t zero2 = pair2(-zero, -zero), inv2 = pair2(inv, inv), neg2 = pair2(-scale, -scale);
    const uint64_t magic2 = pair2(MAGIC, MAGIC);
    uint32_t word = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float2 f = kv4_unpack2<BF16>(w[j]);
        if (BF16 && clamp) {
            f.x = fminf(fmaxf(f.x, -65504.f), 65504.f);
            f.y = fminf(fmaxf(f.y, -65504.f), 65504.f);
        }
        const uint64_t d = add2(pair2(f.x, f.y), zero2);
        uint64_t q = mul2(d, inv2);
        q = fma2(fma2(q, neg2, d), inv2, q);
        q = add2(q, magic2);
        word += static_cast<uint32_t>(q) << (8 * j);
        word += static_cast<uint32_t>(q >> 32) << (8 * j + 4);
    }
    word -= MAGICS;
    codes = finite ? word : 0u;
    pair = finite ? static_cast<uint32_t>(__half_as_ushort(scale_h)) | (static_cast<uint32_t>(__half_as_ushort(zero_h)) << 16)
                  : 0x7fff7fffu;
}

// (token, head) pairs u, u + 1, ..: the token and head of the first and a step
// to the next without a division.
struct Pair {
    unsigned n, h;
    __device__ __forceinline__ Pair(unsigned u, unsigned heads) : n(u / heads), h(u - n * heads) {}
    __device__ __forceinline__ void next(unsigned heads) {
        if (++h == heads) {
            h = 0;
            ++n;
        }
    }
};

template <bool BF16, int NG>
__global__ void __launch_bounds__(CACHE_THREADS) kv4_append_kernel(const CacheArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, kv = lane >> 4, i = lane & 15;
    const unsigned warps = gridDim.x * (CACHE_THREADS / 32), heads = a.Hkv;
    const unsigned pairs = static_cast<unsigned>(a.N) * heads;
    const uint8_t* src = static_cast<const uint8_t*>(kv ? a.v : a.k) + 16 * i;
    const long long stride = 2 * (kv ? a.v_stride : a.k_stride);
    bool bad = false;
    for (unsigned u = (blockIdx.x * (CACHE_THREADS / 32) + (threadIdx.x >> 5)) * CACHE_UNROLL; u < pairs;
         u += warps * CACHE_UNROLL) {
        uint4 raw[CACHE_UNROLL];
        int slot[CACHE_UNROLL];
        unsigned head[CACHE_UNROLL];
        Pair p(u, heads);
#pragma unroll
        for (int x = 0; x < CACHE_UNROLL; ++x) {
            slot[x] = -1;
            head[x] = p.h;
            if (u + x < pairs) {
                slot[x] = __ldg(a.slots + p.n);
                raw[x] = ld_stream(src + p.n * stride + p.h * (2 * KV4_D));
            }
            p.next(heads);
        }
#pragma unroll
        for (int x = 0; x < CACHE_UNROLL; ++x) {
            const int s = checked_slot(slot[x], a.num_blocks, bad);
            if (s < 0) continue;  // the whole warp
            uint32_t codes, pair;
            quantise<BF16, NG>(raw[x], codes, pair);
            const int t = s % KV4_BLOCK;
            uint8_t* rec = a.pool + (static_cast<size_t>(s / KV4_BLOCK) * heads + head[x]) * kv4_record(NG);
            *reinterpret_cast<uint32_t*>(rec + (kv ? kv4_v_word(t, i) : kv4_k_word(t, i))) = codes;
            if (i % (16 / NG) == 0) *reinterpret_cast<uint32_t*>(rec + kv4_param(t, kv, NG, i / (16 / NG))) = pair;
        }
    }
    if (bad) report_error(a.err_flag, CLO_FLAG_BAD_INDEX);
}

// The values of a word's 8 codes.
template <bool BF16>
__device__ __forceinline__ uint4 expand(uint32_t codes, uint32_t pair) {
    // 1024 + code and 1024 + 16 * code as pairs of fp16 (codes 0 and 4, 1 and
    // 5, 2 and 6, 3 and 7), then the codes alone; all exact.
    const __half2 sz = *reinterpret_cast<const __half2*>(&pair);
    __half2 r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t m = ((codes >> (k >= 2 ? 8 : 0)) & ((k & 1) ? 0x00f000f0u : 0x000f000fu)) | 0x64006400u;
        const __half2 h = *reinterpret_cast<const __half2*>(&m);
        r[k] = (k & 1) ? __hfma2(h, __float2half2_rn(0.0625f), __float2half2_rn(-64.f))
                       : __hadd2(h, __float2half2_rn(-1024.f));
    }
    uint32_t o[4];
    if constexpr (BF16) {
        const float2 f = __half22float2(sz);
        float2 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 c = __half22float2(r[k]);
            v[k] = make_float2(fmaf(c.x, f.x, f.y), fmaf(c.y, f.x, f.y));
        }
        o[0] = kv4_pack2<true>(v[0].x, v[1].x);
        o[1] = kv4_pack2<true>(v[2].x, v[3].x);
        o[2] = kv4_pack2<true>(v[0].y, v[1].y);
        o[3] = kv4_pack2<true>(v[2].y, v[3].y);
    } else {
        // One rounding: code * scale + zero is a single fp16 multiply-add.
        uint32_t v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __half2 y = __hfma2(r[k], __low2half2(sz), __high2half2(sz));
            v[k] = *reinterpret_cast<const uint32_t*>(&y);
        }
        o[0] = __byte_perm(v[0], v[1], 0x5410);
        o[1] = __byte_perm(v[2], v[3], 0x5410);
        o[2] = __byte_perm(v[0], v[1], 0x7632);
        o[3] = __byte_perm(v[2], v[3], 0x7632);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool BF16, int NG>
__global__ void __launch_bounds__(CACHE_THREADS) kv4_gather_kernel(const CacheArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, kv = lane >> 4, i = lane & 15;
    const unsigned warps = gridDim.x * (CACHE_THREADS / 32), heads = a.Hkv;
    const unsigned pairs = static_cast<unsigned>(a.N) * heads;
    uint4* dst = static_cast<uint4*>(const_cast<void*>(kv ? a.v : a.k)) + i;
    bool bad = false;
    for (unsigned u = (blockIdx.x * (CACHE_THREADS / 32) + (threadIdx.x >> 5)) * CACHE_UNROLL; u < pairs;
         u += warps * CACHE_UNROLL) {
        uint32_t codes[CACHE_UNROLL], pair[CACHE_UNROLL];
        int slot[CACHE_UNROLL];
        Pair p(u, heads), q = p;
#pragma unroll
        for (int x = 0; x < CACHE_UNROLL; ++x) {
            slot[x] = u + x < pairs ? __ldg(a.slots + p.n) : -1;
            p.next(heads);
        }
#pragma unroll
        for (int x = 0; x < CACHE_UNROLL; ++x) {
            const int s = checked_slot(slot[x], a.num_blocks, bad);
            // Code 0 of scale 0 and zero 0: a row of zeros.
            codes[x] = pair[x] = 0u;
            if (s >= 0) {
                const int t = s % KV4_BLOCK;
                const uint8_t* rec = a.pool + (static_cast<size_t>(s / KV4_BLOCK) * heads + q.h) * kv4_record(NG);
                codes[x] = __ldg(reinterpret_cast<const uint32_t*>(rec + (kv ? kv4_v_word(t, i) : kv4_k_word(t, i))));
                pair[x] = __ldg(reinterpret_cast<const uint32_t*>(rec + kv4_param(t, kv, NG, i / (16 / NG))));
            }
            q.next(heads);
        }
#pragma unroll
        for (int x = 0; x < CACHE_UNROLL; ++x)
            if (u + x < pairs) dst[static_cast<size_t>(u + x) * 16] = expand<BF16>(codes[x], pair[x]);
    }
    if (bad) report_error(a.err_flag, CLO_FLAG_BAD_INDEX);
}

using CacheKernel = void (*)(const CacheArgs);

static clo_status launch_cache(CacheKernel kernel, const CacheArgs& a, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0 || !prepare_kernel(reinterpret_cast<const void*>(kernel), 0)) return CLO_ERR_CUDA;
    const long long units = static_cast<long long>(a.N) * a.Hkv;
    constexpr int per_cta = CACHE_THREADS / 32 * CACHE_UNROLL;
    long long grid = (units + per_cta - 1) / per_cta;
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
    if (static_cast<long long>(N) * Hkv >= (1ll << 31) - (1 << 20) || num_blocks > (1 << 27)) return CLO_ERR_UNSUPPORTED;
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

extern "C" clo_status clo_kv4_append(const clo_kv4_append_args* args, cudaStream_t stream) {
    if (args == nullptr) return CLO_ERR_INVALID_ARG;
    const clo_kv4_append_args& r = *args;
    const clo_status st = check_cache(r.k, r.v, r.dtype, r.slot_map, r.N, r.Hkv, r.d, r.pool, r.num_blocks,
                                      r.block_size, r.group, r.err_flag);
    if (st != CLO_OK) return st;
    const long long row = static_cast<long long>(r.Hkv) * r.d;
    if (r.N > 1 && (r.k_stride < row || r.v_stride < row || r.k_stride % 8 != 0 || r.v_stride % 8 != 0 ||
                    r.k_stride > (1ll << 40) || r.v_stride > (1ll << 40)))
        return CLO_ERR_INVALID_ARG;
    if (r.N == 0) return CLO_OK;
    CacheArgs a{r.k, r.v, r.k_stride, r.v_stride, r.pool, r.slot_map, r.err_flag, r.N, r.Hkv, r.num_blocks};
    const int ng = kv4_groups(r.group);
    return launch_cache(r.dtype == CLO_BF16 ? append_kernel<true>(ng) : append_kernel<false>(ng), a, stream);
}

extern "C" clo_status clo_kv4_gather(const clo_kv4_gather_args* args, cudaStream_t stream) {
    if (args == nullptr) return CLO_ERR_INVALID_ARG;
    const clo_kv4_gather_args& r = *args;
    const clo_status st = check_cache(r.k, r.v, r.dtype, r.slot_map, r.N, r.Hkv, r.d, r.pool, r.num_blocks,
                                      r.block_size, r.group, r.err_flag);
    if (st != CLO_OK) return st;
    if (r.N == 0) return CLO_OK;
    CacheArgs a{r.k, r.v, 0, 0, const_cast<uint8_t*>(r.pool), r.slot_map, r.err_flag, r.N, r.Hkv, r.num_blocks};
    const int ng = kv4_groups(r.group);
    return launch_cache(r.dtype == CLO_BF16 ? gather_kernel<true>(ng) : gather_kernel<false>(ng), a, stream);
}
