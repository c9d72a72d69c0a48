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
// rows of 4 (token, head)s in flight: of one token where the heads divide by 4
// (one slot and one address for all), else 2 heads of 2 tokens or 1 of 4.  The
// rows are loaded without waiting for their slots, and fp32 work is done on
// pairs (the f32x2 instructions).
#include "clo_kv4.cuh"

namespace clo {

constexpr int CACHE_THREADS = 256;
// CTAs an SM (registers: up to 42, and 42 or 32 a thread).  A warp
// takes one group and ends: a grid of one wave whose warps loop measured 8%
// slower on 128K tokens of 8 heads.
constexpr int APPEND_CTAS = 6;
constexpr int gather_ctas(int heads) { return heads == 4 ? 8 : 6; }
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

// Smaller and larger of pairs of 16-bit values of the input's type; NaN where
// there is a NaN.
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

template <bool BF16>
__device__ __forceinline__ uint32_t most2(uint32_t a, uint32_t b) {
    if constexpr (BF16) {
        const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                             *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    } else {
        const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
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
    const uint32_t up = SIGNS ^ most2<BF16>(most2<BF16>(w[0], w[1]), most2<BF16>(w[2], w[3]));
    uint32_t ends = least2<BF16>(__byte_perm(lo, up, 0x5410), __byte_perm(lo, up, 0x7632));
#pragma unroll
    for (int o = 1; o < 16 / NG; o <<= 1) ends = least2<BF16>(ends, __shfl_xor_sync(FULL_MASK, ends, o));
    const float2 e = kv4_unpack2<BF16>(ends);
    float least = e.x, most = -e.y;
    bool finite = true, clamp = false;
    uint32_t zero_h = ends & 0xffffu;
    if (BF16) {
        finite = fabsf(least) < INFINITY && fabsf(most) < INFINITY;
        clamp = least < -65504.f || most > 65504.f;
        least = fminf(fmaxf(least, -65504.f), 65504.f);
        most = fminf(fmaxf(most, -65504.f), 65504.f);
        zero_h = __half_as_ushort(__float2half_rd(least));
    }
    const float zero = BF16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(zero_h))) : least;
    // Rounded up, so that below, where 15 times an fp16 value (exact in fp32)
    // is compared with it, the answer is the exact difference's.
    const float reach = __fsub_ru(most, zero);
    if (!BF16) finite = reach < INFINITY;  // no: infinite or NaN
    // The fp16 value next to reach / 15, moved up if it is below it.
    __half scale_h = __float2half_rn(reach * (1.f / 15.f));
    if (15.f * __half2float(scale_h) < reach)
        scale_h = __ushort_as_half(static_cast<unsigned short>(__half_as_ushort(scale_h) + 1));
    const float scale = __half2float(scale_h);
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
    inv = fminf(inv, 0x1p126f);  // scale 0: every element is the zero
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
    pair = finite ? static_cast<uint32_t>(__half_as_ushort(scale_h)) | (zero_h << 16) : 0x7fff7fffu;
}

// Where a lane's word of codes and its group's pair lie in a record.
struct LaneAt {
    int word, flip, pair;
    __device__ __forceinline__ LaneAt(int kv, int i, int ng)
        : word(kv ? kv4_v_word(0, i) : kv4_k_word(0, i)), flip(kv ? 0x30 : 0), pair(kv4_param(0, kv, ng, i * ng / 16)) {}
    // Token t's: the chunks of a V row change places with t, by an exclusive or.
    __device__ __forceinline__ int word_of(int t) const { return t * KV4_ROW + (word ^ ((t << 3) & flip)); }
    __device__ __forceinline__ int pair_of(int t, int ng) const { return t * 8 * ng + pair; }
};

// A warp's group of (token, head)s: T tokens from n on, H heads from h on.
template <int H>
struct Group {
    static constexpr int T = CACHE_UNROLL / H;
    unsigned n, h;
    __device__ __forceinline__ Group(unsigned u, unsigned heads) {
        const unsigned per_token = heads / H, q = u / per_token;
        n = q * T;
        h = (u - q * per_token) * H;
    }
    static __host__ __device__ long long count(long long N, int heads) { return (N + T - 1) / T * (heads / H); }
};

template <bool BF16, int NG, int H>
__global__ void __launch_bounds__(CACHE_THREADS, APPEND_CTAS) kv4_append_kernel(const CacheArgs a) {
    constexpr int T = Group<H>::T, R = kv4_record(NG);
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, kv = lane >> 4, i = lane & 15;
    const LaneAt lane_at(kv, i, NG);
    const unsigned heads = a.Hkv, N = a.N;
    const unsigned u = blockIdx.x * (CACHE_THREADS / 32) + (threadIdx.x >> 5);
    if (u >= static_cast<unsigned>(Group<H>::count(N, heads))) return;
    const uint8_t* src = static_cast<const uint8_t*>(kv ? a.v : a.k) + 16 * i;
    const long long stride = 2 * (kv ? a.v_stride : a.k_stride);
    const size_t block_bytes = static_cast<size_t>(heads) * R;
    bool bad = false;
    const Group<H> g(u, heads);
    uint4 raw[T][H];
    int slot[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
        slot[t] = -1;
        if (g.n + t < N) {
            slot[t] = a.slots[g.n + t];
            const uint8_t* row = src + (g.n + t) * stride + g.h * (2 * KV4_D);
#pragma unroll
            for (int x = 0; x < H; ++x) raw[t][x] = ld_stream(row + x * (2 * KV4_D));
        }
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int s = checked_slot(slot[t], a.num_blocks, bad);
        if (s < 0) continue;  // the whole warp
        uint8_t* rec = a.pool + (s / KV4_BLOCK) * block_bytes + g.h * R;
        uint32_t* word = reinterpret_cast<uint32_t*>(rec + lane_at.word_of(s % KV4_BLOCK));
        uint32_t* params = reinterpret_cast<uint32_t*>(rec + lane_at.pair_of(s % KV4_BLOCK, NG));
#pragma unroll
        for (int x = 0; x < H; ++x) {
            uint32_t codes, pair;
            quantise<BF16, NG>(raw[t][x], codes, pair);
            word[x * (R / 4)] = codes;
            if (i % (16 / NG) == 0) params[x * (R / 4)] = pair;
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
        // One rounding: code * scale + zero is a single fp16 multiply-add.  Then
        // the values past fp16's largest (the scale is rounded up) are that.
        const __half2 top = __float2half2_rn(65504.f);
        uint32_t v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            __half2 y = __hfma2(r[k], __low2half2(sz), __high2half2(sz));
            y = __hmax2_nan(__hmin2_nan(y, top), __hneg2(top));
            v[k] = *reinterpret_cast<const uint32_t*>(&y);
        }
        o[0] = __byte_perm(v[0], v[1], 0x5410);
        o[1] = __byte_perm(v[2], v[3], 0x5410);
        o[2] = __byte_perm(v[0], v[1], 0x7632);
        o[3] = __byte_perm(v[2], v[3], 0x7632);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool BF16, int NG, int H>
__global__ void __launch_bounds__(CACHE_THREADS, gather_ctas(H)) kv4_gather_kernel(const CacheArgs a) {
    constexpr int T = Group<H>::T, R = kv4_record(NG);
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, kv = lane >> 4, i = lane & 15;
    const LaneAt lane_at(kv, i, NG);
    const unsigned heads = a.Hkv, N = a.N;
    const unsigned u = blockIdx.x * (CACHE_THREADS / 32) + (threadIdx.x >> 5);
    if (u >= static_cast<unsigned>(Group<H>::count(N, heads))) return;
    uint4* dst = static_cast<uint4*>(const_cast<void*>(kv ? a.v : a.k)) + i;
    const size_t block_bytes = static_cast<size_t>(heads) * R;
    bool bad = false;
    const Group<H> g(u, heads);
    uint32_t codes[T][H], pair[T][H];
    int slot[T];
#pragma unroll
    for (int t = 0; t < T; ++t) slot[t] = g.n + t < N ? a.slots[g.n + t] : -1;
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int s = checked_slot(slot[t], a.num_blocks, bad);
        const uint8_t* rec = a.pool + (max(s, 0) / KV4_BLOCK) * block_bytes + g.h * R;
        const int tok = max(s, 0) % KV4_BLOCK;
        const uint32_t* word = reinterpret_cast<const uint32_t*>(rec + lane_at.word_of(tok));
        const uint32_t* params = reinterpret_cast<const uint32_t*>(rec + lane_at.pair_of(tok, NG));
#pragma unroll
        for (int x = 0; x < H; ++x) {
            // Code 0 of scale 0 and zero 0: a row of zeros.
            codes[t][x] = s >= 0 ? word[x * (R / 4)] : 0u;
            pair[t][x] = s >= 0 ? params[x * (R / 4)] : 0u;
        }
    }
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int x = 0; x < H; ++x)
            if (g.n + t < N)
                dst[(static_cast<size_t>(g.n + t) * heads + g.h + x) * 16] = expand<BF16>(codes[t][x], pair[t][x]);
    if (bad) report_error(a.err_flag, CLO_FLAG_BAD_INDEX);
}

using CacheKernel = void (*)(const CacheArgs);

static clo_status launch_cache(CacheKernel kernel, long long groups, const CacheArgs& a, cudaStream_t stream) {
    if (!prepare_kernel(reinterpret_cast<const void*>(kernel), 0)) return CLO_ERR_CUDA;
    const long long grid = (groups + CACHE_THREADS / 32 - 1) / (CACHE_THREADS / 32);
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

template <bool BF16, int H>
static CacheKernel cache_kernel(bool append, int ng) {
    if (append)
        return ng == 1 ? kv4_append_kernel<BF16, 1, H> : ng == 2 ? kv4_append_kernel<BF16, 2, H>
                                                                 : kv4_append_kernel<BF16, 4, H>;
    return ng == 1 ? kv4_gather_kernel<BF16, 1, H> : ng == 2 ? kv4_gather_kernel<BF16, 2, H>
                                                             : kv4_gather_kernel<BF16, 4, H>;
}

template <int H>
static clo_status run_cache_heads(bool append, clo_dtype dtype, int ng, const CacheArgs& a, cudaStream_t stream) {
    return launch_cache(dtype == CLO_BF16 ? cache_kernel<true, H>(append, ng) : cache_kernel<false, H>(append, ng),
                        Group<H>::count(a.N, a.Hkv), a, stream);
}

static clo_status run_cache(bool append, clo_dtype dtype, int ng, const CacheArgs& a, cudaStream_t stream) {
    return a.Hkv % 4 == 0   ? run_cache_heads<4>(append, dtype, ng, a, stream)
           : a.Hkv % 2 == 0 ? run_cache_heads<2>(append, dtype, ng, a, stream)
                            : run_cache_heads<1>(append, dtype, ng, a, stream);
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
    return run_cache(true, r.dtype, kv4_groups(r.group), a, stream);
}

extern "C" clo_status clo_kv4_gather(const clo_kv4_gather_args* args, cudaStream_t stream) {
    if (args == nullptr) return CLO_ERR_INVALID_ARG;
    const clo_kv4_gather_args& r = *args;
    const clo_status st = check_cache(r.k, r.v, r.dtype, r.slot_map, r.N, r.Hkv, r.d, r.pool, r.num_blocks,
                                      r.block_size, r.group, r.err_flag);
    if (st != CLO_OK) return st;
    if (r.N == 0) return CLO_OK;
    CacheArgs a{r.k, r.v, 0, 0, const_cast<uint8_t*>(r.pool), r.slot_map, r.err_flag, r.N, r.Hkv, r.num_blocks};
    return run_cache(false, r.dtype, kv4_groups(r.group), a, stream);
}
