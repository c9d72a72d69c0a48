// clo_paged_select.cu -- the range of each block's keys in 8-bit codes, and the
// blocks that a decode step selects by a score from those ranges.
//
// Mathematics.  For a query s and keys k_t of a block, s . k_t is at most the sum
// over channels of max(s_c * max_t k_tc, s_c * min_t k_tc).  With the ranges and
// the query as whole numbers of at most 127 in size the sum is a whole number
// below 2^24, the same in any order, and one product with the block's scale (a
// single rounding) makes the score.  So a selection depends on its inputs alone,
// not on the split of the work, and equal scores are exactly equal.  A positive
// code meets the largest keys, a negative one the smallest: with the query's
// positive and negative codes apart, each a word of four bytes, the sum is two
// dp4a for every four channels.
#include <math.h>

#include "clo_kv4_math.cuh"  // barriers and bulk copies
#include "clo_paged.cuh"

namespace clo {

// ---------------------------------------------------------------- bounds
// A warp reads a block of one KV head once, 4 KB in 16-byte loads that are all in flight
// together, and writes its record.  65531 tokens of 8 KV heads (134 MB) take 31 us,
// 4.3 TB/s: about 450 instructions a block (16 quotients of a lane pair in fp32 among them)
// and HBM share the time.  Warps that went through several blocks with the next one's
// rows on their way were no faster.

constexpr int BOUNDS_THREADS = 128;

struct BoundsArgs {
    const uint8_t* kc;
    const int32_t* slots;
    uint8_t* bounds;
    int32_t* err_flag;
    int N, Hkv, num_blocks, tokens;  // tokens a warp looks at
};

template <bool BF16>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <bool BF16>
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (BF16) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ int code_of(float x, float div, bool up) {
    const float c = __fdiv_rn(x, div);
    return static_cast<int>(fminf(fmaxf(up ? ceilf(c) : floorf(c), -127.f), 127.f));
}

// The record of one block and head, of its first `count` rows, by a warp: lanes i
// and i + 16 take 16-byte chunk i of the even and of the odd rows.
template <bool BF16>
__device__ __forceinline__ void block_record(const uint8_t* rows, int count, uint8_t* rec, int lane) {
    const int i = lane & 15, odd = lane >> 4;
    uint4 r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        // Rows past the end repeat the first one, which is always there.
        const int row = 2 * j + odd < count ? 2 * j + odd : 0;
        r[j] = *reinterpret_cast<const uint4*>(rows + row * PG_ROW + 16 * i);
    }
    uint32_t hi[4] = {r[0].x, r[0].y, r[0].z, r[0].w}, lo[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
    for (int j = 1; j < 8; ++j) {
        const uint32_t w[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            hi[c] = max2_nan<BF16>(hi[c], w[c]);
            lo[c] = min2_nan<BF16>(lo[c], w[c]);
        }
    }
    float2 top[4], low[4];
    float m = 0.f;
    bool finite = true;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        hi[c] = max2_nan<BF16>(hi[c], __shfl_xor_sync(FULL_MASK, hi[c], 16));
        lo[c] = min2_nan<BF16>(lo[c], __shfl_xor_sync(FULL_MASK, lo[c], 16));
        top[c] = pg_unpack<BF16>(hi[c]);
        low[c] = pg_unpack<BF16>(lo[c]);
        finite &= pg_finite(top[c].x) && pg_finite(top[c].y) && pg_finite(low[c].x) && pg_finite(low[c].y);
        m = fmaxf(m, fmaxf(fmaxf(fabsf(top[c].x), fabsf(top[c].y)), fmaxf(fabsf(low[c].x), fabsf(low[c].y))));
    }
    finite = __all_sync(FULL_MASK, finite);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, off));
    const float scale = finite ? __fdiv_rn(m, 127.f) : INFINITY;
    const float div = scale > 0.f ? scale : 1.f;
    // The lower lanes make the codes of the largest keys, the upper ones those of the smallest.
    uint32_t w[2] = {0u, 0u};  // of channels 8i .. 8i + 3 and 8i + 4 .. 8i + 7
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const float2 a = odd == 0 ? top[2 * x] : low[2 * x], b = odd == 0 ? top[2 * x + 1] : low[2 * x + 1];
        if (finite)
            w[x] = (code_of(a.x, div, odd == 0) & 0xff) | (code_of(a.y, div, odd == 0) & 0xff) << 8 |
                   (code_of(b.x, div, odd == 0) & 0xff) << 16 | static_cast<uint32_t>(code_of(b.y, div, odd == 0) & 0xff) << 24;
    }
    const uint32_t l0 = __shfl_xor_sync(FULL_MASK, w[0], 16), l1 = __shfl_xor_sync(FULL_MASK, w[1], 16);
    if (odd == 0) *reinterpret_cast<uint4*>(rec + 16 * i) = make_uint4(w[0], l0, w[1], l1);
    if (lane == 16) *reinterpret_cast<uint4*>(rec + 256) = make_uint4(__float_as_uint(scale), 0u, 0u, 0u);
}

template <bool BF16>
__global__ void __launch_bounds__(BOUNDS_THREADS) block_bounds_kernel(const BoundsArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long first = (blockIdx.x * static_cast<long long>(BOUNDS_THREADS / 32) + (threadIdx.x >> 5)) * a.tokens;
    const int h = blockIdx.y;
    // Lane l looks at token first + l: is it the last of its block?
    const long long n = first + lane;
    int slot = -1;
    bool last = false, bad = false;
    if (lane < a.tokens && n < a.N) {
        slot = a.slots[n];
        const int next = n + 1 < a.N ? a.slots[n + 1] : -1;
        bad = slot >= 0 && slot >= a.num_blocks * PG_BLOCK;
        last = slot >= 0 && !bad && (slot % PG_BLOCK == PG_BLOCK - 1 || next != slot + 1);
    }
    unsigned todo = __ballot_sync(FULL_MASK, last);
    while (todo != 0) {
        const int s = __shfl_sync(FULL_MASK, slot, __ffs(todo) - 1);
        todo &= todo - 1;
        const size_t at = static_cast<size_t>(s / PG_BLOCK) * a.Hkv + h;
        block_record<BF16>(a.kc + at * PG_BLOCK_BYTES, s % PG_BLOCK + 1, a.bounds + at * PG_RECORD, lane);
    }
    if (bad && h == 0) report_error(a.err_flag, CLO_FLAG_BAD_INDEX);
}

// ---------------------------------------------------------------- scores

constexpr int SCORE_THREADS = 256;
constexpr int SCORE_COLS = SCORE_THREADS / 8;    // columns a CTA scores: 8 lanes a column
constexpr int SCORE_HEADS = 8;                   // KV heads a CTA scores, at most
// Above every score's key: a block that has none, and above those the first and last ones,
// for which n_sel always has room.
constexpr uint32_t KEY_ALWAYS = 0xfffffffeu, KEY_FORCED = 0xffffffffu;

struct SelectArgs {
    const void* q;
    const uint8_t* bounds;
    const int32_t* table;
    const int32_t* ctx_len;
    uint32_t* keys;  // [B * Hkv][key_stride]
    int32_t* sel;
    int32_t* err_flag;
    int Hq, Hkv, G, num_blocks, max_blocks, n_sel, n_first, n_last, key_stride;
};

// The blocks of a request, or -1 for a bad length.
__device__ __forceinline__ int select_blocks(const SelectArgs& a, int r) {
    const int ctx = a.ctx_len[r];
    return ctx < 0 || ctx > a.max_blocks * PG_BLOCK ? -1 : (ctx + PG_BLOCK - 1) / PG_BLOCK;
}

// Unsigned keys in the order of finite floats (-0 as 0); +inf gives KEY_ALWAYS.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x == INFINITY) return KEY_ALWAYS;
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// 32 columns of one request and up to 8 KV heads a CTA.  HBM-bound (272 bytes a record).  A
// block's heads lie side by side: one bulk copy a column brings its records, all 32 at
// once, while the queries' codes are made; then 8 lanes sum up a record.  Three CTAs share
// an SM.  (Loads of 16 bytes a lane into registers had half the bandwidth: a record is not
// a multiple of a sector, and the registers hold too few of them.)
template <bool BF16>
__global__ void __launch_bounds__(SCORE_THREADS, 3) block_score_kernel(const SelectArgs a) {
    extern __shared__ __align__(16) uint8_t records[];  // [SCORE_COLS][heads][PG_RECORD]
    __shared__ __align__(16) uint32_t codes[SCORE_HEADS][2][PG_D / 4];  // positive, negative
    __shared__ unsigned long long bar;
    const uint32_t b = smem_u32(&bar);
    if (threadIdx.x == 0) {
        mbar_init(b);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    const int head_groups = (a.Hkv + SCORE_HEADS - 1) / SCORE_HEADS;
    const int r = blockIdx.y / head_groups, g0 = blockIdx.y % head_groups * SCORE_HEADS;
    const int heads = min(SCORE_HEADS, a.Hkv - g0), bytes = heads * PG_RECORD;
    const int first = blockIdx.x * SCORE_COLS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, u = threadIdx.x & 7;
    // (The table's entry and the length come together; an entry behind the length is not used.)
    int id = -1;
    if (warp == 0 && first + lane < a.max_blocks) id = a.table[static_cast<size_t>(r) * a.max_blocks + first + lane];
    const int nb = select_blocks(a, r);
    if (nb < 0 && blockIdx.x == 0 && threadIdx.x == 0) report_error(a.err_flag, CLO_FLAG_BAD_CTX);
    if (nb <= a.n_sel || first >= nb) return;  // all blocks are selected: no scores
    if (warp == 0) {
        const bool there = first + lane < nb, ok = there && id >= 0 && id < a.num_blocks;
        const unsigned copies = __popc(__ballot_sync(FULL_MASK, ok));
        if (lane == 0) mbar_expect(b, copies * bytes);
        __syncwarp();
        uint8_t* to = records + lane * bytes;
        if (ok) {
            bulk_load(smem_u32(to), a.bounds + (static_cast<size_t>(id) * a.Hkv + g0) * PG_RECORD, bytes, b, l2_evict_first_policy());
        } else if (there) {  // a bad block counts as one without a score
            report_error(a.err_flag, CLO_FLAG_BAD_INDEX);
            for (int h = 0; h < heads; ++h) *reinterpret_cast<float*>(to + h * PG_RECORD + 256) = INFINITY;
        }
    }
    // The queries' codes: a warp a KV head, a lane four channels; the group's heads added up
    // in order.
    if (warp < heads) {
        const uint2* q = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) +
                                                        (static_cast<size_t>(r) * a.Hq + static_cast<size_t>(g0 + warp) * a.G) * PG_D) + lane;
        uint2 w[PG_MAX_G];
#pragma unroll
        for (int h = 0; h < PG_MAX_G; ++h)
            if (h < a.G) w[h] = q[h * (PG_D / 4)];
        float s[4];
#pragma unroll
        for (int h = 0; h < PG_MAX_G; ++h)
            if (h < a.G) {
                const float2 x = pg_unpack<BF16>(w[h].x), y = pg_unpack<BF16>(w[h].y);
                s[0] = h == 0 ? x.x : s[0] + x.x;
                s[1] = h == 0 ? x.y : s[1] + x.y;
                s[2] = h == 0 ? y.x : s[2] + y.x;
                s[3] = h == 0 ? y.y : s[3] + y.y;
            }
        bool finite = pg_finite(s[0]) && pg_finite(s[1]) && pg_finite(s[2]) && pg_finite(s[3]);
        finite = __all_sync(FULL_MASK, finite);
        float m = fmaxf(fmaxf(fabsf(s[0]), fabsf(s[1])), fmaxf(fabsf(s[2]), fabsf(s[3])));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, off));
        const float step = __fdiv_rn(m, 127.f);
        uint32_t pos = 0u, neg = 0u;
        if (finite && step > 0.f) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int code = static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(s[c], step)), -127.f), 127.f));
                pos |= static_cast<uint32_t>(max(code, 0)) << (8 * c);
                neg |= (static_cast<uint32_t>(min(code, 0)) & 0xffu) << (8 * c);
            }
        }
        codes[warp][0][lane] = pos;
        codes[warp][1][lane] = neg;
    }
    __syncthreads();
    if (!mbar_wait(b, 0)) {  // once more, so that no copy comes after the CTA's end
        if (lane == 0) report_error(a.err_flag, CLO_FLAG_TIMEOUT);
        mbar_wait(b, 0);
    }
    const int col = first + (threadIdx.x >> 3);
    const uint8_t* rec = records + (threadIdx.x >> 3) * bytes;
#pragma unroll 2
    for (int h = 0; h < heads; ++h, rec += PG_RECORD) {
        int sum = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // channels 8u .. 8u + 7, then 64 + 8u ..
            const uint4 x = *reinterpret_cast<const uint4*>(rec + 128 * i + 16 * u);
            const uint2 qp = *reinterpret_cast<const uint2*>(&codes[h][0][16 * i + 2 * u]);
            const uint2 qn = *reinterpret_cast<const uint2*>(&codes[h][1][16 * i + 2 * u]);
            sum = __dp4a(static_cast<int>(x.x), static_cast<int>(qp.x), sum);
            sum = __dp4a(static_cast<int>(x.y), static_cast<int>(qn.x), sum);
            sum = __dp4a(static_cast<int>(x.z), static_cast<int>(qp.y), sum);
            sum = __dp4a(static_cast<int>(x.w), static_cast<int>(qn.y), sum);
        }
        sum += __shfl_xor_sync(FULL_MASK, sum, 4);
        sum += __shfl_xor_sync(FULL_MASK, sum, 2);
        sum += __shfl_xor_sync(FULL_MASK, sum, 1);
        if (u == 0 && col < nb) {
            const float scale = *reinterpret_cast<const float*>(rec + 256);
            const bool forced = col < a.n_first || col >= nb - a.n_last;
            a.keys[(static_cast<size_t>(r) * a.Hkv + g0 + h) * a.key_stride + col] =
                forced ? KEY_FORCED : !pg_finite(scale) ? KEY_ALWAYS : score_key(static_cast<float>(sum) * scale);
        }
    }
}

// ---------------------------------------------------------------- selection

constexpr int PICK_THREADS = 1024;
constexpr int PICK_WARPS = PICK_THREADS / 32;
constexpr int PICK_HELD = 8;                             // neighbouring keys a thread takes in a round
constexpr int PICK_ROUND = PICK_THREADS * PICK_HELD;     // columns of a round: 128K tokens
constexpr int PICK_BITS = 11;                            // of a digit: 11, 11 and 10
constexpr int PICK_BINS = 1 << PICK_BITS;

// Sum of x over the threads before this one, and over all (in `total`).
__device__ __forceinline__ int scan_threads(int x, int* warp_sum, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(FULL_MASK, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int w = warp_sum[lane];  // PICK_WARPS == 32
    int all = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(FULL_MASK, all, off);
        if (lane >= off) all += v;
    }
    total = __shfl_sync(FULL_MASK, all, 31);
    const int before = __shfl_sync(FULL_MASK, all - w, warp);
    __syncthreads();  // warp_sum may be written again
    return before + incl - x;
}

// One CTA a (request, KV head).  The n_sel-th largest key is found digit by digit
// (three passes that count the keys that agree with the digits found so far by their next
// one); then the keys above it, and of the equal ones the first, are written in the
// order of the columns.  Up to 8192 columns stay in registers; latency bounds it.
__global__ void __launch_bounds__(PICK_THREADS) block_pick_kernel(const SelectArgs a) {
    __shared__ int hist[PICK_BINS];
    __shared__ int warp_sum[PICK_WARPS];
    __shared__ int found[2];  // digit, keys above it
    static_assert(PICK_WARPS == 32 && PICK_BINS == 2 * PICK_THREADS, "");
    pdl_launch_dependents();
    pdl_wait();
    const int r = blockIdx.x / a.Hkv;
    const int nb = max(select_blocks(a, r), 0);
    int32_t* sel = a.sel + static_cast<size_t>(blockIdx.x) * a.n_sel;
    const int tid = threadIdx.x;
    if (nb <= a.n_sel) {
        for (int i = tid; i < a.n_sel; i += PICK_THREADS) sel[i] = i < nb ? i : -1;
        return;
    }
    const uint32_t* keys = a.keys + static_cast<size_t>(blockIdx.x) * a.key_stride;
    uint32_t key[PICK_HELD];
    const auto load = [&](int base) {  // this thread's keys of a round; a row of keys is padded to 8
#pragma unroll
        for (int j = 0; j < PICK_HELD; j += 4) {
            const int i = base + tid * PICK_HELD + j;
            const uint4 v = i < nb ? *reinterpret_cast<const uint4*>(keys + i) : make_uint4(0u, 0u, 0u, 0u);
            key[j] = v.x;
            key[j + 1] = v.y;
            key[j + 2] = v.z;
            key[j + 3] = v.w;
        }
    };
    const bool once = nb <= PICK_ROUND;
    if (once) load(0);
    uint32_t prefix = 0u;
    int want = a.n_sel;  // how many of the keys that agree with the prefix are selected
#pragma unroll 1
    for (int top = 32; top > 0; top -= PICK_BITS) {  // bits top - width .. top - 1
        const int width = min(PICK_BITS, top), shift = top - width;
        const uint32_t mask = (1u << width) - 1u;
        hist[tid] = 0;
        hist[tid + PICK_THREADS] = 0;
        __syncthreads();
#pragma unroll 1
        for (int base = 0; base < nb; base += PICK_ROUND) {
            if (!once) load(base);
#pragma unroll
            for (int j = 0; j < PICK_HELD; ++j)
                if (base + tid * PICK_HELD + j < nb && (top == 32 || (key[j] >> top) == (prefix >> top)))
                    atomicAdd(&hist[(key[j] >> shift) & mask], 1);
        }
        __syncthreads();
        // Thread t has the bins 2047 - 2t and 2046 - 2t: the largest digits first.
        const int hi = PICK_BINS - 1 - 2 * tid, n_hi = hist[hi], n_lo = hist[hi - 1];
        int total;
        const int above = scan_threads(n_hi + n_lo, warp_sum, total);
        if (above < want && above + n_hi >= want) {
            found[0] = hi;
            found[1] = above;
        } else if (above + n_hi < want && above + n_hi + n_lo >= want) {
            found[0] = hi - 1;
            found[1] = above + n_hi;
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(found[0]) << shift;
        want -= found[1];
    }
    int above = 0, equal = 0;  // keys above and equal ones in earlier rounds
#pragma unroll 1
    for (int base = 0; base < nb; base += PICK_ROUND) {
        if (!once) load(base);
        int n_gt = 0, n_eq = 0;
#pragma unroll
        for (int j = 0; j < PICK_HELD; ++j) {
            const bool in = base + tid * PICK_HELD + j < nb;
            n_gt += in && key[j] > prefix;
            n_eq += in && key[j] == prefix;
        }
        // Both counts are below 2^14 in a round.
        int total;
        const int before = scan_threads(n_gt << 16 | n_eq, warp_sum, total);
        int g0 = above + (before >> 16), e0 = equal + (before & 0xffff);
#pragma unroll
        for (int j = 0; j < PICK_HELD; ++j) {
            const int i = base + tid * PICK_HELD + j;
            if (i >= nb) break;
            if (key[j] > prefix || (key[j] == prefix && e0 < want)) sel[g0 + min(e0, want)] = i;
            g0 += key[j] > prefix;
            e0 += key[j] == prefix;
        }
        above += total >> 16;
        equal += total & 0xffff;
    }
}

}  // namespace clo

using namespace clo;

extern "C" size_t clo_paged_bounds_bytes(int block_size, int d) {
    return block_size == PG_BLOCK && d == PG_D ? PG_RECORD : 0;
}

extern "C" clo_status clo_paged_block_bounds(const clo_paged_block_bounds_args* args, cudaStream_t stream) {
    if (args == nullptr) return CLO_ERR_INVALID_ARG;
    const clo_paged_block_bounds_args& r = *args;
    if (r.N < 0 || r.Hkv < 1 || r.num_blocks < 1 || !pg_dtype_ok(r.dtype)) return CLO_ERR_INVALID_ARG;
    if (r.N > 0 && (r.kc == nullptr || r.slot_map == nullptr || r.bounds == nullptr)) return CLO_ERR_INVALID_ARG;
    if (!pg_aligned(r.kc, 16) || !pg_aligned(r.bounds, 16) || !pg_aligned(r.slot_map, 4) || !pg_aligned(r.err_flag, 4))
        return CLO_ERR_INVALID_ARG;
    if (r.d != PG_D || r.block_size != PG_BLOCK || r.Hkv > 65535 || r.num_blocks > (1 << 26)) return CLO_ERR_UNSUPPORTED;
    if (r.N == 0) return CLO_OK;
    BoundsArgs a{static_cast<const uint8_t*>(r.kc), r.slot_map, r.bounds, r.err_flag, r.N, r.Hkv, r.num_blocks, 0};
    // A warp looks at 16 tokens, about one block of a prompt; at one where that leaves few
    // warps, for the sake of a decode step, in which each token ends a block.  Us with 1 and
    // with 16 tokens a warp, by tokens times heads (1, 8 or 32 heads, the same within 2%):
    //   a token a block   2048: 3.3, 16.2   16384: 8.6, 19.1   32768: 16.6, 33   65536: 39, 51   131072: 74, 79
    //   a prompt          2048: 2.2, 2.1    16384: 4.8, 2.6    32768: 9.1, 3.4   65536: 17, 4.3  131072: 34, 5.5
    a.tokens = static_cast<long long>(r.N) * r.Hkv <= 32768 ? 1 : 16;
    const long long warps = (static_cast<long long>(r.N) + a.tokens - 1) / a.tokens;
    const unsigned grid = static_cast<unsigned>((warps + BOUNDS_THREADS / 32 - 1) / (BOUNDS_THREADS / 32));
    const auto kernel = r.dtype == CLO_BF16 ? block_bounds_kernel<true> : block_bounds_kernel<false>;
    if (!prepare_kernel(reinterpret_cast<const void*>(kernel), 0)) return CLO_ERR_CUDA;
    return launch_pdl(kernel, dim3(grid, r.Hkv), dim3(BOUNDS_THREADS), 0, stream, a) == cudaSuccess ? CLO_OK
                                                                                                   : CLO_ERR_CUDA;
}

static bool select_sizes_ok(int B, int Hkv, int max_blocks) {
    return B >= 0 && B <= PG_MAX_B && Hkv >= 1 && max_blocks >= 1 && max_blocks <= (1 << 20) &&
           static_cast<long long>(B) * Hkv <= 65535 && static_cast<long long>(B) * Hkv * max_blocks < (1ll << 31);
}

// Keys of a row, padded for 16-byte loads.
static int key_stride(int max_blocks) { return (max_blocks + 7) / 8 * 8; }

extern "C" size_t clo_paged_select_workspace_size(int B, int Hkv, int max_blocks) {
    if (!select_sizes_ok(B, Hkv, max_blocks)) return 0;
    return static_cast<size_t>(B) * Hkv * key_stride(max_blocks) * sizeof(uint32_t) + 16;
}

extern "C" clo_status clo_paged_block_select(const clo_paged_block_select_args* args, cudaStream_t stream) {
    if (args == nullptr) return CLO_ERR_INVALID_ARG;
    const clo_paged_block_select_args& r = *args;
    if (r.B < 0 || r.Hq < 1 || r.Hkv < 1 || r.Hq % r.Hkv != 0 || r.num_blocks < 1 || r.max_blocks < 1 || r.n_sel < 1 ||
        r.n_first < 0 || r.n_last < 0 || r.n_first > r.n_sel - r.n_last || !pg_dtype_ok(r.dtype))
        return CLO_ERR_INVALID_ARG;
    if (r.B > 0 && (r.q == nullptr || r.bounds == nullptr || r.block_table == nullptr || r.ctx_len == nullptr || r.sel == nullptr))
        return CLO_ERR_INVALID_ARG;
    if (!pg_aligned(r.q, 16) || !pg_aligned(r.bounds, 16) || !pg_aligned(r.block_table, 4) || !pg_aligned(r.ctx_len, 4) ||
        !pg_aligned(r.sel, 4) || !pg_aligned(r.err_flag, 4))
        return CLO_ERR_INVALID_ARG;
    if (r.d != PG_D || r.block_size != PG_BLOCK || r.Hq / r.Hkv > PG_MAX_G || r.num_blocks > (1 << 26) || r.n_sel > (1 << 20) ||
        !select_sizes_ok(r.B, r.Hkv, r.max_blocks))
        return CLO_ERR_UNSUPPORTED;
    if (r.B == 0) return CLO_OK;
    if (r.workspace == nullptr || r.ws_bytes < clo_paged_select_workspace_size(r.B, r.Hkv, r.max_blocks) ||
        !pg_aligned(r.workspace, 16))
        return CLO_ERR_WORKSPACE;
    const SelectArgs a{r.q, r.bounds, r.block_table, r.ctx_len, static_cast<uint32_t*>(r.workspace), r.sel, r.err_flag,
                       r.Hq, r.Hkv, r.Hq / r.Hkv, r.num_blocks, r.max_blocks, r.n_sel, r.n_first, r.n_last, key_stride(r.max_blocks)};
    const auto score = r.dtype == CLO_BF16 ? block_score_kernel<true> : block_score_kernel<false>;
    const int smem = SCORE_COLS * min(r.Hkv, SCORE_HEADS) * PG_RECORD;
    if (!prepare_kernel(reinterpret_cast<const void*>(score), smem) ||
        !prepare_kernel(reinterpret_cast<const void*>(block_pick_kernel), 0))
        return CLO_ERR_CUDA;
    const unsigned sets = static_cast<unsigned>(r.B) * r.Hkv;
    const unsigned head_groups = static_cast<unsigned>(r.Hkv + SCORE_HEADS - 1) / SCORE_HEADS;
    if (launch_pdl(score, dim3((r.max_blocks + SCORE_COLS - 1) / SCORE_COLS, r.B * head_groups), dim3(SCORE_THREADS), smem,
                   stream, a) !=
        cudaSuccess)
        return CLO_ERR_CUDA;
    return launch_pdl(block_pick_kernel, dim3(sets), dim3(PICK_THREADS), 0, stream, a) == cudaSuccess ? CLO_OK : CLO_ERR_CUDA;
}
