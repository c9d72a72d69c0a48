// clo_kv4_attention.cu -- clo_kv4_paged_decode_attn: decode attention over
// the paged cache held in 4 bits (format: clo_kv4.h).
//
// Mathematics.  With K = code * s + z a score splits into
//     q . K_t = sum_g s_tg (sum_{d in g} q_d code_td) + z_tg (sum_{d in g} q_d):
// the inner sums over codes are matrix products of 4-bit integers, the rest a
// multiply-add a group.  Likewise sum_t p_t V_t = sum_t (p_t s_tg) code_td +
// sum_t p_t z_tg.  So the matrix instructions run on the bare codes.
//   * A code in the low bits of a 16-bit lane *is* an fp16 number, code * 2^-24
//     (a subnormal), and 4 bits further up code * 2^-20: one AND turns a 32-bit
//     word into a pair of exact operands, no conversion and no subtraction.
//     The powers of two are taken out in fp32 afterwards (for K already in the
//     query, whose second half is stored as q / 16).
//   * The queries are scaled by a power of two a row so that their largest
//     element is near 2^13: exact, for bf16 too, but for elements some 2^-27 of
//     the largest.
//   * Online softmax with one reference a query row, the running maximum of
//     x_t + log2(largest V scale of t), x the score in log2 units.  The weights
//     p_t s_tg that are rounded to fp16 for the second product are then at most
//     1 and never all small, whatever the V scales are; l = sum p_t stays in
//     fp32 (p_t < 2^25 as an fp16 scale is at least 2^-24).
//
// Shape.  mma.sync m16n8k16 with 16 tokens on M and 8 query rows (of the
// G * n_q of a KV head) on N for the scores, then channels on M for the second
// product; the operands come out of registers because they are made there (a
// tcgen05 operand would have to be written back to shared memory in 16 bits,
// 4 times the bytes that were read).  The kernel is bound by HBM: at 24 bytes a
// clock and SM the codes need 0.19 of these instructions a clock and n8 tile.
//
// Work split.  A tile is the record of one block and KV head (2176 to 2560
// bytes, K, V and parameters together): one bulk copy.  All tiles of the call
// form one stream, ordered by request, head and position, cut into equal
// ranges, one a warp; each warp keeps a ring of records in flight.  A (request,
// KV head) that lies in one warp's range is finished by that warp alone.  What
// crosses ranges is merged once a CTA at its end, in shared memory, and what
// crosses CTAs leaves one fp32 partial a CTA, merged by a second kernel.  The
// split depends on the lengths alone, so the bits of a result do not depend on
// timing.
#include <math.h>

#include <algorithm>

#include "clo_kv4.cuh"

namespace clo {

constexpr int KV4_WARPS = 4;
constexpr int KV4_THREADS = KV4_WARPS * 32;
constexpr int KV4_STAGES = 4;      // records a warp has room for
constexpr int KV4_MAX_ROWS = 32;   // query rows of a KV head: G * n_q
constexpr int KV4_PIECE_ROW = KV4_D + 4;  // floats of a row of a piece; the four behind: m, l
constexpr int KV4_SMEM_PER_SM = 228 * 1024;  // 1 KB of it reserved for each CTA
constexpr long long KV4_WAIT_CLOCKS = 1ll << 32;  // about 2 s
constexpr uint32_t LOW_CODES = 0x000f000fu, HIGH_CODES = 0x00f000f0u;

// CTAs an SM for NT tiles of 8 query rows (registers: 128, 168, 255 a thread).
__host__ __device__ constexpr int kv4_ctas_per_sm(int nt) { return nt == 1 ? 4 : nt == 2 ? 3 : 2; }

struct Kv4Args {
    const void* q;
    void* out;
    float* lse;
    const uint8_t* pool;
    const int32_t* table;
    const int32_t* ctx_len;
    int32_t* err_flag;
    float* ws_o;    // [2 * CTAs][rows][128] partial sums, head piece and tail piece of each CTA
    float2* ws_ml;  // [2 * CTAs][rows] their (reference, denominator); denominator -1: bad data
    int2* ws_tail;  // [CTAs] (token set, CTAs it covers) of the set that starts in this CTA and goes on, or covers 0
    float scale_log2;
    int max_blocks, num_blocks, B, n_q, Hq, Hkv, G, rows;
};

__device__ __forceinline__ void mbar_init(uint32_t bar) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// False if the phase did not end within KV4_WAIT_CLOCKS.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
    if (mbar_try(bar, parity)) return true;
    const long long t0 = clock64();
    do {
        if (mbar_try(bar, parity)) return true;
    } while (clock64() - t0 < KV4_WAIT_CLOCKS);
    return false;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                          uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], "
        "%4;\n" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// Tiles of request r of one KV head; 0 if it is empty or its length is bad.
__device__ __forceinline__ int kv4_tiles(const Kv4Args& a, int r, bool& bad) {
    const int n = a.ctx_len[r];
    bad = n < 0 || n > a.max_blocks * KV4_BLOCK;
    return bad ? 0 : (n + KV4_BLOCK - 1) / KV4_BLOCK;
}

// prefix[r] = tiles of the requests before r (all heads), r <= B.
__device__ __forceinline__ void kv4_prefix(const Kv4Args& a, int* prefix, int* wsum) {
    const int per = (a.B + KV4_THREADS - 1) / KV4_THREADS;
    const int r0 = min(a.B, static_cast<int>(threadIdx.x) * per), r1 = min(a.B, r0 + per);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool bad, any_bad = false;
    int mine = 0;
    for (int r = r0; r < r1; ++r) {
        mine += kv4_tiles(a, r, bad) * a.Hkv;
        any_bad |= bad;
    }
    if (any_bad && blockIdx.x == 0) report_error(a.err_flag, CLO_FLAG_BAD_CTX);
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(FULL_MASK, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int run = incl - mine;
    for (int w = 0; w < warp; ++w) run += wsum[w];
    if (threadIdx.x == 0) prefix[0] = 0;
    for (int r = r0; r < r1; ++r) {
        run += kv4_tiles(a, r, bad) * a.Hkv;
        prefix[r + 1] = run;
    }
    __syncthreads();
}

// A position in the stream of tiles: tile j of nt of request r's head h.
struct Place {
    int r, h, j, nt;
};

__device__ __forceinline__ Place kv4_place(const int* prefix, int B, int Hkv, int t) {
    int lo = 0, hi = B - 1;  // the last request with prefix[r] <= t: skips empty ones
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= t) lo = mid; else hi = mid - 1;
    }
    Place p;
    p.r = lo;
    p.nt = (prefix[lo + 1] - prefix[lo]) / Hkv;
    p.h = (t - prefix[lo]) / p.nt;
    p.j = t - prefix[lo] - p.h * p.nt;
    return p;
}

// The next tile's place (one past the last tile: r == B, nt == 0).
__device__ __forceinline__ void kv4_next(const int* prefix, int B, int Hkv, Place& p) {
    if (++p.j < p.nt) return;
    p.j = 0;
    if (++p.h < Hkv) return;
    p.h = 0;
    do {
        ++p.r;
    } while (p.r < B && prefix[p.r + 1] == prefix[p.r]);
    p.nt = p.r < B ? (prefix[p.r + 1] - prefix[p.r]) / Hkv : 0;
}

// The queries of one KV head in the layout of the first product's B operand,
// and what their scores need in fp32.
template <int NT, int NG>
struct Queries {
    uint32_t b[NT][4][2][2];  // [n8 tile][word j][low, high codes][register]
    float unit[NT][2];        // fp32 factor of the code sums, columns 2c and 2c + 1
    float sum[NT][2][NG];     // sum of the group's elements (log2 units)
    int limit[NT][2];         // tokens behind the last one that the column does not see
};

template <bool BF16, int NT, int NG>
__device__ __forceinline__ void load_queries(const Kv4Args& a, const Place& p, int lane, Queries<NT, NG>& qs) {
    const int head = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int row = nt * 8 + head;
        const bool has = row < a.rows;
        const int qi = row / a.G, g = row - qi * a.G;
        const size_t at = (static_cast<size_t>(p.r) * a.n_q + qi) * a.Hq + static_cast<size_t>(p.h) * a.G + g;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.q) + at * KV4_D * 2);
        // This lane's channels: 32j + 8c .. + 7 for j = 0 .. 3.
        float x[4][8];
        float top = 0.f;
        float part[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 v = has ? __ldg(src + 4 * j + c) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            part[j] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = kv4_unpack2<BF16>(w[k]);
                x[j][2 * k] = f.x;
                x[j][2 * k + 1] = f.y;
                top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                part[j] += f.x + f.y;
            }
        }
        top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 1));
        top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 2));
        // 2^e brings the largest element into [2^12, 2^13); e is bounded so
        // that 2^e and the factor that undoes it are finite.
        int e = top > 0.f && top < INFINITY ? 12 - ilogbf(top) : 0;
        e = min(max(e, -100), 100);
        const float up = ldexpf(1.f, e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float* y = x[j];
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] *= up;
            qs.b[nt][j][0][0] = pack_half2(y[0], y[4]);
            qs.b[nt][j][0][1] = pack_half2(y[2], y[6]);
            qs.b[nt][j][1][0] = pack_half2(y[1] * 0.0625f, y[5] * 0.0625f);
            qs.b[nt][j][1][1] = pack_half2(y[3] * 0.0625f, y[7] * 0.0625f);
        }
        const float unit = ldexpf(a.scale_log2, 24 - e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            part[j] *= a.scale_log2;
            part[j] += __shfl_xor_sync(FULL_MASK, part[j], 1);
            part[j] += __shfl_xor_sync(FULL_MASK, part[j], 2);
        }
        float group[NG];
#pragma unroll
        for (int g2 = 0; g2 < NG; ++g2) {
            group[g2] = 0.f;
#pragma unroll
            for (int j = 0; j < 4 / NG; ++j) group[g2] += part[g2 * (4 / NG) + j];
        }
#pragma unroll
        for (int col = 0; col < 2; ++col) {
            const int from = (2 * c + col) * 4;
            qs.unit[nt][col] = __shfl_sync(FULL_MASK, unit, from);
#pragma unroll
            for (int g2 = 0; g2 < NG; ++g2) qs.sum[nt][col][g2] = __shfl_sync(FULL_MASK, group[g2], from);
            qs.limit[nt][col] = a.n_q - 1 - min(nt * 8 + 2 * c + col, a.rows - 1) / a.G;
        }
    }
}

// One warp's running softmax of a token set.
template <int NT, int NG>
struct Softmax {
    float m[NT][2];        // reference (log2 units) of columns 2c, 2c + 1
    float l[NT][2];        // this lane's share of sum p
    float z[NT][2][NG];    // this lane's share of sum p z_g
    float o[NT][4][2][4];  // sum p s code: [n8 tile][chunk][low, high codes][register]
};

template <int NT, int NG>
__device__ __forceinline__ void reset(Softmax<NT, NG>& w) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int col = 0; col < 2; ++col) {
            w.m[nt][col] = -INFINITY;
            w.l[nt][col] = 0.f;
#pragma unroll
            for (int g = 0; g < NG; ++g) w.z[nt][col][g] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int hl = 0; hl < 2; ++hl)
#pragma unroll
                for (int k = 0; k < 4; ++k) w.o[nt][c][hl][k] = 0.f;
    }
}

// Takes one record in.  EDGE: it holds tokens that some query does not see;
// `left` counts the tokens from its first one on.
template <int NT, int NG, bool EDGE>
__device__ __forceinline__ void take_tile(const uint8_t* rec, int left, const Queries<NT, NG>& qs,
                                          Softmax<NT, NG>& w, int lane) {
    const int gid = lane >> 2, c = lane & 3;
    // ---- scores of tokens gid and gid + 8 (rows), query rows 2c and 2c + 1 of each n8 tile
    const uint4 k0 = *reinterpret_cast<const uint4*>(rec + gid * KV4_ROW + c * 16);
    const uint4 k1 = *reinterpret_cast<const uint4*>(rec + (gid + 8) * KV4_ROW + c * 16);
    const uint32_t kw0[4] = {k0.x, k0.y, k0.z, k0.w}, kw1[4] = {k1.x, k1.y, k1.z, k1.w};
    float2 kp[2][NG], vp[2][NG];  // (scale, zero) of both tokens
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const uint32_t* par = reinterpret_cast<const uint32_t*>(rec + kv4_param(gid + 8 * t, 0, NG, 0));
        uint32_t raw[2 * NG];
        if constexpr (NG == 1) {
            const uint2 u = *reinterpret_cast<const uint2*>(par);
            raw[0] = u.x, raw[1] = u.y;
        } else {
#pragma unroll
            for (int k = 0; k < NG / 2; ++k) {
                const uint4 u = reinterpret_cast<const uint4*>(par)[k];
                raw[4 * k] = u.x, raw[4 * k + 1] = u.y, raw[4 * k + 2] = u.z, raw[4 * k + 3] = u.w;
            }
        }
        // What lies behind the last token may be anything, NaN among it.
        const bool there = !EDGE || gid + 8 * t < left;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const uint32_t rk = there ? raw[g] : 0u, rv = there ? raw[NG + g] : 0u;
            kp[t][g] = __half22float2(*reinterpret_cast<const __half2*>(&rk));
            vp[t][g] = __half22float2(*reinterpret_cast<const __half2*>(&rv));
        }
    }
    float x[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[nt][k] = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[nt][k] = 0.f;
#pragma unroll
        for (int jj = 0; jj < 4 / NG; ++jj) {
            const int j = g * (4 / NG) + jj;
            const uint32_t lo[4] = {kw0[j] & LOW_CODES, kw1[j] & LOW_CODES, (kw0[j] >> 8) & LOW_CODES,
                                    (kw1[j] >> 8) & LOW_CODES};
            const uint32_t hi[4] = {kw0[j] & HIGH_CODES, kw1[j] & HIGH_CODES, (kw0[j] >> 8) & HIGH_CODES,
                                    (kw1[j] >> 8) & HIGH_CODES};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_16816(s[nt], lo, qs.b[nt][j][0][0], qs.b[nt][j][0][1]);
                mma_16816(s[nt], hi, qs.b[nt][j][1][0], qs.b[nt][j][1][1]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) x[nt][k] = fmaf(kp[k >> 1][g].x, s[nt][k], x[nt][k]);
    }
    float big[2];  // log2 of the largest V scale of each token
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        float v = vp[t][0].x;
#pragma unroll
        for (int g = 1; g < NG; ++g) v = fmaxf(v, vp[t][g].x);
        big[t] = fmaxf(__log2f(v), -24.f);
    }
    float p[NT][4];
    bool moved = false;
    float al[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int t = k >> 1, col = k & 1;
            float y = x[nt][k] * qs.unit[nt][col];
#pragma unroll
            for (int g = 0; g < NG; ++g) y = fmaf(kp[t][g].y, qs.sum[nt][col][g], y);
            if (EDGE && gid + 8 * t >= left - qs.limit[nt][col]) y = -INFINITY;
            x[nt][k] = y;
            top[col] = fmaxf(top[col], y + big[t]);
        }
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) {
            top[0] = fmaxf(top[0], __shfl_xor_sync(FULL_MASK, top[0], off));
            top[1] = fmaxf(top[1], __shfl_xor_sync(FULL_MASK, top[1], off));
        }
#pragma unroll
        for (int col = 0; col < 2; ++col) {
            const float mn = fmaxf(w.m[nt][col], top[col]);
            const float ref = mn == -INFINITY ? 0.f : mn;
            al[nt][col] = fast_exp2(w.m[nt][col] - ref);
            moved |= al[nt][col] != 1.f;
            w.m[nt][col] = mn;
            p[nt][col] = fast_exp2(x[nt][col] - ref);
            p[nt][2 + col] = fast_exp2(x[nt][2 + col] - ref);
        }
    }
    if (__any_sync(FULL_MASK, moved)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int col = 0; col < 2; ++col) {
                w.l[nt][col] *= al[nt][col];
#pragma unroll
                for (int g = 0; g < NG; ++g) w.z[nt][col][g] *= al[nt][col];
            }
#pragma unroll
            for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                for (int hl = 0; hl < 2; ++hl)
#pragma unroll
                    for (int k = 0; k < 4; ++k) w.o[nt][ch][hl][k] *= al[nt][k & 1];
        }
    }
    // ---- weights in the layout of the second product's B operand, a group each
    uint32_t pb[NT][NG][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int col = 0; col < 2; ++col) w.l[nt][col] += p[nt][col] + p[nt][2 + col];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = k >> 1, col = k & 1;
                // A query that does not see a token takes nothing from it, not even a NaN.
                const bool sees = !EDGE || gid + 8 * t < left - qs.limit[nt][col];
                y[k] = sees ? p[nt][k] * vp[t][g].x : 0.f;
                w.z[nt][col][g] += sees ? p[nt][k] * vp[t][g].y : 0.f;
            }
            pb[nt][g][0] = movmatrix_trans(pack_half2(y[0], y[1]));  // tokens 0-7
            pb[nt][g][1] = movmatrix_trans(pack_half2(y[2], y[3]));  // tokens 8-15
        }
    }
    // ---- second product: channels 32 ch + 4 gid + 0..3 of chunk ch
    const int tok = lane & 15, half = lane >> 4;
    const uint32_t vbase = smem_u32(rec) + KV4_CODES + tok * KV4_ROW;
#pragma unroll
    for (int cp = 0; cp < 2; ++cp) {
        uint32_t v[4];  // chunk 2cp: tokens 0-7, 8-15; chunk 2cp + 1: the same
        ldmatrix_x4_trans(v, vbase + (((2 * cp + half) ^ ((tok >> 1) & 3)) << 4));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int ch = 2 * cp + k, g = ch * NG / 4;
            const uint32_t a0 = v[2 * k], a1 = v[2 * k + 1];
            const uint32_t lo[4] = {a0 & LOW_CODES, (a0 >> 8) & LOW_CODES, a1 & LOW_CODES, (a1 >> 8) & LOW_CODES};
            const uint32_t hi[4] = {a0 & HIGH_CODES, (a0 >> 8) & HIGH_CODES, a1 & HIGH_CODES,
                                    (a1 >> 8) & HIGH_CODES};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_16816(w.o[nt][ch][0], lo, pb[nt][g][0], pb[nt][g][1]);
                mma_16816(w.o[nt][ch][1], hi, pb[nt][g][0], pb[nt][g][1]);
            }
        }
    }
}

// Row of the outputs and of lse for query row `row` of request r's KV head h.
__device__ __forceinline__ size_t kv4_out_row(const Kv4Args& a, int r, int h, int row) {
    const int qi = row / a.G, g = row - qi * a.G;
    return (static_cast<size_t>(r) * a.n_q + qi) * a.Hq + static_cast<size_t>(h) * a.G + g;
}

template <bool BF16>
__device__ __forceinline__ void store4(const Kv4Args& a, size_t row, int ch4, float4 v, float inv, bool none) {
    uint2 pk = make_uint2(0u, 0u);
    if (!none) {
        pk.x = kv4_pack2<BF16>(v.x * inv, v.y * inv);
        pk.y = kv4_pack2<BF16>(v.z * inv, v.w * inv);
    }
    reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + row * KV4_D * 2)[ch4] = pk;
}

__device__ __forceinline__ float kv4_lse(float m, float l, bool none) {
    return none ? -INFINITY : (m + log2f(l)) * LN2;
}

// Ends a token set in this warp: writes the outputs (piece == nullptr) or
// leaves the sums in `piece`, [rows][KV4_PIECE_ROW] floats.
template <bool BF16, int NT, int NG>
__device__ __forceinline__ void end_set(const Kv4Args& a, const Softmax<NT, NG>& w, int r, int h, bool bad,
                                        float* piece, int lane) {
    const int gid = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int col = 0; col < 2; ++col) {
            float l = w.l[nt][col];
            float z[NG];
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) l += __shfl_xor_sync(FULL_MASK, l, off);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                z[g] = w.z[nt][col][g];
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1) z[g] += __shfl_xor_sync(FULL_MASK, z[g], off);
            }
            const int row = nt * 8 + 2 * c + col;
            if (row >= a.rows) continue;
            const float m = w.m[nt][col];
            const bool none = bad || l == 0.f;
            const float inv = none ? 0.f : 1.f / l;
            const size_t orow = piece == nullptr ? kv4_out_row(a, r, h, row) : 0;
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
                const float zg = z[ch * NG / 4];
                const float4 o = make_float4(fmaf(w.o[nt][ch][0][col], 0x1p24f, zg), fmaf(w.o[nt][ch][1][col], 0x1p20f, zg),
                                             fmaf(w.o[nt][ch][0][2 + col], 0x1p24f, zg),
                                             fmaf(w.o[nt][ch][1][2 + col], 0x1p20f, zg));
                if (piece == nullptr)
                    store4<BF16>(a, orow, ch * 8 + gid, o, inv, none);
                else
                    *reinterpret_cast<float4*>(piece + row * KV4_PIECE_ROW + ch * 32 + gid * 4) = o;
            }
            if (gid == 0) {
                if (piece == nullptr) {
                    if (a.lse != nullptr) a.lse[orow] = kv4_lse(m, l, none);
                } else {
                    piece[row * KV4_PIECE_ROW + KV4_D] = m;
                    piece[row * KV4_PIECE_ROW + KV4_D + 1] = bad ? -1.f : l;
                }
            }
        }
}

// Shared memory of a CTA, in bytes from its start.
struct Kv4Layout {
    int ring, piece, bars, prefix, total;  // ring and piece: bytes a warp
};

__host__ __device__ inline Kv4Layout kv4_layout(int ng, int rows, int B) {
    Kv4Layout y;
    const int piece = rows * KV4_PIECE_ROW * static_cast<int>(sizeof(float));
    const int ring = KV4_STAGES * kv4_record(ng);
    y.ring = ((ring > piece ? ring : piece) + 127) / 128 * 128;  // the last piece takes the ring's place
    y.piece = (piece + 15) / 16 * 16;
    y.bars = KV4_WARPS * (y.ring + y.piece);
    y.prefix = y.bars + KV4_WARPS * KV4_STAGES * 8;
    y.total = y.prefix + (B + 1) * static_cast<int>(sizeof(int));
    return y;
}

template <bool BF16, int NT, int NG>
__global__ void __launch_bounds__(KV4_THREADS, kv4_ctas_per_sm(NT)) kv4_attn_kernel(const Kv4Args a) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int wsum[KV4_WARPS];
    __shared__ int piece_set[2 * KV4_WARPS];  // token set of each warp's first and last piece, or -1
    constexpr int R = kv4_record(NG);
    const Kv4Layout y = kv4_layout(NG, a.rows, a.B);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* ring = smem + warp * y.ring;
    float* first_piece = reinterpret_cast<float*>(smem + KV4_WARPS * y.ring + warp * y.piece);
    const uint32_t bars = smem_u32(smem + y.bars) + warp * KV4_STAGES * 8;
    int* prefix = reinterpret_cast<int*>(smem + y.prefix);

    if (lane < KV4_STAGES) mbar_init(bars + lane * 8);
    if (lane < 2) piece_set[2 * warp + lane] = -1;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    pdl_wait();
    pdl_launch_dependents();
    kv4_prefix(a, prefix, wsum);

    // Requests without a token (or with a bad length) get zeros.
    for (int r = blockIdx.x; r < a.B; r += gridDim.x) {
        if (prefix[r + 1] != prefix[r]) continue;
        const size_t row0 = static_cast<size_t>(r) * a.n_q * a.Hq;
        for (int i = threadIdx.x; i < a.n_q * a.Hq * (KV4_D / 8); i += KV4_THREADS)
            (reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + row0 * KV4_D * 2))[i] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse != nullptr)
            for (int i = threadIdx.x; i < a.n_q * a.Hq; i += KV4_THREADS) a.lse[row0 + i] = -INFINITY;
    }

    // Warp g of W takes tiles [N g / W, N (g + 1) / W).
    const long long N = prefix[a.B];
    const long long W = min(static_cast<long long>(gridDim.x) * KV4_WARPS, N);
    const long long g0 = static_cast<long long>(blockIdx.x) * KV4_WARPS;
    const long long g = g0 + warp;
    const int t0 = g < W ? static_cast<int>(N * g / W) : 0;
    const int t1 = g < W ? static_cast<int>(N * (g + 1) / W) : 0;
    if (t0 < t1) {
        const uint64_t policy = l2_evict_first_policy();
        Place pl = kv4_place(prefix, a.B, a.Hkv, t0), ps = pl;  // loading, computing
        // Block ids: lane i holds entry `base` + i of the loading request's
        // row, and the 32 after them.
        int base = 0, ids = 0, ids_next = 0;
        auto load_ids = [&](int at) {
            return at + lane < pl.nt ? __ldg(a.table + static_cast<size_t>(pl.r) * a.max_blocks + at + lane) : 0;
        };
        auto start_ids = [&]() {
            base = pl.j;
            ids = load_ids(base);
            ids_next = load_ids(base + 32);
        };
        start_ids();
        uint32_t bad_slots = 0;  // stages whose record does not exist
        auto issue = [&](int stage) {
            if (pl.j - base == 32) {
                base += 32;
                ids = ids_next;
                ids_next = load_ids(base + 32);
            }
            const int id = __shfl_sync(FULL_MASK, ids, pl.j - base);
            const bool ok = id >= 0 && id < a.num_blocks;
            bad_slots = ok ? bad_slots & ~(1u << stage) : bad_slots | (1u << stage);
            if (lane == 0) {
                const uint32_t bar = bars + stage * 8;
                if (ok) {
                    mbar_expect(bar, R);
                    bulk_load(smem_u32(ring) + stage * R,
                              a.pool + (static_cast<size_t>(id) * a.Hkv + pl.h) * R, R, bar, policy);
                } else {
                    mbar_arrive(bar);
                }
            }
            const int r_before = pl.r, h_before = pl.h;
            kv4_next(prefix, a.B, a.Hkv, pl);
            if (pl.r != r_before) {
                if (pl.r < a.B) start_ids();
            } else if (pl.h != h_before) {
                start_ids();
            }
        };
        int issued = t0;
        for (; issued < t1 && issued - t0 < KV4_STAGES; ++issued) issue(issued - t0);

        Queries<NT, NG> qs;
        Softmax<NT, NG> w;
        bool bad = false, fresh = true;
        int set_start = t0;  // first tile of the current set in this range
        int n_tok = 0;
        int stage = 0;
        uint32_t parity = 0;
        for (int t = t0; t < t1; ++t) {
            if (fresh) {
                n_tok = __ldg(a.ctx_len + ps.r);
                load_queries<BF16, NT, NG>(a, ps, lane, qs);
                reset(w);
                bad = false;
                fresh = false;
                set_start = t;
            }
            const bool came = mbar_wait(bars + stage * 8, parity);
            if (!came) {
                if (lane == 0) report_error(a.err_flag, CLO_FLAG_TIMEOUT);
                bad = true;
            }
            const int left = n_tok - ps.j * KV4_BLOCK;
            if ((bad_slots >> stage) & 1u) {
                bad = true;
                if (lane == 0) report_error(a.err_flag, CLO_FLAG_BAD_INDEX);
            } else if (came) {
                const uint8_t* rec = ring + stage * R;
                if (left >= KV4_BLOCK + a.n_q - 1)
                    take_tile<NT, NG, false>(rec, left, qs, w, lane);
                else
                    take_tile<NT, NG, true>(rec, left, qs, w, lane);
            }
            __syncwarp();
            if (issued < t1) {
                issue(stage);
                ++issued;
            }
            if (++stage == KV4_STAGES) {
                stage = 0;
                parity ^= 1;
            }
            const bool set_done = ps.j + 1 == ps.nt, last = t + 1 == t1;
            if (set_done || last) {
                const bool whole = set_done && t - set_start == ps.j;  // all of its tiles were here
                float* piece = whole ? nullptr : last ? reinterpret_cast<float*>(ring) : first_piece;
                if (lane == 0 && !whole) piece_set[2 * warp + (last ? 1 : 0)] = ps.r * a.Hkv + ps.h;
                end_set<BF16, NT, NG>(a, w, ps.r, ps.h, bad, piece, lane);
                fresh = true;
            }
            kv4_next(prefix, a.B, a.Hkv, ps);
        }
    }
    __syncthreads();

    // The CTA's pieces, in the order of the stream; those of one token set are
    // next to each other.
    const int c0 = g0 < W ? static_cast<int>(N * g0 / W) : 0;
    const int c1 = g0 < W ? static_cast<int>(N * min(g0 + KV4_WARPS, W) / W) : 0;
    int tail_set = 0, tail_ctas = 0;
    for (int i = 0; i < 2 * KV4_WARPS;) {
        const int set = piece_set[i];
        int end = i + 1;
        if (set >= 0) {
            // -1 entries between two pieces of a set: a warp that has one piece only
            for (int k = end; k < 2 * KV4_WARPS; ++k) {
                if (piece_set[k] == set) end = k + 1;
                else if (piece_set[k] >= 0) break;
            }
            const int r = set / a.Hkv, h = set - r * a.Hkv;
            const int nt = (prefix[r + 1] - prefix[r]) / a.Hkv;
            const int s0 = prefix[r] + h * nt, s1 = s0 + nt;  // its tiles
            const bool done = s0 >= c0 && s1 <= c1;
            const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (s0 < c0 ? 0 : 1);
            if (s0 >= c0 && s1 > c1) {
                tail_set = set;
                tail_ctas = static_cast<int>((static_cast<long long>(s1) * W - 1) / N / KV4_WARPS) -
                            static_cast<int>(blockIdx.x) + 1;
            }
            for (int it = threadIdx.x; it < a.rows * (KV4_D / 4); it += KV4_THREADS) {
                const int row = it / (KV4_D / 4), col = it % (KV4_D / 4);
                float M = -INFINITY;
                bool bad = false;
                for (int k = i; k < end; ++k)
                    if (piece_set[k] == set) {
                        const float* pc = reinterpret_cast<const float*>(
                            (k & 1) ? smem + (k >> 1) * y.ring : smem + KV4_WARPS * y.ring + (k >> 1) * y.piece);
                        M = fmaxf(M, pc[row * KV4_PIECE_ROW + KV4_D]);
                        bad |= pc[row * KV4_PIECE_ROW + KV4_D + 1] == -1.f;
                    }
                float L = 0.f;
                float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
                const float ref = M == -INFINITY ? 0.f : M;
                for (int k = i; k < end; ++k)
                    if (piece_set[k] == set) {
                        const float* pc = reinterpret_cast<const float*>(
                            (k & 1) ? smem + (k >> 1) * y.ring : smem + KV4_WARPS * y.ring + (k >> 1) * y.piece);
                        const float e = fast_exp2(pc[row * KV4_PIECE_ROW + KV4_D] - ref);
                        const float4 v = *reinterpret_cast<const float4*>(pc + row * KV4_PIECE_ROW + 4 * col);
                        L = fmaf(pc[row * KV4_PIECE_ROW + KV4_D + 1], e, L);
                        O.x = fmaf(v.x, e, O.x);
                        O.y = fmaf(v.y, e, O.y);
                        O.z = fmaf(v.z, e, O.z);
                        O.w = fmaf(v.w, e, O.w);
                    }
                if (done) {
                    const bool none = bad || L == 0.f;
                    const size_t orow = kv4_out_row(a, r, h, row);
                    store4<BF16>(a, orow, col, O, none ? 0.f : 1.f / L, none);
                    if (a.lse != nullptr && col == 0) a.lse[orow] = kv4_lse(M, L, none);
                } else {
                    *reinterpret_cast<float4*>(a.ws_o + (slot * a.rows + row) * KV4_D + 4 * col) = O;
                    if (col == 0) a.ws_ml[slot * a.rows + row] = make_float2(M, bad ? -1.f : L);
                }
            }
        }
        i = end;
    }
    if (threadIdx.x == 0) a.ws_tail[blockIdx.x] = make_int2(tail_set, tail_ctas);
}

// Block (c, row) merges query row `row` of the token set that starts in CTA c
// of the main kernel and goes on: its tail piece and the head pieces of the
// CTAs behind it, in a fixed order.  A lane holds 4 channels; the warps take
// the pieces in turn.
template <bool BF16>
__global__ void __launch_bounds__(KV4_THREADS) kv4_merge_kernel(const Kv4Args a) {
    __shared__ float sm_m[KV4_WARPS], sm_l[KV4_WARPS];
    __shared__ float4 sm_o[KV4_WARPS][32];
    pdl_launch_dependents();
    pdl_wait();
    const int2 tail = a.ws_tail[blockIdx.x];
    if (tail.y == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = blockIdx.y;
    float M = -INFINITY, L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    bool bad = false;
    constexpr int U = 4;  // pieces a warp loads at a time
    for (int p0 = warp; p0 < tail.y; p0 += KV4_WARPS * U) {
        float2 ml[U];
        float4 v[U];
        float mx = M;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = p0 + u * KV4_WARPS;
            ml[u] = make_float2(-INFINITY, 0.f);
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p < tail.y) {
                const size_t slot = 2 * (static_cast<size_t>(blockIdx.x) + p) + (p == 0 ? 1 : 0);
                ml[u] = a.ws_ml[slot * a.rows + row];
                v[u] = reinterpret_cast<const float4*>(a.ws_o + (slot * a.rows + row) * KV4_D)[lane];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mx = fmaxf(mx, ml[u].x);
            bad |= ml[u].y == -1.f;
        }
        const float ref = mx == -INFINITY ? 0.f : mx;
        float e = fast_exp2(M - ref);
        L *= e, O.x *= e, O.y *= e, O.z *= e, O.w *= e;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            e = fast_exp2(ml[u].x - ref);
            L = fmaf(ml[u].y, e, L);
            O.x = fmaf(v[u].x, e, O.x);
            O.y = fmaf(v[u].y, e, O.y);
            O.z = fmaf(v[u].z, e, O.z);
            O.w = fmaf(v[u].w, e, O.w);
        }
        M = mx;
    }
    if (lane == 0) {
        sm_m[warp] = M;
        sm_l[warp] = L;
    }
    sm_o[warp][lane] = O;
    bad = __syncthreads_or(bad) != 0;
    if (warp != 0) return;
    float top = M;
#pragma unroll
    for (int x = 1; x < KV4_WARPS; ++x) top = fmaxf(top, sm_m[x]);
    const float ref = top == -INFINITY ? 0.f : top;
    L = 0.f;
    O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < KV4_WARPS; ++x) {
        const float e = fast_exp2(sm_m[x] - ref);
        const float4 v = sm_o[x][lane];
        L = fmaf(sm_l[x], e, L);
        O.x = fmaf(v.x, e, O.x);
        O.y = fmaf(v.y, e, O.y);
        O.z = fmaf(v.z, e, O.z);
        O.w = fmaf(v.w, e, O.w);
    }
    const bool none = bad || L == 0.f;
    const int r = tail.x / a.Hkv, h = tail.x - r * a.Hkv;
    const size_t orow = kv4_out_row(a, r, h, row);
    store4<BF16>(a, orow, lane, O, none ? 0.f : 1.f / L, none);
    if (a.lse != nullptr && lane == 0) a.lse[orow] = kv4_lse(top, L, none);
}

using Kv4Kernel = void (*)(const Kv4Args);

template <bool BF16, int NT>
static Kv4Kernel attn_kernel_ng(int ng) {
    return ng == 1 ? kv4_attn_kernel<BF16, NT, 1> : ng == 2 ? kv4_attn_kernel<BF16, NT, 2> : kv4_attn_kernel<BF16, NT, 4>;
}
template <bool BF16>
static Kv4Kernel attn_kernel(int nt, int ng) {
    return nt == 1 ? attn_kernel_ng<BF16, 1>(ng) : nt == 2 ? attn_kernel_ng<BF16, 2>(ng) : attn_kernel_ng<BF16, 4>(ng);
}

// n8 tiles of the kernel that takes this many query rows.
static int kv4_row_tiles(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

// One wave at the most: what the workspace is sized for.
static int kv4_most_ctas(int rows) { return device_sm_count() * kv4_ctas_per_sm(kv4_row_tiles(rows)); }

static size_t round256(size_t x) { return (x + 255) / 256 * 256; }

static size_t kv4_workspace(int ctas, int rows) {
    const size_t slots = 2 * static_cast<size_t>(ctas) * rows;
    return round256(slots * KV4_D * sizeof(float)) + round256(slots * sizeof(float2)) +
           round256(static_cast<size_t>(ctas) * sizeof(int2));
}

}  // namespace clo

using namespace clo;

extern "C" size_t clo_kv4_paged_workspace_size(int B, int n_q, int Hq, int Hkv, int d, int num_ctas) {
    if (B < 0 || n_q < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || d != KV4_D || num_ctas < 0) return 0;
    if (static_cast<long long>(Hq / Hkv) * n_q > KV4_MAX_ROWS) return 0;
    const int rows = Hq / Hkv * n_q;
    const int ctas = num_ctas > 0 ? num_ctas : kv4_most_ctas(rows);
    return ctas > 0 ? kv4_workspace(ctas, rows) : 0;
}

extern "C" clo_status clo_kv4_paged_decode_attn(const void* q, clo_dtype dtype, const uint8_t* pool,
                                                const int32_t* block_table, int max_blocks,
                                                const int32_t* ctx_len, int num_blocks, int B, int n_q,
                                                int Hq, int Hkv, int d, int block_size, int group,
                                                float scale, void* out, float* lse, void* workspace,
                                                size_t ws_bytes, int32_t* err_flag,
                                                const clo_attn_opts* opts, cudaStream_t stream) {
    if (B < 0 || n_q < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_blocks < 1 || num_blocks < 1)
        return CLO_ERR_INVALID_ARG;
    if (dtype != CLO_F16 && dtype != CLO_BF16) return CLO_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !isfinite(scale)) return CLO_ERR_INVALID_ARG;
    if (opts != nullptr && opts->num_ctas < 0) return CLO_ERR_INVALID_ARG;
    if (B > 0 && (q == nullptr || pool == nullptr || block_table == nullptr || ctx_len == nullptr || out == nullptr))
        return CLO_ERR_INVALID_ARG;
    if (!kv4_aligned(q, 16) || !kv4_aligned(pool, 16) || !kv4_aligned(out, 16) || !kv4_aligned(block_table, 4) ||
        !kv4_aligned(ctx_len, 4) || !kv4_aligned(lse, 4) || !kv4_aligned(err_flag, 4))
        return CLO_ERR_INVALID_ARG;
    const int ng = kv4_groups(group);
    if (d != KV4_D || block_size != KV4_BLOCK || ng == 0 || B > KV4_MAX_B ||
        static_cast<long long>(Hq / Hkv) * n_q > KV4_MAX_ROWS)
        return CLO_ERR_UNSUPPORTED;
    const long long tiles = static_cast<long long>(B) * Hkv * max_blocks;  // at most: the lengths are on the device
    if (tiles >= (1ll << 31) || max_blocks > (1 << 26)) return CLO_ERR_UNSUPPORTED;
    if (opts != nullptr && opts->num_ctas > (1 << 20)) return CLO_ERR_UNSUPPORTED;
    if (B == 0) return CLO_OK;

    Kv4Args a;
    a.rows = Hq / Hkv * n_q;
    const int smem = kv4_layout(ng, a.rows, B).total;
    // One wave: as many CTAs an SM as registers and shared memory allow.
    const int per_sm = std::min(kv4_ctas_per_sm(kv4_row_tiles(a.rows)), KV4_SMEM_PER_SM / (smem + 1024 + 128));
    int ctas = opts != nullptr && opts->num_ctas > 0 ? opts->num_ctas : device_sm_count() * per_sm;
    const long long most = (tiles + KV4_WARPS - 1) / KV4_WARPS;
    if (ctas > most) ctas = static_cast<int>(most);
    if (workspace == nullptr || !kv4_aligned(workspace, 16) ||
        ws_bytes < clo_kv4_paged_workspace_size(B, n_q, Hq, Hkv, d, opts != nullptr ? opts->num_ctas : 0))
        return CLO_ERR_WORKSPACE;
    if (ctas <= 0) return CLO_ERR_CUDA;

    const size_t slots = 2 * static_cast<size_t>(ctas) * a.rows;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.ws_o = reinterpret_cast<float*>(ws);
    a.ws_ml = reinterpret_cast<float2*>(ws + round256(slots * KV4_D * sizeof(float)));
    a.ws_tail = reinterpret_cast<int2*>(ws + round256(slots * KV4_D * sizeof(float)) + round256(slots * sizeof(float2)));
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.pool = pool;
    a.table = block_table;
    a.ctx_len = ctx_len;
    a.err_flag = err_flag;
    a.scale_log2 = scale * LOG2E;
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    a.B = B;
    a.n_q = n_q;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    const int nt = kv4_row_tiles(a.rows);
    const Kv4Kernel kernel = dtype == CLO_BF16 ? attn_kernel<true>(nt, ng) : attn_kernel<false>(nt, ng);
    const Kv4Kernel merge = dtype == CLO_BF16 ? kv4_merge_kernel<true> : kv4_merge_kernel<false>;
    if (!prepare_kernel(reinterpret_cast<const void*>(kernel), kv4_layout(ng, a.rows, KV4_MAX_B).total) ||
        !prepare_kernel(reinterpret_cast<const void*>(merge), 0))
        return CLO_ERR_CUDA;
    if (opts != nullptr && opts->ev_begin != nullptr && !record_event(opts->ev_begin, stream)) return CLO_ERR_CUDA;
    if (launch_pdl(kernel, dim3(ctas), dim3(KV4_THREADS), smem, stream, a) != cudaSuccess) return CLO_ERR_CUDA;
    if (opts != nullptr && opts->ev_end != nullptr && !record_event(opts->ev_end, stream)) return CLO_ERR_CUDA;
    if (ctas > 1 &&
        launch_pdl(merge, dim3(ctas - 1, a.rows), dim3(KV4_THREADS), 0, stream, a) != cudaSuccess)
        return CLO_ERR_CUDA;
    return CLO_OK;
}
