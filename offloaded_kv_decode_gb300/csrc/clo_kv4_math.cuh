// clo_kv4_math.cuh -- what a warp does in decode attention over the paged cache
// held in 4 bits (format: clo_kv4.h): queries in, records in, sums out.
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
//   * Online softmax with one reference m a query row, p_t = 2^(x_t - m), x the
//     score in log2 units.  m follows 2^6 below the maximum of x_t + log2(largest
//     V scale of t, in size), and only when a unit gets 2^14 above it: the weights
//     p_t s_tg that are rounded to fp16 for the second product are then below
//     2^15 and the largest of them not below 2^6, whatever the V scales are, most
//     units need no reduction over lanes, and the sums are hardly ever rescaled.
//     l = sum p_t stays in fp32 (p_t < 2^39 as an fp16 scale is at least 2^-24).
//     (With the maximum itself for m, weights 2^-25 of the largest were lost:
//     1e-3 of bf16 outputs, V scales 0.2, with 128K tokens in a warp beside one
//     of ten times their scale and a score 16 above theirs; now under 1e-4.)
//   * That rounding is the one that costs accuracy.  For fp16 outputs the sums
//     are arranged so that it meets V's codes from the middle of their range,
//         sum_t (p_t s_tg)~ (code_td - 7.5) + sum_t p_t (z_tg + 7.5 s_tg),
//     ~ the rounding: the first product and z take the 7.5 (p s)~ away again.
//     Outputs are then 2.4e-4 off the 64-bit ones in the 2-norm, 2.1e-4 of which
//     is their own rounding, against 3.4e-4, for 2 to 6% of the time (128 ragged
//     multi-head requests: 217 us against 207).  Beside a bf16 output's own
//     rounding, 1.7e-3, neither shows, and it is left out.
//
// Shape.  mma.sync m16n8k16 with 16 tokens on M and 8 query rows (of the
// G * n_q of a KV head) on N for the scores, then channels on M for the second
// product; the operands come out of registers because they are made there (a
// tcgen05 operand would have to be written back to shared memory in 16 bits,
// 4 times the bytes that were read).
#pragma once

#include <math.h>

#include "clo_kv4.cuh"

namespace clo {

constexpr int KV4_WARPS = 4;
constexpr int KV4_THREADS = KV4_WARPS * 32;
constexpr int KV4_UNIT = 2 * KV4_BLOCK;  // tokens of a unit
constexpr int KV4_MAX_ROWS = 32;   // query rows of a KV head: G * n_q
constexpr int KV4_PIECE_ROW = KV4_D + 4;  // floats of a row of a piece; the four behind: m, l
constexpr int KV4_SMEM_PER_SM = 228 * 1024;
constexpr int KV4_SMEM_RESERVED = 1024 + 256;  // of a CTA: the system's, and the static arrays
constexpr long long KV4_WAIT_CLOCKS = 1ll << 32;  // about 2 s
// How far x + log2(V scale) lies above the reference when this moves, and how far
// it may get: weights up to 2^14 of fp16's 2^16, and down to its least steps of
// 2^-24 for those 2^-30 of the largest.
constexpr float KV4_LIFT = 6.f, KV4_SLACK = 14.f;
constexpr uint32_t LOW_CODES = 0x000f000fu, HIGH_CODES = 0x00f000f0u;

// CTAs of 4 warps that an SM's registers hold for NT tiles of 8 query rows (128,
// 168, 255 a thread).
__host__ __device__ constexpr int kv4_ctas_per_sm(int nt) { return nt == 1 ? 4 : nt == 2 ? 3 : 2; }

// Units a warp's ring has room for: what fits beside the others' at 4 CTAs an SM.
__host__ __device__ constexpr int kv4_stages(int ng) { return ng == 4 ? 2 : 3; }

struct Kv4Args {
    const void* q;
    void* out;
    float* lse;
    const uint8_t* pool;
    const int32_t* table;
    const int32_t* ctx_len;
    int32_t* err_flag;
    float* ws_o;    // [2 * CTAs][rows][128] partial sums, head piece and tail piece of each CTA
    float* ws_first;  // [warps][rows][KV4_PIECE_ROW] piece of the set that ends in a warp but began before it
    float2* ws_ml;  // [2 * CTAs][rows] their (reference, denominator); denominator -1: bad data
    int2* ws_cut;   // what the merge finds its work by: see kv4_merge_kernel
    float scale_log2;
    int max_blocks, num_blocks, B, n_q, Hq, Hkv, G, rows;
    bool by_set;    // ws_cut is by token set, else by CTA
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
// For a whole warp: all of it goes on, or none.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    return __all_sync(FULL_MASK, mbar_wait(bar, parity));
}
// After a wait that ran out: waits, with the same limit, for the other stages'
// copies, so that none lands in memory that is used for something else by then.
template <int STAGES>
__device__ __noinline__ void give_up(int32_t* err_flag, uint32_t bars, int stage, uint32_t parity, int lane) {
    if (lane == 0) report_error(err_flag, CLO_FLAG_TIMEOUT);
    for (int s = 0; s < STAGES; ++s)
        if (s != stage) mbar_wait(bars + s * 8, s > stage ? parity : parity ^ 1u);
    __syncwarp();
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                          uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], "
        "%4;\n" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// The queries of one KV head.  The B operand of the first product: one n8 tile
// is kept in registers, more in the warp's shared memory.  What the scores need
// in fp32, in shared memory: a row's factor of the code sums, and the sum of
// each group's elements (log2 units).
template <int NT, int NG>
struct Queries {
    static constexpr bool kShared = NT > 1;
    uint4 reg[kShared ? 1 : 4];  // word j: low codes' two registers, high codes' two
    float* sm;                   // [NT * 8] factors, [NG][NT * 8] sums, then operands [NT][4][32]

    __device__ __forceinline__ uint4* sm_operands() const {
        return reinterpret_cast<uint4*>(sm + (1 + NG) * NT * 8);
    }
    __device__ __forceinline__ uint4 operand(int nt, int j, int lane) const {
        if constexpr (kShared) return sm_operands()[(nt * 4 + j) * 32 + lane];
        else return reg[j];
    }
    // Of columns 2c and 2c + 1.
    __device__ __forceinline__ float2 factor(int nt, int c) const {
        return *reinterpret_cast<const float2*>(sm + nt * 8 + 2 * c);
    }
    __device__ __forceinline__ float2 sum(int nt, int g, int c) const {
        return *reinterpret_cast<const float2*>(sm + (1 + g) * NT * 8 + nt * 8 + 2 * c);
    }
};

__host__ __device__ constexpr int kv4_query_bytes(int nt, int ng) {
    return (1 + ng) * nt * 8 * 4 + (nt > 1 ? nt * 4 * 32 * 16 : 0);
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float kv4_power2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];\n" ::"l"(p)); }

template <bool BF16, int NT, int NG>
__device__ __forceinline__ void load_queries(const Kv4Args& a, int r, int h, int lane, Queries<NT, NG>& qs) {
    const int head = lane >> 2, c = lane & 3;
    __syncwarp();  // the last set's are no longer read
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int row = nt * 8 + head;
        const bool has = row < a.rows;
        const int qi = row / a.G, g = row - qi * a.G;
        const size_t at = (static_cast<size_t>(r) * a.n_q + qi) * a.Hq + static_cast<size_t>(h) * a.G + g;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.q) + at * KV4_D * 2);
        // This lane's channels: 32j + 8c .. + 7 for j = 0 .. 3.
        uint4 raw[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) raw[j] = has ? src[4 * j + c] : make_uint4(0u, 0u, 0u, 0u);
        float top = 0.f;
        float part[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
            part[j] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = kv4_unpack2<BF16>(w[k]);
                top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                part[j] += f.x + f.y;
            }
        }
        top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 1));
        top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 2));
        // 2^e brings the largest element into [2^12, 2^13); e is bounded so
        // that 2^e and the factor that undoes it are finite.
        const int e = min(max(139 - static_cast<int>(__float_as_uint(top) >> 23), -100), 100);
        const float up = kv4_power2(e), up16 = kv4_power2(e - 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f0 = kv4_unpack2<BF16>(raw[j].x), f1 = kv4_unpack2<BF16>(raw[j].y);
            const float2 f2 = kv4_unpack2<BF16>(raw[j].z), f3 = kv4_unpack2<BF16>(raw[j].w);
            uint4 o;
            o.x = pack_half2(f0.x * up, f2.x * up);      // channels 0, 4
            o.y = pack_half2(f1.x * up, f3.x * up);      // 2, 6
            o.z = pack_half2(f0.y * up16, f2.y * up16);  // 1, 5
            o.w = pack_half2(f1.y * up16, f3.y * up16);  // 3, 7
            if constexpr (Queries<NT, NG>::kShared) qs.sm_operands()[(nt * 4 + j) * 32 + lane] = o;
            else qs.reg[j] = o;
        }
        float group[NG];
#pragma unroll
        for (int g2 = 0; g2 < NG; ++g2) group[g2] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            part[j] *= a.scale_log2;
            part[j] += __shfl_xor_sync(FULL_MASK, part[j], 1);
            part[j] += __shfl_xor_sync(FULL_MASK, part[j], 2);
            group[j * NG / 4] += part[j];
        }
        if (c == 0) {
            float* u = qs.sm + nt * 8 + head;
            u[0] = a.scale_log2 * kv4_power2(24 - e);
#pragma unroll
            for (int g2 = 0; g2 < NG; ++g2) u[(1 + g2) * NT * 8] = group[g2];
        }
    }
    __syncwarp();
}

// One warp's running softmax of a token set.
template <int NT, int NG>
struct Softmax {
    float m[NT][2];        // reference (log2 units) of columns 2c, 2c + 1
    float l[NT][2];        // this lane's share of sum p
    float z[NT][2][NG];    // this lane's share of sum p z_g (fp16 outputs: p (z_g + 7.5 s_g) - 7.5 (p s_g)~)
    float o[NT][4][2][4];  // sum p s code, but for what is in z: [n8 tile][chunk][low, high codes][register]
};

template <int NT, int NG>
__device__ __forceinline__ void reset(Softmax<NT, NG>& w) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int col = 0; col < 2; ++col) {
            w.m[nt][col] = 0.f;
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

// 2^x and log2(x) in one instruction each; neither sees a subnormal that
// matters (weights below 2^-126, V scales below 2^-24).
__device__ __forceinline__ float kv4_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float kv4_log2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// As mma_16816 and movmatrix_trans, but not volatile: they depend on their
// operands alone, and the compiler may interleave them.
__device__ __forceinline__ void kv4_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t kv4_transpose(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(a));
    return d;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}\n" : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
        " mul.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}\n" : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
        " add.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}\n" : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ __half2 kv4_half2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }

// The NG (scale, zero) pairs of one token's K (kv = 0) or V, as stored.
template <int NG>
__device__ __forceinline__ void load_params(const uint8_t* rec, int t, int kv, bool there, uint32_t (&p)[NG]) {
    const uint8_t* at = rec + kv4_param(t, kv, NG, 0);
    if constexpr (NG == 1) {
        p[0] = *reinterpret_cast<const uint32_t*>(at);
    } else if constexpr (NG == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(at);
        p[0] = u.x, p[1] = u.y;
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(at);
        p[0] = u.x, p[1] = u.y, p[2] = u.z, p[3] = u.w;
    }
    // What lies behind the last token may be anything, NaN among it.
#pragma unroll
    for (int g = 0; g < NG; ++g) p[g] = there ? p[g] : 0u;
}

// Takes NB records in.  Rows are tokens gid and gid + 8 of each record, columns
// query rows 2c and 2c + 1 of each n8 tile.  first: nothing has been taken in
// yet.  EDGE: there are tokens that some query does not see; `left` counts the
// tokens from the first record's first one on.
template <bool BF16, int NT, int NG, int NB, bool EDGE>
__device__ __forceinline__ void take_records(const uint8_t* rec, int left, bool first, const Kv4Args& a,
                                             const Queries<NT, NG>& qs, Softmax<NT, NG>& w, int lane) {
    constexpr int R = kv4_record(NG);
    const int gid = lane >> 2, c = lane & 3;
    // Tokens behind the last one that a column does not see.
    auto limit = [&](int nt, int col) { return a.n_q - 1 - min(nt * 8 + 2 * c + col, a.rows - 1) / a.G; };
    auto sees = [&](int nt, int row, int col) { return !EDGE || gid + 8 * row < left - limit(nt, col); };
    auto there = [&](int row) { return !EDGE || gid + 8 * row < left; };

    // ---- scores in log2 units, relative to the reference
    float x[NT][NB][4];  // [n8 tile][record][row of the record, column]
    float big[2 * NB];   // log2 of the largest V scale of a row
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const uint4 k0 = *reinterpret_cast<const uint4*>(rec + b * R + gid * KV4_ROW + c * 16);
        const uint4 k1 = *reinterpret_cast<const uint4*>(rec + b * R + (gid + 8) * KV4_ROW + c * 16);
        const uint32_t kw0[4] = {k0.x, k0.y, k0.z, k0.w}, kw1[4] = {k1.x, k1.y, k1.z, k1.w};
        uint32_t kp[2][NG];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint32_t vp[NG];
            load_params<NG>(rec + b * R, gid + 8 * t, 0, there(2 * b + t), kp[t]);
            load_params<NG>(rec + b * R, gid + 8 * t, 1, there(2 * b + t), vp);
            // Scales of either sign.
            __half2 most = NG == 1 ? kv4_half2(vp[0]) : __habs2(kv4_half2(vp[0]));
#pragma unroll
            for (int g = 1; g < NG; ++g) most = __hmax2(most, __habs2(kv4_half2(vp[g])));
            big[2 * b + t] = fmaxf(kv4_log2(fabsf(__low2float(most))), -24.f);
        }
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
                    const uint4 q = qs.operand(nt, j, lane);
                    kv4_mma(s[nt], lo, q.x, q.y);
                    kv4_mma(s[nt], hi, q.z, q.w);
                }
            }
            const float f[2] = {__low2float(kv4_half2(kp[0][g])), __low2float(kv4_half2(kp[1][g]))};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const float2 ff = make_float2(f[k >> 1], f[k >> 1]), ss = make_float2(s[nt][k], s[nt][k + 1]);
                    const float2 y = g == 0 ? mul2(ff, ss) : fma2(ff, ss, make_float2(x[nt][b][k], x[nt][b][k + 1]));
                    x[nt][b][k] = y.x;
                    x[nt][b][k + 1] = y.y;
                }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float2 factor = qs.factor(nt, c);
            float2 y[2];
            const float2 ref = make_float2(-w.m[nt][0], -w.m[nt][1]);
#pragma unroll
            for (int t = 0; t < 2; ++t) y[t] = fma2(make_float2(x[nt][b][2 * t], x[nt][b][2 * t + 1]), factor, ref);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float2 sum = qs.sum(nt, g, c);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float z = __high2float(kv4_half2(kp[t][g]));
                    y[t] = fma2(make_float2(z, z), sum, y[t]);
                }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                x[nt][b][2 * t] = y[t].x;
                x[nt][b][2 * t + 1] = y[t].y;
            }
        }
    }
    bool hot = first;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float over = -INFINITY;
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
            float* v = &x[nt][t >> 1][2 * (t & 1)];
            if (EDGE && !sees(nt, t, 0)) v[0] = -INFINITY;
            if (EDGE && !sees(nt, t, 1)) v[1] = -INFINITY;
            const float2 y = add2(make_float2(v[0], v[1]), make_float2(big[t], big[t]));
            over = fmaxf(over, fmaxf(y.x, y.y));
        }
        hot |= over > KV4_SLACK;
    }
    if (__any_sync(FULL_MASK, hot)) {  // the reference moves
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int col = 0; col < 2; ++col) {
                float top = -INFINITY;
#pragma unroll
                for (int t = 0; t < 2 * NB; ++t) top = fmaxf(top, x[nt][t >> 1][2 * (t & 1) + col] + big[t]);
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, off));
                // At the first records to below their maximum (0 where a column sees nothing), later only up.
                const float by = first ? (top == -INFINITY ? 0.f : top - KV4_LIFT) : fmaxf(top - KV4_LIFT, 0.f);
                const float al = first ? 0.f : kv4_exp2(-by);
                w.m[nt][col] += by;
                w.l[nt][col] *= al;
#pragma unroll
                for (int g = 0; g < NG; ++g) w.z[nt][col][g] *= al;
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                    for (int hl = 0; hl < 2; ++hl) {
                        w.o[nt][ch][hl][col] *= al;
                        w.o[nt][ch][hl][2 + col] *= al;
                    }
#pragma unroll
                for (int t = 0; t < 2 * NB; ++t) x[nt][t >> 1][2 * (t & 1) + col] -= by;
            }
    }

    // ---- weights, and their product with V a record and a group at a time
    const int tok = lane & 15, half = lane >> 4;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[nt][b][k] = kv4_exp2(x[nt][b][k]);
            const float2 l = add2(make_float2(w.l[nt][0], w.l[nt][1]), add2(make_float2(x[nt][b][0], x[nt][b][1]),
                                                                            make_float2(x[nt][b][2], x[nt][b][3])));
            w.l[nt][0] = l.x;
            w.l[nt][1] = l.y;
        }
        uint32_t vp[2][NG];
#pragma unroll
        for (int t = 0; t < 2; ++t) load_params<NG>(rec + b * R, gid + 8 * t, 1, there(2 * b + t), vp[t]);
        const uint32_t vbase = smem_u32(rec) + b * R + KV4_CODES + tok * KV4_ROW;
        uint32_t v[4];       // chunk 2cp: tokens 0-7, 8-15; chunk 2cp + 1: the same
        uint32_t pb[NT][2];  // the second product's B operand
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {  // channels 32 ch + 4 gid + 0..3
            if (ch % (4 / NG) == 0) {
                const int g = ch * NG / 4;
                float2 f[2] = {__half22float2(kv4_half2(vp[0][g])), __half22float2(kv4_half2(vp[1][g]))};
                if constexpr (!BF16) {
                    const float2 mid = fma2(make_float2(f[0].x, f[1].x), make_float2(7.5f, 7.5f), make_float2(f[0].y, f[1].y));
                    f[0].y = mid.x, f[1].y = mid.y;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float y[4];
                    if constexpr (EDGE) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            // A query that does not see a token takes nothing from it, not even a NaN.
                            const bool in = sees(nt, 2 * b + (k >> 1), k & 1);
                            float& z = w.z[nt][k & 1][g];
                            y[k] = in ? x[nt][b][k] * f[k >> 1].x : 0.f;
                            z = in ? fmaf(x[nt][b][k], f[k >> 1].y, z) : z;
                        }
                    } else {
                        float2 z = make_float2(w.z[nt][0][g], w.z[nt][1][g]);
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const float2 p = make_float2(x[nt][b][2 * t], x[nt][b][2 * t + 1]);
                            const float2 v2 = mul2(p, make_float2(f[t].x, f[t].x));
                            y[2 * t] = v2.x;
                            y[2 * t + 1] = v2.y;
                            z = fma2(p, make_float2(f[t].y, f[t].y), z);
                        }
                        w.z[nt][0][g] = z.x;
                        w.z[nt][1][g] = z.y;
                    }
                    const uint32_t yr[2] = {pack_half2(y[0], y[1]), pack_half2(y[2], y[3])};
                    if constexpr (!BF16) {  // a code counts from 7.5
                        float2 z = make_float2(w.z[nt][0][g], w.z[nt][1][g]);
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            z = fma2(__half22float2(kv4_half2(yr[t])), make_float2(-7.5f, -7.5f), z);
                        w.z[nt][0][g] = z.x;
                        w.z[nt][1][g] = z.y;
                    }
                    pb[nt][0] = kv4_transpose(yr[0]);  // tokens 0-7
                    pb[nt][1] = kv4_transpose(yr[1]);  // tokens 8-15
                }
            }
            if ((ch & 1) == 0) ldmatrix_x4_trans(v, vbase + (((ch + half) ^ ((tok >> 1) & 3)) << 4));
            const uint32_t a0 = v[2 * (ch & 1)], a1 = v[2 * (ch & 1) + 1];
            const uint32_t lo[4] = {a0 & LOW_CODES, (a0 >> 8) & LOW_CODES, a1 & LOW_CODES, (a1 >> 8) & LOW_CODES};
            const uint32_t hi[4] = {a0 & HIGH_CODES, (a0 >> 8) & HIGH_CODES, a1 & HIGH_CODES, (a1 >> 8) & HIGH_CODES};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                kv4_mma(w.o[nt][ch][0], lo, pb[nt][0], pb[nt][1]);
                kv4_mma(w.o[nt][ch][1], hi, pb[nt][0], pb[nt][1]);
            }
        }
    }
}

// Takes out of a warp's sums of p s code what the channels of a group have in
// common (the mean of the first lanes' channels) and adds it to sum p z.  The
// codes are not negative, so the sums grow with every token, and the matrix
// instructions cut each addition to the accumulator off, toward zero: over many
// tokens the loss is as large as the output, in which the sums of codes and
// zeros all but cancel (50000 tokens a warp, V of mean 0: 5 to 30%).  What is
// left in the accumulators after this is of the outputs' own size.  The kernel
// that gives a token set a cluster has at most 32 units a warp and goes without.
template <int NT, int NG>
__device__ __forceinline__ void level_sums(Softmax<NT, NG>& w, int lane) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float2 mean = make_float2(0.f, 0.f);  // of columns 2c and 2c + 1
#pragma unroll
            for (int ch = g * 4 / NG; ch < (g + 1) * 4 / NG; ++ch)
#pragma unroll
                for (int hl = 0; hl < 2; ++hl) {
                    const float* o = w.o[nt][ch][hl];
                    const float unit = (hl == 0 ? 0x1p24f : 0x1p20f) * NG / 16.f;
                    mean = fma2(add2(make_float2(o[0], o[1]), make_float2(o[2], o[3])), make_float2(unit, unit), mean);
                }
            mean.x = __shfl_sync(FULL_MASK, mean.x, lane & 3);
            mean.y = __shfl_sync(FULL_MASK, mean.y, lane & 3);
            w.z[nt][0][g] += lane < 4 ? mean.x : 0.f;
            w.z[nt][1][g] += lane < 4 ? mean.y : 0.f;
#pragma unroll
            for (int ch = g * 4 / NG; ch < (g + 1) * 4 / NG; ++ch)
#pragma unroll
                for (int hl = 0; hl < 2; ++hl) {
                    float* o = w.o[nt][ch][hl];
                    const float unit = hl == 0 ? -0x1p-24f : -0x1p-20f;
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const float2 x = fma2(mean, make_float2(unit, unit), make_float2(o[k], o[k + 1]));
                        o[k] = x.x;
                        o[k + 1] = x.y;
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
        pk.x = kv4_pack2_finite<BF16>(v.x * inv, v.y * inv);
        pk.y = kv4_pack2_finite<BF16>(v.z * inv, v.w * inv);
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
            const float m = l == 0.f ? -INFINITY : w.m[nt][col];  // a query that saw nothing
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

// Sums of pieces of one query row's 4 channels, in order; l = -1 marks
// bad data, and l = 0 with m = -inf a piece without a token.
struct Sums {
    float M = -INFINITY, L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    template <int P>
    __device__ __forceinline__ void take(const float2 (&ml)[P], const float4 (&v)[P]) {
        bool bad = L == -1.f;
        float top = M;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            top = fmaxf(top, ml[p].x);
            bad |= ml[p].y == -1.f;
        }
        const float ref = top == -INFINITY ? 0.f : top, keep = kv4_exp2(M - ref);
        M = top;
        L *= keep, O.x *= keep, O.y *= keep, O.z *= keep, O.w *= keep;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const float e = kv4_exp2(ml[p].x - ref);
            L = fmaf(ml[p].y, e, L);
            O.x = fmaf(v[p].x, e, O.x);
            O.y = fmaf(v[p].y, e, O.y);
            O.z = fmaf(v[p].z, e, O.z);
            O.w = fmaf(v[p].w, e, O.w);
        }
        if (bad) L = -1.f;
    }
    template <bool BF16>
    __device__ __forceinline__ void write(const Kv4Args& a, int r, int h, int row, int col) const {
        const bool none = L == -1.f || L == 0.f;
        const size_t orow = kv4_out_row(a, r, h, row);
        store4<BF16>(a, orow, col, O, none ? 0.f : 1.f / L, none);
        if (a.lse != nullptr && col == 0) a.lse[orow] = kv4_lse(M, L, none);
    }
};

// The kernel that gives each token set a cluster (clo_kv4_sets.cu): the CTAs of
// one, 0 where the even split is the faster way; and its launch.
int kv4_set_cluster(const Kv4Args& a, int ng);
cudaError_t kv4_launch_sets(const Kv4Args& a, int ng, bool bf16, int cluster, cudaStream_t stream);

// n8 tiles of the kernel that takes this many query rows.
inline int kv4_row_tiles(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

}  // namespace clo
