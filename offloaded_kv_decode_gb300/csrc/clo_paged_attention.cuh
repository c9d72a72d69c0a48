// clo_paged_attention.cuh -- the attention over the 16-bit paged cache: its
// arguments, which tokens a query row sees and where they lie, and the attention
// of one row by one warp.
#pragma once

#include "clo_paged.cuh"

namespace clo {

struct PagedAttnArgs {
    const uint8_t* q;
    const uint8_t* kc;
    const uint8_t* vc;
    uint8_t* out;
    float* lse;
    const int32_t* table;
    const int32_t* ctx_len;
    const int32_t* offsets;  // dense: the requests' rows
    const int32_t* sel;      // sparse: [B][Hkv][n_sel] columns of the table
    int32_t* err_flag;
    long long q_stride, kv_block, kv_head, kv_token;  // bytes
    long long unit_block, unit_head;  // kv_block and kv_head in units of their greatest common divisor
    float scale_log2;
    int B, N, Hq, Hkv, G, num_blocks, max_blocks, n_sel;
    int tt, shift;  // tokens of a tile of rows; unit of weights (clo_paged_attention.cu)
};

// A request as the kernels take it.
struct PagedReq {
    int row0;   // its first row of q
    int n;      // rows
    int ctx;    // cached tokens; 0 for a bad length
    bool bad;   // a bad length, or bad offsets
};

template <bool SPARSE>
__device__ __forceinline__ PagedReq paged_request(const PagedAttnArgs& a, int r) {
    PagedReq q;
    q.ctx = a.ctx_len[r];
    q.bad = q.ctx < 0 || q.ctx > a.max_blocks * PG_BLOCK;
    if (q.bad) q.ctx = 0;
    if constexpr (SPARSE) {
        q.row0 = r;
        q.n = 1;
    } else {
        const int first = a.offsets[r], end = a.offsets[r + 1];
        const bool ok = first >= 0 && first <= end && end <= a.N;
        q.row0 = ok ? first : 0;
        q.n = ok ? end - first : 0;
        q.bad |= !ok;
    }
    return q;
}

// Places (16 tokens each) that row i of a request goes over, and the tokens it
// sees in place p: dense, the blocks in order up to its own token; sparse, the
// selected blocks.
template <bool SPARSE>
__device__ __forceinline__ int paged_sees(const PagedReq& q, int i) {
    return SPARSE ? q.ctx : max(q.ctx - (q.n - 1 - i), 0);
}
template <bool SPARSE>
__device__ __forceinline__ int paged_places(const PagedAttnArgs& a, int sees) {
    const int nb = (sees + PG_BLOCK - 1) / PG_BLOCK;
    return SPARSE ? min(nb, a.n_sel) : nb;
}

// Place p of KV head h: block id * 32 + tokens seen there; 0 for a place that is
// left out, -1 for a bad one.
template <bool SPARSE>
__device__ __forceinline__ int paged_place(const PagedAttnArgs& a, int r, int h, int sees, int p) {
    int col = p;
    if constexpr (SPARSE) {
        col = a.sel[(static_cast<size_t>(r) * a.Hkv + h) * a.n_sel + p];
        if (col == -1) return 0;
        if (col < 0 || col >= (sees + PG_BLOCK - 1) / PG_BLOCK) return -1;
    }
    const int id = a.table[static_cast<size_t>(r) * a.max_blocks + col];
    if (id < 0 || id >= a.num_blocks) return -1;
    return id * 32 + min(sees - col * PG_BLOCK, PG_BLOCK);
}

// A pair of results in 16 bits.  Rounded weights may take an fp16 sum past the
// largest V by a little: finite ones stop at 65504.
template <bool BF16>
__device__ __forceinline__ uint32_t pg_pack_out(float lo, float hi) {
    if constexpr (BF16) {
        return pg_pack<true>(lo, hi);
    } else {
        const float top = 65504.f;
        const float x = fabsf(lo) <= 66000.f ? fminf(fmaxf(lo, -top), top) : lo;
        const float y = fabsf(hi) <= 66000.f ? fminf(fmaxf(hi, -top), top) : hi;
        return pg_pack<false>(x, y);
    }
}

// The attention of one query row by one warp, token after token in fp32: lane l
// holds channels 4l .. 4l + 3.  Slow, and without any value of a token that the
// row does not see.  `mine`: of this lane's channels those that are not finite so far are
// written (what made one so stays in it, and leaves the others right).  The row's lse is
// left: values do not enter it, and blocks that make different channels anew share it.
// bf16 values reach 2^128, and so would sums of a few: a channel whose sum passes 2^100 goes
// on in units of 2^64, in which a sum of 2^24 values stays below 2^88.
template <bool BF16, bool SPARSE>
__device__ __noinline__ void paged_row(const PagedAttnArgs& a, int r, const PagedReq& req, int i, int head, int lane, bool mine) {
    const int h = head / a.G;
    const size_t row = static_cast<size_t>(req.row0) + i;
    const uint2 qw = *reinterpret_cast<const uint2*>(a.q + static_cast<long long>(row) * a.q_stride + head * PG_ROW + lane * 8);
    const float2 q0 = pg_unpack<BF16>(qw.x), q1 = pg_unpack<BF16>(qw.y);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    float unit[4] = {1.f, 1.f, 1.f, 1.f};  // of what is added to o, 1 or 2^-64
    const int sees = paged_sees<SPARSE>(req, i), places = paged_places<SPARSE>(a, sees);
    bool bad = false;
    for (int p = 0; p < places; ++p) {
        const int at = paged_place<SPARSE>(a, r, h, sees, p);
        if (at < 0) {
            bad = true;
            continue;
        }
        const long long base = static_cast<long long>(at / 32) * a.kv_block + h * a.kv_head + lane * 8;
        for (int t = 0; t < at % 32; ++t) {
            const uint2 kw = *reinterpret_cast<const uint2*>(a.kc + base + t * a.kv_token);
            const float2 k0 = pg_unpack<BF16>(kw.x), k1 = pg_unpack<BF16>(kw.y);
            float x = q0.x * k0.x + q0.y * k0.y + q1.x * k1.x + q1.y * k1.y;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(FULL_MASK, x, off);
            x *= a.scale_log2;
            const float mn = fmaxf(m, x);
            const float old = m == -INFINITY ? 0.f : exp2f(m - mn), w = x == -INFINITY ? 0.f : exp2f(x - mn);
            const uint2 vw = *reinterpret_cast<const uint2*>(a.vc + base + t * a.kv_token);
            const float2 v0 = pg_unpack<BF16>(vw.x), v1 = pg_unpack<BF16>(vw.y);
            l = l * old + w;
            const float v[4] = {v0.x, v0.y, v1.x, v1.y};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                o[c] = o[c] * old + w * (v[c] * unit[c]);
                if (BF16 && unit[c] == 1.f && fabsf(o[c]) > 0x1p100f) {
                    unit[c] = 0x1p-64f;
                    o[c] *= unit[c];
                }
            }
            m = mn;
        }
    }
    if (bad && lane == 0) report_error(a.err_flag, CLO_FLAG_BAD_INDEX);
    const bool none = bad || l == 0.f;
    const float inv = none ? 0.f : 1.f / l;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = none ? 0.f : o[c] * inv * (unit[c] == 1.f ? 1.f : 0x1p64f);
    if (!mine) return;
    uint2* const out = reinterpret_cast<uint2*>(a.out + (row * a.Hq + head) * PG_ROW + lane * 8);
    const uint2 first = *out;
    const float2 f0 = pg_unpack<BF16>(first.x), f1 = pg_unpack<BF16>(first.y);
    *out = make_uint2(pg_pack_out<BF16>(pg_finite(f0.x) ? f0.x : o[0], pg_finite(f0.y) ? f0.y : o[1]),
                      pg_pack_out<BF16>(pg_finite(f1.x) ? f1.x : o[2], pg_finite(f1.y) ? f1.y : o[3]));
}

}  // namespace clo
