// clo_kv4_attention.cu -- clo_kv4_paged_decode_attn: decode attention over
// the paged cache held in 4 bits (format: clo_kv4.h).
//
// One CTA a (request, KV head, query row); its warps take the tokens in turn,
// a lane 4 channels of a row, with an online softmax a warp and one merge of
// the warps at the end.
#include <math.h>

#include "clo_kv4.cuh"

namespace clo {

constexpr int KV4_WARPS = 8;
constexpr int KV4_MAX_ROWS = 32;  // query rows a KV head: G * n_q

struct Kv4Args {
    const void* q;
    void* out;
    float* lse;
    const uint8_t* pool;
    const int32_t* table;
    const int32_t* ctx_len;
    int32_t* err_flag;
    float scale;
    int max_blocks, num_blocks, B, n_q, Hq, Hkv, G;
};

template <bool BF16, int NG>
__global__ void __launch_bounds__(KV4_WARPS * 32) kv4_attn_kernel(const Kv4Args a) {
    __shared__ float sm_m[KV4_WARPS], sm_l[KV4_WARPS], sm_o[KV4_WARPS][KV4_D];
    __shared__ int sm_bad;
    pdl_launch_dependents();
    pdl_wait();
    if (threadIdx.x == 0) sm_bad = 0;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.x / a.Hkv, h = blockIdx.x - r * a.Hkv;
    const int qi = blockIdx.y / a.G, g = blockIdx.y - qi * a.G;
    const size_t row = (static_cast<size_t>(r) * a.n_q + qi) * a.Hq + static_cast<size_t>(h) * a.G + g;
    int n = a.ctx_len[r];
    const bool bad_len = n < 0 || n > a.max_blocks * KV4_BLOCK;
    if (bad_len && threadIdx.x == 0) report_error(a.err_flag, CLO_FLAG_BAD_CTX);
    n = bad_len ? 0 : n;
    const int see = n - (a.n_q - 1 - qi);
    const uint2 qw = reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.q) + row * KV4_D * 2)[lane];
    const float2 q01 = kv4_unpack2<BF16>(qw.x), q23 = kv4_unpack2<BF16>(qw.y);
    const int i = lane >> 1, sh = (lane & 1) * 16, grp = lane / (32 / NG);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    // Every block of the request is checked, also behind what this query sees.
    for (int t = warp; t < n; t += KV4_WARPS) {
        const int id = a.table[static_cast<size_t>(r) * a.max_blocks + t / KV4_BLOCK];
        if (id < 0 || id >= a.num_blocks) {
            if (lane == 0) {
                report_error(a.err_flag, CLO_FLAG_BAD_INDEX);
                atomicOr(&sm_bad, 1);
            }
            continue;
        }
        if (t >= see) continue;
        const int tt = t % KV4_BLOCK;
        const uint8_t* rec = a.pool + (static_cast<size_t>(id) * a.Hkv + h) * kv4_record(NG);
        const uint32_t kc = *reinterpret_cast<const uint32_t*>(rec + kv4_k_word(tt, i)) >> sh;
        const uint32_t vc = *reinterpret_cast<const uint32_t*>(rec + kv4_v_word(tt, i)) >> sh;
        const float2 kp = __half22float2(*reinterpret_cast<const __half2*>(rec + kv4_param(tt, 0, NG, grp)));
        const float2 vp = __half22float2(*reinterpret_cast<const __half2*>(rec + kv4_param(tt, 1, NG, grp)));
        const float qv[4] = {q01.x, q01.y, q23.x, q23.y};
        float x = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) x = fmaf(qv[j], fmaf(static_cast<float>((kc >> (4 * j)) & 15u), kp.x, kp.y), x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(FULL_MASK, x, off);
        x *= a.scale * LOG2E;
        const float mn = fmaxf(m, x);
        const float al = fast_exp2(m - mn), p = fast_exp2(x - mn);
        l = fmaf(l, al, p);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = fmaf(o[j], al, p * fmaf(static_cast<float>((vc >> (4 * j)) & 15u), vp.x, vp.y));
        m = mn;
    }
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sm_o[warp][4 * lane + j] = o[j];
    __syncthreads();
    if (warp != 0) return;
    float M = -INFINITY, L = 0.f, O[4] = {0.f, 0.f, 0.f, 0.f};
    for (int w = 0; w < KV4_WARPS; ++w) M = fmaxf(M, sm_m[w]);
    for (int w = 0; w < KV4_WARPS; ++w) {
        if (sm_m[w] == -INFINITY && sm_l[w] == 0.f) continue;
        const float e = fast_exp2(sm_m[w] - M);
        L = fmaf(sm_l[w], e, L);
        for (int j = 0; j < 4; ++j) O[j] = fmaf(sm_o[w][4 * lane + j], e, O[j]);
    }
    const bool none = sm_bad != 0 || L == 0.f;
    const float inv = none ? 0.f : 1.f / L;
    uint2 pk;
    pk.x = none ? 0u : kv4_pack2<BF16>(O[0] * inv, O[1] * inv);
    pk.y = none ? 0u : kv4_pack2<BF16>(O[2] * inv, O[3] * inv);
    reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + row * KV4_D * 2)[lane] = pk;
    if (a.lse != nullptr && lane == 0) a.lse[row] = none ? -INFINITY : (M + log2f(L)) * LN2;
}

template <bool BF16>
static void (*attn_kernel(int ng))(const Kv4Args) {
    return ng == 1 ? kv4_attn_kernel<BF16, 1> : ng == 2 ? kv4_attn_kernel<BF16, 2> : kv4_attn_kernel<BF16, 4>;
}

}  // namespace clo

using namespace clo;

extern "C" size_t clo_kv4_paged_workspace_size(int B, int n_q, int Hq, int Hkv, int d, int num_ctas) {
    if (B < 0 || n_q < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || d != KV4_D || num_ctas < 0) return 0;
    if (static_cast<long long>(Hq / Hkv) * n_q > KV4_MAX_ROWS) return 0;
    return 256;
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
    if (static_cast<long long>(B) * Hkv * max_blocks >= (1ll << 31) || max_blocks > (1 << 26))
        return CLO_ERR_UNSUPPORTED;
    if (B == 0) return CLO_OK;
    const size_t need = clo_kv4_paged_workspace_size(B, n_q, Hq, Hkv, d, opts != nullptr ? opts->num_ctas : 0);
    if (workspace == nullptr || ws_bytes < need || !kv4_aligned(workspace, 16)) return CLO_ERR_WORKSPACE;

    Kv4Args a;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.pool = pool;
    a.table = block_table;
    a.ctx_len = ctx_len;
    a.err_flag = err_flag;
    a.scale = scale;
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    a.B = B;
    a.n_q = n_q;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    const auto kernel = dtype == CLO_BF16 ? attn_kernel<true>(ng) : attn_kernel<false>(ng);
    if (!prepare_kernel(reinterpret_cast<const void*>(kernel), 0)) return CLO_ERR_CUDA;
    if (opts != nullptr && opts->ev_begin != nullptr && !record_event(opts->ev_begin, stream)) return CLO_ERR_CUDA;
    if (launch_pdl(kernel, dim3(static_cast<unsigned>(B) * Hkv, a.G * n_q), dim3(KV4_WARPS * 32), 0, stream, a) !=
        cudaSuccess)
        return CLO_ERR_CUDA;
    if (opts != nullptr && opts->ev_end != nullptr && !record_event(opts->ev_end, stream)) return CLO_ERR_CUDA;
    return CLO_OK;
}
