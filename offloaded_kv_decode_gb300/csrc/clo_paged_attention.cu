// clo_paged_attention.cu -- attention of chunks of new tokens over the 16-bit
// paged cache, and decode attention over selected blocks of it.
#include <math.h>

#include "clo_paged_attention.cuh"

namespace clo {

constexpr int ROWS_THREADS = 256;

// A warp a (query row, head).
template <bool BF16, bool SPARSE>
__global__ void __launch_bounds__(ROWS_THREADS) paged_rows_kernel(const PagedAttnArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long warps = static_cast<long long>(gridDim.x) * (ROWS_THREADS / 32);
    const long long w0 = blockIdx.x * static_cast<long long>(ROWS_THREADS / 32) + (threadIdx.x >> 5);
    for (int r = 0; r < a.B; ++r) {
        const PagedReq req = paged_request<SPARSE>(a, r);
        if (req.bad && w0 == 0 && lane == 0) report_error(a.err_flag, CLO_FLAG_BAD_CTX);
        for (long long w = w0; w < static_cast<long long>(req.n) * a.Hq; w += warps)
            paged_row<BF16, SPARSE>(a, r, req, static_cast<int>(w / a.Hq), static_cast<int>(w % a.Hq), lane);
    }
}

static clo_status run_paged_attention(const PagedAttnArgs& a, bool sparse, clo_dtype dtype, const clo_attn_opts* opts,
                                      cudaStream_t stream) {
    const auto kernel = dtype == CLO_BF16 ? (sparse ? paged_rows_kernel<true, true> : paged_rows_kernel<true, false>)
                                          : (sparse ? paged_rows_kernel<false, true> : paged_rows_kernel<false, false>);
    if (!prepare_kernel(reinterpret_cast<const void*>(kernel), 0)) return CLO_ERR_CUDA;
    if (opts != nullptr && opts->ev_begin != nullptr && !record_event(opts->ev_begin, stream)) return CLO_ERR_CUDA;
    if (launch_pdl(kernel, dim3(device_sm_count() * 8), dim3(ROWS_THREADS), 0, stream, a) != cudaSuccess) return CLO_ERR_CUDA;
    if (opts != nullptr && opts->ev_end != nullptr && !record_event(opts->ev_end, stream)) return CLO_ERR_CUDA;
    return CLO_OK;
}

constexpr int CHUNK_MAX_CTAS = 4095;
constexpr int CHUNK_ROWS = 256;  // rows (query, head of the group) a CTA works on at once
// Workspace a CTA: two partial results of 256 rows, and 128 bytes that say of what.
constexpr size_t CHUNK_WS_CTA = 2 * CHUNK_ROWS * (PG_D * sizeof(float) + sizeof(float2)) + 128;

}  // namespace clo

using namespace clo;

extern "C" size_t clo_paged_chunk_workspace_size(int Hq, int Hkv, int d, int num_ctas) {
    if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > PG_MAX_G || d != PG_D || num_ctas < 0 || num_ctas > CHUNK_MAX_CTAS)
        return 0;
    const int ctas = num_ctas > 0 ? num_ctas : device_sm_count();
    return static_cast<size_t>(ctas) * CHUNK_WS_CTA;
}

// What both calls check.
static clo_status check_paged(const void* q, const void* kc, const void* vc, const int32_t* table, const int32_t* ctx,
                              const int32_t* lists, const void* out, const float* lse, const void* ws, size_t ws_bytes,
                              const int32_t* err_flag, const clo_attn_opts* opts, clo_dtype dtype, float scale, int B,
                              long long rows, int Hq, int Hkv, int d, int num_blocks, int block_size, int max_blocks) {
    if (B < 0 || rows < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || num_blocks < 1 || max_blocks < 1 || !pg_dtype_ok(dtype))
        return CLO_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !isfinite(scale)) return CLO_ERR_INVALID_ARG;
    if (opts != nullptr && opts->num_ctas < 0) return CLO_ERR_INVALID_ARG;
    if (B > 0 && rows > 0 && (q == nullptr || kc == nullptr || vc == nullptr || table == nullptr || ctx == nullptr ||
                              lists == nullptr || out == nullptr))
        return CLO_ERR_INVALID_ARG;
    for (const void* p : {q, kc, vc, out})
        if (!pg_aligned(p, 16)) return CLO_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(table), static_cast<const void*>(ctx), static_cast<const void*>(lists),
                          static_cast<const void*>(lse), static_cast<const void*>(err_flag)})
        if (!pg_aligned(p, 4)) return CLO_ERR_INVALID_ARG;
    if (d != PG_D || block_size != PG_BLOCK || Hq / Hkv > PG_MAX_G || B > PG_MAX_B || rows * Hq >= (1ll << 31) ||
        max_blocks > (1 << 20) || num_blocks > (1 << 26) || (opts != nullptr && opts->num_ctas > CHUNK_MAX_CTAS))
        return CLO_ERR_UNSUPPORTED;
    if (B > 0 && rows > 0) {
        const size_t need = clo_paged_chunk_workspace_size(Hq, Hkv, d, opts != nullptr ? opts->num_ctas : 0);
        if (need == 0) return CLO_ERR_CUDA;
        if (ws == nullptr || ws_bytes < need || !pg_aligned(ws, 16)) return CLO_ERR_WORKSPACE;
    }
    return CLO_OK;
}

extern "C" clo_status clo_paged_chunk_attn(const clo_paged_chunk_attn_args* args, cudaStream_t stream) {
    if (args == nullptr) return CLO_ERR_INVALID_ARG;
    const clo_paged_chunk_attn_args& r = *args;
    const clo_status st = check_paged(r.q, r.kc, r.vc, r.block_table, r.ctx_len, r.offsets, r.out, r.lse, r.workspace, r.ws_bytes,
                                      r.err_flag, r.opts, r.dtype, r.scale, r.B, r.N, r.Hq, r.Hkv, r.d, r.num_blocks,
                                      r.block_size, r.max_blocks);
    if (st != CLO_OK) return st;
    if (r.B == 0 || r.N == 0) return CLO_OK;
    const long long row = static_cast<long long>(r.Hq) * r.d;
    if (r.N > 1 && (r.q_stride < row || r.q_stride % 8 != 0 || r.q_stride > (1ll << 38))) return CLO_ERR_INVALID_ARG;
    long long kb = r.kv_block, kh = r.kv_head, kt = r.kv_token;
    if (kb == 0 && kh == 0 && kt == 0) {
        kt = r.d;
        kh = static_cast<long long>(PG_BLOCK) * r.d;
        kb = kh * r.Hkv;
    }
    for (const long long s : {kb, kh, kt})
        if (s < r.d || s % 8 != 0 || s > (1ll << 38)) return CLO_ERR_INVALID_ARG;
    // The output may be the queries only row for row.
    if (r.out == r.q && r.N > 1 && r.q_stride != row) return CLO_ERR_INVALID_ARG;
    PagedAttnArgs a{};
    a.q = static_cast<const uint8_t*>(r.q);
    a.kc = static_cast<const uint8_t*>(r.kc);
    a.vc = static_cast<const uint8_t*>(r.vc);
    a.out = static_cast<uint8_t*>(r.out);
    a.lse = r.lse;
    a.table = r.block_table;
    a.ctx_len = r.ctx_len;
    a.offsets = r.offsets;
    a.err_flag = r.err_flag;
    a.q_stride = r.N > 1 ? 2 * r.q_stride : 0;
    a.kv_block = 2 * kb;
    a.kv_head = 2 * kh;
    a.kv_token = 2 * kt;
    a.scale_log2 = r.scale * LOG2E;
    a.B = r.B;
    a.N = r.N;
    a.Hq = r.Hq;
    a.Hkv = r.Hkv;
    a.G = r.Hq / r.Hkv;
    a.num_blocks = r.num_blocks;
    a.max_blocks = r.max_blocks;
    return run_paged_attention(a, false, r.dtype, r.opts, stream);
}

extern "C" clo_status clo_paged_sparse_decode_attn(const clo_paged_sparse_attn_args* args, cudaStream_t stream) {
    if (args == nullptr) return CLO_ERR_INVALID_ARG;
    const clo_paged_sparse_attn_args& r = *args;
    const clo_status st = check_paged(r.q, r.kc, r.vc, r.block_table, r.ctx_len, r.sel, r.out, r.lse, r.workspace, r.ws_bytes,
                                      r.err_flag, r.opts, r.dtype, r.scale, r.B, r.B, r.Hq, r.Hkv, r.d, r.num_blocks,
                                      r.block_size, r.max_blocks);
    if (st != CLO_OK) return st;
    if (r.n_sel < 1) return CLO_ERR_INVALID_ARG;
    if (static_cast<long long>(r.B) * r.Hkv * r.n_sel >= (1ll << 31)) return CLO_ERR_UNSUPPORTED;
    if (r.B == 0) return CLO_OK;
    PagedAttnArgs a{};
    a.q = static_cast<const uint8_t*>(r.q);
    a.kc = static_cast<const uint8_t*>(r.kc);
    a.vc = static_cast<const uint8_t*>(r.vc);
    a.out = static_cast<uint8_t*>(r.out);
    a.lse = r.lse;
    a.table = r.block_table;
    a.ctx_len = r.ctx_len;
    a.sel = r.sel;
    a.err_flag = r.err_flag;
    a.q_stride = 2ll * r.Hq * r.d;
    a.kv_token = PG_ROW;
    a.kv_head = PG_BLOCK_BYTES;
    a.kv_block = static_cast<long long>(PG_BLOCK_BYTES) * r.Hkv;
    a.scale_log2 = r.scale * LOG2E;
    a.B = r.B;
    a.N = r.B;
    a.Hq = r.Hq;
    a.Hkv = r.Hkv;
    a.G = r.Hq / r.Hkv;
    a.num_blocks = r.num_blocks;
    a.max_blocks = r.max_blocks;
    a.n_sel = r.n_sel;
    return run_paged_attention(a, true, r.dtype, r.opts, stream);
}
