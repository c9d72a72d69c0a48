// clo_paged_rope.cu -- rotary positions on new tokens' queries and keys, and
// their K and V into the 16-bit paged cache, in one pass over the projections'
// output.
//
// Mathematics.  A pair of channels turns by pos * f.  With f in units of 2^-64 of
// a turn, pos * f modulo 2^64 is one 64-bit product that is exact whatever the
// position; its top 32 bits, as a signed number, are the angle in (-1/2, 1/2)
// turns to 2^-32, which sincospif takes.  No table of cosines is read, no
// position is too far.
//
// A token's rows (query, key and value heads) are cut into units of 32 bytes: two
// 16-byte chunks that hold both sides of 8 pairs (channels 8u .. and rot/2 + 8u ..,
// or 16u .. 16u + 15 for neighbours in pairs).  The CTA makes the sines and cosines
// of its token once, in shared memory, while the rows are on their way; 8 threads
// move a row.  The work is one read and one write of every row, and HBM bounds it: 65536
// tokens of 32 and 8 heads take 265 us (6.1 TB/s).  5003 tokens of 40 and 8 heads take 29.4 us
// in a graph, 4.9 TB/s, with one axis and 29.6 with three.
#include <math.h>

#include "clo_paged.cuh"

namespace clo {

constexpr int ROPE_THREADS = 128;
constexpr int ROPE_ROWS = ROPE_THREADS / 8;   // rows a CTA moves at once
constexpr int ROPE_AHEAD = 3;                 // rows a thread keeps in flight
constexpr int ROPE_MAX_TOKENS = 16;           // tokens a CTA takes where they have few rows

struct RopeArgs {
    const uint8_t* q;
    const uint8_t* k;
    const uint8_t* v;
    uint8_t* q_out;
    long long q_stride, k_stride, v_stride, q_out_stride;  // bytes
    const int32_t* pos;
    const clo_rope_pair* pairs;
    const int32_t* slots;
    uint8_t* kc;
    uint8_t* vc;
    int32_t* err_flag;
    int N, axes, half, Hq, Hkv, num_blocks, tokens;  // half = rot / 2; tokens a CTA
};

// Byte offsets of the two chunks of unit u of a row.
template <bool INTER>
__device__ __forceinline__ void unit_chunks(int u, int half, int& c0, int& c1) {
    if constexpr (INTER) {
        c0 = 32 * u;
        c1 = c0 + 16;
    } else {
        const int units = half / 8;  // units that turn; the others take the rest of the row in order
        c0 = u < units ? 16 * u : 32 * u;
        c1 = u < units ? 16 * u + 2 * half : c0 + 16;
    }
}

// Turns the 8 pairs of a unit; cs holds their 8 cosines and then, 64 floats on, sines.
template <bool BF16, bool INTER>
__device__ __forceinline__ void turn_unit(uint4& x, uint4& y, const float* cs) {
    const float4 ca = *reinterpret_cast<const float4*>(cs), cb = *reinterpret_cast<const float4*>(cs + 4);
    const float4 sa = *reinterpret_cast<const float4*>(cs + 64), sb = *reinterpret_cast<const float4*>(cs + 68);
    const float c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
    const float s[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
    uint32_t* wx = reinterpret_cast<uint32_t*>(&x);
    uint32_t* wy = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = pg_unpack<BF16>(wx[i]), b = pg_unpack<BF16>(wy[i]);
        if constexpr (INTER) {  // words of x are pairs 0..3, of y 4..7
            wx[i] = pg_pack<BF16>(a.x * c[i] - a.y * s[i], a.x * s[i] + a.y * c[i]);
            wy[i] = pg_pack<BF16>(b.x * c[4 + i] - b.y * s[4 + i], b.x * s[4 + i] + b.y * c[4 + i]);
        } else {  // word i holds one side of pairs 2i and 2i + 1
            wx[i] = pg_pack<BF16>(a.x * c[2 * i] - b.x * s[2 * i], a.y * c[2 * i + 1] - b.y * s[2 * i + 1]);
            wy[i] = pg_pack<BF16>(a.x * s[2 * i] + b.x * c[2 * i], a.y * s[2 * i + 1] + b.y * c[2 * i + 1]);
        }
    }
}

template <bool BF16, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS) rope_append_kernel(const RopeArgs a) {
    __shared__ __align__(16) float cs[ROPE_MAX_TOKENS][128];  // cosines, then sines, of a token's pairs
    __shared__ int slot_of[ROPE_MAX_TOKENS];
    pdl_launch_dependents();
    pdl_wait();
    const int n0 = blockIdx.x * a.tokens;
    const int tokens = min(a.tokens, a.N - n0);
    const int heads = a.Hq + 2 * a.Hkv;
    const int rows = tokens * heads;
    const int u = threadIdx.x & 7;
    int c0, c1;
    unit_chunks<INTER>(u, a.half, c0, c1);

    // Row i of the CTA: its token, its place in the inputs.
    auto source = [&](int i, int& t, int& h) {
        t = i / heads;
        h = i - t * heads;
        const long long n = n0 + t;
        return h < a.Hq             ? a.q + n * a.q_stride + h * PG_ROW
               : h < a.Hq + a.Hkv   ? a.k + n * a.k_stride + (h - a.Hq) * PG_ROW
                                    : a.v + n * a.v_stride + (h - a.Hq - a.Hkv) * PG_ROW;
    };
    uint4 x[ROPE_AHEAD], y[ROPE_AHEAD];
    auto load = [&](int first) {
#pragma unroll
        for (int j = 0; j < ROPE_AHEAD; ++j) {
            const int i = first + j * ROPE_ROWS;
            if (i < rows) {
                int t, h;
                const uint8_t* src = source(i, t, h);
                x[j] = *reinterpret_cast<const uint4*>(src + c0);
                y[j] = *reinterpret_cast<const uint4*>(src + c1);
            }
        }
    };
    int row = threadIdx.x >> 3;
    load(row);  // on their way while the sines are made

    bool bad = false;
    for (int i = threadIdx.x; i < tokens * a.half; i += ROPE_THREADS) {
        const int t = i / a.half, p = i - t * a.half;
        const clo_rope_pair pr = a.pairs[p];
        const bool axis_ok = pr.axis >= 0 && pr.axis < a.axes;
        bad |= !axis_ok;
        const int32_t pos = a.pos[static_cast<size_t>(axis_ok ? pr.axis : 0) * a.N + n0 + t];
        const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(pos)) * pr.turns;
        // Half turns in [-1, 1): the top 32 bits as a signed number, times 2^-31.
        const float half_turns = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 4.656612873077393e-10f;
        float s, c;
        sincospif(half_turns, &s, &c);
        cs[t][p] = c;
        cs[t][64 + p] = s;
    }
    if (static_cast<int>(threadIdx.x) < tokens) {
        const int s = a.slots[n0 + threadIdx.x];
        const bool ok = s >= 0 && s < a.num_blocks * PG_BLOCK;
        bad |= s < -1 || (s >= 0 && !ok);
        slot_of[threadIdx.x] = ok ? s : -1;
    }
    __syncthreads();
    const bool turns = u < a.half / 8;
    for (; row < rows; row += ROPE_AHEAD * ROPE_ROWS) {
#pragma unroll
        for (int j = 0; j < ROPE_AHEAD; ++j) {
            const int i = row + j * ROPE_ROWS;
            if (i >= rows) break;
            const int t = i / heads, h = i - t * heads;
            if (turns && h < a.Hq + a.Hkv) turn_unit<BF16, INTER>(x[j], y[j], &cs[t][8 * u]);
            uint8_t* dst;
            if (h < a.Hq) {
                dst = a.q_out + static_cast<long long>(n0 + t) * a.q_out_stride + h * PG_ROW;
            } else {
                const int s = slot_of[t], g = h < a.Hq + a.Hkv ? h - a.Hq : h - a.Hq - a.Hkv;
                if (s < 0) continue;
                const long long r = (static_cast<long long>(s / PG_BLOCK) * a.Hkv + g) * PG_BLOCK + s % PG_BLOCK;
                dst = (h < a.Hq + a.Hkv ? a.kc : a.vc) + r * PG_ROW;
            }
            *reinterpret_cast<uint4*>(dst + c0) = x[j];
            *reinterpret_cast<uint4*>(dst + c1) = y[j];
        }
        load(row + ROPE_AHEAD * ROPE_ROWS);
    }
    if (bad) report_error(a.err_flag, CLO_FLAG_BAD_INDEX);
}

// Whether rows of `row` bytes, `stride` apart, of the two tensors share bytes
// (taken as whole ranges).
static bool ranges_meet(const void* p, long long ps, long long prow, const void* q, long long qs, long long qrow,
                        int N) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + static_cast<uintptr_t>((N - 1) * qs + qrow) && b < a + static_cast<uintptr_t>((N - 1) * ps + prow);
}

}  // namespace clo

using namespace clo;

extern "C" clo_status clo_rope_pairs(const double* inv_freq, const int32_t* axis, int n, clo_rope_pair* pairs) {
    if (n < 0 || (n > 0 && (inv_freq == nullptr || pairs == nullptr))) return CLO_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        if (!(fabs(inv_freq[i]) < 1048576.0) || (axis != nullptr && (axis[i] < 0 || axis[i] >= 4)))
            return CLO_ERR_INVALID_ARG;
    // 1 / (2 pi) * 2^128, in two words.
    constexpr uint64_t C_HIGH = 0x28be60db9391054aull, C_LOW = 0x7f09d5f47d4d3770ull;
    for (int i = 0; i < n; ++i) {
        int e = 0;
        const double f = frexp(fabs(inv_freq[i]), &e);
        const uint64_t m = static_cast<uint64_t>(ldexp(f, 53));  // |inv_freq| = m * 2^(e - 53)
        // m / (2 pi) * 2^64, below 2^115, without its fraction.
        const unsigned __int128 p = static_cast<unsigned __int128>(m) * C_HIGH +
                                    static_cast<uint64_t>((static_cast<unsigned __int128>(m) * C_LOW) >> 64);
        const int shift = 53 - e;  // at least 33
        uint64_t turns = 0;
        if (shift < 128) {
            const unsigned __int128 q = p >> (shift - 1);  // rounded by the last bit that goes
            turns = static_cast<uint64_t>((q >> 1) + (q & 1));
        }
        pairs[i].turns = inv_freq[i] < 0 ? 0 - turns : turns;
        pairs[i].axis = axis != nullptr ? axis[i] : 0;
        pairs[i].reserved = 0;
    }
    return CLO_OK;
}

extern "C" clo_status clo_paged_rope_append(const clo_paged_rope_append_args* args, cudaStream_t stream) {
    if (args == nullptr) return CLO_ERR_INVALID_ARG;
    const clo_paged_rope_append_args& r = *args;
    if (r.N < 0 || r.Hq < 0 || r.Hkv < 1 || r.num_blocks < 1 || r.axes < 1 || r.rot < 0 || !pg_dtype_ok(r.dtype))
        return CLO_ERR_INVALID_ARG;
    if ((r.q == nullptr) != (r.q_out == nullptr)) return CLO_ERR_INVALID_ARG;
    const int Hq = r.q == nullptr ? 0 : r.Hq;
    if (r.N > 0 && (r.k == nullptr || r.v == nullptr || r.pos == nullptr || (r.pairs == nullptr && r.rot > 0) ||
                    r.slot_map == nullptr || r.kc == nullptr || r.vc == nullptr))
        return CLO_ERR_INVALID_ARG;
    for (const void* p : {r.q, r.k, r.v, static_cast<const void*>(r.q_out), static_cast<const void*>(r.kc),
                          static_cast<const void*>(r.vc), static_cast<const void*>(r.pairs)})
        if (!pg_aligned(p, 16)) return CLO_ERR_INVALID_ARG;
    if (!pg_aligned(r.pos, 4) || !pg_aligned(r.slot_map, 4) || !pg_aligned(r.err_flag, 4)) return CLO_ERR_INVALID_ARG;
    if (r.d != PG_D || r.block_size != PG_BLOCK || r.rot > PG_D || r.rot % 16 != 0 || r.axes > 4)
        return CLO_ERR_UNSUPPORTED;
    const long long heads = static_cast<long long>(Hq) + 2ll * r.Hkv;
    if (r.N * heads >= (1ll << 31) - (1 << 20) || heads > (1 << 20) || r.num_blocks > (1 << 26))
        return CLO_ERR_UNSUPPORTED;
    if (r.N == 0) return CLO_OK;
    RopeArgs a{};
    const auto stride_ok = [&](long long s, int h) {
        return r.N == 1 || (s >= static_cast<long long>(h) * r.d && s % 8 == 0 && s <= (1ll << 40));
    };
    if ((Hq > 0 && (!stride_ok(r.q_stride, Hq) || !stride_ok(r.q_out_stride, Hq))) || !stride_ok(r.k_stride, r.Hkv) ||
        !stride_ok(r.v_stride, r.Hkv))
        return CLO_ERR_INVALID_ARG;
    const long long one = r.N > 1;
    a.q_stride = one * 2 * r.q_stride;
    a.k_stride = one * 2 * r.k_stride;
    a.v_stride = one * 2 * r.v_stride;
    a.q_out_stride = one * 2 * r.q_out_stride;
    if (Hq > 0) {
        // In place, or apart: q_out in the same rows as q, or beside them.  (Inputs
        // that interleave with q_out's rows in one fused buffer are told apart by
        // rows: see below.)
        const long long qrow = static_cast<long long>(Hq) * PG_ROW, krow = static_cast<long long>(r.Hkv) * PG_ROW;
        const bool same = r.q == r.q_out && a.q_stride == a.q_out_stride;
        const auto apart = [&](const void* p, long long ps, long long prow) {
            if (!ranges_meet(r.q_out, a.q_out_stride, qrow, p, ps, prow, r.N)) return true;
            // Ranges that meet are apart only as columns of the same rows.
            if (ps != a.q_out_stride || r.N == 1) return false;
            const long long gap = (static_cast<long long>(reinterpret_cast<uintptr_t>(p)) -
                                   static_cast<long long>(reinterpret_cast<uintptr_t>(r.q_out))) % ps;
            const long long at = gap < 0 ? gap + ps : gap;  // where p's row starts after a row of q_out
            return at >= qrow && at + prow <= ps;
        };
        if ((!same && !apart(r.q, a.q_stride, qrow)) || !apart(r.k, a.k_stride, krow) || !apart(r.v, a.v_stride, krow))
            return CLO_ERR_INVALID_ARG;
    }
    a.q = static_cast<const uint8_t*>(r.q);
    a.k = static_cast<const uint8_t*>(r.k);
    a.v = static_cast<const uint8_t*>(r.v);
    a.q_out = static_cast<uint8_t*>(r.q_out);
    a.pos = r.pos;
    a.pairs = r.pairs;
    a.slots = r.slot_map;
    a.kc = static_cast<uint8_t*>(r.kc);
    a.vc = static_cast<uint8_t*>(r.vc);
    a.err_flag = r.err_flag;
    a.N = r.N;
    a.axes = r.axes;
    a.half = r.rot / 2;
    a.Hq = Hq;
    a.Hkv = r.Hkv;
    a.num_blocks = r.num_blocks;
    // A token a CTA, or as many as fill its threads.
    a.tokens = heads >= ROPE_ROWS ? 1 : static_cast<int>((ROPE_ROWS + heads - 1) / heads);
    const unsigned grid = static_cast<unsigned>((r.N + a.tokens - 1) / a.tokens);
    const auto kernel = r.dtype == CLO_BF16
                            ? (r.interleaved ? rope_append_kernel<true, true> : rope_append_kernel<true, false>)
                            : (r.interleaved ? rope_append_kernel<false, true> : rope_append_kernel<false, false>);
    if (!prepare_kernel(reinterpret_cast<const void*>(kernel), 0)) return CLO_ERR_CUDA;
    return launch_pdl(kernel, dim3(grid), dim3(ROPE_THREADS), 0, stream, a) == cudaSuccess ? CLO_OK : CLO_ERR_CUDA;
}
