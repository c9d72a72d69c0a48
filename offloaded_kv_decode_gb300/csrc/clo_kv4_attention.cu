// clo_kv4_attention.cu -- clo_kv4_paged_decode_attn: decode attention over
// the paged cache held in 4 bits (format: clo_kv4.h; a warp's work:
// clo_kv4_math.cuh).
//
// There are two kernels; clo_kv4_sets.cu says when the other one is taken.
//
// Work split.  A unit is 32 tokens of one KV head: the records of two blocks
// (2176 to 2560 bytes each, K, V and parameters together), a bulk copy each.
// All units of the call form one stream, ordered by request, head and
// position, cut into equal ranges, one a warp; each warp keeps a ring of units
// in flight.  A (request, KV head) that lies in one warp's range is finished by
// that warp alone.  What crosses ranges is merged once a CTA at its end, and
// what crosses CTAs leaves one fp32 partial a CTA, merged by a second kernel.
// The split depends on the lengths, the table's width and the grid alone, so the
// bits of a result do not depend on timing.
#include <algorithm>

#include "clo_kv4_math.cuh"

namespace clo {

constexpr int KV4_MAX_CTAS = 4095;       // of 16 warps: warps squared stay in 32 bits
constexpr int KV4_FLAT_WARPS = 16;       // of a CTA, at most
constexpr int KV4_FLAT_SMEM = 225 * 1024;     // dynamic, at most
constexpr int KV4_FLAT_RESERVED = 1024 + 1536;  // beside it: the system's, and the static arrays
constexpr int KV4_MERGE_THREADS = 512;
constexpr int KV4_MERGE_UNROLL = 8;
// What starting and ending a token set costs a warp, in units.  With 2, 4, 6 and
// 8: 32 requests of 1 to 4096 tokens (8 KV heads, 16 query rows each) 43.2, 41.2,
// 39.6 and 39.2 us; 24 of 1 to 16384 (32 rows) 118, 113, 109 and 109; 128 of 1 to
// 8192 (4 rows) 119.4, 118.9, 118.9 and 119.7.  Without it, 128 requests of 128
// to 4096 tokens took a third longer.
constexpr int KV4_SET_COST = 6;
// Units that a warp's accumulators take in before what the channels have in
// common is taken out of them (level_sums).  16 requests of 32K tokens (4 query
// rows a KV head) 94 us, against 99 in one loop without it, with 32 query rows
// and 16K tokens 139 against 137; every 32 units measured the same.
constexpr int KV4_LEVEL_UNITS = 16;

// Units of request r of one KV head; 0 if it is empty or its length is bad.
__device__ __forceinline__ int kv4_units(const Kv4Args& a, int r, bool& bad) {
    const int n = a.ctx_len[r];
    bad = n < 0 || n > a.max_blocks * KV4_BLOCK;
    return bad ? 0 : (n + KV4_UNIT - 1) / KV4_UNIT;
}

// The stream the warps share: each token set (request, KV head) with a token
// is KV4_SET_COST steps for its start and end, then a step a unit.  prefix[r] =
// steps of the requests before r (all heads), r <= B.
__device__ __forceinline__ int kv4_steps(const Kv4Args& a, int r, bool& bad) {
    const int n = kv4_units(a, r, bad);
    return n > 0 ? (n + KV4_SET_COST) * a.Hkv : 0;
}

__device__ __forceinline__ void kv4_prefix(const Kv4Args& a, int* prefix, int* wsum) {
    const int per = (a.B + blockDim.x - 1) / blockDim.x;
    const int r0 = min(a.B, static_cast<int>(threadIdx.x) * per), r1 = min(a.B, r0 + per);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool bad, any_bad = false;
    int mine = 0;
    for (int r = r0; r < r1; ++r) {
        const int steps = kv4_steps(a, r, bad);
        prefix[r + 1] = steps;
        mine += steps;
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
        run += prefix[r + 1];
        prefix[r + 1] = run;
    }
    __syncthreads();
}

// W warps share N steps equally: warp g from at(g) on, that is floor(N g / W), in
// 32 bits.  (Equal shares although the warps of an SM do not advance alike: each
// of its schedulers prefers the oldest of its warps, which ends a third earlier
// than the youngest.  Weighing the shares by age measured 3 to 8% slower.)
struct Kv4Split {
    unsigned N, W, each, rest;
    __device__ __forceinline__ Kv4Split(int steps, unsigned warps) : N(steps), W(min(warps, N)) {
        each = W > 0 ? N / W : 0u;
        rest = N - each * W;
    }
    __device__ __forceinline__ int at(unsigned g) const { return g < W ? each * g + rest * g / W : N; }
    // The warp that step t < N belongs to.
    __device__ __forceinline__ unsigned owner(int t) const {
        unsigned g = min(W - 1, static_cast<unsigned>(static_cast<float>(t) / static_cast<float>(N) * static_cast<float>(W)));
        while (g > 0 && at(g) > t) --g;
        while (g + 1 < W && at(g + 1) <= t) ++g;
        return g;
    }
};

// A unit: j of nt of request r's head h.
struct Place {
    int r, h, j, nt;
};

// The first unit at step t or behind it (r == B: there is none).
__device__ __forceinline__ Place kv4_place(const int* prefix, int B, int Hkv, int t) {
    Place p;
    if (t >= prefix[B]) {
        p.r = B;
        p.h = p.j = p.nt = 0;
        return p;
    }
    int lo = 0, hi = B - 1;  // the last request with prefix[r] <= t: skips empty ones
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int steps = (prefix[lo + 1] - prefix[lo]) / Hkv;
    p.r = lo;
    p.nt = steps - KV4_SET_COST;
    p.h = (t - prefix[lo]) / steps;
    p.j = max(t - prefix[lo] - p.h * steps - KV4_SET_COST, 0);
    return p;
}

// The first unit of the next set (r == B: there is none).
__device__ __forceinline__ void kv4_next_set(const int* prefix, int B, int Hkv, Place& p) {
    p.j = 0;
    if (++p.h < Hkv) return;
    p.h = 0;
    do {
        ++p.r;
    } while (p.r < B && prefix[p.r + 1] == prefix[p.r]);
    p.nt = p.r < B ? (prefix[p.r + 1] - prefix[p.r]) / Hkv - KV4_SET_COST : 0;
}

// Asks for the queries of a set ahead of its start.
__device__ __forceinline__ void prefetch_queries(const Kv4Args& a, const Place& p, int lane) {
    for (int line = lane; line < 2 * a.rows; line += 32) {
        const int qi = (line >> 1) / a.G, g = (line >> 1) - qi * a.G;
        const size_t at = (static_cast<size_t>(p.r) * a.n_q + qi) * a.Hq + static_cast<size_t>(p.h) * a.G + g;
        prefetch_l1(static_cast<const uint8_t*>(a.q) + at * KV4_D * 2 + (line & 1) * 128);
    }
}

// Shared memory of a CTA, in bytes from its start.
struct Kv4Layout {
    int ring, warp, bars, prefix, total;  // ring, warp: bytes of a warp's ring, and with its queries
};

__host__ __device__ inline Kv4Layout kv4_layout(int warps, int nt, int ng, int rows, int B) {
    Kv4Layout y;
    y.ring = kv4_stages(ng) * 2 * kv4_record(ng);
    const int piece = rows * KV4_PIECE_ROW * static_cast<int>(sizeof(float));
    const int both = y.ring + kv4_query_bytes(nt, ng);
    y.warp = ((both > piece ? both : piece) + 127) / 128 * 128;  // the last piece takes their place
    y.bars = warps * y.warp;
    y.prefix = y.bars + warps * kv4_stages(ng) * 8;
    y.total = y.prefix + (B + 1) * static_cast<int>(sizeof(int));
    return y;
}

// All warps of an SM in one CTA, so that their pieces meet in shared memory and
// the prefix sums are made once an SM: 16 requests of 64K tokens 212 us against
// 219 with CTAs of 4 warps.  With 4 n8 tiles of queries (8 warps an SM) two CTAs
// of 4 are faster: 16 requests of 16K tokens and 32 query rows 127 us against 136.
__host__ __device__ constexpr int kv4_flat_ctas(int nt) { return nt == 4 ? 2 : 1; }
__host__ __device__ constexpr int kv4_flat_warps(int nt) { return 4 * kv4_ctas_per_sm(nt) / kv4_flat_ctas(nt); }

template <bool BF16, int NT, int NG>
__global__ void __launch_bounds__(kv4_flat_warps(NT) * 32, kv4_flat_ctas(NT)) kv4_attn_kernel(const Kv4Args a) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int wsum[KV4_FLAT_WARPS];
    __shared__ Place walks[KV4_FLAT_WARPS][3];
    __shared__ int4 piece_of[2 * KV4_FLAT_WARPS];  // (token set, request, its units' first step, the step behind them) of
                                              // each warp's first and last piece; set -1: none
    constexpr int R = kv4_record(NG), STAGES = kv4_stages(NG);
    const int warps = blockDim.x >> 5, threads = blockDim.x;
    const Kv4Layout y = kv4_layout(warps, NT, NG, a.rows, a.B);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* ring = smem + warp * y.warp;
    const uint32_t bars = smem_u32(smem + y.bars) + warp * STAGES * 8;
    int* prefix = reinterpret_cast<int*>(smem + y.prefix);

    if (lane < STAGES) mbar_init(bars + lane * 8);
    if (lane < 2) piece_of[2 * warp + lane] = make_int4(-1, 0, 0, 0);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    pdl_wait();
    kv4_prefix(a, prefix, wsum);

    // Requests without a token (or with a bad length) get zeros.
    for (int r = blockIdx.x; r < a.B; r += gridDim.x) {
        if (prefix[r + 1] != prefix[r]) continue;
        const size_t row0 = static_cast<size_t>(r) * a.n_q * a.Hq;
        for (int i = threadIdx.x; i < a.n_q * a.Hq * (KV4_D / 8); i += threads)
            (reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + row0 * KV4_D * 2))[i] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse != nullptr)
            for (int i = threadIdx.x; i < a.n_q * a.Hq; i += threads) a.lse[row0 + i] = -INFINITY;
        if (a.by_set)
            for (int h = threadIdx.x; h < a.Hkv; h += threads) a.ws_cut[r * a.Hkv + h] = make_int2(0, 0);
    }

    // Warp g takes the units of steps [split.at(g), split.at(g + 1)).
    const Kv4Split split(prefix[a.B], gridDim.x * warps);
    const unsigned g0 = blockIdx.x * warps, g = g0 + warp;
    const int x0 = split.at(g), x1 = split.at(g + 1);
    // Where this warp's range begins and ends, and where its loads and its
    // computation stand: read when one goes on to another token set.
    Place* const walk = walks[warp];
    float* first_piece = a.ws_first + static_cast<size_t>(g) * a.rows * KV4_PIECE_ROW;
    const Place begin = kv4_place(prefix, a.B, a.Hkv, x0);
    // ---- loads.  Lane i holds entry `at0` + i of the row of block ids; the next
    // unit is entries at0 + at and the one behind it.
    int ids = 0, at = 0, to_load = 0;     // to_load: units of this set that are still to load
    const uint8_t* head_pool = nullptr;   // the pool from this KV head's record on
    const int32_t* row = nullptr;         // the request's ids from at0 on, and how many there are
    int row_left = 0;
    auto load_ids = [&]() {
        if (lane < row_left) ids = row[lane];
        if (lane == 0 && row_left > 32) prefetch_l1(row + 32);
        at = 0;
    };
    auto start_row = [&](const Place& p) {
        row = a.table + static_cast<size_t>(p.r) * a.max_blocks + 2 * p.j;
        row_left = (a.ctx_len[p.r] + KV4_BLOCK - 1) / KV4_BLOCK - 2 * p.j;
        head_pool = a.pool + static_cast<size_t>(p.h) * R;
        load_ids();
    };
    if (x0 < x1 && begin.r < a.B) {
        start_row(begin);
        const Place end = kv4_place(prefix, a.B, a.Hkv, x1);
        const bool one_set = begin.r == end.r && begin.h == end.h;
        to_load = (one_set ? end.j : begin.nt) - begin.j;
        if (lane == 0) {
            walk[0] = walk[1] = begin;
            walk[2] = end;
        }
        __syncwarp();
    }
    if (to_load > 0) {
        const uint64_t policy = l2_evict_first_policy();
        uint32_t bad_slots = 0;  // stages with a record that does not exist
        const size_t block_bytes = static_cast<size_t>(a.Hkv) * R;
        auto issue = [&](int stage) {
            if (at == 32) {
                row += 32;
                row_left -= 32;
                load_ids();
            }
            // Lanes 0 and 1 take the unit's two blocks; the second may be behind the last one.
            const int id = __shfl_sync(FULL_MASK, ids, at + (lane & 1));
            const bool exists = at + (lane & 1) < row_left;
            const bool ok = exists && static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks);
            const uint32_t have = __ballot_sync(FULL_MASK, ok) & 3u;
            bad_slots &= ~(1u << stage);
            if (__any_sync(FULL_MASK, exists && !ok)) bad_slots |= 1u << stage;
            const uint32_t bar = bars + stage * 8;
            if (lane == 0) {
                if (have != 0u) mbar_expect(bar, have == 3u ? 2 * R : R);
                else mbar_arrive(bar);
            }
            __syncwarp();
            if (lane < 2 && ok)
                bulk_load(smem_u32(ring) + (2 * stage + lane) * R, head_pool + id * block_bytes, R, bar, policy);
            at += 2;
            if (--to_load == 0) {  // on to the next set, if its first unit is this warp's
                Place p = walk[0];
                const Place end = walk[2];
                if (p.r == end.r && p.h == end.h) return;
                kv4_next_set(prefix, a.B, a.Hkv, p);
                if (p.r == a.B || (p.r == end.r && p.h == end.h && end.j == 0)) return;
                __syncwarp();
                if (lane == 0) walk[0] = p;
                __syncwarp();
                start_row(p);
                to_load = p.r == end.r && p.h == end.h ? end.j : p.nt;
                prefetch_queries(a, p, lane);
            }
        };
#pragma unroll 1
        for (int i = 0; i < STAGES && to_load > 0; ++i) issue(i);

        // ---- computation
        Queries<NT, NG> qs;
        qs.sm = reinterpret_cast<float*>(ring + y.ring);
        Softmax<NT, NG> w;
        int stage = 0;
        uint32_t parity = 0;
        bool lost = false;  // a record did not come: no more loads, and all that follows is bad
        for (bool last = false; !last;) {  // a token set, or the part of it in this range
            load_queries<BF16, NT, NG>(a, walk[1].r, walk[1].h, lane, qs);
            reset(w);
            bool bad = false, first = true;
            int units, left;  // still to take in; tokens from the next unit's first one on
            {
                const Place p = walk[1], end = walk[2];
                units = (p.r == end.r && p.h == end.h ? end.j : p.nt) - p.j;
                left = a.ctx_len[p.r] - p.j * KV4_UNIT;
            }
            while (units > 0 && !lost) {
                for (int todo = min(units, KV4_LEVEL_UNITS); todo > 0; --todo, --units, left -= KV4_UNIT) {
                    if (!warp_wait(bars + stage * 8, parity)) {
                        lost = true;
                        break;
                    }
                    if (((bad_slots >> stage) & 1u) == 0u) {
                        const uint8_t* rec = ring + 2 * stage * R;
                        constexpr int NB = NT >= 2 ? 1 : 2;  // registers
#pragma unroll
                        for (int b = 0; b < 2; b += NB) {
                            const int from_here = left - b * KV4_BLOCK;
                            if (from_here >= NB * KV4_BLOCK + a.n_q - 1)
                                take_records<BF16, NT, NG, NB, false>(rec + b * R, from_here, first && b == 0, a, qs, w, lane);
                            else if (from_here > 0)
                                take_records<BF16, NT, NG, NB, true>(rec + b * R, from_here, first && b == 0, a, qs, w, lane);
                        }
                        first = false;
                    } else {
                        bad = true;
                        if (lane == 0) report_error(a.err_flag, CLO_FLAG_BAD_INDEX);
                    }
                    __syncwarp();
                    if (to_load > 0) issue(stage);
                    if (++stage == STAGES) {
                        stage = 0;
                        parity ^= 1;
                    }
                }
                if (units > 0) level_sums(w, lane);
            }
            bad |= lost;
            Place p = walk[1];
            const Place end = walk[2];
            const int set = p.r * a.Hkv + p.h, r = p.r, h = p.h, nt = p.nt;
            const int s0 = prefix[r] + h * (nt + KV4_SET_COST) + KV4_SET_COST;  // the first unit's step
            const bool ends_here = !(p.r == end.r && p.h == end.h), whole = ends_here && p.j == 0;
            last = !ends_here;
            if (ends_here) {
                kv4_next_set(prefix, a.B, a.Hkv, p);
                last = p.r == a.B || (p.r == end.r && p.h == end.h && end.j == 0);
            }
            __syncwarp();
            if (lane == 0) {
                walk[1] = p;
                if (!whole) piece_of[2 * warp + (last ? 1 : 0)] = make_int4(set, r, s0, s0 + nt);
                else if (a.by_set) a.ws_cut[set] = make_int2(0, 0);
            }
            __syncwarp();
            if (lost && last) give_up<STAGES>(a.err_flag, bars, stage, parity, lane);
            float* piece = whole ? nullptr : last ? reinterpret_cast<float*>(ring) : first_piece;
            end_set<BF16, NT, NG>(a, w, r, h, bad, piece, lane);
        }
    }
    // Dependents start here, not earlier: blocks of the merge that wait on an SM
    // would hold registers that CTAs of this grid or the next one need.
    pdl_launch_dependents();
    __syncthreads();

    // The CTA's pieces, a token set at a time.  A warp's last piece is in shared
    // memory, its first one (written in this CTA too) in the workspace; lane k
    // holds the set of piece k.
    const int c0 = split.at(g0), c1 = split.at(g0 + warps);  // the CTA's steps
    const int set_of = lane < 2 * warps ? piece_of[lane].x : -1;
    uint32_t todo = __ballot_sync(FULL_MASK, set_of >= 0);
    int tail_set = 0, tail_ctas = 0;
#pragma unroll 1
    while (todo != 0u) {
        const int4 piece = piece_of[__ffs(todo) - 1];
        const uint32_t mine = __ballot_sync(FULL_MASK, set_of == piece.x);
        todo &= ~mine;
        const int set = piece.x, r = piece.y, s0 = piece.z, s1 = piece.w, h = set - r * a.Hkv;
        const bool starts = s0 >= c0, goes_on = s1 > c1;
        const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (starts ? 1 : 0);
        int covers = 0;
        if (starts && goes_on) {
            covers = static_cast<int>(split.owner(s1 - 1) / warps) - static_cast<int>(blockIdx.x) + 1;
            tail_set = set;
            tail_ctas = covers;
        }
        if (a.by_set && starts && threadIdx.x == 0) a.ws_cut[set] = make_int2(blockIdx.x, covers);
        for (int it = threadIdx.x; it < a.rows * (KV4_D / 4); it += threads) {
            const int row = it / (KV4_D / 4), col = it % (KV4_D / 4);
            Sums sums;
            for (uint32_t left = mine; left != 0u;) {
                constexpr int P = 8;  // read at a time
                float2 ml[P];
                float4 v[P];
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    ml[p] = make_float2(-INFINITY, 0.f);
                    v[p] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (left != 0u) {
                        const int k = __ffs(left) - 1;
                        left &= left - 1;
                        const float* pc = (k & 1) ? reinterpret_cast<const float*>(smem + (k >> 1) * y.warp)
                                                  : a.ws_first + static_cast<size_t>(g0 + (k >> 1)) * a.rows * KV4_PIECE_ROW;
                        ml[p] = *reinterpret_cast<const float2*>(pc + row * KV4_PIECE_ROW + KV4_D);
                        v[p] = *reinterpret_cast<const float4*>(pc + row * KV4_PIECE_ROW + 4 * col);
                    }
                }
                sums.take<P>(ml, v);
            }
            if (starts && !goes_on) {
                sums.write<BF16>(a, r, h, row, col);
            } else {
                *reinterpret_cast<float4*>(a.ws_o + (slot * a.rows + row) * KV4_D + 4 * col) = sums.O;
                if (col == 0) a.ws_ml[slot * a.rows + row] = make_float2(sums.M, sums.L);
            }
        }
    }
    if (!a.by_set && threadIdx.x == 0) a.ws_cut[blockIdx.x] = make_int2(tail_set, tail_ctas);
}

// Merges the token sets that are cut by CTA boundaries, a query row of one an
// item: the tail piece of the CTA it starts in and the head pieces of those
// behind it, in a fixed order.  ws_cut, by token set: (CTA it starts in, CTAs
// it covers, 0 if nothing is to merge); by CTA: (the set that starts in this one
// and goes on, CTAs it covers).  An item has `share` warps (a power of 2), which
// take its pieces in turn, KV4_MERGE_UNROLL loads in flight each; a lane holds 4
// channels.
template <bool BF16>
__global__ void __launch_bounds__(KV4_MERGE_THREADS) kv4_merge_kernel(const Kv4Args a, int items, int share) {
    constexpr int WARPS = KV4_MERGE_THREADS / 32, U = KV4_MERGE_UNROLL;
    __shared__ float2 sm_ml[WARPS];
    __shared__ float4 sm_o[WARPS][32];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp & (share - 1);
    const int item = blockIdx.x * (WARPS / share) + warp / share;
    const int where = item / a.rows, row = item - where * a.rows;
    const int2 cut = item < items ? a.ws_cut[where] : make_int2(0, 0);
    const int set = a.by_set ? where : cut.x, cta = a.by_set ? cut.x : where, pieces = cut.y;
    Sums sums;
    for (int p0 = part; p0 < pieces; p0 += share * U) {
        float2 ml[U];
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = p0 + u * share;
            ml[u] = make_float2(-INFINITY, 0.f);
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p < pieces) {
                const size_t slot = 2 * (static_cast<size_t>(cta) + p) + (p == 0 ? 1 : 0);
                ml[u] = a.ws_ml[slot * a.rows + row];
                v[u] = reinterpret_cast<const float4*>(a.ws_o + (slot * a.rows + row) * KV4_D)[lane];
            }
        }
        sums.take<U>(ml, v);
    }
    if (share > 1) {
        if (lane == 0) sm_ml[warp] = make_float2(sums.M, sums.L);
        sm_o[warp][lane] = sums.O;
        __syncthreads();
        if (part != 0) return;
        for (int x = 1; x < share; ++x) {
            const float2 ml[1] = {sm_ml[warp + x]};
            const float4 v[1] = {sm_o[warp + x][lane]};
            sums.take<1>(ml, v);
        }
    }
    if (pieces == 0) return;
    const int r = set / a.Hkv, h = set - r * a.Hkv;
    sums.write<BF16>(a, r, h, row, lane);
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

static size_t round256(size_t x) { return (x + 255) / 256 * 256; }

static size_t kv4_workspace(int ctas, int rows) {
    const size_t slots = 2 * static_cast<size_t>(ctas) * rows;
    return round256(slots * KV4_D * sizeof(float)) + round256(slots * sizeof(float2)) +
           round256(static_cast<size_t>(ctas) * sizeof(int2)) +
           static_cast<size_t>(ctas) * kv4_flat_warps(kv4_row_tiles(rows)) * rows * KV4_PIECE_ROW * sizeof(float);
}

}  // namespace clo

using namespace clo;

extern "C" size_t clo_kv4_paged_workspace_size(int B, int n_q, int Hq, int Hkv, int d, int num_ctas) {
    if (B < 0 || n_q < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || d != KV4_D || num_ctas < 0) return 0;
    if (static_cast<long long>(Hq / Hkv) * n_q > KV4_MAX_ROWS) return 0;
    const int rows = Hq / Hkv * n_q;
    const int ctas = num_ctas > 0 ? num_ctas : device_sm_count() * kv4_flat_ctas(kv4_row_tiles(rows));
    return ctas > 0 ? kv4_workspace(ctas, rows) : 0;
}

extern "C" clo_status clo_kv4_paged_decode_attn(const clo_kv4_attn_args* args, cudaStream_t stream) {
    if (args == nullptr) return CLO_ERR_INVALID_ARG;
    const void* q = args->q;
    const uint8_t* pool = args->pool;
    const int32_t *block_table = args->block_table, *ctx_len = args->ctx_len;
    int32_t* err_flag = args->err_flag;
    void *out = args->out, *workspace = args->workspace;
    float* lse = args->lse;
    const size_t ws_bytes = args->ws_bytes;
    const clo_attn_opts* opts = args->opts;
    const clo_dtype dtype = args->dtype;
    const float scale = args->scale;
    const int B = args->B, n_q = args->n_q, Hq = args->Hq, Hkv = args->Hkv, d = args->d;
    const int num_blocks = args->num_blocks, block_size = args->block_size, max_blocks = args->max_blocks;
    const int group = args->group;
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
    const long long blocks = static_cast<long long>(B) * Hkv * max_blocks;
    const long long units = static_cast<long long>(B) * Hkv * ((max_blocks + 1) / 2);  // at most: the lengths are on the device
    if (blocks >= (1ll << 31) || max_blocks > (1 << 26) ||
        units + static_cast<long long>(B) * Hkv * KV4_SET_COST >= (1ll << 31))
        return CLO_ERR_UNSUPPORTED;
    if (opts != nullptr && opts->num_ctas > KV4_MAX_CTAS) return CLO_ERR_UNSUPPORTED;
    if (B == 0) return CLO_OK;

    Kv4Args a;
    a.rows = Hq / Hkv * n_q;
    const int nt = kv4_row_tiles(a.rows);
    // As many warps as shared memory allows, in one wave.
    int warps = kv4_flat_warps(nt);
    while (warps > 4 && kv4_layout(warps, nt, ng, a.rows, B).total > KV4_FLAT_SMEM) warps -= 4;
    const int smem = kv4_layout(warps, nt, ng, a.rows, B).total;
    const int per_sm = std::min(kv4_flat_ctas(nt), KV4_SMEM_PER_SM / (smem + KV4_FLAT_RESERVED));
    int ctas = opts != nullptr && opts->num_ctas > 0 ? opts->num_ctas : device_sm_count() * std::max(per_sm, 1);
    const long long most = (units + warps - 1) / warps;  // a unit a warp
    if (ctas > most) ctas = static_cast<int>(most);
    if (workspace == nullptr || !kv4_aligned(workspace, 16) ||
        ws_bytes < clo_kv4_paged_workspace_size(B, n_q, Hq, Hkv, d, opts != nullptr ? opts->num_ctas : 0))
        return CLO_ERR_WORKSPACE;
    if (ctas <= 0) return CLO_ERR_CUDA;

    // Few sets are cut into many pieces each: the merge goes by set.  Many
    // are cut into two or three: it goes by the cuts between CTAs.
    const int sets = B * Hkv;
    a.by_set = sets < ctas;
    // Enough warps an item to load the pieces of an average set at once.
    int share = 1;
    while (share < KV4_MERGE_THREADS / 32 && share * KV4_MERGE_UNROLL < ctas / sets + 1) share *= 2;
    const int items = (a.by_set ? sets : ctas - 1) * a.rows;
    const int per_block = KV4_MERGE_THREADS / 32 / share;
    const size_t slots = 2 * static_cast<size_t>(ctas) * a.rows;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.ws_o = reinterpret_cast<float*>(ws);
    a.ws_ml = reinterpret_cast<float2*>(ws + round256(slots * KV4_D * sizeof(float)));
    a.ws_cut = reinterpret_cast<int2*>(ws + round256(slots * KV4_D * sizeof(float)) + round256(slots * sizeof(float2)));
    a.ws_first = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a.ws_cut) +
                                          round256(static_cast<size_t>(ctas) * sizeof(int2)));
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
    const int cluster = opts != nullptr && opts->num_ctas > 0 ? 0 : kv4_set_cluster(a, ng);
    if (cluster > 0) {
        if (opts != nullptr && opts->ev_begin != nullptr && !record_event(opts->ev_begin, stream)) return CLO_ERR_CUDA;
        if (kv4_launch_sets(a, ng, dtype == CLO_BF16, cluster, stream) != cudaSuccess) return CLO_ERR_CUDA;
        if (opts != nullptr && opts->ev_end != nullptr && !record_event(opts->ev_end, stream)) return CLO_ERR_CUDA;
        return CLO_OK;
    }
    const Kv4Kernel kernel = dtype == CLO_BF16 ? attn_kernel<true>(nt, ng) : attn_kernel<false>(nt, ng);
    const auto merge = dtype == CLO_BF16 ? kv4_merge_kernel<true> : kv4_merge_kernel<false>;
    if (!prepare_kernel(reinterpret_cast<const void*>(kernel), KV4_FLAT_SMEM) ||
        !prepare_kernel(reinterpret_cast<const void*>(merge), 0))
        return CLO_ERR_CUDA;
    if (opts != nullptr && opts->ev_begin != nullptr && !record_event(opts->ev_begin, stream)) return CLO_ERR_CUDA;
    if (launch_pdl(kernel, dim3(ctas), dim3(warps * 32), smem, stream, a) != cudaSuccess) return CLO_ERR_CUDA;
    if (opts != nullptr && opts->ev_end != nullptr && !record_event(opts->ev_end, stream)) return CLO_ERR_CUDA;
    if (ctas > 1 &&
        launch_pdl(merge, dim3((items + per_block - 1) / per_block), dim3(KV4_MERGE_THREADS), 0, stream, a, items, share) !=
            cudaSuccess)
        return CLO_ERR_CUDA;
    return CLO_OK;
}
