// clo_paged_attention.cu -- attention of chunks of new tokens over the 16-bit
// paged cache, and decode attention over selected blocks of it.
//
// Work.  A request's rows of one KV head (its new tokens times the G heads of the
// group) are cut into tiles of as many whole tokens as fit 128 rows, and two tiles are
// an item.  An item goes over the tokens that its last row sees, 128 at a time.  All
// items of a call, weighed by their tokens, are shared out evenly, one contiguous range
// a CTA and one CTA an SM; each CTA works its range out by itself from the lengths.  An
// item that a border cuts leaves a partial result for each piece (sums, reference,
// denominator), which paged_merge_kernel joins.  So few rows over a long context occupy
// every SM, and a long prompt costs each SM the same.
//
// A CTA has two streams, each a warpgroup with its own scores and sums in tensor memory
// (4 x 128 columns: all of it).  An item of two tiles of rows gives one to each stream,
// and both go over every tile of tokens, so the tensor cores work on one stream's
// products while the other's weights are made.  An item of one tile gives the streams
// alternate tiles of tokens, and their sums are added up at its end.  A row belongs to
// one thread: no shuffles.  Besides:
//   warp 8   brings K and V tiles into a ring of five (a copy a block, whatever the
//            cache's strides), in the order in which the products take them;
//   warp 9   issues the products: S = Q K^T, both from shared memory, and O += P V with
//            P from tensor memory, where it takes the place of S;
//   warp 10  brings the rows of q;
//   warp 11  tells the others their pieces of work, ahead of time.
//
// What bounds it, and the figures (one GB300).  Many rows: the chain of one stream, the
// products of its tile (16 instructions, about 1250 clocks for the 1024 they are worth:
// Q K^T reads both operands from shared memory) and its softmax (1130 clocks for 128 scores
// a thread: exponentials, conversions and sums together), with about 700 clocks of
// hand-overs between the two; 1.5 us a pair of tiles.  4096 tokens after 61440 with 32
// query heads take 2.71 to 2.93 ms from idle (1.45 to 1.57 PFLOP/s, 0.77 to 0.83 of the measured
// burst rate of bf16 products; the tensor pipe is busy 72% of the time) and 3.2 to 3.4 ms back to
// back, under the power limit (1.25 to 1.33, 0.73 to 0.77 of the sustained rate).  Few rows:
// HBM; 64 requests of 8001 tokens and 8 KV heads, a token each, take 308 us (6.8 TB/s), one of
// 128K 89 us (6.0).  Short calls: about 3 us until the first copies, 2 a piece's end, 4 for the
// join.
//   Tried and not kept: two warpgroups a stream, 64 scores a thread (+4%: the exponentials
// take as long, and more warps wait); the maximum beside the weights instead of before them
// (+4%); the first half of a tile's weights handed over early (+3%); one lane of a warp, or
// none, asking a barrier that others wait for (+3 to 6%); asking without suspending the warp
// (+18%, in one thread alone); results turned within the warp so that a store writes whole
// lines (+1 to 3%).
// Softmax: with a reference that lies 2^6 below a maximum seen so far and moves only when
// a score passes it by 2^14, weights up to 2^14 fit fp16 and those down to 2^-31 of
// the largest still count, and sums in tensor memory are seldom rescaled.
//
// Weights in 16 bits: each is off by half a step, 2^-9 or 2^-12 of itself, and so is a row of a
// few tokens, where the roundings of many do not cancel out.  In tiles of rows that see up to
// CH_FINE tiles of tokens what the rounding took off is a second set of weights, and both meet
// V: half again as many products in items that have few (a prompt of 2000 tokens takes 62 us
// instead of 59; one of 300 with a query head a KV head 16.3 instead of 14.3), and bf16 results
// of short contexts are off by their own rounding alone.
//
// What a row does not see.  Scores are replaced before anything is made of them.  A
// weight of 0 does not hide a V that is not finite: rows of V behind the item's
// last token are zeroed as they are brought in; one between a row's last token and
// the item's can only make the row's result not finite, so such results are looked at
// again at the end and made anew by paged_row where a V that they do not see is
// not finite (nothing of this runs on results that are finite).
//
// Values near bf16's largest.  Weights of up to 2^14 times 2^24 values keep sums in fp32
// finite below 2^90 alone.  So a bf16 result that is not finite is made anew too where a V
// from 2^90 on is among what its item goes over.
//
// Every wait has a limit (about 2 s); one that runs out ends the CTA's work in order.
#include <math.h>

#include <atomic>

#include "clo_kv4_math.cuh"  // barriers, fp32 pairs
#include "clo_paged_attention.cuh"
#include "clo_tcgen05.cuh"

namespace clo {

constexpr int CH_TILE = 128;                      // tokens of a K or V tile; rows of a Q tile
constexpr int CH_PLACES = CH_TILE / PG_BLOCK;     // blocks of a tile
constexpr int CH_HALF = CH_TILE * 128;            // bytes of 64 channels of a tile
constexpr int CH_TILE_BYTES = 2 * CH_HALF;
constexpr int CH_STAGES = 5;
constexpr int CHUNK_ROWS = 2 * CH_TILE;           // rows of an item, at most
constexpr int CH_ROLES = 8;                       // warps of the softmax; behind them: copies, products, queries, pieces
constexpr int CH_THREADS = 384;
constexpr int CH_REGS = 168;                      // a thread at launch: 65536 / 384, in eights
constexpr int CH_REGS_SOFTMAX = 200, CH_REGS_REST = 104;  // (with 216 and 72 the thread of the products spills)
static_assert(2 * CH_REGS_SOFTMAX + CH_REGS_REST <= 3 * CH_REGS, "a split may not ask for more than the launch has");
// Weights, in tokens of an item of two tiles of rows.  Fitted to the CTAs' times in mixed
// steps: a tile of tokens takes 1.5 us with two tiles of rows and 1.15 us with one, an item
// 6 and 4.5 us beside its tiles.  (A mixed step of 64 requests takes 844 us on average over
// six draws; with 256 tokens an item 919, with equal weights for both kinds 981 to 928.)
constexpr int CH_FIXED = 512;                     // an item, beside its tokens
constexpr int CH_ONE = 12;                        // a token of an item of one tile of rows, in 16ths
constexpr int CH_LEAST = 384;                     // what is worth a CTA of its own
constexpr int CH_JOIN = 640;                      // cutting an item (partial results, the join)
constexpr float CH_LIFT = 6.f, CH_SLACK = 14.f;   // log2 units: see above
constexpr int CH_FINE = 1;                        // tiles of tokens up to which weights come in two parts: see above
constexpr int CH_SMALL = 2048;                    // shared memory beside the tiles
constexpr int CH_SMEM = CHUNK_ROWS * PG_ROW + CH_STAGES * CH_TILE_BYTES + CH_SMALL + 1024;
constexpr int CH_PIECES = 4;                      // pieces told ahead
constexpr int MERGE_THREADS = 256;

// Where a range starts or ends: tile `cut` of item (request, KV head, item).
struct ChunkPos {
    int r, h, j, cut;
};

struct ChunkWs {
    float4* o;    // [CTA][head piece, tail piece][32][256 rows]: 4 channels of each row together
    float2* ml;   // [CTA][2][256] reference and denominator; denominator -1: bad data
    int4* desc;   // [CTA][8]: see CH_DESC
};
// Of a CTA: where its share starts and ends; flags: x head piece (of an item that starts
// in an earlier share), y tail piece (of one that ends in a later share), w look again; for
// the tail piece, the CTA in whose share the item ends, its request's first row and rows.
enum { DESC_START, DESC_END, DESC_FLAGS, DESC_TAIL };

struct alignas(16) ChunkSmall {
    unsigned long long told[CH_PIECES], heard[CH_PIECES];
    unsigned long long full[CH_STAGES], empty[CH_STAGES], q_full, q_empty, s_full[2], p_ready[2], o_full[2], x_full, x_empty, drain;
    ChunkPos start, end;
    int4 piece[CH_PIECES][3];
    PagedReq first;  // the request that the share starts in
    int4 tail;       // DESC_TAIL
    uint32_t tmem;
    int dead;      // a wait ran out
    int again;     // a complete item has a result that is not finite
    int copied, asked;  // tiles and queries whose copies were issued
    int odd;       // a request is bad
    int bad[8];    // by item: a place that could not be read
    float2 ml1[CH_TILE];  // stream 1's reference and denominator, for items with one tile of rows
};
static_assert(sizeof(ChunkSmall) <= CH_SMALL, "");

// ---------------------------------------------------------------- shares

// Tokens of a tile of rows.
__host__ __device__ __forceinline__ int tile_tokens(int G) { return CH_TILE / G; }

// Tokens that the last row of item j sees (sparse: the selected places' length).
template <bool SPARSE>
__device__ __forceinline__ int item_sees(const PagedAttnArgs& a, const PagedReq& q, int j) {
    if constexpr (SPARSE) return paged_places<true>(a, q.ctx) * PG_BLOCK;
    else return max(q.ctx - q.n + static_cast<int>(min(static_cast<unsigned>(q.n), 2u * (j + 1) * a.tt)), 0);
}
__device__ __forceinline__ int items_of(const PagedAttnArgs& a, const PagedReq& q) {
    return static_cast<int>((static_cast<unsigned>(q.n) + 2 * a.tt - 1) / (2 * a.tt));
}

// The weights of a request's items of one KV head, in tokens (or 2^shift of them, so
// that all of a call's weights stay below 2^31): item j weighs the tokens before the
// new ones, CH_FIXED and the new ones up to its end.
struct Weights {
    unsigned each, last;  // each = without the part that rises
    int items, tt, shift;
    __device__ unsigned before(int j) const {  // items 0 .. j - 1
        return j < items ? j * each + rise(j) : all();
    }
    __device__ unsigned all() const { return items == 0 ? 0 : (items - 1) * each + rise(items - 1) + last; }
    __device__ unsigned rise(int j) const {
        return static_cast<unsigned>((static_cast<unsigned long long>(j) * (j + 1) * tt) >> shift);
    }
};
template <bool SPARSE>
__device__ __forceinline__ Weights weights_of(const PagedAttnArgs& a, const PagedReq& q) {
    Weights w;
    w.tt = a.tt;
    w.shift = a.shift;
    w.items = items_of(a, q);
    const int base = SPARSE ? 0 : max(q.ctx - q.n, 0);
    w.each = max((base + CH_FIXED) >> a.shift, 1);
    const int seen = SPARSE ? item_sees<true>(a, q, 0) : base + q.n;
    const bool one = q.n - (w.items - 1) * 2 * a.tt <= a.tt;
    w.last = max(((one ? seen / 16 * CH_ONE : seen) + CH_FIXED) >> a.shift, 1);
    return w;
}

// What a CTA knows of the requests while it finds its share, in the ring's memory.
struct Shares {
    unsigned weight[PG_MAX_B + 1];  // of the requests before
    int items[PG_MAX_B + 1];        // of all heads
    PagedReq req[PG_MAX_B];
    unsigned warp_weight[CH_THREADS / 32];
    int warp_items[CH_THREADS / 32], warp_most[CH_THREADS / 32];
};
static_assert(sizeof(Shares) <= CH_STAGES * CH_TILE_BYTES, "");

// How a call's work is shared out over `grid` CTAs.  Cut: even shares of the weight,
// wherever they fall.  Whole items, where that is as good: one a CTA if there are enough
// CTAs, else even shares up to items' starts.  A cut costs CH_JOIN, a whole item up to
// its own weight more than the even share.
struct Split {
    bool whole, by_item;
    int ctas;
    unsigned each, more;  // CTA c's share starts at weight each * c + min(c, more)
    __device__ Split(unsigned all, int items, int most, int grid, int shift) {
        const unsigned least = max(CH_LEAST >> shift, 1);
        by_item = items <= grid;
        whole = by_item ? most <= static_cast<int>(max(all / grid, least)) + (CH_JOIN >> shift) : most <= (CH_JOIN >> shift);
        by_item &= whole;
        ctas = items == 0 ? 0 : by_item ? items : whole ? grid : max(min(grid, static_cast<int>(all / least)), 1);
        if (!whole && ctas > items && items > 0) ctas -= ctas % items;  // items of one size: pieces of one size
        each = ctas > 0 ? all / ctas : 0;
        more = all - each * ctas;
    }
    __device__ unsigned start(int c) const { return each * c + min(static_cast<unsigned>(c), more); }
    // The CTA whose share weight x belongs to.
    __device__ int owner(unsigned x) const {
        return static_cast<int>(x < (each + 1) * more ? x / (each + 1) : more + (x - (each + 1) * more) / each);
    }
};

// Item `x` (counted over the heads) of request r.
__device__ __forceinline__ ChunkPos item_at(const PagedAttnArgs& a, const PagedReq& q, int r, int x) {
    const int n = items_of(a, q);
    return ChunkPos{r, x / n, x % n, 0};
}

// Where weight `rest` of request r lies; whole: the item that starts there or behind.
template <bool SPARSE>
__device__ ChunkPos weight_at(const PagedAttnArgs& a, const PagedReq& q, int r, unsigned rest, bool whole) {
    const Weights w = weights_of<SPARSE>(a, q);
    const unsigned head = w.all();
    const int h = static_cast<int>(rest / head);
    rest -= h * head;
    int lo = 0, hi = w.items - 1;  // the last j with before(j) <= rest
#pragma unroll 1
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (w.before(mid) <= rest) lo = mid;
        else hi = mid - 1;
    }
    const int tiles = (item_sees<SPARSE>(a, q, lo) + CH_TILE - 1) / CH_TILE;
    const float part = __fdividef(static_cast<float>(rest - w.before(lo)), static_cast<float>(w.before(lo + 1) - w.before(lo)));
    ChunkPos p{r, h, lo, max(min(static_cast<int>(part * tiles), tiles - 1), 0)};
    if (whole && rest > w.before(lo)) {
        p = ChunkPos{r, h, lo + 1, 0};
        if (p.j == w.items) p = h + 1 < a.Hkv ? ChunkPos{r, h + 1, 0, 0} : ChunkPos{r + 1, 0, 0, 0};
    }
    return p;
}

// One piece of work: tiles lo .. hi - 1 of an item of `tiles`.
struct Piece {
    PagedReq q;
    int r, h, j, lo, hi;
    int marks;   // the item's tiles; bits 30 + s: stream s makes weights in two parts (with one
                 // tile of rows both say so).  One register: with two the softmax spills.
    int tokens;  // of the item
    int sees;    // tokens of the item's last row
    __device__ int tiles() const { return marks & 0x3fffffff; }
    __device__ bool whole() const { return lo == 0 && hi == tiles(); }
    __device__ bool two(const PagedAttnArgs& a) const { return tokens > a.tt; }
    // (Behind CH_FINE tiles of tokens all of such a stream's weights are 0.)
    __device__ bool fine(int s, int t) const { return t < CH_FINE && (static_cast<unsigned>(marks) >> (30 + s) & 1) != 0; }
};

// The pieces from `start` to `end`, in order.
template <bool SPARSE>
struct Walk {
    PagedReq q;
    ChunkPos at, end;
    int items;
    bool loaded;
    __device__ Walk(const ChunkPos& s, const ChunkPos& e) : at(s), end(e), items(0), loaded(false) {}
    __device__ Walk(const PagedAttnArgs& a, const ChunkPos& s, const ChunkPos& e, const PagedReq& first)
        : q(first), at(s), end(e), items(items_of(a, first)), loaded(true) {}
    __device__ bool next(const PagedAttnArgs& a, Piece& p) {
        while (at.r < a.B) {
            if (at.r > end.r) return false;
            if (!loaded) {
                q = paged_request<SPARSE>(a, at.r);
                items = items_of(a, q);
                loaded = true;
            }
            if (items > 0 && at.h < a.Hkv) break;
            at = ChunkPos{at.r + 1, 0, 0, 0};
            loaded = false;
        }
        if (at.r >= a.B) return false;
        if (at.r == end.r && (at.h > end.h || (at.h == end.h && at.j > end.j))) return false;
        const bool at_end = at.r == end.r && at.h == end.h && at.j == end.j;
        if (at_end && end.cut <= at.cut) return false;
        p.q = q;
        p.r = at.r;
        p.h = at.h;
        p.j = at.j;
        p.sees = item_sees<SPARSE>(a, q, at.j);
        p.marks = (p.sees + CH_TILE - 1) / CH_TILE;
        p.tokens = min(2 * a.tt, q.n - at.j * 2 * a.tt);
        p.lo = at.cut;
        p.hi = at_end ? min(end.cut, p.marks) : p.marks;
        at.cut = 0;
        if (++at.j == items) {
            at.j = 0;
            ++at.h;
        }
        return true;
    }
};

// Row (tile of rows * 128 + row of the tile) of item j: its token among the
// request's new ones and its head in the group; whether there is such a row.
__device__ __forceinline__ bool row_of(const PagedAttnArgs& a, int j, int tokens, int row, int& token, int& g) {
    const int x = row & (CH_TILE - 1), t = x / a.G;
    const int i = (row >> 7) * a.tt + t;
    g = x - t * a.G;
    token = 2 * j * a.tt + i;
    return t < a.tt && i < tokens;
}

// Whether results that are not finite may be due to more than what their rows see; with fp16
// values and the same tokens for all rows they are not.  (Sums of weights that are NaN always are.)
__host__ __device__ constexpr bool ch_again(bool bf16, bool sparse) { return bf16 || !sparse; }

// ---------------------------------------------------------------- small parts

__device__ __forceinline__ void mbar_init_n(uint32_t bar, int n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(n) : "memory");
}
// False if the wait ran out, here or in another warp.
__device__ __forceinline__ bool ch_wait(unsigned long long& bar, uint32_t parity, ChunkSmall* sm) {
    const uint32_t b = smem_u32(&bar);
    if (mbar_try(b, parity)) return true;
    const long long t0 = clock64();
    do {
        if (mbar_try(b, parity)) return true;
        if (*reinterpret_cast<volatile int*>(&sm->dead) != 0) return false;
    } while (clock64() - t0 < KV4_WAIT_CLOCKS);
    *reinterpret_cast<volatile int*>(&sm->dead) = 1;
    return false;
}
__device__ __forceinline__ bool ch_warp_wait(unsigned long long& bar, uint32_t parity, ChunkSmall* sm) {
    return __all_sync(FULL_MASK, ch_wait(bar, parity, sm));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int R>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(R)); }

// ---------------------------------------------------------------- pieces of work

// The pieces of a CTA, as warp 11 tells them: each role takes them in turn.
struct Pieces {
    ChunkSmall* sm;
    int it = 0;
    // For a whole warp (lane) or for one thread of it (lane = -1).
    __device__ __forceinline__ bool next(Piece& p, int lane) {
        const int slot = it % CH_PIECES;
        const uint32_t parity = it / CH_PIECES & 1;
        ++it;
        if (lane < 0 ? !ch_wait(sm->told[slot], parity, sm) : !ch_warp_wait(sm->told[slot], parity, sm)) return false;
        const int4 x = sm->piece[slot][0], y = sm->piece[slot][1], z = sm->piece[slot][2];
        p.q = PagedReq{x.x, x.y, x.z, false};
        p.r = x.w;
        p.h = y.x;
        p.j = y.y;
        p.lo = y.z;
        p.hi = y.w;
        p.marks = z.x;
        p.tokens = z.y;
        p.sees = z.z;
        if (lane >= 0) __syncwarp();
        if (lane <= 0) mbar_arrive(smem_u32(&sm->heard[slot]));
        return p.tokens > 0;  // else that was the end
    }
};

// Where offsets descend the others' requests may overlap, and with more than 2 N rows the
// weights' sums, made for N, might pass 32 bits: such a call has no pieces.
__device__ __noinline__ bool too_many_rows(const int32_t* offsets, int B, int N) {
    long long rows = 0;
#pragma unroll 1
    for (int r = 0; r < B; ++r) {
        const int first = offsets[r], end = offsets[r + 1];
        if (first >= 0 && first <= end && end <= N) rows += end - first;
    }
    return rows > 2ll * N;
}

template <bool SPARSE>
__device__ __forceinline__ void tell_pieces(const PagedAttnArgs& a, ChunkSmall* sm, Walk<SPARSE>& walk) {  // one thread
    for (int it = 0;; ++it) {
        const int slot = it % CH_PIECES;
        Piece p;
        const bool more = walk.next(a, p);
        if (!more) p.tokens = 0;
        if (!ch_wait(sm->heard[slot], (it / CH_PIECES & 1) ^ 1, sm)) return;
        sm->piece[slot][0] = make_int4(p.q.row0, p.q.n, p.q.ctx, p.r);
        sm->piece[slot][1] = make_int4(p.h, p.j, p.lo, p.hi);
        // By what the last row of a stream's own tile sees, be that the first of an item's two or not.
        const int first_sees = p.sees - (p.two(a) ? p.tokens - a.tt : 0);
        const unsigned fine = (first_sees <= CH_FINE * CH_TILE ? 1u << 30 : 0u) | (p.sees <= CH_FINE * CH_TILE ? 1u << 31 : 0u);
        sm->piece[slot][2] = make_int4(static_cast<int>(p.marks | fine), p.tokens, p.sees, 0);
        mbar_arrive(smem_u32(&sm->told[slot]));
        if (!more) return;
    }
}

// ---------------------------------------------------------------- the copying warp

template <bool SPARSE>
struct Loader {
    const PagedAttnArgs& a;
    const CUtensorMap *mk, *mv;
    ChunkSmall* sm;
    uint32_t ring;
    int lane;
    int it = 0;  // tiles brought so far

    // A tile's 8 places are lanes 8 (t % 4) .. of `places`.
    __device__ bool tile(const Piece& p, bool is_v, int t, int places, int slot) {
        const int stage = it % CH_STAGES;
        if (!ch_warp_wait(sm->empty[stage], (it / CH_STAGES & 1) ^ 1, sm)) return false;
        ++it;
        const uint32_t dst = ring + stage * CH_TILE_BYTES, bar = smem_u32(&sm->full[stage]);
        const int mine = __shfl_sync(FULL_MASK, places, (t & 3) * CH_PLACES + (lane & 7));
        if (__any_sync(FULL_MASK, mine < 0) && lane == 0) {  // (before the arrival below)
            *reinterpret_cast<volatile int*>(&sm->bad[slot]) = 1;
            report_error(a.err_flag, CLO_FLAG_BAD_INDEX);
        }
        const int rows = mine < 0 ? 0 : mine & 31, id = mine >> 5;
        const bool copy = is_v ? rows == PG_BLOCK : rows > 0;
        const unsigned copied = __ballot_sync(FULL_MASK, copy) & 0xffu;
        if (is_v && copied != 0xffu) {
            // Rows that nobody sees are zeros: a weight of 0 times what lies there need
            // not be 0.
            for (int b = 0; b < CH_PLACES; ++b) {
                const int brows = __shfl_sync(FULL_MASK, rows, b), bid = __shfl_sync(FULL_MASK, id, b);
                if (brows == PG_BLOCK) continue;
                const long long base = brows > 0 ? static_cast<long long>(bid) * a.kv_block + p.h * a.kv_head : 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int row = (lane >> 4) + 2 * k, c = lane & 15;
                    const uint4 x = row < brows ? *reinterpret_cast<const uint4*>(a.vc + base + row * a.kv_token + c * 16)
                                                : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t to = dst + b * PG_BLOCK_BYTES + (row >> 3) * 2048 + (c >> 3) * 1024 + (row & 7) * 128 +
                                        (((c & 7) ^ (row & 7)) << 4);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(to), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w)
                                 : "memory");
                }
            }
            async_proxy_fence();
            __syncwarp();
        }
        if (lane == 0) mbar_expect(bar, __popc(copied) * PG_BLOCK_BYTES);
        __syncwarp();
        if (lane < CH_PLACES && copy)
            tma_load_5d(dst + lane * PG_BLOCK_BYTES, is_v ? mv : mk, bar, 0, 0, 0, 0, static_cast<int>(id * a.unit_block + p.h * a.unit_head));
        return true;
    }

    __device__ bool piece(const Piece& p, int slot) {
        const int n = p.hi - p.lo, ahead = p.two(a) ? 1 : 2;
        const int sees = SPARSE ? p.q.ctx : p.sees, last = paged_places<SPARSE>(a, sees);
        // Places of four tiles a register: of the group that K is in, the one before, and on
        // their way the next one's blocks and (sparse) the columns of the one after that.
        const int nb = (sees + PG_BLOCK - 1) / PG_BLOCK;
        const auto column = [&](int group) {
            const int x = group * 32 + lane;
            if constexpr (SPARSE) return x < last ? a.sel[(static_cast<size_t>(p.r) * a.Hkv + p.h) * a.n_sel + x] : -1;
            else return x < last ? x : -1;
        };
        const auto block = [&](int col) {
            return col >= 0 && col < nb ? a.table[static_cast<size_t>(p.r) * a.max_blocks + col] : -1;
        };
        const auto pack = [&](int col, int id) {
            const bool bad = col < -1 || col >= nb || (col >= 0 && (id < 0 || id >= a.num_blocks));
            return bad ? -1 : col < 0 ? 0 : id * 32 + min(sees - col * PG_BLOCK, PG_BLOCK);
        };
        int group = p.lo >> 2;
        int cur_col = column(group), next_col = column(group + 1), after_col = column(group + 2);
        int cur_id = block(cur_col), next_id = block(next_col);
        int cur = pack(cur_col, cur_id), prev = 0;
        const auto k_tile = [&](int t) {
            if ((t >> 2) != group) {
                ++group;
                prev = cur;
                cur = pack(next_col, next_id);
                next_col = after_col;
                next_id = block(next_col);
                after_col = column(group + 2);
            }
            return tile(p, false, t, cur, slot);
        };
        for (int i = 0; i < min(ahead, n); ++i)
            if (!k_tile(p.lo + i)) return false;
        for (int i = 0; i < n; ++i) {
            const int t = p.lo + i;
            if (!tile(p, true, t, (t >> 2) == group ? cur : prev, slot)) return false;
            if (i + ahead < n && !k_tile(t + ahead)) return false;
        }
        return true;
    }
};

// ---------------------------------------------------------------- the thread that issues products

template <bool BF16>
struct Issuer {
    ChunkSmall* sm;
    uint32_t q, ring, tmem;
    int tt;
    int it = 0;              // tiles taken so far
    uint32_t p_count0 = 0, p_count1 = 0;
    uint32_t q_count = 0;

    __device__ bool wait(unsigned long long& bar, uint32_t parity) { return ch_wait(bar, parity, sm); }
    __device__ int take() { return it++; }
    __device__ bool here(int x) { return wait(sm->full[x % CH_STAGES], x / CH_STAGES & 1); }
    __device__ void release(int x) { tc_commit(smem_u32(&sm->empty[x % CH_STAGES])); }
    // S of stream s = Q of row tile qt times K of tile x.
    __device__ void scores(int s, int qt, int x) {
        const uint64_t k = tc_tile(ring + (x % CH_STAGES) * CH_TILE_BYTES, 16, 2048), qa = tc_tile(q + qt * CH_TILE_BYTES, 16, 1024);
        const uint32_t d = tmem + s * CH_TILE;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t off = (i & 3) * 32;
            tc_mma(d, tc_ahead(qa, ((i >> 2) * CH_HALF + off) >> 4), tc_ahead(k, ((i >> 2) * 1024 + off) >> 4), tc_shape(BF16, CH_TILE, CH_TILE, false), i > 0);
        }
        tc_commit(smem_u32(&sm->s_full[s]));
    }
    // O of stream s (+)= its weights times V of tile x.
    __device__ void sums(int s, int x, bool add, bool fine) {
        const uint64_t v = tc_tile(ring + (x % CH_STAGES) * CH_TILE_BYTES, 1024, 2048);
        const uint32_t d = tmem + (2 + s) * CH_TILE, w = tmem + s * CH_TILE;
        tc_mma_ts(d, w, v, tc_shape(BF16, CH_TILE, CH_TILE, true), add);
#pragma unroll
        for (int i = 1; i < 8; ++i)
            tc_mma_ts(d, w + 8 * i, tc_ahead(v, i * PG_BLOCK_BYTES >> 4), tc_shape(BF16, CH_TILE, CH_TILE, true), true);
        if (fine)
#pragma unroll 1
            for (int i = 0; i < 8; ++i)
                tc_mma_ts(d, w + 64 + 8 * i, tc_ahead(v, i * PG_BLOCK_BYTES >> 4), tc_shape(BF16, CH_TILE, CH_TILE, true), true);
    }
    __device__ bool weights(int s) {
        const uint32_t count = s == 0 ? p_count0++ : p_count1++;
        if (!wait(sm->p_ready[s], count & 1)) return false;
        tc_fence_after();
        return true;
    }

    __device__ bool piece(const Piece& p) {
        const int n = p.hi - p.lo;
        if (!wait(sm->q_full, q_count++ & 1)) return false;
        tc_fence_after();
        if (p.tokens > tt) {
            int k = take();
            if (!here(k)) return false;
            scores(0, 0, k);
            scores(1, 1, k);
            release(k);
            if (n == 1) tc_commit(smem_u32(&sm->q_empty));
            for (int i = 0; i < n; ++i) {
                const int v = take();
                const bool more = i + 1 < n;
                if (more) k = take();
                if (!here(v)) return false;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (!weights(s)) return false;
                    sums(s, v, i > 0, p.fine(s, p.lo + i));
                    if (s == 1) release(v);
                    if (more) {
                        if (s == 0 && !here(k)) return false;
                        scores(s, s, k);
                    } else {
                        tc_commit(smem_u32(&sm->o_full[s]));
                    }
                }
                if (more) release(k);
                if (i + 2 == n) tc_commit(smem_u32(&sm->q_empty));
            }
        } else {
            for (int i = 0; i < min(n, 2); ++i) {
                const int k = take();
                if (!here(k)) return false;
                scores(i, 0, k);
                release(k);
            }
            if (n <= 2) tc_commit(smem_u32(&sm->q_empty));
            for (int i = 0; i < n; ++i) {
                const int s = i & 1, v = take();
                const bool more = i + 2 < n;
                const int k = more ? take() : 0;
                if (!here(v) || !weights(s)) return false;
                sums(s, v, i >= 2, p.fine(1, p.lo + i));
                release(v);
                if (more) {
                    if (!here(k)) return false;
                    scores(s, 0, k);
                    release(k);
                    if (i + 3 == n) tc_commit(smem_u32(&sm->q_empty));
                } else {
                    tc_commit(smem_u32(&sm->o_full[s]));
                }
            }
        }
        return true;
    }
};

// ---------------------------------------------------------------- the softmax warpgroups

template <bool BF16, bool SPARSE>
struct RowSoftmax {
    const PagedAttnArgs& a;
    const ChunkWs& ws;
    ChunkSmall* sm;
    int s;            // stream
    int tid;          // thread of the warpgroup: the row of its tile
    uint32_t tmem;    // this warp's lanes of column 0
    uint32_t s_count = 0, o_count0 = 0, o_count1 = 0, x_count = 0, e_count = 0;
    int piece_count = 0;

    // The weights of one tile of tokens from their scores.  sees: tokens of the
    // tile that the row sees; first: of this piece.
    template <bool FINE>
    __device__ __forceinline__ void tile(int sees, uint32_t place_rows, bool masked, bool first, float& ref, float& sum) {
        float x[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_load32(x[c], tmem + s * CH_TILE + 32 * c);
        tmem_wait_load();
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_loaded32(x[c]);
        if (masked) {
            if constexpr (SPARSE) {
                // place_rows of lanes 0 .. 7: the tokens of each place
#pragma unroll
                for (int b = 0; b < CH_PLACES; ++b) {
                    const int rows = __shfl_sync(FULL_MASK, place_rows, b);
#pragma unroll
                    for (int i = 0; i < PG_BLOCK; ++i)
                        if (i >= rows) x[b / 2][(b & 1) * 16 + i] = -INFINITY;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (32 * c + i >= sees) x[c][i] = -INFINITY;
            }
        }
        float m[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            m[c] = fmaxf(x[c][0], x[c][1]);
#pragma unroll
            for (int i = 2; i < 32; i += 2) m[c] = fmaxf(m[c], fmaxf(x[c][i], x[c][i + 1]));
        }
        const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * a.scale_log2;
        if (first) {
            ref = top == -INFINITY ? top : top - CH_LIFT;
            sum = 0.f;
        } else {
            const bool moves = top - CH_SLACK > ref;
            if (__any_sync(FULL_MASK, moves)) {
                // The sums of the earlier tiles are complete: the product that made these
                // scores came after them.
                const float to = moves ? top - CH_LIFT : ref;
                const float f = moves ? ex2(ref - to) : 1.f;
                ref = to;
                sum *= f;
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    float o[16];
                    const uint32_t at = tmem + (2 + s) * CH_TILE + 16 * c;
                    asm volatile(
                        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                        "%14, %15}, [%16];\n tcgen05.wait::ld.sync.aligned;\n"
                        : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]), "=f"(o[6]), "=f"(o[7]),
                          "=f"(o[8]), "=f"(o[9]), "=f"(o[10]), "=f"(o[11]), "=f"(o[12]), "=f"(o[13]), "=f"(o[14]), "=f"(o[15])
                        : "r"(at)
                        : "memory");
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] *= f;
                    asm volatile(
                        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                        "%14, %15, %16};\n" ::"r"(at),
                        "f"(o[0]), "f"(o[1]), "f"(o[2]), "f"(o[3]), "f"(o[4]), "f"(o[5]), "f"(o[6]), "f"(o[7]), "f"(o[8]),
                        "f"(o[9]), "f"(o[10]), "f"(o[11]), "f"(o[12]), "f"(o[13]), "f"(o[14]), "f"(o[15])
                        : "memory");
                }
            }
        }
        const float r = ref == -INFINITY ? 0.f : ref;
        const float2 scale = make_float2(a.scale_log2, a.scale_log2), minus = make_float2(-r, -r);
        float2 l[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        if constexpr (!FINE) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int c = 2 * half + i / 16, k = 2 * (i & 15);
                    float2 y = fma2(make_float2(x[c][k], x[c][k + 1]), scale, minus);
                    y = make_float2(ex2(y.x), ex2(y.y));
                    w[i] = pg_pack<BF16>(y.x, y.y);
                    l[i & 1] = add2(l[i & 1], y);
                }
                tmem_store32(tmem + s * CH_TILE + 32 * half, w);
            }
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t w[16], rest[16];  // the weights, and what their rounding took off
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float2 y = fma2(make_float2(x[c][2 * i], x[c][2 * i + 1]), scale, minus);
                    y = make_float2(ex2(y.x), ex2(y.y));
                    w[i] = pg_pack<BF16>(y.x, y.y);
                    const float2 z = pg_unpack<BF16>(w[i]);
                    rest[i] = pg_pack<BF16>(y.x - z.x, y.y - z.y);
                    l[i & 1] = add2(l[i & 1], y);
                }
                tmem_store16(tmem + s * CH_TILE + 16 * c, w);
                tmem_store16(tmem + s * CH_TILE + 64 + 16 * c, rest);
            }
        }
        l[0] = add2(l[0], l[1]);
        sum += l[0].x + l[0].y;
        tmem_wait_store();
        tc_fence_before();
        __syncwarp();
        if ((tid & 31) == 0) mbar_arrive(smem_u32(&sm->p_ready[s]));
    }

    // Writes a row's result: out and lse of a whole item, else its piece's sums.
    template <typename Load>
    __device__ __forceinline__ void write(const Piece& p, int row, bool bad, float ref, float sum, Load load) {
        int token, g;
        const bool valid = row_of(a, p.j, p.tokens, row, token, g);
        const size_t place = (static_cast<size_t>(p.q.row0) + token) * a.Hq + p.h * a.G + g;
        const bool whole = p.whole();
        const size_t slot = static_cast<size_t>(blockIdx.x) * 2 + (p.lo == 0);
        const bool none = bad || !(sum != 0.f);  // (a NaN is something)
        const float inv = none ? 0.f : 1.f / sum;
        float odd = 0.f;  // turns NaN with a value that is not finite
        if (!__any_sync(FULL_MASK, valid)) return;
        // (Not unrolled: this runs once a piece, and its instructions come from far.)
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            float o[32];
            load(o, c);
            if (whole) {
                uint32_t w[16];
                float2 sink = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 x = mul2(make_float2(o[2 * i], o[2 * i + 1]), make_float2(inv, inv));
                    sink = fma2(x, make_float2(0.f, 0.f), sink);
                    w[i] = none ? 0u : kv4_pack2_finite<BF16>(x.x, x.y);  // (see pg_pack_out)
                }
                sink.x += sink.y;
                if (!none && sink.x != 0.f) {  // something is not finite
                    odd = sink.x;
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] = pg_pack_out<BF16>(o[2 * i] * inv, o[2 * i + 1] * inv);
                }
                if (valid) {  // whole sectors: a thread's row lies apart from its neighbours'
                    uint8_t* dst = a.out + place * PG_ROW + c * 64;
                    const bool sectors = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (!sectors) {
                            reinterpret_cast<uint4*>(dst)[2 * i] = make_uint4(w[8 * i], w[8 * i + 1], w[8 * i + 2], w[8 * i + 3]);
                            reinterpret_cast<uint4*>(dst)[2 * i + 1] = make_uint4(w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]);
                        } else
                        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst + 32 * i), "r"(w[8 * i]),
                                     "r"(w[8 * i + 1]), "r"(w[8 * i + 2]), "r"(w[8 * i + 3]), "r"(w[8 * i + 4]), "r"(w[8 * i + 5]),
                                     "r"(w[8 * i + 6]), "r"(w[8 * i + 7])
                                     : "memory");
                }
            } else if (valid) {
                float4* dst = ws.o + (slot * 32 + c * 8) * CHUNK_ROWS + row;
#pragma unroll
                for (int i = 0; i < 8; ++i) dst[i * CHUNK_ROWS] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
        }
        if (!valid) return;
        if (whole) {
            if (a.lse != nullptr) a.lse[place] = none ? -INFINITY : (ref + log2f(sum)) * LN2;
            if (ch_again(BF16, SPARSE) && odd != 0.f && sum == sum) *reinterpret_cast<volatile int*>(&sm->again) = 1;
        } else {
            ws.ml[slot * CHUNK_ROWS + row] = make_float2(ref, bad ? -1.f : sum);
        }
    }

    __device__ bool piece(const Piece& p) {
        const int n = p.hi - p.lo;
        const bool two = p.two(a);
        const int row = two ? s * CH_TILE + tid : tid;
        if (n == 0) {  // no row of the item sees a token
            if (two || s == 0) write(p, row, false, -INFINITY, 0.f, [](float (&o)[32], int) {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0.f;
            });
            return true;
        }
        const int lane = tid & 31;
        int token, g;
        const bool valid = row_of(a, p.j, p.tokens, row, token, g);
        // Rows past the item's (their results are not used) see everything.
        const int sees = SPARSE || !valid ? 0x7fffffff : paged_sees<false>(p.q, token);
        const int places = SPARSE ? paged_places<true>(a, p.q.ctx) : 0;
        const int nb = (p.q.ctx + PG_BLOCK - 1) / PG_BLOCK;
        const auto column = [&](int t) {  // sparse: lanes 0 .. 7, the column of each place
            const int x = t * CH_PLACES + (lane & 7);
            return x < places ? a.sel[(static_cast<size_t>(p.r) * a.Hkv + p.h) * a.n_sel + x] : -1;
        };
        const bool idle = !__any_sync(FULL_MASK, valid);
        float ref = -INFINITY, sum = 0.f;
        const int step = two ? 1 : 2, t0 = p.lo + (two ? 0 : s);
        int next_col = SPARSE && t0 < p.hi ? column(t0) : 0;
        for (int t = t0; t < p.hi; t += step) {
            // (The next tile's columns are on their way; nothing waits for them here.)
            const int col = next_col;
            if (SPARSE && t + step < p.hi) next_col = column(t + step);
            const int rows_here = col >= 0 && col < nb ? min(p.q.ctx - col * PG_BLOCK, PG_BLOCK) : 0;
            const int seen = sees - t * CH_TILE;
            const bool masked = SPARSE ? __any_sync(FULL_MASK, rows_here != PG_BLOCK) : __any_sync(FULL_MASK, seen < CH_TILE);
            if (!ch_warp_wait(sm->s_full[s], s_count++ & 1, sm)) return false;
            if (idle) {  // nobody reads what becomes of these rows
                if (lane == 0) mbar_arrive(smem_u32(&sm->p_ready[s]));
                continue;
            }
            tc_fence_after();
            if (p.fine(s, t)) tile<true>(seen, rows_here, masked, t == t0, ref, sum);
            else tile<false>(seen, rows_here, masked, t == t0, ref, sum);
        }
        const bool second = two || n > 1;  // stream 1 had tiles
        if (s == 0 || two) {
            if (!ch_warp_wait(sm->o_full[s], (s == 0 ? o_count0 : o_count1) & 1, sm)) return false;
            if (s == 0 && !two && second && !ch_warp_wait(sm->o_full[1], o_count1 & 1, sm)) return false;
        }
        ++o_count0;
        if (second) ++o_count1;
        const bool bad = *reinterpret_cast<volatile int*>(&sm->bad[piece_count & 7]) != 0;
        ++piece_count;
        tc_fence_after();
        if (two || !second) {
            if (s == 1 && !two) return true;
            write(p, row, bad, ref, sum, [&](float (&o)[32], int c) {
                tmem_load32(o, tmem + (2 + s) * CH_TILE + 32 * c);
                tmem_wait_load();
                tmem_loaded32(o);
            });
            tc_fence_before();
            return true;
        }
        // One tile of rows: stream 0 adds stream 1's sums to its own.
        if (s == 1) {
            sm->ml1[tid] = make_float2(ref, sum);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm->x_full));
            return ch_warp_wait(sm->x_empty, e_count++ & 1, sm);
        }
        if (!ch_warp_wait(sm->x_full, x_count++ & 1, sm)) return false;
        const volatile float* ml1 = reinterpret_cast<const volatile float*>(&sm->ml1[tid]);
        const float2 other = make_float2(ml1[0], ml1[1]);
        const float to = fmaxf(ref, other.x);
        const float f0 = ref == -INFINITY ? 0.f : ex2(ref - to), f1 = other.x == -INFINITY ? 0.f : ex2(other.x - to);
        write(p, row, bad, to, sum * f0 + other.y * f1, [&](float (&o)[32], int c) {
            float o1[32];
            tmem_load32(o, tmem + 2 * CH_TILE + 32 * c);
            tmem_load32(o1, tmem + 3 * CH_TILE + 32 * c);
            tmem_wait_load();
            tmem_loaded32(o);
            tmem_loaded32(o1);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = o[i] * f0 + o1[i] * f1;
        });
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm->x_empty));
        return true;
    }
};

// ---------------------------------------------------------------- the main kernel

template <bool BF16, bool SPARSE>
__global__ void __launch_bounds__(CH_THREADS, 1)
    paged_chunk_kernel(const PagedAttnArgs a, const ChunkWs ws, const __grid_constant__ CUtensorMap map_q,
                       const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
    extern __shared__ uint8_t raw[];
    uint8_t* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint8_t* ring = base + CHUNK_ROWS * PG_ROW;
    ChunkSmall* sm = reinterpret_cast<ChunkSmall*>(ring + CH_STAGES * CH_TILE_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < CH_STAGES; ++i) {
            mbar_init_n(smem_u32(&sm->full[i]), 1);
            mbar_init_n(smem_u32(&sm->empty[i]), 1);
        }
        for (int i = 0; i < CH_PIECES; ++i) {
            mbar_init_n(smem_u32(&sm->told[i]), 1);
            mbar_init_n(smem_u32(&sm->heard[i]), 11);  // eight warps, copies, products, queries
        }
        mbar_init_n(smem_u32(&sm->q_full), 1);
        mbar_init_n(smem_u32(&sm->q_empty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init_n(smem_u32(&sm->s_full[i]), 1);
            mbar_init_n(smem_u32(&sm->p_ready[i]), 4);
            mbar_init_n(smem_u32(&sm->o_full[i]), 1);
        }
        mbar_init_n(smem_u32(&sm->x_full), 4);
        mbar_init_n(smem_u32(&sm->x_empty), 4);
        mbar_init_n(smem_u32(&sm->drain), 1);
        sm->dead = sm->again = sm->copied = sm->asked = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == CH_ROLES + 1) tmem_alloc(smem_u32(&sm->tmem), 4 * CH_TILE);
    if (threadIdx.x == CH_ROLES * 32) sm->odd = 0;
    __syncwarp();
    if (threadIdx.x == (CH_ROLES + 2) * 32) {
        tma_prefetch(&map_q);
        tma_prefetch(&map_k);
        tma_prefetch(&map_v);
    }
    pdl_wait();
    pdl_launch_dependents();

    // The share: warp 0 finds its end, warp 8 its start.
    const int cta = blockIdx.x;
    Shares& sh = *reinterpret_cast<Shares*>(ring);
    const bool finder = warp == 0 || warp == 8;
    const bool one_warp = a.B <= 32;  // a request a lane; else summed up by all threads
    PagedReq req{0, 0, 0, false};
    unsigned weight = 0, weight1 = 0;  // up to and with this thread's requests; of those alone
    int items = 0, items1 = 0, most = 0;
    const auto add = [&](const PagedReq& q) {
        const Weights w = weights_of<SPARSE>(a, q);
        weight += w.all() * a.Hkv;
        items += w.items * a.Hkv;
        if (w.items > 0) most = max(most, static_cast<int>(w.last));
    };
    if (!one_warp || finder) {
        const int per = one_warp ? 1 : (a.B + CH_THREADS - 1) / CH_THREADS;
        const int r0 = (one_warp ? lane : static_cast<int>(threadIdx.x)) * per, r1 = min(a.B, r0 + per);
        if (!SPARSE && !one_warp) __syncthreads();  // (odd)
        bool bad = false;
#pragma unroll 1
        for (int r = r0; r < r1; ++r) {
            req = paged_request<SPARSE>(a, r);
            bad |= req.bad;
            if (!one_warp) sh.req[r] = req;
            add(req);
        }
        if (bad) {
            if (cta == 0) report_error(a.err_flag, CLO_FLAG_BAD_CTX);
            *reinterpret_cast<volatile int*>(&sm->odd) = 1;
        }
        weight1 = weight;
        items1 = items;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const unsigned v = __shfl_up_sync(FULL_MASK, weight, off);
            const int n = __shfl_up_sync(FULL_MASK, items, off);
            if (lane >= off) {
                weight += v;
                items += n;
            }
        }
        most = __reduce_max_sync(FULL_MASK, most);
        if (!one_warp) {
            if (lane == 31) {
                sh.warp_weight[warp] = weight;
                sh.warp_items[warp] = items;
                sh.warp_most[warp] = most;
            }
            __syncthreads();
            weight -= weight1;
            items -= items1;
            for (int w = 0; w < warp; ++w) {
                weight += sh.warp_weight[w];
                items += sh.warp_items[w];
            }
            if (threadIdx.x == 0) {
                sh.weight[0] = 0;
                sh.items[0] = 0;
            }
#pragma unroll 1
            for (int r = r0; r < r1; ++r) {
                add(sh.req[r]);
                sh.weight[r + 1] = weight;
                sh.items[r + 1] = items;
            }
            __syncthreads();
            most = __reduce_max_sync(FULL_MASK, lane < CH_THREADS / 32 ? sh.warp_most[lane] : 0);
        }
    }
    if (finder) {
        const unsigned all = one_warp ? __shfl_sync(FULL_MASK, weight, 31) : sh.weight[a.B];
        const int n = one_warp ? __shfl_sync(FULL_MASK, items, 31) : sh.items[a.B];
        const Split split(all, n, most, gridDim.x, a.shift);
        const int c = cta + (warp == 0);
        ChunkPos p{a.B, 0, 0, 0};
        PagedReq q{0, 0, 0, false};
        int4 tail = make_int4(0, 0, 0, 0);
        if (c < split.ctas) {
            // The request: the first whose end lies behind the start's weight or item.
            const unsigned x = split.start(c);
            int r;
            unsigned w0;
            int i0;
            if (one_warp) {
                r = __popc(__ballot_sync(FULL_MASK, split.by_item ? items <= c : weight <= x));
                w0 = __shfl_sync(FULL_MASK, weight - weight1, r);
                i0 = __shfl_sync(FULL_MASK, items - items1, r);
                q.row0 = __shfl_sync(FULL_MASK, req.row0, r);
                q.n = __shfl_sync(FULL_MASK, req.n, r);
                q.ctx = __shfl_sync(FULL_MASK, req.ctx, r);
            } else {
                int lo = 0, hi = a.B - 1;
#pragma unroll 1
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (split.by_item ? sh.items[mid + 1] > c : sh.weight[mid + 1] > x) hi = mid;
                    else lo = mid + 1;
                }
                r = lo;
                w0 = sh.weight[r];
                i0 = sh.items[r];
                q = sh.req[r];
            }
            p = split.by_item ? item_at(a, q, r, c - i0) : weight_at<SPARSE>(a, q, r, x - w0, split.whole);
            if (warp == 0 && p.cut > 0) {
                const Weights w = weights_of<SPARSE>(a, q);
                tail = make_int4(split.owner(w0 + p.h * w.all() + w.before(p.j + 1) - 1), q.row0, q.n, q.ctx);
            }
            if (p.r != r) q = p.r < a.B ? paged_request<SPARSE>(a, p.r) : PagedReq{0, 0, 0, false};
        }
        if (lane == 0) {
            if (warp == 0) {
                sm->end = p;
                sm->tail = tail;
            } else {
                sm->start = p;
                sm->first = q;
            }
        }
        if (warp == 8 && p.r < a.B && q.n > 0) {  // the first places' blocks, on their way while the roles begin
            const int x = p.cut * CH_PLACES + lane;
            if (!SPARSE && x < paged_places<SPARSE>(a, item_sees<SPARSE>(a, q, p.j)))
                prefetch_l1(a.table + static_cast<size_t>(p.r) * a.max_blocks + x);
            if (SPARSE && x < paged_places<SPARSE>(a, q.ctx))
                prefetch_l1(a.sel + (static_cast<size_t>(p.r) * a.Hkv + p.h) * a.n_sel + x);
        }
    }
    tc_fence_before();
    async_proxy_fence();  // copies will write where the weights lie
    __syncthreads();
    tc_fence_after();
    const ChunkPos start = sm->start, end = sm->end;
    const uint32_t tmem = sm->tmem;
    Pieces pieces{sm};
    Piece p;

    if (warp < CH_ROLES) {
        regs_up<CH_REGS_SOFTMAX>();  // (granted once the other four warps have given theirs up)
        RowSoftmax<BF16, SPARSE> w{a, ws, sm, warp >> 2, static_cast<int>(threadIdx.x) & 127,
                                tmem + (static_cast<uint32_t>(warp & 3) << 21)};
        while (pieces.next(p, lane))
            if (!w.piece(p)) break;
    } else {
        regs_down<CH_REGS_REST>();
        if (warp == CH_ROLES) {
            Loader<SPARSE> w{a, &map_k, &map_v, sm, smem_u32(ring), lane};
            int head = 0, tail = 0, count = 0;
            bool ok = true;
            while (ok && pieces.next(p, lane)) {
                if (p.lo > 0) head = 1;
                else if (p.hi < p.tiles()) tail = 1;
                if (p.hi == p.lo) continue;
                if (lane == 0) *reinterpret_cast<volatile int*>(&sm->bad[count & 7]) = 0;
                ok = w.piece(p, count & 7);
                ++count;
            }
            if (lane == 0) {
                int4* d = ws.desc + static_cast<size_t>(cta) * 8;
                d[DESC_START] = make_int4(start.r, start.h, start.j, start.cut);
                d[DESC_END] = make_int4(end.r, end.h, end.j, end.cut);
                d[DESC_FLAGS] = make_int4(head, tail, 0, 0);
                d[DESC_TAIL] = sm->tail;
            }
            if (lane == 0) sm->copied = w.it;
        } else if (warp == CH_ROLES + 1) {
            if (lane == 0) {
                Issuer<BF16> w{sm, smem_u32(base), smem_u32(ring), tmem, a.tt};
                bool ok = true;
                while (ok && pieces.next(p, -1))
                    if (p.hi > p.lo) ok = w.piece(p);
            }
            __syncwarp();
        } else if (warp == CH_ROLES + 2 && lane == 0) {
            uint32_t count = 0;
            bool ok = true;
            while (ok && pieces.next(p, -1)) {
                if (p.hi == p.lo) continue;
                ok = ch_wait(sm->q_empty, (count & 1) ^ 1, sm);
                if (!ok) break;
                ++count;
                // Rows of tokens behind the request's are others'; they make rows that nobody uses.
                const int tiles = p.two(a) ? 2 : 1, bytes = a.tt * a.G * PG_ROW;
                mbar_expect(smem_u32(&sm->q_full), tiles * bytes);
                for (int t = 0; t < tiles; ++t)
                    for (int half = 0; half < 2; ++half)
                        tma_load_4d(smem_u32(base) + t * CH_TILE_BYTES + half * CH_HALF, &map_q, smem_u32(&sm->q_full), 0, half,
                                    p.h * a.G, p.q.row0 + (2 * p.j + t) * a.tt);
            }
            sm->asked = count;
        } else if (warp == CH_ROLES + 3 && lane == 0) {
            Walk<SPARSE> walk(a, start, end, sm->first);
            if (!SPARSE && sm->odd != 0 && too_many_rows(a.offsets, a.B, a.N)) walk.at.r = a.B;
            tell_pieces<SPARSE>(a, sm, walk);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (sm->dead != 0) {  // what is in flight ends before the memory is given up (or the limits run out)
        if (warp == CH_ROLES && lane == 0) {
            report_error(a.err_flag, CLO_FLAG_TIMEOUT);
            for (int x = max(sm->copied - CH_STAGES, 0); x < sm->copied; ++x)
                mbar_wait(smem_u32(&sm->full[x % CH_STAGES]), x / CH_STAGES & 1);
            if (sm->asked > 0) mbar_wait(smem_u32(&sm->q_full), (sm->asked - 1) & 1);
        } else if (warp == CH_ROLES + 1 && lane == 0) {
            tc_commit(smem_u32(&sm->drain));
            mbar_wait(smem_u32(&sm->drain), 0);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        ws.desc[static_cast<size_t>(cta) * 8 + DESC_FLAGS].w = sm->again;
    }
    if (warp == CH_ROLES + 1) {
        tc_fence_after();
        tmem_free(tmem, 4 * CH_TILE);
    }
}

// ---------------------------------------------------------------- joining pieces, looking again

// Whether V of a token in [from, to), which some row does not see, is not finite; a warp.
template <bool BF16>
__device__ bool hidden_odd(const PagedAttnArgs& a, int r, int h, int from, int to, int lane) {
    bool odd = false;
    for (int t = from; t < to; ++t) {
        const int at = paged_place<false>(a, r, h, to, t / PG_BLOCK);
        if (at < 0) continue;
        const uint2 w = *reinterpret_cast<const uint2*>(a.vc + static_cast<long long>(at / 32) * a.kv_block + h * a.kv_head +
                                                        (t % PG_BLOCK) * a.kv_token + lane * 8);
        const float2 x = pg_unpack<BF16>(w.x), y = pg_unpack<BF16>(w.y);
        odd |= !(pg_finite(x.x) && pg_finite(x.y) && pg_finite(y.x) && pg_finite(y.y));
    }
    return __any_sync(FULL_MASK, odd);
}

// Whether a V from place `from` on among the first `sees` tokens (sparse: of the selected
// places) is finite and 2^90 or larger (exponents 217 to 254); the block.
template <bool BF16, bool SPARSE>
__device__ __noinline__ bool large_values(const PagedAttnArgs& a, int r, int h, int from, int sees) {
    const int lane = threadIdx.x & 31, places = paged_places<SPARSE>(a, sees);
    bool large = false;
#pragma unroll 1
    for (int first = from + (threadIdx.x & ~31); first < places; first += MERGE_THREADS) {
        const int mine = first + lane < places ? paged_place<SPARSE>(a, r, h, sees, first + lane) : 0;
#pragma unroll 1
        for (int p = 0; p < min(places - first, 32); ++p) {
            const int at = __shfl_sync(FULL_MASK, mine, p);
            if (at <= 0) continue;
            const uint8_t* v = a.vc + static_cast<long long>(at / 32) * a.kv_block + h * a.kv_head + (lane & 15) * 16;
            uint4 x[PG_BLOCK / 2];
#pragma unroll
            for (int i = 0; i < PG_BLOCK / 2; ++i) {
                const int t = 2 * i + (lane >> 4);  // (a row behind the last token repeats the first)
                x[i] = *reinterpret_cast<const uint4*>(v + (t < at % 32 ? t : 0) * a.kv_token);
            }
#pragma unroll
            for (int i = 0; i < PG_BLOCK / 2; ++i) {
                const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int c = 0; c < 4; ++c) large |= ((w[c] & 0x7fffu) - 0x6c80u < 0x1300u) | ((w[c] >> 16 & 0x7fffu) - 0x6c80u < 0x1300u);
            }
        }
    }
    return __syncthreads_or(large) != 0;
}

// Makes what is not finite of a row's result anew if that may come from what the row does not
// see, or from values so `large` that their sums were not finite.  `mine`: this lane's
// channels are written.
template <bool BF16, bool SPARSE>
__device__ __noinline__ void look_again(const PagedAttnArgs& a, const PagedReq& q, int r, int h, int j, int token, int g, int lane,
                                        bool mine, bool large) {
    if constexpr (!SPARSE) large = large || hidden_odd<BF16>(a, r, h, paged_sees<false>(q, token), item_sees<false>(a, q, j), lane);
    if (large) paged_row<BF16, SPARSE>(a, r, q, token, h * a.G + g, lane, mine);
}

// Whole items of a CTA's share that have results that are not finite: the block's rows of each.
// (Apart from the kernel, whose registers it would take.)
template <bool BF16, bool SPARSE>
__device__ __noinline__ void look_at_items(const PagedAttnArgs& a, const int4* desc) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 s = desc[DESC_START], e = desc[DESC_END];
    Walk<SPARSE> walk(ChunkPos{s.x, s.y, s.z, s.w}, ChunkPos{e.x, e.y, e.z, e.w});
    Piece p;
    int r = -1, h = 0, looked = 0;  // places of request r and head h that were looked at
    bool large = false;
    while (walk.next(a, p)) {
        if (!p.whole()) continue;
        if (p.r != r || p.h != h) {
            r = p.r;
            h = p.h;
            looked = 0;
            large = false;
        }
        // (A warp has at most 8 rows: the grid has 4 blocks an item or more.)
        const int row0 = blockIdx.y * (MERGE_THREADS / 32) + warp, step = gridDim.y * (MERGE_THREADS / 32);
        unsigned odd = 0;
        int token, g;
#pragma unroll 1
        for (int k = 0; row0 + k * step < CHUNK_ROWS; ++k) {
            if (!row_of(a, p.j, p.tokens, row0 + k * step, token, g)) continue;
            const size_t place = (static_cast<size_t>(p.q.row0) + token) * a.Hq + p.h * a.G + g;
            const uint2 w = *reinterpret_cast<const uint2*>(a.out + place * PG_ROW + lane * 8);
            const float2 x = pg_unpack<BF16>(w.x), y = pg_unpack<BF16>(w.y);
            if (__any_sync(FULL_MASK, !(pg_finite(x.x) && pg_finite(x.y) && pg_finite(y.x) && pg_finite(y.y)))) odd |= 1u << k;
        }
        if (BF16 && __syncthreads_or(odd) && !large) {
            // (A request's later items see the tokens of the earlier ones and more.)
            large = large_values<BF16, SPARSE>(a, r, h, looked, SPARSE ? p.q.ctx : p.sees);
            looked = p.sees / PG_BLOCK;
        }
        for (; odd != 0; odd &= odd - 1) {
            row_of(a, p.j, p.tokens, row0 + (__ffs(odd) - 1) * step, token, g);
            look_again<BF16, SPARSE>(a, p.q, p.r, p.h, p.j, token, g, lane, true, large);
        }
    }
}

// Block (c, y) joins the pieces of the item that starts in CTA c's share and ends in a
// later one's, for ROWS of its rows and 4 * NI of the channels.  Lanes are rows, and with ROWS
// = 8 four subsets of the pieces; a warp holds 4 channels of its rows, NI / 8 times.
template <bool BF16, bool SPARSE, int ROWS, int NI>
__global__ void __launch_bounds__(MERGE_THREADS, SPARSE ? 3 : 2) paged_merge_kernel(const PagedAttnArgs a, const ChunkWs ws, int ctas) {
    constexpr int SUBS = 32 / ROWS, K = NI / 8, AHEAD = 8 / K;
    __shared__ int odd_row[ROWS];
    __shared__ uint2 result[ROWS][NI + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    const int c = blockIdx.x;
    const int4* desc = ws.desc + static_cast<size_t>(c) * 8;
    const int4 flags = desc[DESC_FLAGS], e = desc[DESC_END], tail = desc[DESC_TAIL];
    if (flags.y != 0) {
        // Item e of request e.x: its pieces are c's tail and the head pieces of the CTAs up
        // to tail.x (one with too small a share has none).
        const PagedReq q{tail.y, tail.z, tail.w, false};
        const int tokens = min(2 * a.tt, q.n - e.z * 2 * a.tt);
        const int ib = blockIdx.y % (32 / NI), row0 = blockIdx.y / (32 / NI) * ROWS;
        int token, g;
        if (row_of(a, e.z, tokens, row0, token, g)) {  // else no row of the block is one
            if (static_cast<int>(threadIdx.x) < ROWS) odd_row[threadIdx.x] = 0;
            __syncthreads();
            const int end = min(tail.x, ctas - 1), row = row0 + lane % ROWS;
            const bool valid = row_of(a, e.z, tokens, row, token, g);
            float m = -INFINITY, l = 0.f;
            float4 o[K];
#pragma unroll
            for (int k = 0; k < K; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            bool bad = false;
            for (int x = c + lane / ROWS; x <= end; x += AHEAD * SUBS) {
                float2 ml[AHEAD];
                float4 v[AHEAD][K];
                bool there[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const int y = min(x + i * SUBS, end);
                    there[i] = valid && x + i * SUBS <= end && (y == c || ws.desc[static_cast<size_t>(y) * 8 + DESC_FLAGS].x != 0);
                    const size_t slot = static_cast<size_t>(y) * 2 + (y == c);
                    ml[i] = ws.ml[slot * CHUNK_ROWS + row];
#pragma unroll
                    for (int k = 0; k < K; ++k) v[i][k] = ws.o[(slot * 32 + ib * NI + warp + 8 * k) * CHUNK_ROWS + row];
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    if (!there[i]) continue;
                    bad |= ml[i].y < 0.f;
                    if (ml[i].x == -INFINITY && ml[i].y == 0.f) continue;  // sums of nothing (NaN is something)
                    const float to = fmaxf(m, ml[i].x);
                    const float f = m == -INFINITY ? 0.f : ex2(m - to), w = ex2(ml[i].x - to);
                    l = l * f + ml[i].y * w;
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        o[k].x = o[k].x * f + v[i][k].x * w;
                        o[k].y = o[k].y * f + v[i][k].y * w;
                        o[k].z = o[k].z * f + v[i][k].z * w;
                        o[k].w = o[k].w * f + v[i][k].w * w;
                    }
                    m = to;
                }
            }
#pragma unroll
            for (int off = ROWS; off < 32; off <<= 1) {
                const float m2 = __shfl_xor_sync(FULL_MASK, m, off), l2 = __shfl_xor_sync(FULL_MASK, l, off);
                bad |= __shfl_xor_sync(FULL_MASK, static_cast<int>(bad), off) != 0;
                const float to = fmaxf(m, m2);
                const float f = m == -INFINITY ? 0.f : ex2(m - to), w = m2 == -INFINITY ? 0.f : ex2(m2 - to);
                l = l * f + l2 * w;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    o[k].x = o[k].x * f + __shfl_xor_sync(FULL_MASK, o[k].x, off) * w;
                    o[k].y = o[k].y * f + __shfl_xor_sync(FULL_MASK, o[k].y, off) * w;
                    o[k].z = o[k].z * f + __shfl_xor_sync(FULL_MASK, o[k].z, off) * w;
                    o[k].w = o[k].w * f + __shfl_xor_sync(FULL_MASK, o[k].w, off) * w;
                }
                m = to;
            }
            const bool none = bad || !(l != 0.f);
            const float inv = none ? 0.f : 1.f / l;
            const auto place_of = [&](int t, int gg) { return (static_cast<size_t>(q.row0) + t) * a.Hq + e.y * a.G + gg; };
            if (lane < ROWS) {
                float odd = 0.f;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float y[4] = {none ? 0.f : o[k].x * inv, none ? 0.f : o[k].y * inv, none ? 0.f : o[k].z * inv,
                                        none ? 0.f : o[k].w * inv};
                    odd += (y[0] + y[1] + y[2] + y[3]) * 0.f;
                    result[lane][warp + 8 * k] = make_uint2(pg_pack_out<BF16>(y[0], y[1]), pg_pack_out<BF16>(y[2], y[3]));
                }
                if (odd != 0.f && valid && l == l) odd_row[lane] = 1;
                if (a.lse != nullptr && valid && warp == 0 && ib == 0)
                    a.lse[place_of(token, g)] = none ? -INFINITY : (m + log2f(l)) * LN2;
            }
            __syncthreads();
            for (int x = threadIdx.x; x < ROWS * NI; x += MERGE_THREADS) {
                int t, gg;
                if (row_of(a, e.z, tokens, row0 + x / NI, t, gg))
                    reinterpret_cast<uint2*>(a.out + place_of(t, gg) * PG_ROW)[ib * NI + x % NI] = result[x / NI][x % NI];
            }
            if constexpr (ch_again(BF16, SPARSE)) {
                // (The rows made anew are written after these.)
                const bool some = __syncthreads_or(threadIdx.x < ROWS && odd_row[threadIdx.x] != 0) != 0;
                const bool large = BF16 && some && large_values<BF16, SPARSE>(a, e.x, e.y, 0, SPARSE ? q.ctx : item_sees<SPARSE>(a, q, e.z));
                for (int x = warp; x < ROWS; x += MERGE_THREADS / 32) {
                    int t, gg;
                    if (odd_row[x] != 0 && row_of(a, e.z, tokens, row0 + x, t, gg))
                        look_again<BF16, SPARSE>(a, q, e.x, e.y, e.z, t, gg, lane, lane / NI == ib, large);
                }
            }
        }
    }
    if constexpr (ch_again(BF16, SPARSE))
        if (flags.w != 0) look_at_items<BF16, SPARSE>(a, desc);
}

// ---------------------------------------------------------------- host

// The cache as copies of a block and head, 4 KB, into units of 8 tokens x 64 channels
// (128-byte-swizzled): those of channels 0 .. 63 and 64 .. 127 of tokens 0 .. 7, then of
// tokens 8 .. 15.  So 8-token groups of either half lie 2048 bytes apart throughout a
// tile, as the products want them, with one copy a block: with a copy for each half (2 KB)
// the copies alone took 1.5 us a tile of K and V.  Blocks and heads share the fifth dimension, in
// units of what divides both strides.
static bool make_map(CUtensorMap* map, const PagedAttnArgs& a, const uint8_t* x, bool bf16, long long unit, long long units) {
    const TensorMapEncode encode = tensor_map_encode();
    if (encode == nullptr) return false;
    const cuuint64_t dims[5] = {64, 8, 2, 2, static_cast<cuuint64_t>(units)};
    const cuuint64_t strides[4] = {static_cast<cuuint64_t>(a.kv_token), 128, static_cast<cuuint64_t>(8 * a.kv_token),
                                   static_cast<cuuint64_t>(unit)};
    const cuuint32_t box[5] = {64, 8, 2, 2, 1}, one[5] = {1, 1, 1, 1, 1};
    return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
                  const_cast<uint8_t*>(x), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as copies of a tile of rows (a.tt tokens, a group's heads) x 64 channels.
static bool make_query_map(CUtensorMap* map, const PagedAttnArgs& a, bool bf16) {
    const TensorMapEncode encode = tensor_map_encode();
    if (encode == nullptr) return false;
    const cuuint64_t dims[4] = {64, 2, static_cast<cuuint64_t>(a.Hq), static_cast<cuuint64_t>(a.N)};
    const cuuint64_t strides[3] = {128, PG_ROW, static_cast<cuuint64_t>(a.q_stride)};
    const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(a.G), static_cast<cuuint32_t>(a.tt)}, one[4] = {1, 1, 1, 1};
    return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<uint8_t*>(a.q), dims,
                  strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workspace a CTA: two pieces' results of 256 rows, and 128 bytes that say of what.
constexpr size_t CHUNK_WS_CTA = 2 * CHUNK_ROWS * (PG_D * sizeof(float) + sizeof(float2)) + 128;

template <bool BF16, bool SPARSE>
static clo_status run_paged(PagedAttnArgs a, void* workspace, const clo_attn_opts* opts, cudaStream_t stream) {
    const auto main = paged_chunk_kernel<BF16, SPARSE>;
    // The roles' registers are taken from those of the launch: with fewer the softmax warps would
    // wait for ever.
    static std::atomic<bool> looked{false};
    if (!looked.load(std::memory_order_relaxed)) {
        cudaFuncAttributes attr;
        if (cudaFuncGetAttributes(&attr, main) != cudaSuccess || attr.numRegs < CH_REGS) return CLO_ERR_CUDA;
        looked.store(true, std::memory_order_relaxed);
    }
    // No item weighs more than the longest request, the new tokens and CH_FIXED.
    const double items = (a.N / (2.0 * a.tt) + min(a.B, a.N)) * a.Hkv;
    const double most = items * (CH_FIXED + (SPARSE ? 16.0 * a.n_sel : 16.0 * a.max_blocks + a.N));
    a.shift = 0;
    while (most / static_cast<double>(1ll << a.shift) >= 1.0e9) ++a.shift;
    // The joining kernel: few rows may have many pieces, so they are spread over more
    // blocks and lanes.
    const long long rows = SPARSE ? a.G : static_cast<long long>(a.N) * a.G;
    const bool few = SPARSE || (rows <= 64 && a.N <= a.tt);
    auto merge = paged_merge_kernel<BF16, SPARSE, 8, 8>;
    if constexpr (!SPARSE)
        if (!few) merge = paged_merge_kernel<BF16, false, 32, 32>;
    const unsigned y = few ? static_cast<unsigned>((rows + 7) / 8) * 4 : CHUNK_ROWS / 32;
    if (!prepare_kernel(reinterpret_cast<const void*>(main), CH_SMEM) ||
        !prepare_kernel(reinterpret_cast<const void*>(merge), 0))
        return CLO_ERR_CUDA;
    const int ctas = opts != nullptr && opts->num_ctas > 0 ? opts->num_ctas : device_sm_count();
    long long unit = a.kv_block, rest = a.kv_head;
    while (rest != 0) {
        const long long x = unit % rest;
        unit = rest;
        rest = x;
    }
    a.unit_block = a.kv_block / unit;
    a.unit_head = a.kv_head / unit;
    const long long units = (a.num_blocks - 1) * a.unit_block + (a.Hkv - 1) * a.unit_head + 1;
    if (units >= (1ll << 31)) return CLO_ERR_UNSUPPORTED;
    CUtensorMap map_q, map_k, map_v;
    if (ctas <= 0 || !make_query_map(&map_q, a, BF16) || !make_map(&map_k, a, a.kc, BF16, unit, units) ||
        !make_map(&map_v, a, a.vc, BF16, unit, units))
        return CLO_ERR_CUDA;
    ChunkWs ws;
    ws.o = static_cast<float4*>(workspace);
    ws.ml = reinterpret_cast<float2*>(ws.o + static_cast<size_t>(ctas) * 2 * CHUNK_ROWS * (PG_D / 4));
    ws.desc = reinterpret_cast<int4*>(ws.ml + static_cast<size_t>(ctas) * 2 * CHUNK_ROWS);
    if (opts != nullptr && opts->ev_begin != nullptr && !record_event(opts->ev_begin, stream)) return CLO_ERR_CUDA;
    if (launch_pdl(main, dim3(ctas), dim3(CH_THREADS), CH_SMEM, stream, a, ws, map_q, map_k, map_v) != cudaSuccess) return CLO_ERR_CUDA;
    if (opts != nullptr && opts->ev_end != nullptr && !record_event(opts->ev_end, stream)) return CLO_ERR_CUDA;
    return launch_pdl(merge, dim3(ctas, y), dim3(MERGE_THREADS), 0, stream, a, ws, ctas) == cudaSuccess ? CLO_OK : CLO_ERR_CUDA;
}

static clo_status run_paged_attention(const PagedAttnArgs& a, bool sparse, clo_dtype dtype, void* workspace, const clo_attn_opts* opts,
                                      cudaStream_t stream) {
    if (dtype == CLO_BF16) return sparse ? run_paged<true, true>(a, workspace, opts, stream) : run_paged<true, false>(a, workspace, opts, stream);
    return sparse ? run_paged<false, true>(a, workspace, opts, stream) : run_paged<false, false>(a, workspace, opts, stream);
}

constexpr int CHUNK_MAX_CTAS = 4095;

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
    if (d != PG_D || block_size != PG_BLOCK || Hq / Hkv > PG_MAX_G || B > PG_MAX_B || rows * Hq >= (1ll << 29) ||
        max_blocks > (1 << 20) || num_blocks > (1 << 26) || (opts != nullptr && opts->num_ctas > CHUNK_MAX_CTAS))
        return CLO_ERR_UNSUPPORTED;
    if (B > 0 && rows > 0) {
        const size_t need = clo_paged_chunk_workspace_size(Hq, Hkv, d, opts != nullptr ? opts->num_ctas : 0);
        if (need == 0) return CLO_ERR_CUDA;
        if (ws == nullptr || ws_bytes < need || !pg_aligned(ws, 16)) return CLO_ERR_WORKSPACE;
    }
    return CLO_OK;
}

// Whether ranges of `pn` and `qn` 16-bit elements share any.
static bool meet(const void* p, long long pn, const void* q, long long qn) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + 2 * static_cast<uintptr_t>(qn) && b < a + 2 * static_cast<uintptr_t>(pn);
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
    for (const long long s : {kb, kh, 16 * kt})
        if (s < r.d || s % 8 != 0 || s > (1ll << 38)) return CLO_ERR_INVALID_ARG;
    if (kt < r.d || kt % 8 != 0) return CLO_ERR_INVALID_ARG;
    if (meet(r.q, (r.N - 1) * (r.N > 1 ? r.q_stride : 0) + row, r.out, r.N * row)) return CLO_ERR_INVALID_ARG;
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
    a.q_stride = 2 * (r.N > 1 ? r.q_stride : row);
    a.kv_block = 2 * kb;
    a.kv_head = 2 * kh;
    a.kv_token = 2 * kt;
    a.scale_log2 = r.scale * LOG2E;
    a.B = r.B;
    a.N = r.N;
    a.Hq = r.Hq;
    a.Hkv = r.Hkv;
    a.G = r.Hq / r.Hkv;
    a.tt = tile_tokens(a.G);
    a.num_blocks = r.num_blocks;
    a.max_blocks = r.max_blocks;
    return run_paged_attention(a, false, r.dtype, r.workspace, r.opts, stream);
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
    const long long elements = static_cast<long long>(r.B) * r.Hq * r.d;
    if (meet(r.q, elements, r.out, elements)) return CLO_ERR_INVALID_ARG;
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
    a.tt = tile_tokens(a.G);
    a.num_blocks = r.num_blocks;
    a.max_blocks = r.max_blocks;
    a.n_sel = r.n_sel;
    return run_paged_attention(a, true, r.dtype, r.workspace, r.opts, stream);
}
