// clo_paged_plan.cu -- clo_paged_plan: block table, slot map and free ring of
// a step, from the requests' lengths.
//
// The mathematics are prefix sums over the requests: of the new tokens (the
// offsets), of the blocks needed (where a request's blocks start in the free
// ring) and, once it is known who is served, of the blocks given back.  The
// served requests among those that need something are a prefix of them (a
// request fails when a running sum passes a limit, and the sums do not fall),
// so what they take from the ring is contiguous.
//
// Latency bounds it: a few KB in, a few KB to a few MB out, and one chain of
// load, two scans, ring read and store.  So it is one launch.  Every CTA does
// the scans over all B <= 4096 requests by itself (three coalesced loads a
// request out of L2), which costs less than handing them round, and then the
// CTAs share the entries to write: one CTA where few tokens are new, one
// cluster of 8 where many are.  The cluster's barrier between the reads of
// the lengths and ring state and the writes of the new ones lets those be
// updated in place.
#include "clo_kv4.cuh"

namespace clo {

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_PER = KV4_MAX_B / PLAN_THREADS;  // requests a thread, at most
constexpr int PLAN_CLUSTER = 8;
constexpr int PLAN_MAX_NEW = 1 << 30;  // strided 32-bit loops stay in range

// Exclusive sums of two 32-bit counts a thread (each total below 2^31) over
// the block, as the two halves of one 64-bit sum; total gets the block's.
__device__ __forceinline__ unsigned long long plan_scan(unsigned long long v, unsigned long long* wsum,
                                                        unsigned long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned long long u = __shfl_up_sync(FULL_MASK, incl, off);
        if (lane >= off) incl += u;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        unsigned long long w = wsum[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const unsigned long long u = __shfl_up_sync(FULL_MASK, w, off);
            if (lane >= off) w += u;
        }
        wsum[lane] = w;
    }
    __syncthreads();
    const unsigned long long before = (warp > 0 ? wsum[warp - 1] : 0ull) + incl - v;
    total = wsum[PLAN_THREADS / 32 - 1];
    __syncthreads();  // wsum is used again
    return before;
}

__device__ __forceinline__ unsigned long long plan_pair(int lo, int hi) {
    return static_cast<unsigned long long>(static_cast<unsigned>(lo)) |
           (static_cast<unsigned long long>(static_cast<unsigned>(hi)) << 32);
}

// The last r with sums[r] <= i (sums ascending, sums[0] = 0, i < sums[n]):
// the request that owns item i.
__device__ __forceinline__ int plan_owner(const int* sums, int n, int i) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sums[mid] <= i) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ int plan_blocks(int tokens) { return (tokens + KV4_BLOCK - 1) / KV4_BLOCK; }

// Entry `head + j` of the ring, head < size, j < size.
__device__ __forceinline__ int plan_wrap(int head, int j, int size) {
    const unsigned x = static_cast<unsigned>(head) + static_cast<unsigned>(j);
    return static_cast<int>(x >= static_cast<unsigned>(size) ? x - static_cast<unsigned>(size) : x);
}

__global__ void __launch_bounds__(PLAN_THREADS) paged_plan_kernel(const clo_paged_plan_args a) {
    extern __shared__ int psm[];
    __shared__ unsigned long long wsum[32];
    const int B = a.B;
    int* off = psm;               // [B + 1] new tokens before request r
    int* taken = off + B + 1;     // [B + 1] blocks taken before it
    int* given = taken + B + 1;   // [B + 1] blocks given back before it
    int* first = given + B + 1;   // [B] position of its first new token, or -1
    int* had = first + B;         // [B] blocks it had
    int* has = had + B;           // [B] blocks it has

    pdl_launch_dependents();
    pdl_wait();
    int head = a.ring_in[0], count = a.ring_in[1];
    const bool ring_ok = head >= 0 && head < a.ring_size && count >= 0 && count <= a.ring_size;
    const int ring0 = head, ring1 = count;
    const int take_back = ring_ok ? a.ring_size - count : 0;  // entries it has room for
    if (!ring_ok) head = count = 0;

    const int room = a.max_blocks * KV4_BLOCK;
    const int per = (B + PLAN_THREADS - 1) / PLAN_THREADS;
    const int r0 = threadIdx.x * per;
    int len[PLAN_PER], keep[PLAN_PER], add[PLAN_PER], need[PLAN_PER];
    bool good[PLAN_PER];
    int my_add = 0, my_need = 0;
#pragma unroll
    for (int x = 0; x < PLAN_PER; ++x) {
        const int r = r0 + x;
        len[x] = keep[x] = add[x] = need[x] = 0;
        good[x] = true;
        if (x < per && r < B) {
            len[x] = a.len_in[r];
            keep[x] = a.keep != nullptr ? a.keep[r] : len[x];
            add[x] = a.add[r];
            good[x] = keep[x] >= 0 && keep[x] <= len[x] && len[x] <= room && add[x] >= 0 &&
                      add[x] <= room - keep[x];
            if (!good[x]) add[x] = 0;
            else need[x] = max(plan_blocks(keep[x] + add[x]) - plan_blocks(len[x]), 0);
            my_add += add[x];
            my_need += need[x];
        }
    }
    unsigned long long total;
    const unsigned long long before = plan_scan(plan_pair(my_add, my_need), wsum, total);
    int tok = static_cast<int>(before & 0xffffffffu), blk = static_cast<int>(before >> 32);
    int flags = ring_ok ? 0 : CLO_FLAG_BAD_INDEX;
    int my_taken = 0, my_given = 0;
#pragma unroll
    for (int x = 0; x < PLAN_PER; ++x) {
        const int r = r0 + x;
        if (x < per && r < B) {
            off[r] = tok;
            tok += add[x];
            blk += need[x];
            const bool served = good[x] && (add[x] == 0 || (tok <= a.max_new && blk <= count));
            if (!served) {
                flags |= good[x] ? CLO_FLAG_NO_ROOM : CLO_FLAG_BAD_CTX;
                need[x] = 0;
            }
            const int now = served ? keep[x] + add[x] : len[x];
            // A bad length owns no table column here, whatever it says.
            had[r] = good[x] ? plan_blocks(len[x]) : 0;
            has[r] = good[x] ? plan_blocks(now) : 0;
            first[r] = served ? keep[x] : -1;
            len[x] = now;
            my_taken += need[x];
            my_given += max(had[r] - has[r], 0);
        }
    }
    unsigned long long moved;
    const unsigned long long moved_before = plan_scan(plan_pair(my_taken, my_given), wsum, moved);
    int t = static_cast<int>(moved_before & 0xffffffffu), g = static_cast<int>(moved_before >> 32);
#pragma unroll
    for (int x = 0; x < PLAN_PER; ++x) {
        const int r = r0 + x;
        if (x < per && r < B) {
            taken[r] = t;
            given[r] = g;
            t += need[x];
            g += max(had[r] - has[r], 0);
        }
    }
    const int n_tok = static_cast<int>(total & 0xffffffffu);
    const int n_taken = static_cast<int>(moved & 0xffffffffu);
    const int n_given = static_cast<int>(moved >> 32);
    const int n_back = min(n_given, take_back);
    if (n_back < n_given) flags |= CLO_FLAG_BAD_INDEX;
    if (threadIdx.x == 0) {
        off[B] = n_tok;
        taken[B] = n_taken;
        given[B] = n_given;
    }
    // Every CTA has read the lengths and the ring's state; from here on they
    // may be overwritten.
    if (gridDim.x > 1) {
        asm volatile("barrier.cluster.arrive.aligned;\n" ::: "memory");
        asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
    } else {
        __syncthreads();
    }

    const int tid = blockIdx.x * PLAN_THREADS + threadIdx.x, nthr = gridDim.x * PLAN_THREADS;
    if (blockIdx.x == 0) {
        if (flags != 0) report_error(a.err_flag, flags);
#pragma unroll
        for (int x = 0; x < PLAN_PER; ++x) {
            const int r = r0 + x;
            if (x < per && r < B) {
                a.len_out[r] = len[x];
                a.start[r] = first[r];
                a.offsets[r] = off[r];
            }
        }
        if (threadIdx.x == 0) {
            a.offsets[B] = n_tok;
            a.ring_out[0] = ring_ok ? plan_wrap(head, n_taken, a.ring_size) : ring0;
            a.ring_out[1] = ring_ok ? count - n_taken + n_back : ring1;
        }
    }
    // Blocks taken: column had + j of a row is the ring's entry head + (blocks taken before) + j.
    for (int i = tid; i < n_taken; i += nthr) {
        const int r = plan_owner(taken, B, i);
        a.block_table[static_cast<long long>(r) * a.max_blocks + had[r] + (i - taken[r])] =
            a.free_ring[plan_wrap(head, i, a.ring_size)];
    }
    // Blocks given back go behind the free ones; those are taken from its other end.
    for (int i = tid; i < n_back; i += nthr) {
        const int r = plan_owner(given, B, i);
        a.free_ring[plan_wrap(plan_wrap(head, count, a.ring_size), i, a.ring_size)] =
            a.block_table[static_cast<long long>(r) * a.max_blocks + has[r] + (i - given[r])];
    }
    // Slots, and the padding behind them.
    bool bad = false;
    for (int i = tid; i < a.max_new; i += nthr) {
        int slot = -1;
        if (i < n_tok) {
            const int r = plan_owner(off, B, i);
            if (first[r] >= 0) {
                const int pos = first[r] + i - off[r], col = pos / KV4_BLOCK;
                const int id = col < had[r]
                                   ? a.block_table[static_cast<long long>(r) * a.max_blocks + col]
                                   : a.free_ring[plan_wrap(head, taken[r] + col - had[r], a.ring_size)];
                const bool ok = id >= 0 && id < (1 << 27);
                bad |= !ok;
                slot = ok ? id * KV4_BLOCK + pos % KV4_BLOCK : -1;
            }
        }
        a.slot_map[i] = slot;
    }
    if (bad) report_error(a.err_flag, CLO_FLAG_BAD_INDEX);
}

}  // namespace clo

using namespace clo;

extern "C" clo_status clo_paged_plan(const clo_paged_plan_args* args, cudaStream_t stream) {
    if (args == nullptr) return CLO_ERR_INVALID_ARG;
    const clo_paged_plan_args& a = *args;
    if (a.B < 0 || a.max_blocks < 1 || a.ring_size < 1 || a.max_new < 0) return CLO_ERR_INVALID_ARG;
    if (a.free_ring == nullptr || a.ring_in == nullptr || a.ring_out == nullptr || a.offsets == nullptr ||
        (a.max_new > 0 && a.slot_map == nullptr))
        return CLO_ERR_INVALID_ARG;
    if (a.B > 0 && (a.len_in == nullptr || a.add == nullptr || a.block_table == nullptr ||
                    a.len_out == nullptr || a.start == nullptr))
        return CLO_ERR_INVALID_ARG;
    for (const int32_t* p : {a.len_in, a.keep, a.add, static_cast<const int32_t*>(a.block_table),
                             static_cast<const int32_t*>(a.free_ring), a.ring_in,
                             static_cast<const int32_t*>(a.ring_out), static_cast<const int32_t*>(a.len_out),
                             static_cast<const int32_t*>(a.start), static_cast<const int32_t*>(a.offsets),
                             static_cast<const int32_t*>(a.slot_map), static_cast<const int32_t*>(a.err_flag)})
        if (!kv4_aligned(p, 4)) return CLO_ERR_INVALID_ARG;
    if (a.block_size != KV4_BLOCK || a.B > KV4_MAX_B || a.max_new > PLAN_MAX_NEW || a.ring_size > PLAN_MAX_NEW)
        return CLO_ERR_UNSUPPORTED;
    if (static_cast<long long>(a.B > 0 ? a.B : 1) * a.max_blocks * KV4_BLOCK >= (1ll << 31))
        return CLO_ERR_UNSUPPORTED;
    const size_t smem = (6 * static_cast<size_t>(a.B) + 3) * sizeof(int);
    if (!prepare_kernel(reinterpret_cast<const void*>(paged_plan_kernel),
                        static_cast<int>((6 * static_cast<size_t>(KV4_MAX_B) + 3) * sizeof(int))))
        return CLO_ERR_CUDA;
    // One CTA writes 4096 slots in the time that a cluster's launch adds.
    const unsigned ctas = a.max_new > 4 * PLAN_THREADS ? PLAN_CLUSTER : 1;
    return launch_pdl_cluster(paged_plan_kernel, dim3(ctas), dim3(PLAN_THREADS), smem, stream, ctas, a) ==
                   cudaSuccess
               ? CLO_OK
               : CLO_ERR_CUDA;
}
