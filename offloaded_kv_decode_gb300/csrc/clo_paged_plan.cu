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
// load, scan, ring read and store.  paged_plan_kernel does all of it in one
// launch where few tokens are new (decoding): one CTA with a thread a request or
// a few, one scan of the three sums where everybody is served, a second one
// only after a refusal.  Where many tokens are new (prompts) it leaves the
// slots to paged_slots_kernel, which spreads them over all SMs and works from
// the plan's outputs, and where many blocks are, a cluster of 8 CTAs, which
// all do the scans, shares the table's entries.  Reads of the lengths and the
// ring's state end at a barrier before the new ones are written, so those can
// be updated in place.
#include <algorithm>

#include "clo_kv4.cuh"

namespace clo {

constexpr int PLAN_MAX_THREADS = 1024;
constexpr int PLAN_PER = KV4_MAX_B / PLAN_MAX_THREADS;  // requests a thread, at most
constexpr int PLAN_CLUSTER = 8;
constexpr int PLAN_MAX_NEW = 1 << 30;  // strided 32-bit loops stay in range
constexpr int SLOTS_THREADS = 256;
constexpr int PLAN_SLOTS_HERE = 4096;   // most slots that the plan's own CTA writes
constexpr int PLAN_FEW = 16;            // new tokens that a request's thread writes by itself
constexpr int PLAN_BLOCKS_HERE = 2048;  // most blocks that one CTA moves

// Exclusive sums over the block of three 32-bit counts a thread (each total
// below 2^31): two as the halves of one 64-bit sum, and a third.
struct PlanSums {
    unsigned long long two;
    int third;
};

__device__ __forceinline__ PlanSums plan_scan(PlanSums v, PlanSums* wsum, PlanSums& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    PlanSums incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned long long u = __shfl_up_sync(FULL_MASK, incl.two, off);
        const int x = __shfl_up_sync(FULL_MASK, incl.third, off);
        if (lane >= off) {
            incl.two += u;
            incl.third += x;
        }
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    // Every warp sums the warps before it (a lane each).
    PlanSums w = lane < nw ? wsum[lane] : PlanSums{0ull, 0};
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned long long u = __shfl_up_sync(FULL_MASK, w.two, off);
        const int x = __shfl_up_sync(FULL_MASK, w.third, off);
        if (lane >= off) {
            w.two += u;
            w.third += x;
        }
    }
    total.two = __shfl_sync(FULL_MASK, w.two, 31);
    total.third = __shfl_sync(FULL_MASK, w.third, 31);
    PlanSums before;
    before.two = incl.two - v.two;
    before.third = incl.third - v.third;
    const unsigned long long u = __shfl_sync(FULL_MASK, w.two, max(warp - 1, 0));
    const int x = __shfl_sync(FULL_MASK, w.third, max(warp - 1, 0));
    if (warp > 0) {
        before.two += u;
        before.third += x;
    }
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

__device__ __forceinline__ int plan_slot(int id, int pos, bool& bad) {
    const bool ok = id >= 0 && id < (1 << 27);
    bad |= !ok;
    return ok ? id * KV4_BLOCK + pos % KV4_BLOCK : -1;
}

__global__ void __launch_bounds__(PLAN_MAX_THREADS) paged_plan_kernel(const clo_paged_plan_args a, bool with_slots) {
    extern __shared__ int psm[];
    __shared__ PlanSums wsum[2][32];
    __shared__ int free_ids[PLAN_MAX_THREADS];  // the ring's first free entries
    const int B = a.B, threads = blockDim.x;
    int* off = psm;               // [B + 1] new tokens before request r
    int* taken = off + B + 1;     // [B + 1] blocks taken before it
    int* given = taken + B + 1;   // [B + 1] blocks given back before it
    int* first = given + B + 1;   // [B] position of its first new token, or -1
    int* had = first + B;         // [B] blocks it had
    int* has = had + B;           // [B] blocks it has

    pdl_launch_dependents();
    pdl_wait();
    int head = a.ring_in[0], count = a.ring_in[1];

    const int room = a.max_blocks * KV4_BLOCK;
    const int per = (B + threads - 1) / threads;
    const int r0 = threadIdx.x * per;
    int len[PLAN_PER], keep[PLAN_PER], add[PLAN_PER], need[PLAN_PER], gave[PLAN_PER];
    int part[PLAN_PER];  // the block that the first new token goes on in, if it has tokens already
    bool good[PLAN_PER];
    bool few = true;     // no request has more new tokens than PLAN_FEW
    int my_add = 0, my_need = 0, my_gave = 0;
#pragma unroll
    for (int x = 0; x < PLAN_PER; ++x) {
        const int r = r0 + x;
        len[x] = keep[x] = add[x] = need[x] = gave[x] = part[x] = 0;
        good[x] = true;
        if (x < per && r < B) {
            len[x] = a.len_in[r];
            keep[x] = a.keep != nullptr ? a.keep[r] : len[x];
            add[x] = a.add[r];
            good[x] = keep[x] >= 0 && keep[x] <= len[x] && len[x] <= room && add[x] >= 0 &&
                      add[x] <= room - keep[x];
            if (!good[x]) {
                add[x] = 0;
            } else {
                const int more = plan_blocks(keep[x] + add[x]) - plan_blocks(len[x]);
                need[x] = max(more, 0);
                gave[x] = max(-more, 0);
                // Read while the sums are made.
                if (add[x] > 0 && keep[x] % KV4_BLOCK != 0)
                    part[x] = a.block_table[static_cast<long long>(r) * a.max_blocks + keep[x] / KV4_BLOCK];
            }
            few = few && add[x] <= PLAN_FEW;
            my_add += add[x];
            my_need += need[x];
            my_gave += gave[x];
        }
    }
    const bool ring_ok = head >= 0 && head < a.ring_size && count >= 0 && count <= a.ring_size;
    const int ring0 = head, ring1 = count;
    const int take_back = ring_ok ? a.ring_size - count : 0;  // entries it has room for
    if (!ring_ok) head = count = 0;
    if (static_cast<int>(threadIdx.x) < count)
        free_ids[threadIdx.x] = a.free_ring[plan_wrap(head, threadIdx.x, a.ring_size)];

    PlanSums total;
    const PlanSums before = plan_scan({plan_pair(my_add, my_need), my_gave}, wsum[0], total);
    const int n_tok = static_cast<int>(total.two & 0xffffffffu);
    int n_taken = static_cast<int>(total.two >> 32), n_given = total.third;
    const bool refused = n_tok > a.max_new || n_taken > count;  // somebody is
    int tok = static_cast<int>(before.two & 0xffffffffu), blk = static_cast<int>(before.two >> 32);
    int t = blk, g = before.third;
    int flags = ring_ok ? 0 : CLO_FLAG_BAD_INDEX;
    int my_taken = 0;
    my_gave = 0;
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
                need[x] = gave[x] = 0;
            }
            const int now = served ? keep[x] + add[x] : len[x];
            // A bad length owns no table column here, whatever it says.
            had[r] = good[x] ? plan_blocks(len[x]) : 0;
            has[r] = good[x] ? plan_blocks(now) : 0;
            first[r] = served ? keep[x] : -1;
            len[x] = now;
            my_taken += need[x];
            my_gave += gave[x];
        }
    }
    if (refused) {  // uniform over the block: what the served ones move
        PlanSums moved;
        const PlanSums m = plan_scan({plan_pair(my_taken, 0), my_gave}, wsum[1], moved);
        t = static_cast<int>(m.two & 0xffffffffu);
        g = m.third;
        n_taken = static_cast<int>(moved.two & 0xffffffffu);
        n_given = moved.third;
    }
#pragma unroll
    for (int x = 0; x < PLAN_PER; ++x) {
        const int r = r0 + x;
        if (x < per && r < B) {
            taken[r] = t;
            given[r] = g;
            t += need[x];
            g += gave[x];
        }
    }
    const int n_back = min(n_given, take_back);
    if (n_back < n_given) flags |= CLO_FLAG_BAD_INDEX;
    if (threadIdx.x == 0) {
        off[B] = n_tok;
        taken[B] = n_taken;
        given[B] = n_given;
    }
    few = __syncthreads_and(few) != 0;
    // Every CTA has read the lengths and the ring's state; from here on they
    // may be overwritten.
    if (gridDim.x > 1) {
        asm volatile("barrier.cluster.arrive.aligned;\n" ::: "memory");
        asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
    }

    const int tid = blockIdx.x * threads + threadIdx.x, nthr = gridDim.x * threads;
    // Blocks given back go behind the free ones; those are taken from its
    // other end.  The reads of a thread's first two go out before the rest.
    const int tail = plan_wrap(head, count, a.ring_size);
    auto given_entry = [&](int i) {
        const int r = plan_owner(given, B, i);
        return a.block_table[static_cast<long long>(r) * a.max_blocks + has[r] + (i - given[r])];
    };
    int back[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (tid + k * nthr < n_back) back[k] = given_entry(tid + k * nthr);

    bool bad = false;
    if (few && gridDim.x == 1) {
        // Each thread writes its requests' blocks and slots itself.
        auto ring_entry = [&](int i) {
            return i < threads ? free_ids[i] : a.free_ring[plan_wrap(head, i, a.ring_size)];
        };
#pragma unroll
        for (int x = 0; x < PLAN_PER; ++x) {
            const int r = r0 + x;
            if (x >= per || r >= B) continue;
            const long long row = static_cast<long long>(r) * a.max_blocks;
            for (int j = 0; j < need[x]; ++j) a.block_table[row + had[r] + j] = ring_entry(taken[r] + j);
            int col = keep[x] / KV4_BLOCK, id = part[x];
            for (int j = 0; with_slots && j < add[x] && off[r] + j < a.max_new; ++j) {
                int slot = -1;
                if (first[r] >= 0) {
                    const int pos = keep[x] + j;
                    if (pos % KV4_BLOCK == 0) {
                        col = pos / KV4_BLOCK;
                        id = col < had[r] ? a.block_table[row + col] : ring_entry(taken[r] + col - had[r]);
                    }
                    slot = plan_slot(id, pos, bad);
                }
                a.slot_map[off[r] + j] = slot;
            }
        }
        for (int i = n_tok + tid; with_slots && i < a.max_new; i += nthr) a.slot_map[i] = -1;
    } else {
        for (int i = tid; with_slots && i < a.max_new; i += nthr) {
            int slot = -1;
            if (i < n_tok) {
                const int r = plan_owner(off, B, i);
                if (first[r] >= 0) {
                    const int pos = first[r] + i - off[r], col = pos / KV4_BLOCK;
                    const int id = col < had[r]
                                       ? a.block_table[static_cast<long long>(r) * a.max_blocks + col]
                                       : a.free_ring[plan_wrap(head, taken[r] + col - had[r], a.ring_size)];
                    slot = plan_slot(id, pos, bad);
                }
            }
            a.slot_map[i] = slot;
        }
        // Column had + j of a row is the ring's entry head + (blocks taken before) + j.
        for (int i = tid; i < n_taken; i += nthr) {
            const int r = plan_owner(taken, B, i);
            a.block_table[static_cast<long long>(r) * a.max_blocks + had[r] + (i - taken[r])] =
                a.free_ring[plan_wrap(head, i, a.ring_size)];
        }
    }
    if (bad) flags |= CLO_FLAG_BAD_INDEX;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (tid + k * nthr < n_back) a.free_ring[plan_wrap(tail, tid + k * nthr, a.ring_size)] = back[k];
    for (int i = tid + 2 * nthr; i < n_back; i += nthr)
        a.free_ring[plan_wrap(tail, i, a.ring_size)] = given_entry(i);
    if (blockIdx.x == 0) {
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
    if (flags != 0) report_error(a.err_flag, flags);
}

// The slots of a plan that paged_plan_kernel has made, from its outputs.  A
// thread makes 4 neighbouring ones at a time.
__global__ void __launch_bounds__(SLOTS_THREADS) paged_slots_kernel(const clo_paged_plan_args a) {
    extern __shared__ int psm[];
    const int B = a.B;
    int* off = psm;             // [B + 1]
    int* first = off + B + 1;   // [B]
    pdl_launch_dependents();
    pdl_wait();
    for (int r = threadIdx.x; r <= B; r += SLOTS_THREADS) {
        off[r] = a.offsets[r];
        if (r < B) first[r] = a.start[r];
    }
    __syncthreads();
    const int n_tok = off[B];
    const bool wide = (reinterpret_cast<uintptr_t>(a.slot_map) & 15u) == 0;
    const int step = gridDim.x * SLOTS_THREADS * 4;
    bool bad = false;
    for (int i0 = (blockIdx.x * SLOTS_THREADS + threadIdx.x) * 4; i0 < a.max_new; i0 += step) {
        int slot[4] = {-1, -1, -1, -1};
        if (i0 < n_tok) {
            int r = plan_owner(off, B, i0);
            int col = -1, id = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + k;
                if (i < n_tok && i < a.max_new) {
                    while (i >= off[r + 1]) {  // on to the next request with new tokens
                        ++r;
                        col = -1;
                    }
                    if (first[r] >= 0) {
                        const int pos = first[r] + i - off[r];
                        if (pos / KV4_BLOCK != col) {
                            col = pos / KV4_BLOCK;
                            id = a.block_table[static_cast<long long>(r) * a.max_blocks + col];
                        }
                        slot[k] = plan_slot(id, pos, bad);
                    }
                }
            }
        }
        if (wide && i0 + 4 <= a.max_new) {
            *reinterpret_cast<int4*>(a.slot_map + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i0 + k < a.max_new) a.slot_map[i0 + k] = slot[k];
        }
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
    const int sms = device_sm_count();
    if (sms <= 0 ||
        !prepare_kernel(reinterpret_cast<const void*>(paged_plan_kernel),
                        static_cast<int>((6 * static_cast<size_t>(KV4_MAX_B) + 3) * sizeof(int))))
        return CLO_ERR_CUDA;
    const size_t smem = (6 * static_cast<size_t>(a.B) + 3) * sizeof(int);
    // Enough threads for the requests, and to move a request's blocks at once.
    const int threads = a.B <= 32 ? PLAN_MAX_THREADS / 4 : PLAN_MAX_THREADS;
    const bool slots_here = a.max_new <= PLAN_SLOTS_HERE;
    const unsigned ctas = a.max_new > PLAN_BLOCKS_HERE * KV4_BLOCK ? PLAN_CLUSTER : 1;
    if (launch_pdl_cluster(paged_plan_kernel, dim3(ctas), dim3(ctas > 1 ? PLAN_MAX_THREADS : threads), smem, stream,
                           ctas, a, slots_here) != cudaSuccess)
        return CLO_ERR_CUDA;
    if (slots_here) return CLO_OK;
    if (!prepare_kernel(reinterpret_cast<const void*>(paged_slots_kernel), 0)) return CLO_ERR_CUDA;
    const long long per_cta = SLOTS_THREADS * 4;
    const long long grid = std::min((a.max_new + per_cta - 1) / per_cta, static_cast<long long>(sms) * 4);
    return launch_pdl(paged_slots_kernel, dim3(static_cast<unsigned>(grid)), dim3(SLOTS_THREADS),
                      (2 * static_cast<size_t>(a.B) + 1) * sizeof(int), stream, a) == cudaSuccess
               ? CLO_OK
               : CLO_ERR_CUDA;
}
