// clo_kv4_sets.cu -- the kernel of clo_kv4_paged_decode_attn that gives each
// token set (request, KV head) to a cluster of its own (a warp's work:
// clo_kv4_math.cuh; the other kernel, which shares all units out evenly:
// clo_kv4_attention.cu).
//
// A cluster is 1 to 8 CTAs; the set's units are cut evenly over its warps.  A
// CTA's warps meet in shared memory, the CTAs in the cluster's (distributed
// shared memory), where each then finishes a part of the outputs: one launch,
// no workspace, no prefix sums and searches, and a fixed order of the sums.  It
// is the faster one in three cases.
//   * Short contexts, where the time is latency.  One request of 1024 tokens (8
//     KV heads, 4 query heads each): 5.0 us against 11.5; 8 requests of 4096:
//     16.1 against 19.2; 64 of 1024: 20.5 against 28.4.
//   * Many sets, several for each place a CTA has, where the hardware's order of
//     CTAs levels the load better than an equal split does (the warps of an SM
//     do not advance alike).  4096 sets of 2048 tokens: 197 us against 209; of
//     4096: 374 and 389; of 128 to 4096: 217 both.  No order of CTAs levels
//     sets of any length: with one request of 128K tokens among 79 of up to 2048
//     (32 KV heads) 1115 us against 170.  So there is a limit here too, by the
//     table's width.
//   * Sets that nearly fill the places, up to about 2048 tokens: 64 requests of
//     2048 tokens 34.5 us against 40.9, of 1 to 2048 29.5 against 30.3; with 16
//     query rows 48 requests 39.0 against 46.7 and 35.6 against 34.5, with 32
//     rows 36 of 1 to 2048 43 against 63.
// With a place or two for each long set the even split wins: 128 sets of 64K
// tokens 211 us against 249, 1024 of 1 to 8192 tokens 123 against 150, 512 of 1
// to 4096 tokens 43 against 54, 384 of 1 to 2048 24.5 against 27.5.
#include <algorithm>

#include "clo_kv4_math.cuh"

namespace clo {

constexpr int SET_MAX_CLUSTER = 8;
// Where the even split wins, by measurement.
constexpr int SET_WARP_UNITS = 12;       // more units a warp, the sets all at once
constexpr int SET_WARP_UNITS_MANY = 16;  // the same with 0.75 to 1 and 1.25 to 4 sets a place
// The same from 4 sets a place on.  2560 sets of 1 to 4096 tokens (4 query rows
// each, up to 32 units a warp) 154 us against 150, of 1 to 8192 tokens 290
// against 268; with one row and 3200 sets 191 against 192, and 363 against 350.
constexpr int SET_WARP_UNITS_MOST = 32;
// Sets for each place and unit (by the table's width), with over 2 sets a place: a
// CTA's start and end cost as much as some units.  8 KV heads, 4 query rows each:
// 256 requests of 1 to 32 tokens 14.8 us against 10.5, of 1 to 96 17.1 against
// 18.1, of 1 to 224 19.7 against 25.5; 600 of 1 to 160 39.2 against 36.1, of 1 to
// 224 42.8 and 42.5.  16 rows, 200 requests: of 1 to 96 tokens 26.7 against 23.2,
// of 1 to 128 27 and 27.5; 32 rows: of 1 to 32 62 against 35, of 1 to 160 79
// against 109.
constexpr float SET_MOST_A_UNIT = 1.15f;

__device__ __forceinline__ unsigned cluster_size() {
    unsigned n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;\n" : "=r"(n));
    return n;
}
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctaid.x;\n" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, unsigned rank) {
    uint32_t d;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(d) : "r"(addr), "r"(rank));
    return d;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];\n"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 cluster_load2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];\n" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// Shared memory of a CTA, in bytes from its start.
struct SetLayout {
    int ring, warp, sums, bars, total;  // ring, warp: bytes of a warp's ring, and with its queries
};

__host__ __device__ inline SetLayout set_layout(int nt, int ng, int rows, int cluster) {
    SetLayout y;
    y.ring = kv4_stages(ng) * 2 * kv4_record(ng);
    const int piece = rows * KV4_PIECE_ROW * static_cast<int>(sizeof(float));
    const int both = y.ring + kv4_query_bytes(nt, ng);
    y.warp = ((both > piece ? both : piece) + 127) / 128 * 128;  // the warp's piece takes their place
    y.sums = KV4_WARPS * y.warp;
    y.bars = y.sums + (cluster > 1 ? (piece + 15) / 16 * 16 : 0);
    y.total = y.bars + KV4_WARPS * kv4_stages(ng) * 8;
    return y;
}

template <bool BF16, int NT, int NG>
__global__ void __launch_bounds__(KV4_THREADS, kv4_ctas_per_sm(NT)) kv4_set_kernel(const Kv4Args a) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int has_piece[KV4_WARPS];
    constexpr int R = kv4_record(NG), STAGES = kv4_stages(NG);
    const unsigned ctas = cluster_size(), rank = cluster_rank();
    const SetLayout y = set_layout(NT, NG, a.rows, ctas);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* ring = smem + warp * y.warp;
    const uint32_t bars = smem_u32(smem + y.bars) + warp * STAGES * 8;
    const int set = blockIdx.x / ctas, r = set / a.Hkv, h = set - r * a.Hkv;

    if (lane < STAGES) mbar_init(bars + lane * 8);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    __syncwarp();
    pdl_launch_dependents();
    pdl_wait();
    int n = a.ctx_len[r];
    if (n < 0 || n > a.max_blocks * KV4_BLOCK) {
        if (threadIdx.x == 0 && rank == 0) report_error(a.err_flag, CLO_FLAG_BAD_CTX);
        n = 0;
    }
    const int units = (n + KV4_UNIT - 1) / KV4_UNIT, blocks = (n + KV4_BLOCK - 1) / KV4_BLOCK;
    const int warps = ctas * KV4_WARPS, w_at = rank * KV4_WARPS + warp;
    const int u0 = units * w_at / warps, u1 = units * (w_at + 1) / warps;
    if (lane == 0) has_piece[warp] = u0 < u1;
    if (u0 < u1) {
        const int32_t* row = a.table + static_cast<size_t>(r) * a.max_blocks;
        const uint64_t policy = l2_evict_first_policy();
        const uint8_t* head_pool = a.pool + static_cast<size_t>(h) * R;
        const size_t block_bytes = static_cast<size_t>(a.Hkv) * R;
        // Lane i holds the id of block 2u + i, u the first of 16 units; the
        // second block of a unit may be behind the last one.
        int id = -1;
        bool exists = false, ok = false;
        auto load_ids = [&](int u) {
            const int entry = 2 * u + lane;
            exists = entry < blocks;
            id = exists ? row[entry] : -1;
            ok = exists && id >= 0 && id < a.num_blocks;
        };
        load_ids(u0);
        uint32_t bad_slots = 0;  // stages with a record that does not exist
        // Loads unit u0 + k: lanes 2k and 2k + 1 of its 16.
        auto issue = [&](int k) {
            const int stage = k % STAGES, at = 2 * (k & 15);
            if ((k & 15) == 0 && k > 0) load_ids(u0 + k);
            const uint32_t have = (__ballot_sync(FULL_MASK, ok) >> at) & 3u, bar = bars + stage * 8;
            const uint32_t wrong = (__ballot_sync(FULL_MASK, exists && !ok) >> at) & 3u;
            bad_slots = (bad_slots & ~(1u << stage)) | (wrong != 0u ? 1u << stage : 0u);
            if (lane == at) {
                if (have != 0u) mbar_expect(bar, have == 3u ? 2 * R : R);
                else mbar_arrive(bar);
            }
            __syncwarp();
            if ((lane & 30) == at && ok)
                bulk_load(smem_u32(ring) + (2 * stage + (lane & 1)) * R, head_pool + id * block_bytes, R, bar, policy);
        };
        const int mine = u1 - u0;
        for (int k = 0; k < STAGES && k < mine; ++k) issue(k);

        Queries<NT, NG> qs;
        qs.sm = reinterpret_cast<float*>(ring + y.ring);
        load_queries<BF16, NT, NG>(a, r, h, lane, qs);
        Softmax<NT, NG> w;
        reset(w);
        bool bad = false, first = true;
        int k = 0;
#pragma unroll 1
        for (; k < mine; ++k) {
            const int stage = k % STAGES, left = n - (u0 + k) * KV4_UNIT;
            if (!warp_wait(bars + stage * 8, (k / STAGES) & 1)) break;
            if (((bad_slots >> stage) & 1u) != 0u) {
                bad = true;
                if (lane == 0) report_error(a.err_flag, CLO_FLAG_BAD_INDEX);
            } else {
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
            }
            __syncwarp();
            if (k + STAGES < mine) issue(k + STAGES);
        }
        if (k < mine) {  // a record did not come
            bad = true;
            give_up<STAGES>(a.err_flag, bars, k % STAGES, (k / STAGES) & 1, lane);
        }
        __syncwarp();
        end_set<BF16, NT, NG>(a, w, r, h, bad, reinterpret_cast<float*>(ring), lane);
    }
    __syncthreads();

    // The CTA's sums, from its warps' pieces.
    float* sums = reinterpret_cast<float*>(smem + y.sums);
    for (int it = threadIdx.x; it < a.rows * (KV4_D / 4); it += KV4_THREADS) {
        const int row = it / (KV4_D / 4), col = it % (KV4_D / 4);
        float2 ml[KV4_WARPS];
        float4 v[KV4_WARPS];
#pragma unroll
        for (int p = 0; p < KV4_WARPS; ++p) {
            ml[p] = make_float2(-INFINITY, 0.f);
            v[p] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (has_piece[p]) {
                const float* pc = reinterpret_cast<const float*>(smem + p * y.warp) + row * KV4_PIECE_ROW;
                ml[p] = *reinterpret_cast<const float2*>(pc + KV4_D);
                v[p] = *reinterpret_cast<const float4*>(pc + 4 * col);
            }
        }
        Sums s;
        s.take<KV4_WARPS>(ml, v);
        if (ctas == 1) {
            s.write<BF16>(a, r, h, row, col);
        } else {
            *reinterpret_cast<float4*>(sums + row * KV4_PIECE_ROW + 4 * col) = s.O;
            if (col == 0) *reinterpret_cast<float2*>(sums + row * KV4_PIECE_ROW + KV4_D) = make_float2(s.M, s.L);
        }
    }
    if (ctas == 1) return;  // uniform over the grid

    // The set's: each CTA finishes a part of the rows' channels.
    cluster_sync_all();
    uint32_t at[SET_MAX_CLUSTER];
#pragma unroll
    for (int c = 0; c < SET_MAX_CLUSTER; ++c)
        at[c] = cluster_map(smem_u32(sums), c < static_cast<int>(ctas) ? c : 0);
    for (int it = rank * KV4_THREADS + threadIdx.x; it < a.rows * (KV4_D / 4); it += ctas * KV4_THREADS) {
        const int row = it / (KV4_D / 4), col = it % (KV4_D / 4);
        float2 ml[SET_MAX_CLUSTER];
        float4 v[SET_MAX_CLUSTER];
#pragma unroll
        for (int c = 0; c < SET_MAX_CLUSTER; ++c) {
            ml[c] = make_float2(-INFINITY, 0.f);
            v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < static_cast<int>(ctas)) {
                ml[c] = cluster_load2(at[c] + (row * KV4_PIECE_ROW + KV4_D) * 4);
                v[c] = cluster_load4(at[c] + (row * KV4_PIECE_ROW + 4 * col) * 4);
            }
        }
        Sums s;
        s.take<SET_MAX_CLUSTER>(ml, v);
        s.write<BF16>(a, r, h, row, col);
    }
    cluster_sync_all();  // no CTA leaves while another reads its shared memory
}

template <bool BF16, int NT>
static void (*set_kernel_ng(int ng))(const Kv4Args) {
    return ng == 1 ? kv4_set_kernel<BF16, NT, 1> : ng == 2 ? kv4_set_kernel<BF16, NT, 2> : kv4_set_kernel<BF16, NT, 4>;
}
template <bool BF16>
static void (*set_kernel(int nt, int ng))(const Kv4Args) {
    return nt == 1   ? set_kernel_ng<BF16, 1>(ng)
           : nt == 2 ? set_kernel_ng<BF16, 2>(ng)
                     : set_kernel_ng<BF16, 4>(ng);
}

// A cluster large enough for a unit a warp, but no larger than lets every set
// start at once; 0 where the even split is faster.  Lengths are on the device:
// the table's width stands for them.
int kv4_set_cluster(const Kv4Args& a, int ng) {
    const long long units = (a.max_blocks + 1) / 2, sets = static_cast<long long>(a.B) * a.Hkv;
    const int nt = kv4_row_tiles(a.rows), sms = device_sm_count();
    auto places = [&](int cluster) {  // CTAs that run at once
        const int smem = set_layout(nt, ng, a.rows, cluster).total + KV4_SMEM_RESERVED;
        return static_cast<long long>(sms) * std::min(kv4_ctas_per_sm(nt), KV4_SMEM_PER_SM / smem);
    };
    int cluster = 1;
    while (cluster < SET_MAX_CLUSTER && units > static_cast<long long>(cluster) * KV4_WARPS &&
           sets * cluster * 2 <= places(2))
        cluster *= 2;
    const long long a_warp = (units + cluster * KV4_WARPS - 1) / (cluster * KV4_WARPS), room = places(cluster);
    const bool filled = sets * cluster <= room && sets * cluster * 4 >= room * 3;
    if (sets * cluster * 4 <= room * 5)
        return a_warp <= (filled ? SET_WARP_UNITS_MANY : SET_WARP_UNITS) ? cluster : 0;
    if (sets > 2 * room && sets > SET_MOST_A_UNIT * room * units) return 0;
    return a_warp <= (sets >= 4 * room ? SET_WARP_UNITS_MOST : SET_WARP_UNITS_MANY) ? cluster : 0;
}

cudaError_t kv4_launch_sets(const Kv4Args& a, int ng, bool bf16, int cluster, cudaStream_t stream) {
    const int nt = kv4_row_tiles(a.rows);
    const auto kernel = bf16 ? set_kernel<true>(nt, ng) : set_kernel<false>(nt, ng);
    const int smem = set_layout(nt, ng, a.rows, cluster).total;
    if (!prepare_kernel(reinterpret_cast<const void*>(kernel), set_layout(nt, ng, KV4_MAX_ROWS, 2).total))
        return cudaErrorUnknown;
    return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(a.B) * a.Hkv * cluster), dim3(KV4_THREADS), smem, stream,
                              static_cast<unsigned>(cluster), a);
}

}  // namespace clo
