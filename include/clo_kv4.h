/*
 * clo_kv4.h -- C ABI of libclo's paged KV cache held in 4 bits: the block
 * plan of a step, the write of new tokens, the read-back in 16 bits and the
 * decode attention over the cache.
 *
 * A decode step of a paged cache is four things: which blocks and slots the
 * new tokens of each request get (clo_paged_plan), their K and V written
 * there (clo_kv4_append), the attention of the new queries over every cached
 * token (clo_kv4_paged_decode_attn), and, for a prompt computed in chunks
 * with a 16-bit attention of the caller's own, the tokens before the chunk read
 * back (clo_kv4_gather).  The paged cache and its block table are those of
 * clo_paged_decode_attn (clo.h); a token's slot is
 *     block * block_size + (position % block_size).
 * In 4 bits a cached token takes 136 to 160 bytes a KV head instead of 512,
 * so a step reads, and an offloaded cache moves, 3.2 to 3.8 times less.
 *
 * Conventions: those of clo.h (device pointers owned by the caller, row-major
 * layouts, asynchronous on `stream`, host validation before any launch,
 * data-dependent errors ORed into *err_flag, no allocation, no exception
 * across the interface).  The data type of 16-bit tensors is an argument
 * (clo_dtype).  d (head dimension) must be 128 and block_size 16 in this
 * build.  Each call takes its arguments in a struct, which it only reads
 * before it returns; a program that makes a call again each step keeps one.
 *
 * The cache.  pool is [num_blocks][Hkv][R] bytes: a record of
 * R = clo_kv4_block_bytes(16, 128, group) bytes holds the 16 tokens of one
 * block and one KV head.  Each row of 128 channels is cut into NG = 128/group
 * groups (group = 32, 64 or 128 channels); each token has, for K and for V,
 * one pair (scale, zero) of fp16 a group, and one code 0..15 a channel:
 *     value = code * scale + zero.
 * (clo_kv4_append writes no negative scale, but a record may hold one.)
 * A record is
 *   bytes    0..1023  K codes, 64 bytes a token: 32-bit word 4c + j of a row
 *                     holds channels 32j + 8c .. 32j + 8c + 7;
 *   bytes 1024..2047  V codes, 64 bytes a token: channels 32c .. 32c + 31 of
 *                     token t are the 16-byte chunk c ^ ((t >> 1) & 3) of its
 *                     row, in order;
 *   bytes 2048..R-1   the pairs, [16 tokens][K, V][NG], scale first;
 * channel 8w + i of the eight in a word is at its bits 4i .. 4i + 3.  (The
 * order of the words and chunks is the one in which the attention's matrix
 * instructions take them without a shuffle.)  A pool may start uninitialised:
 * what no append has written is never used.
 */
#ifndef CLO_KV4_H_
#define CLO_KV4_H_

#include "clo.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum clo_dtype {
    CLO_F16 = 0, /* IEEE binary16 */
    CLO_BF16 = 1 /* bfloat16 */
} clo_dtype;

/* ORed into *err_flag by clo_paged_plan when a request got no room. */
#define CLO_FLAG_NO_ROOM 0x10 /* the free blocks or the slot map ran out */

/* Bytes of one record of the cache, or 0 for sizes this build does not have. */
size_t clo_kv4_block_bytes(int block_size, int d, int group);

/*
 * clo_paged_plan -- the block table and slot map of a step, made on the GPU
 * from the requests' lengths.  Request r has len_in[r] cached tokens in the
 * blocks table[r][0 .. ceil(len/16)).  The step keeps the first keep[r] of
 * them (drafted tokens that were rejected are dropped this way; 0 ends a
 * request) and gives it add[r] new ones.  With nb(x) = ceil(x / block_size):
 *   - the new length is keep + add;
 *   - if nb(keep + add) > nb(len), that many blocks are taken from the free
 *     ring, in the order of the requests, into columns nb(len) .. of its row;
 *   - if it is smaller, the blocks of columns nb(keep + add) .. nb(len) - 1
 *     go back to the ring, in the order of the requests and columns (the row
 *     itself is left as it is), and can be taken from the next call on;
 *   - its j-th new token is token offsets[r] + j of the step's batch, where
 *     offsets[r] = add[0] + .. + add[r-1], and
 *     slot_map[offsets[r] + j] = table[r][p / 16] * 16 + p % 16, p = keep + j.
 * The entries of slot_map behind the last new token are set to -1, which
 * clo_kv4_append and clo_kv4_gather skip: a captured step of a fixed number
 * of tokens can be padded.
 * A request is left as it was (len_out = len_in, start = -1, nothing taken or
 * given back, -1 in the slots of its new tokens) if
 *   - its numbers are bad: not 0 <= keep <= len <= max_blocks * 16, add < 0 or
 *     keep + add > max_blocks * 16 (CLO_FLAG_BAD_CTX; such a request counts as
 *     add = 0 in offsets), or
 *   - it has new tokens and there is no room: the new tokens up to and with
 *     its own are more than max_new, or the blocks that the good requests up
 *     to and with it need are more than the ring has (CLO_FLAG_NO_ROOM).
 * len_in:  [B] int32.  keep: [B] int32, or NULL for keep = len.  add: [B] int32.
 * block_table: [B][max_blocks] int32, updated in place.
 * free_ring: [ring_size] int32 block ids, updated in place; ring_size is at
 *          least the number of blocks that exist.  The free blocks are the
 *          ring_in[1] entries from ring_in[0] on, round the end.
 * ring_in, ring_out: [2] int32 (first entry, count) before and after.  A
 *          state out of range counts as an empty ring that takes nothing, and
 *          blocks given back to a full one are dropped (CLO_FLAG_BAD_INDEX).
 * len_out: [B] int32.  start: [B] int32, the position of the first new token,
 *          or -1.  offsets: [B + 1] int32.  slot_map: [max_new] int32 (may be
 *          NULL when max_new == 0).
 * len_out may be len_in, and ring_out may be ring_in; other arrays may not
 * overlap.
 * Requires block_size == 16, 0 <= B <= 4096, B * max_blocks * 16 < 2^31,
 * max_new <= 2^30, ring_size <= 2^30.
 * With B == 0 the padding, offsets[0] = 0 and ring_out are still written.
 */
typedef struct clo_paged_plan_args {
    const int32_t* len_in;
    const int32_t* keep;
    const int32_t* add;
    int32_t* block_table;
    int32_t* free_ring;
    const int32_t* ring_in;
    int32_t* ring_out;
    int32_t* len_out;
    int32_t* start;
    int32_t* offsets;
    int32_t* slot_map;
    int32_t* err_flag;
    int B;
    int block_size;
    int max_blocks;
    int ring_size;
    int max_new;
} clo_paged_plan_args;

clo_status clo_paged_plan(const clo_paged_plan_args* args, cudaStream_t stream);

/*
 * clo_kv4_append -- writes the K and V rows of N new tokens into the cache.
 * Row n goes to slot slot_map[n].  For each group of channels, with x its
 * values:
 *     zero = min x, rounded down to fp16,
 *     scale = (max x - zero) / 15, rounded up to fp16,
 *     code = (x - zero) / scale, rounded to the nearest integer (ties to
 *            even), 0 where scale is 0.
 * So no code is cut off and an element is off by at most scale / 2.  A group
 * with a NaN or an infinity gets scale = zero = NaN and reads back as NaN.
 * bf16 values beyond +-65504 are taken as +-65504.
 * k, v:     [N][Hkv][d] of type `dtype`; rows of consecutive tokens are
 *           k_stride / v_stride elements apart (a multiple of 8, at least
 *           Hkv * d), so both may be parts of a fused projection's output.
 * slot_map: [N] int32, distinct slots; -1 skips the row.  Any other slot
 *           outside [0, num_blocks * 16) sets CLO_FLAG_BAD_INDEX and skips it.
 * Requires k, v and pool 16-byte aligned, N * Hkv < 2^31 - 2^20.
 */
typedef struct clo_kv4_append_args {
    const void* k;
    const void* v;
    long long k_stride;
    long long v_stride;
    const int32_t* slot_map;
    uint8_t* pool;
    int32_t* err_flag;
    clo_dtype dtype;
    int N;
    int Hkv;
    int d;
    int num_blocks;
    int block_size;
    int group;
} clo_kv4_append_args;

clo_status clo_kv4_append(const clo_kv4_append_args* args, cudaStream_t stream);

/*
 * clo_kv4_gather -- reads the rows of N slots back in 16 bits: what the
 * attention takes as their K and V, code * scale + zero rounded to the nearest
 * value of `dtype` (for bf16 by way of fp32).  In fp16 a value beyond +-65504 is
 * read as +-65504: the scale is rounded up, so the code of a group's largest
 * element may stand for up to 64 more.
 * slot_map: [N] int32; a slot may repeat.  -1 gives a row of zeros, any other
 *           slot outside [0, num_blocks * 16) too (and CLO_FLAG_BAD_INDEX).
 * k, v:     [N][Hkv][d] of type `dtype`, contiguous, 16-byte aligned.
 */
typedef struct clo_kv4_gather_args {
    const uint8_t* pool;
    const int32_t* slot_map;
    void* k;
    void* v;
    int32_t* err_flag;
    clo_dtype dtype;
    int N;
    int Hkv;
    int d;
    int num_blocks;
    int block_size;
    int group;
} clo_kv4_gather_args;

clo_status clo_kv4_gather(const clo_kv4_gather_args* args, cudaStream_t stream);

/* Workspace bytes clo_kv4_paged_decode_attn needs when run with num_ctas CTAs
 * (0 = the default grid on the current device); 0 for invalid sizes.  It needs
 * no initialisation and may be reused by later calls on the same stream. */
size_t clo_kv4_paged_workspace_size(int B, int n_q, int Hq, int Hkv, int d, int num_ctas);

/*
 * clo_kv4_paged_decode_attn -- decode attention over the 4-bit paged cache
 * for the last n_q tokens of each request (1 for plain decoding, more when
 * drafted tokens are scored at once).  ctx_len[r] counts every cached token,
 * the last n_q among them: query i of request r sees the tokens
 * t < ctx_len[r] - (n_q - 1 - i), and
 *     o = sum_t softmax_t(scale * q . K_t) V_t,  lse = log sum_t exp(scale * q . K_t),
 * zeros and -inf for a query that sees no token.  fp16 outputs beyond +-65504
 * are +-65504.  Nothing behind the last token a query sees enters its result,
 * whatever it holds.
 * q:           [B][n_q][Hq][d] of type `dtype`; bf16 elements beyond +-2^112
 *              may overflow to NaN.
 * pool:        the cache; block_table: [B][max_blocks] int32 entries in
 *              [0, num_blocks); ctx_len: [B] int32 in [0, max_blocks * 16].
 * out:         [B][n_q][Hq][d] of type `dtype`; may be q.
 * lse:         [B][n_q][Hq] fp32 or NULL.
 * workspace:   >= clo_kv4_paged_workspace_size(...) bytes, 16-byte aligned.
 * err_flag, opts: as for clo_paged_decode_attn; opts->num_ctas > 0 also picks
 *              the kernel that shares all tokens out evenly, where for short
 *              contexts a cluster for each request and KV head is the default;
 *              the events bracket whichever runs (a bad block zeroes the
 *              queries of that request and KV head, a bad length those of the
 *              request; a record that does not arrive within about 2 s, which
 *              says that the GPU is in trouble, sets CLO_FLAG_TIMEOUT and
 *              zeroes what needed it).
 * Sums are in fp32.  The weights are rounded to fp16 once, times V's scale; the
 * largest lie between 2^6 and 2^15 there, and what is 2^-31 of them counts as 0.
 * The same call on the same kind of GPU gives the same bits each time.  The order
 * of the sums, and with it the last bits, depends on every request's length, on
 * max_blocks, num_ctas and the number of SMs.
 * More than 32 query rows a KV head take several calls: the queries 0 .. i of
 * each request with ctx_len less n_q - 1 - i (0 if that is negative), then the
 * rest with ctx_len.
 * Requires d == 128, block_size == 16, (Hq / Hkv) * n_q <= 32, B <= 4096,
 * B * Hkv * max_blocks < 2^31, opts->num_ctas <= 4095.
 */
typedef struct clo_kv4_attn_args {
    const void* q;
    const uint8_t* pool;
    const int32_t* block_table;
    const int32_t* ctx_len;
    void* out;
    float* lse;
    void* workspace;
    size_t ws_bytes;
    int32_t* err_flag;
    const clo_attn_opts* opts;
    clo_dtype dtype;
    float scale;
    int B;
    int n_q;
    int Hq;
    int Hkv;
    int d;
    int num_blocks;
    int block_size;
    int max_blocks;
    int group;
} clo_kv4_attn_args;

clo_status clo_kv4_paged_decode_attn(const clo_kv4_attn_args* args, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CLO_KV4_H_ */
