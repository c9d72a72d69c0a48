/*
 * clo_paged.h -- C ABI of libclo's paged KV cache held in 16 bits: what writes
 * it, what a prompt computes on it and what a long decode step reads of it.
 *
 * clo_paged_decode_attn (clo.h) attends one fp16 query a request to such a
 * cache.  Around it, a serving step needs
 *   - the new tokens' queries and keys turned by their positions, and K and V
 *     written to the slots that clo_paged_plan gave (clo_paged_rope_append);
 *   - the attention of each request's new tokens, one or thousands, over its
 *     cached tokens, themselves among them (clo_paged_chunk_attn);
 *   - for long contexts, a selection of blocks by a score that reads a
 *     fifteenth of the keys' bytes (clo_paged_block_bounds,
 *     clo_paged_block_select) and the decode attention over the selected
 *     blocks alone (clo_paged_sparse_decode_attn).  It is to a paged cache what
 *     clo_topk_retrieve and the Cache Buffer are to an offloaded one.
 *
 * Conventions: those of clo.h (device pointers owned by the caller,
 * asynchronous on `stream`, host validation before any launch, data-dependent
 * errors ORed into *err_flag, no allocation, no exception across the
 * interface) and clo_kv4.h (argument structs, which a call only reads before it
 * returns; the type of 16-bit tensors is an argument).  d (head dimension) must
 * be 128 and block_size 16 in this build, Hq / Hkv at most 8.
 *
 * The cache is kc and vc, [num_blocks][Hkv][16][128]; token t of request r is row
 * t % 16 of block block_table[r][t / 16], and its slot is block * 16 + t % 16.
 */
#ifndef CLO_PAGED_H_
#define CLO_PAGED_H_

#include "clo.h"
#include "clo_kv4.h" /* clo_dtype */

#ifdef __cplusplus
extern "C" {
#endif

/* How a pair of channels turns with the position: by turns * 2^-64 of a full
 * turn for each step of position axis `axis`. */
typedef struct clo_rope_pair {
    uint64_t turns;
    int32_t axis;
    int32_t reserved; /* 0 */
} clo_rope_pair;

/*
 * clo_rope_pairs -- the table for clo_paged_rope_append, made on the host once
 * for a model: pairs[i].turns = inv_freq[i] / (2 pi) * 2^64, rounded to the
 * nearest whole number, modulo 2^64.  pos * turns modulo 2^64 is then the exact
 * fraction of a turn, so far positions lose nothing: after 2^20 steps the angle
 * is off by 2e-13, where 32-bit angles are off by up to 0.06.
 * inv_freq: [n] host fp64, finite and below 2^20 in size (radians a position;
 *           theta^(-2i/rot), scaled as the model scales them).
 * axis:     [n] host int32 in [0, 4), or NULL for axis 0 throughout.
 * pairs:    [n] host output, to be copied to the device by the caller.
 */
clo_status clo_rope_pairs(const double* inv_freq, const int32_t* axis, int n, clo_rope_pair* pairs);

/*
 * clo_paged_rope_append -- rotary positions for N new tokens and their K and V
 * into the cache.  With a token's positions pos[axis] and t_i = 2 pi * (turns_i *
 * pos[axis_i] / 2^64), every head's pair i of a query or key (a_i, b_i) becomes
 *     (a_i cos t_i - b_i sin t_i, a_i sin t_i + b_i cos t_i),
 * in fp32, rounded once.  Pair i is channels (i, i + rot / 2), or with
 * `interleaved` (2i, 2i + 1); channels from rot on are left as they are.
 * The queries go to q_out, K and V to row slot % 16 of block slot / 16.
 * q, q_out: [N][Hq][d] (both NULL: keys and values alone); k, v: [N][Hkv][d], of
 *           type `dtype`; rows of consecutive tokens are *_stride elements apart
 *           (a multiple of 8, at least a row), so they may be parts of a fused
 *           projection's output.  q_out may be q (with its stride); it may not
 *           overlap the inputs otherwise.
 * pos:      [axes][N] int32, any value: 1 axis for text, 3 for time, height and
 *           width.
 * pairs:    [rot / 2] (device), 16-byte aligned; an axis outside [0, axes) counts
 *           as 0 and sets CLO_FLAG_BAD_INDEX.  May be NULL when rot == 0.
 * slot_map: [N] int32, distinct slots; -1 skips K and V of the token (its query
 *           is turned all the same).  Any other slot outside [0, num_blocks * 16)
 *           does too and sets CLO_FLAG_BAD_INDEX.
 * kc, vc:   the cache.
 * Requires 16-byte aligned tensors, rot a multiple of 16 in [0, 128], 1 <= axes <=
 * 4, N * (Hq + 2 Hkv) < 2^31 - 2^20.  Hq need not be a multiple of Hkv.
 */
typedef struct clo_paged_rope_append_args {
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    long long q_stride;
    long long k_stride;
    long long v_stride;
    long long q_out_stride;
    const int32_t* pos;
    const clo_rope_pair* pairs;
    const int32_t* slot_map;
    void* kc;
    void* vc;
    int32_t* err_flag;
    clo_dtype dtype;
    int N;
    int axes;
    int rot;
    int interleaved;
    int Hq;
    int Hkv;
    int d;
    int num_blocks;
    int block_size;
} clo_paged_rope_append_args;

clo_status clo_paged_rope_append(const clo_paged_rope_append_args* args, cudaStream_t stream);

/* Workspace bytes clo_paged_chunk_attn needs when run with num_ctas CTAs (0 =
 * the default, one a multiprocessor); 0 for invalid sizes.  It needs no
 * initialisation and may be reused by later calls on the same stream. */
size_t clo_paged_chunk_workspace_size(int Hq, int Hkv, int d, int num_ctas);

/*
 * clo_paged_chunk_attn -- attention of the last n_r tokens of each request over
 * its cached tokens, themselves among them: n_r = offsets[r + 1] - offsets[r],
 * rows offsets[r] .. offsets[r + 1] - 1 of q.  ctx_len[r] counts every cached
 * token, the n_r new ones included: row offsets[r] + i sees the tokens
 * t < ctx_len[r] - (n_r - 1 - i), and
 *     o = sum_t softmax_t(scale * q . K_t) V_t,  lse = log sum_t exp(scale * q . K_t),
 * zeros and -inf for a row that sees no token.  Any mixture of prompts, chunks
 * of prompts and decoding requests is one call.  Nothing behind the last token a
 * row sees enters its result, whatever it holds; fp16 outputs beyond +-65504 are
 * +-65504.  bf16 values may be as large as the type holds.  Rows whose first sums are not
 * finite, by a value that they do not see or by values from 2^90 on, are made anew token by
 * token: right, but slow.
 * q:           [N][Hq][d] of type `dtype`, rows q_stride elements apart (a
 *              multiple of 8, at least Hq * d).
 * kc, vc:      [num_blocks][Hkv][16][d] of type `dtype` with the strides
 *              kv_block, kv_head, kv_token (elements, multiples of 8, the same
 *              for both; 0 for all three: contiguous).  Rows of clo_kv4_gather
 *              [16 * num_blocks][Hkv][d] are such a cache, with strides
 *              16 * Hkv * d, d, Hkv * d.
 * block_table: [B][max_blocks] int32 entries in [0, num_blocks).
 * ctx_len:     [B] int32 in [0, max_blocks * 16].
 * offsets:     [B + 1] int32, not descending, in [0, N], as clo_paged_plan writes
 *              them.  Rows of no request are left as they were.
 * out:         [N][Hq][d] of type `dtype`, contiguous, apart from q.
 *              lse: [N][Hq] fp32 or NULL.
 * workspace:   >= clo_paged_chunk_workspace_size(...) bytes, 16-byte aligned.
 * err_flag:    a length out of range or offsets that descend or leave [0, N] set
 *              CLO_FLAG_BAD_CTX: a bad length zeroes the request's rows, and
 *              requests with bad offsets are passed over, all requests if the
 *              others' rows come to more than 2 N.  A bad block sets
 *              CLO_FLAG_BAD_INDEX and zeroes the rows (of that KV head) that see it,
 *              and it may zero other rows of the request and KV head.  A copy or a
 *              product that does not end within about 2 s, which says that the GPU
 *              is in trouble, sets CLO_FLAG_TIMEOUT; the outputs are then undefined.
 * opts:        optional: num_ctas, at most 4095; the events bracket the main kernel.
 * One fp16 token a request over a contiguous cache is also what clo_paged_decode_attn
 * computes.  With 4 query heads a KV head or more this call is the faster one (1.05 to 2.8
 * times) up to B * Hkv of 2000, but for a few thousand cached tokens in all, and for contexts
 * of several thousand tokens; with 1, or from there on where contexts are below 1000 tokens,
 * that one is (up to 2.2 times).  With 2 or 3 they are about equal.
 * Scores and sums are in fp32; the weights are rounded to `dtype` for the product
 * with V (which may take a result off by half a step of `dtype` of the values' size,
 * beside its own rounding), in fp16 after a factor that keeps what is 2^-31 of the
 * largest; in tiles of rows (a request's new tokens in groups of floor(128 Hkv / Hq))
 * whose last one sees at most 128 tokens, to twice the bits.  The same call on the same
 * kind of GPU gives the same bits each time.
 * Requires d == 128, block_size == 16, Hq / Hkv <= 8, B <= 4096, N * Hq < 2^29,
 * max_blocks <= 2^20, num_blocks <= 2^26, scale > 0, strides of at most 2^38 (kv_token
 * 2^34) and a cache that spans less than 2^31 times the greatest common divisor of
 * kv_block and kv_head.
 */
typedef struct clo_paged_chunk_attn_args {
    const void* q;
    const void* kc;
    const void* vc;
    long long q_stride;
    long long kv_block;
    long long kv_head;
    long long kv_token;
    const int32_t* block_table;
    const int32_t* ctx_len;
    const int32_t* offsets;
    void* out;
    float* lse;
    void* workspace;
    size_t ws_bytes;
    int32_t* err_flag;
    const clo_attn_opts* opts;
    clo_dtype dtype;
    float scale;
    int B;
    int N;
    int Hq;
    int Hkv;
    int d;
    int num_blocks;
    int block_size;
    int max_blocks;
} clo_paged_chunk_attn_args;

clo_status clo_paged_chunk_attn(const clo_paged_chunk_attn_args* args, cudaStream_t stream);

/* Bytes of one record of block bounds: [num_blocks][Hkv][272] bytes for a cache.
 * Bytes 8w .. 8w + 3 hold the codes of the largest keys of channels 4w .. 4w + 3,
 * bytes 8w + 4 .. 8w + 7 those of the smallest, as signed bytes; bytes 256..259
 * their fp32 scale; 260..271 zeros. */
size_t clo_paged_bounds_bytes(int block_size, int d);

/*
 * clo_paged_block_bounds -- the range of the keys, channel by channel, of the
 * blocks that a step's new tokens went to, from K as it lies in the cache (after
 * clo_paged_rope_append with the same slot_map).  With M the largest magnitude
 * among the block's keys (up to and with its last new token) and
 *     scale = M / 127 (fp32),
 *     code of a channel's largest  = its quotient by scale (fp32), rounded up,
 *     code of a channel's smallest = its quotient by scale (fp32), rounded down,
 * both limited to +-127.  A block with a NaN or an infinity gets codes of 0 and
 * the scale +inf: it is selected before those with a score.
 * kc:       [num_blocks][Hkv][16][d] of type `dtype`, contiguous.
 * slot_map: [N] int32.  A request's new tokens follow one another, as
 *           clo_paged_plan writes them: the last entry of a run of consecutive
 *           slots within one block names the block and the last of its tokens (a
 *           block's new tokens make one run; where two name a block its record is
 *           undefined).  Negative slots are skipped, any other outside [0, num_blocks * 16) too
 *           (and CLO_FLAG_BAD_INDEX).
 * bounds:   [num_blocks][Hkv][272] uint8, 16-byte aligned; records of other blocks
 *           are left as they are.
 */
typedef struct clo_paged_block_bounds_args {
    const void* kc;
    const int32_t* slot_map;
    uint8_t* bounds;
    int32_t* err_flag;
    clo_dtype dtype;
    int N;
    int Hkv;
    int d;
    int num_blocks;
    int block_size;
} clo_paged_block_bounds_args;

clo_status clo_paged_block_bounds(const clo_paged_block_bounds_args* args, cudaStream_t stream);

/* Workspace bytes of clo_paged_block_select (the scores); 0 for invalid sizes. */
size_t clo_paged_select_workspace_size(int B, int Hkv, int max_blocks);

/*
 * clo_paged_block_select -- the blocks that a decode step attends to, for each
 * request and KV head.  With s = the sum of the group's queries (fp32, added in
 * the order of the heads), M its largest magnitude and code_c = s_c / (M / 127)
 * (fp32, rounded to the nearest, ties to even, limited to +-127; 0 where M is 0
 * or anything in s is not finite), block b has the score
 *     scale_b * sum_c max(code_c * largest_c, code_c * smallest_c),
 * the whole numbers exact and the product in fp32.  In exact numbers this is an
 * upper bound of the summed score s . K_t that clo_topk_retrieve ranks tokens by.
 * The first n_first blocks of a request and the last n_last, the one being
 * filled among them, are always selected.  Of the others those without a finite
 * scale or entry come next (see bounds and block_table), with those whose score is
 * beyond fp32, then those with the highest scores, equal ones going to the lower
 * block, until there are n_sel.  A request with no more than n_sel blocks has them
 * all.
 * q:           [B][Hq][d] of type `dtype`, contiguous.
 * bounds:      as clo_paged_block_bounds writes them.
 * block_table, ctx_len: as for clo_paged_decode_attn.  A block out of range sets
 *              CLO_FLAG_BAD_INDEX and counts as one without a finite scale (what
 *              attends to it reports it); a bad length sets CLO_FLAG_BAD_CTX and
 *              selects nothing.  A copy that does not end within about 2 s sets
 *              CLO_FLAG_TIMEOUT; sel is then undefined.
 * sel:         [B][Hkv][n_sel] int32 output: columns of block_table, ascending,
 *              then -1.
 * workspace:   >= clo_paged_select_workspace_size(B, Hkv, max_blocks) bytes, 16-byte
 *              aligned.
 * Requires n_first, n_last >= 0, 1 <= n_sel, n_first + n_last <= n_sel <= 2^20,
 * B <= 4096, B * Hkv <= 65535, B * Hkv * max_blocks < 2^31, max_blocks <= 2^20.
 */
typedef struct clo_paged_block_select_args {
    const void* q;
    const uint8_t* bounds;
    const int32_t* block_table;
    const int32_t* ctx_len;
    int32_t* sel;
    void* workspace;
    size_t ws_bytes;
    int32_t* err_flag;
    clo_dtype dtype;
    int B;
    int Hq;
    int Hkv;
    int d;
    int num_blocks;
    int block_size;
    int max_blocks;
    int n_sel;
    int n_first;
    int n_last;
} clo_paged_block_select_args;

clo_status clo_paged_block_select(const clo_paged_block_select_args* args, cudaStream_t stream);

/*
 * clo_paged_sparse_decode_attn -- clo_paged_decode_attn over some blocks of each
 * request and KV head: the first min(n_sel, ceil(ctx_len[r] / 16)) entries of
 * sel[r][g], columns of block_table in any order (a column that is named twice
 * counts twice, an entry of -1 is skipped).  Of a column the tokens below
 * ctx_len[r] are attended to; other entries outside [0, ceil(ctx_len[r] / 16))
 * and bad blocks set CLO_FLAG_BAD_INDEX and zero the outputs of that request and KV
 * head, as do bad lengths (CLO_FLAG_BAD_CTX) those of the request.  With every
 * column in sel the result is that of the dense attention.
 * q, out:    [B][Hq][d] of type `dtype`, contiguous, apart from one another.
 *            lse: [B][Hq] fp32 or NULL.
 * workspace: >= clo_paged_chunk_workspace_size(Hq, Hkv, d, num_ctas) bytes,
 *            16-byte aligned.
 * Sums are in fp32; the weights are rounded to `dtype` for the product with V.  Large bf16
 * values: as for clo_paged_chunk_attn.
 * Requires d == 128, block_size == 16, Hq / Hkv <= 8, B <= 4096, B * Hq < 2^29,
 * num_blocks <= 2^26, max_blocks <= 2^20, B * Hkv * n_sel < 2^31, scale > 0.
 */
typedef struct clo_paged_sparse_attn_args {
    const void* q;
    const void* kc;
    const void* vc;
    const int32_t* block_table;
    const int32_t* ctx_len;
    const int32_t* sel;
    void* out;
    float* lse;
    void* workspace;
    size_t ws_bytes;
    int32_t* err_flag;
    const clo_attn_opts* opts;
    clo_dtype dtype;
    float scale;
    int B;
    int Hq;
    int Hkv;
    int d;
    int num_blocks;
    int block_size;
    int max_blocks;
    int n_sel;
} clo_paged_sparse_attn_args;

clo_status clo_paged_sparse_decode_attn(const clo_paged_sparse_attn_args* args, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CLO_PAGED_H_ */
