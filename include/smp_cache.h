/*
 * smp_cache.h -- C ABI of libsmp, second part: the target model's side of a
 * speculative decoding step over a paged key/value cache held in 8 bits.
 *
 * One step of a batch: smp_block_plan gives every token of the step its place
 * in the cache, smp_qk_norm_rope prepares the step's queries and keys,
 * smp_cache_append writes keys and values, smp_cache_attention reads the
 * cache, and smp_spec_verify or smp_spec_verify_probs (smp.h) checks the
 * drafts; the accepted lengths are the next step's `lens`.
 *
 * The conventions are those of smp.h: calls are asynchronous on the caller's
 * stream, allocate nothing, may be captured in a CUDA graph, and report what
 * the host can see as a return code before anything is launched.  Problems
 * that only the device can see OR a flag into the optional device status
 * word, which the call clears first; what the affected request or token then
 * gets is said at each call.
 *
 * The cache.  `num_blocks` blocks of `block_size` tokens.  A block of one
 * head is contiguous: codes k[num_blocks, kv_heads, block_size, head_dim] and
 * v likewise, one byte per element, and one positive binary32 scale per block
 * and head, k_scale[num_blocks, kv_heads] and v_scale likewise; an element is
 * code * scale.  Token t of request b lies in block block_table[b, t /
 * block_size] at offset t % block_size; its slot is block * block_size +
 * offset.  Codes are SMP_CACHE_E4M3 (4 exponent bits, 3 mantissa bits, no
 * infinities, largest 448) or SMP_CACHE_I8 (-127 .. 127).
 */
#ifndef SMP_CACHE_H
#define SMP_CACHE_H

#include "smp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest head dimension of the cache and of smp_qk_norm_rope. */
#define SMP_MAX_HEAD_DIM 256

typedef enum smp_cache_type {
    SMP_CACHE_E4M3 = 0,
    SMP_CACHE_I8 = 1
} smp_cache_type;

/* Flags OR-ed into the device status word, beside those of smp.h. */
#define SMP_ROW_BAD_LENGTH 16    /* a length, count, position or slot out of range */
#define SMP_ROW_NO_CAPACITY 32   /* not enough free blocks, or more tokens than the step holds */
#define SMP_ROW_BAD_BLOCK 64     /* a block id outside [0, num_blocks) */

/*
 * A cache as the calls take it: device pointers and sizes, read on the host
 * during the call.
 *   k, v               device, [num_blocks, kv_heads, block_size, head_dim]
 *                      bytes, contiguous, 16-byte aligned.
 *   k_scale, v_scale   device, [num_blocks, kv_heads] float.
 *   block_size         a power of two, 16 .. 256.
 *   head_dim           a multiple of 16, 16 .. SMP_MAX_HEAD_DIM.
 *   type               smp_cache_type.
 */
typedef struct smp_cache {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int32_t num_blocks;
    int32_t kv_heads;
    int32_t block_size;
    int32_t head_dim;
    int32_t type;
} smp_cache;

/*
 * smp_block_plan -- where the tokens of one step go: blocks for the requests
 * that outgrow theirs, and for every token its request, position and slot.
 * Request b has lens[b] tokens in the cache and adds add[b]; it needs
 * ceil((lens + add) / block_size) blocks and holds held[b].  Missing blocks
 * are taken from the free list in request order: request b's i-th new block
 * is free_blocks[*free_head + (new blocks of requests before b) + i].
 *
 *   lens, add, held  device, [batch] int32.  A request is valid when lens, add
 *                  >= 0, ceil(lens / block_size) <= held <= table_stride and
 *                  the blocks it needs are <= table_stride.
 *   free_blocks    device, [free_count] int32 block ids; free_head: device, one
 *                  int32, the ids used so far (0 .. free_count).
 *   block_table    device, [batch, table_stride] int32, read at the blocks a
 *                  request holds and written at the new ones only.
 *   max_tokens     capacity of the per-token outputs (0: no tokens, tables
 *                  are not extended).
 *   out_lens, out_held  device, [batch] int32: lens + add and the blocks held
 *                  after the step; out_free_head: device, one int32.
 *   out_start      device, [batch + 1] int32: first token of each request.
 *   out_position, out_request  device, [max_tokens] int32, out_slot device,
 *                  [max_tokens] int64: for token t = out_start[b] + i the
 *                  position lens[b] + i, the request b and the slot; -1 past
 *                  the last token, so that a captured step of a fixed size
 *                  can run with fewer.
 *   batch 0 .. 2^24; num_blocks 1 ..; max_tokens and free_count 0 .. 2^31-2;
 *   outputs must not overlap inputs.
 * An invalid request adds nothing (SMP_ROW_BAD_LENGTH): its length and blocks
 * stay.  When tokens or free blocks run out, the first request that does not
 * fit and all later ones that add tokens add nothing (SMP_ROW_NO_CAPACITY).
 * A block id outside [0, num_blocks) gives its tokens the slot -1
 * (SMP_ROW_BAD_BLOCK).
 */
smp_status smp_block_plan(const int32_t* lens, const int32_t* add, const int32_t* held, int32_t batch,
                          const int32_t* free_blocks, int32_t free_count, const int32_t* free_head,
                          int32_t* block_table, int32_t table_stride, int32_t block_size, int32_t num_blocks,
                          int32_t max_tokens, int32_t* out_lens, int32_t* out_held, int32_t* out_free_head,
                          int32_t* out_start, int32_t* out_position, int32_t* out_request, int64_t* out_slot,
                          int32_t* status, void* stream);

/*
 * smp_qk_norm_rope -- the norm of every query and key head and the position
 * rotation, in one pass.  For a head x of head_dim elements at position t:
 *   y_i = x_i * w_i / sqrt(mean_j x_j^2 + eps)
 * and, for the first rotary_dim = 2r elements, pairs (a, b) become
 *   (a cos - b sin, b cos + a sin)
 * with cos = table[t, j], sin = table[t, r + j] and pair j = (y_j, y_{r+j}),
 * or (y_2j, y_2j+1) when `interleaved` is not 0.  Sums and products are in
 * binary32; results are rounded once to the elements' type.
 *
 *   q, k           device, [tokens, q_heads | k_heads, head_dim] elements of
 *                  `dtype`; heads contiguous, tokens q_stride / k_stride
 *                  elements apart.  k may be NULL with k_heads = 0.
 *   q_weight, k_weight  device, [head_dim] float, or NULL (all ones).
 *   table          device, [table_rows, rotary_dim] float: cosines, then sines.
 *   rotary_dim     even, 0 .. head_dim; 0: no rotation (table may be NULL).
 *   positions      device, [tokens] int32.  A negative position marks padding:
 *                  the token's outputs are not written.  A position >=
 *                  table_rows gives NaN outputs and SMP_ROW_BAD_LENGTH.
 *   out_q, out_k   device, like q and k with their own strides; may be q and k
 *                  themselves with the same strides (in place), and must not
 *                  overlap them otherwise.
 *   head_dim 1 .. SMP_MAX_HEAD_DIM; tokens * (q_heads + k_heads) 0 .. 2^31-1;
 *   strides at least heads * head_dim.
 */
smp_status smp_qk_norm_rope(const void* q, const void* k, int32_t tokens, int32_t q_heads, int32_t k_heads,
                            int32_t head_dim, int64_t q_stride, int64_t k_stride, smp_dtype dtype,
                            const float* q_weight, const float* k_weight, float eps, const float* table,
                            int32_t table_rows, int32_t rotary_dim, int32_t interleaved, const int32_t* positions,
                            void* out_q, void* out_k, int64_t out_q_stride, int64_t out_k_stride, int32_t* status,
                            void* stream);

/*
 * smp_cache_append -- keys and values of the step's tokens into the cache.
 * Consecutive tokens whose slots follow one another inside one block form a
 * run.  For a run and a head, with amax the largest finite |x| of the run's
 * tokens and top the type's largest code (448 or 127):
 *   s = 2^e, the smallest power of two >= 2^-100 with amax <= top * s; if the
 *   run starts at an offset > 0, s = max(s, the block's scale), and when that
 *   is more than the block's scale the codes before the run are encoded again
 *   as round(code * old scale / s).
 *   code = round(x / s), to the nearest code, ties to even.
 * With power-of-two scales the division is exact, and encoding e4m3 codes
 * again only rounds those that become subnormal.
 *
 *   k, v         device, [tokens, kv_heads, head_dim] elements of `dtype`, heads
 *                contiguous, tokens k_stride / v_stride elements apart.
 *   slots        device, [tokens] int64.  A negative slot is padding: the token
 *                is skipped.  A slot >= num_blocks * block_size is skipped with
 *                SMP_ROW_BAD_LENGTH.  The tokens of one block must form one run
 *                (as smp_block_plan orders them): two runs of one call in the
 *                same block race on its scale, and the block's contents are
 *                then undefined.
 * Infinities become the largest code of their sign; NaN becomes e4m3's NaN
 * code, or the i8 code 0; either sets SMP_ROW_NONFINITE.
 */
smp_status smp_cache_append(const smp_cache* cache, const void* k, const void* v, int32_t tokens, int64_t k_stride,
                            int64_t v_stride, smp_dtype dtype, const int64_t* slots, int32_t* status, void* stream);

/*
 * smp_cache_attention_workspace_bytes -- device workspace that
 * smp_cache_attention needs on the current device for these sizes (0 if they
 * are invalid).  At most 64 MiB on a GPU of 160 SMs.
 */
size_t smp_cache_attention_workspace_bytes(int32_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                           int32_t batch);

/*
 * smp_cache_attention -- causal attention of the step's queries over the cache.
 * Request b has lens[b] tokens in the cache (the step's own included) and the
 * queries of tokens start[b] .. start[b + 1] - 1, its last ones: query i of n
 * is at position p = lens[b] - n + i and sees the keys j <= p, and only those
 * j > p - window when window > 0.  For query head h, with key head g = h /
 * (q_heads / kv_heads):
 *   out = sum_j softmax_j(scale * q . k_j) v_j
 * over the visible keys; a query that sees none gets zeros (lse -inf).
 * Scores, sums and the weighted values are held in binary32; a key, a query
 * and a weight enter their products with at least bf16's precision (binary32
 * queries: 22 bits), weights far below a row's largest (p_j times the value
 * scale) with an error of at most 2^-33 of it.  That holds for value scales of
 * 2^-92 to 2^92; for those down to 2^-100, the least that smp_cache_append
 * writes, the error is at most 2^-25.  Cache positions that a query does not
 * see do not influence its result, whatever bytes they hold, and neither do
 * the scales of blocks of which it sees nothing.
 *
 *   q            device, [tokens, q_heads, head_dim] of `dtype`, heads
 *                contiguous, tokens q_stride elements apart.
 *   start        device, [batch + 1] int32, non-decreasing, start[batch] <=
 *                tokens; output rows of tokens at or past start[batch] are not
 *                written.  lens: device, [batch] int32.
 *   block_table  device, [batch, table_stride] int32.
 *   out          device, like q, tokens out_stride elements apart; must not
 *                overlap q.  out_lse: device, [tokens, q_heads] float, the
 *                natural logarithm of the sum of exp(scale * q . k_j), or NULL.
 *   q_heads a multiple of kv_heads; batch 0 .. 2^20; window >= 0; scale finite.
 *   workspace    device, of smp_cache_attention_workspace_bytes(...) bytes,
 *                16-byte aligned; scratch, no initial contents needed; calls
 *                that overlap on the GPU must not share it.
 * A start out of order or out of range makes its request's queries none, and a
 * length below 0 or above table_stride * block_size is cut to that range
 * (SMP_ROW_BAD_LENGTH); keys of a block id outside [0, num_blocks) are not
 * visible (SMP_ROW_BAD_BLOCK).  Ids of blocks that the window of every query
 * has left are not looked at: their pages may have been given back.
 */
smp_status smp_cache_attention(const smp_cache* cache, const void* q, int32_t tokens, int32_t q_heads,
                               int64_t q_stride, smp_dtype dtype, const int32_t* start, const int32_t* lens,
                               int32_t batch, const int32_t* block_table, int32_t table_stride, float scale,
                               int32_t window, void* out, int64_t out_stride, float* out_lse, int32_t* status,
                               void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SMP_CACHE_H */
