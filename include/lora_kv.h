/*
 * lora_kv.h -- the attention of a mixed multi-LoRA batch, between the q/k/v
 * projections and the o projection: the step's block tables and slot maps,
 * rotary positions, a paged cache of K and V in 4 bits, attention over that
 * cache, and attention over whole prompts.
 *
 * The cache lives in fixed-size blocks addressed through tables of block ids,
 * as adapters live in pages ([MLSP] "Unified Paging Architecture" and [MLSA]
 * "S-LoRA unified paging": adapters and KV cache share one pool of pages; the
 * source titles are those of lora.h).  A block may be a page of a lora_pool_t:
 * base = the pool's base, block_stride = the page's bytes, num_blocks = the
 * pool's pages, and the page ids that lora_cache_admit hands out are the
 * block ids.
 *
 * The general rules of lora.h hold: device pointers unless a comment says
 * host, caller-owned buffers, asynchronous enqueue on `stream` (whose device
 * must be the current one and the one the buffers are on), host checks before
 * anything is enqueued, no allocation, no exception.  Data-dependent
 * conditions never abort: they set flags (LORA_KV_FLAG_*).
 *
 * Element types: LORA_DTYPE_BF16 (q, k, v and outputs bf16) or
 * LORA_DTYPE_F32.  Scores, softmax statistics and every accumulation are
 * fp32.  With bf16 each softmax weight is rounded to bf16 (by at most 2^-8 of
 * it) for its product with V, as the bf16 matrix instructions take it; the sum
 * that divides the result is of the rounded weights, so that the weights sum
 * to one (rows that see one and the same V return it).  With fp32 weights
 * keep 24 bits.  Scores may be of any size, as long as scale * log2(e) * q.K
 * stays within fp32's range.
 */
#ifndef LORA_KV_H
#define LORA_KV_H

#include <stddef.h>
#include <stdint.h>

#include "lora.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_KV_UNIT 16          /* tokens per record of the cache */
#define LORA_KV_GROUP 32         /* values that share one scale */
#define LORA_KV_MAX_HEAD_DIM 256 /* head_dim: a multiple of 32 up to this */
#define LORA_KV_MAX_HEADS 1024   /* query heads */
#define LORA_KV_MAX_SEQS (1 << 16)

/* Heads of a batch of token rows: element (token t, head h, dim d) at
 * data[t*token_stride + h*head_stride + d].  Strides in elements, multiples
 * of 16 bytes, data 16-byte aligned; views into a fused projection's rows
 * (token_stride larger than heads*head_dim) are fine. */
typedef struct {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
  int32_t heads;
} lora_heads_t;

/* Paged 4-bit cache of one layer.  Block b is at base + b*block_stride bytes
 * (block_stride >= lora_kv_block_bytes, multiple of 16) and holds
 * block_tokens tokens (16, 32, 64, 128 or 256) of every kv head, as records
 * [kv head][unit of 16 tokens].  A record, with nc = head_dim/32:
 *   K codes  256*nc bytes  [16 t][4 g][nc c][4 b]  low nibble dim 32c+8g+2b,
 *                          high nibble that dim + 1, of the unit's token t
 *   V codes  256*nc bytes  [4 g][16 d][nc c][4 j]  low nibble dim 32c+d, high
 *                          nibble dim 32c+16+d, of the unit's token 4g+j
 *   K scales  16*nc bytes  [16 t][nc c]
 *   V scales  16*nc bytes  [16 t][nc c]
 * A value is code * 2^(scale byte - 127); codes are 1 sign, 2 exponent and 1
 * fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6.  Each token's 32 consecutive dims
 * share a scale: the smallest power of two 2^e, -95 <= e <= 124, with
 * max|x| <= 7 * 2^e (so that saturating at 6 costs no more than the rounding
 * between 4 and 6 does); codes are x / 2^e rounded to nearest, ties to the
 * even code. */
typedef struct {
  void* base;
  int64_t block_stride;
  int32_t num_blocks;
  int32_t block_tokens;
  int32_t num_kv_heads;
  int32_t head_dim;
} lora_kv_cache_t;

/* Bytes of one block (0 for an unsupported geometry). */
size_t lora_kv_block_bytes(int32_t block_tokens, int32_t num_kv_heads, int32_t head_dim);

/* One step's batch: which rows of q/k/v belong to which request, where their
 * K and V go, and the work plan of lora_kv_attend.  Device arrays carved from
 * one caller buffer by lora_kv_batch_init; built by lora_kv_build once per
 * step and read by every layer's calls.  T tokens and B requests of the
 * step may be anything up to max_tokens and max_seqs.
 *   q_indptr[B+1]  token rows of request i: q_indptr[i] .. q_indptr[i+1]-1
 *   kv_len[B]      cached tokens of request i after the step
 *   token_seq[T]   the row's request, -1 for rows behind the last request's
 *   positions[T]   the row's position in its request, -1 likewise
 *   slots[T]       block id * block_tokens + offset in the block, or -1
 *   counts[16]     see LORA_KV_COUNT_* */
typedef struct {
  int32_t max_tokens;
  int32_t max_seqs;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t* q_indptr;
  int32_t* kv_len;
  int32_t* token_seq;
  int32_t* positions;
  int32_t* slots;
  int32_t* counts;
  int32_t* plan;
} lora_kv_batch_t;

#define LORA_KV_COUNT_TOKENS 0     /* rows that belong to a request */
#define LORA_KV_COUNT_NEW_BLOCKS 1 /* blocks asked of the free list */
#define LORA_KV_COUNT_ITEMS 2      /* work items of 16 rows (per kv head) */
#define LORA_KV_COUNT_PARTS 3      /* partial results (16 rows of one chunk each) */
#define LORA_KV_COUNT_CHUNK 4      /* cached tokens per work item */
#define LORA_KV_COUNT_MID 5        /* work items of 32 rows (per kv head) */
#define LORA_KV_COUNT_WIDE 6       /* work items of 128 rows (per kv head) */
#define LORA_KV_COUNT_FLAGS 8
#define LORA_KV_FLAG_LENGTH 1     /* a negative length, or one past the table's row (cut) */
#define LORA_KV_FLAG_TOKENS 2     /* more new tokens than the call's T (the rest has no rows) */
#define LORA_KV_FLAG_FREE_LIST 4  /* the free list ran out (slots of the rest are -1) */
#define LORA_KV_FLAG_BLOCK_RANGE 8 /* a block id outside the cache (slot -1; not attended) */
#define LORA_KV_FLAG_NONFINITE 16 /* lora_kv_append saw an infinity or NaN in K or V */
#define LORA_KV_FLAG_BATCH 32     /* the batch, or its shared plan, was not built for this call */
#define LORA_KV_FLAG_GROUPS 64    /* lora_kv_share: a group outside the requests, or a negative length (not shared) */

/* Bytes of the buffer (0 outside the limits: max_tokens in [0,
 * LORA_MAX_TOKENS], max_seqs in [1, LORA_KV_MAX_SEQS], num_q_heads a multiple
 * of num_kv_heads up to LORA_KV_MAX_HEADS, head_dim as in the cache, and
 * max_tokens * num_q_heads / 16 + max_seqs * num_kv_heads + 8192 < 2^21 work
 * items). */
size_t lora_kv_batch_size(int32_t max_tokens, int32_t max_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                          int32_t head_dim);
/* Carve the buffer (device, 16-byte aligned).  Enqueues nothing.  Errors:
 * INVALID_ARG, UNSUPPORTED, ALIGNMENT, WORKSPACE. */
lora_status_t lora_kv_batch_init(void* buf, size_t bytes, int32_t max_tokens, int32_t max_seqs, int32_t num_q_heads,
                                 int32_t num_kv_heads, int32_t head_dim, lora_kv_batch_t* out);

/* Build the batch from request lengths: request i has ctx_len[i] cached
 * tokens and brings new_len[i] more (0 is allowed).  Its rows follow request
 * i-1's; row j of it has position ctx_len[i] + j and lies in block
 * position / block_tokens of its table row.  Blocks that the new tokens need
 * and the cached ones do not fill are taken from free_blocks (num_free ids)
 * in the order of requests, then of positions, and written into block_table
 * [B][table_stride], of which table_width entries are used; entries of
 * cached blocks are read and kept, all others left as they are.  The call
 * changes no other input, so the same call gives the same batch again; the
 * caller moves on by adding new_len to ctx_len and by dropping the first
 * counts[LORA_KV_COUNT_NEW_BLOCKS] ids of the free list.
 * T: rows of the step's tensors.  Rows behind the last request's (T larger
 * than the sum of new_len: a padded batch) get -1 everywhere and no call
 * touches them.
 * free_blocks may be NULL when num_free is 0.  No input may reach into the
 * batch's own buffer (the next step's ctx_len is a copy of kv_len, not kv_len).
 * Errors: INVALID_ARG, WORKSPACE (B or T past the capacity), UNSUPPORTED
 * (block_tokens; num_blocks*block_tokens past 2^31; table_width*block_tokens
 * past 2^30), HIP. */
lora_status_t lora_kv_build(const int32_t* ctx_len, const int32_t* new_len, int32_t B, int32_t T,
                            int32_t* block_table, int64_t table_stride, int32_t table_width,
                            const int32_t* free_blocks, int32_t num_free, int32_t num_blocks, int32_t block_tokens,
                            const lora_kv_batch_t* batch, void* stream);

/* Rotary positions.  Pair i of a head's first rot_dim dims is (i, i +
 * rot_dim/2) in the half layout and (2i, 2i+1) in the interleaved one; at
 * position p it becomes
 *   (x c - y s, y c + x s),  c = scale cos(p f_i),  s = scale sin(p f_i)
 * with f_i = inv_freq[i] (device, rot_dim/2 doubles, radians per position).
 * Dims from rot_dim on are passed through.  Angles are reduced in 64 bits,
 * whatever the position; K is rotated in 64 bits and rounded once, so that
 * the codes of lora_kv_append do not depend on how a product was summed; fp32
 * Q likewise, bf16 Q in fp32 before its one rounding. */
#define LORA_ROPE_HALF 0
#define LORA_ROPE_INTERLEAVED 1
typedef struct {
  const double* inv_freq;
  int32_t rot_dim; /* even, 2 .. head_dim */
  int32_t layout;
  double scale;
} lora_rope_t;

/* Host helper: the frequencies of a model, scaled for contexts longer than
 * the `original` positions it was trained on by `factor` >= 1, and the scale
 * of cos and sin.  With f_i = theta^(-2i/rot_dim):
 *   NONE    f_i
 *   LINEAR  f_i / factor                          (positions interpolated)
 *   NTK     f_i of theta * factor^(rot/(rot-2))   (base stretched)
 *   YARN    f_i keep_i + f_i/factor (1 - keep_i), keep_i falling from 1 to 0
 *           over the pairs i between those that turn `high` and `low` times
 *           over `original` positions; scale 0.1 ln(factor) + 1
 *   BANDS   f_i mix_i + f_i/factor (1 - mix_i), mix_i = (turns_i - low) /
 *           (high - low) cut to [0, 1], turns_i = original f_i / (2 pi)
 * low, high: 0 takes the defaults, 1 and 32 (YARN) or 1 and 4 (BANDS).
 * out: host, rot_dim/2 doubles; scale: host.  Errors: INVALID_ARG. */
#define LORA_ROPE_SCALING_NONE 0
#define LORA_ROPE_SCALING_LINEAR 1
#define LORA_ROPE_SCALING_NTK 2
#define LORA_ROPE_SCALING_YARN 3
#define LORA_ROPE_SCALING_BANDS 4
lora_status_t lora_rope_frequencies(int32_t rot_dim, double theta, int32_t scaling, double factor, double original,
                                    double low, double high, double* out, double* scale);

/* Rotate q and k (either may have heads = 0 with data NULL) into q_out and
 * k_out, which may be q and k themselves but not overlap them otherwise.
 * positions: device [T]; rows with a negative position are not written.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED, HIP. */
lora_status_t lora_rope(const lora_heads_t* q, const lora_heads_t* q_out, const lora_heads_t* k,
                        const lora_heads_t* k_out, const int32_t* positions, int32_t T, int32_t head_dim,
                        int32_t dtype, const lora_rope_t* rope, void* stream);

/* Rotate q into q_out and put the rotated k (as lora_rope would round it)
 * and v into the cache at `slots` in 4 bits, in one launch.  rope NULL: no
 * rotation (q and positions are not used and may be NULL).  q NULL or with 0
 * heads: only the cache is written.  Rows with a slot of -1, or outside the
 * cache, are not cached; rows with a negative position are left out wholly.
 * No two rows of a call may have the same slot.  A NaN is cached as 0 and an
 * infinity as its group's largest value of that sign, and either sets
 * LORA_KV_FLAG_NONFINITE in *flags (device, may be NULL).
 * Errors as lora_rope. */
lora_status_t lora_kv_append(const lora_heads_t* q, const lora_heads_t* q_out, const lora_heads_t* k,
                             const lora_heads_t* v, const int32_t* positions, const int32_t* slots, int32_t T,
                             int32_t dtype, const lora_rope_t* rope, const lora_kv_cache_t* cache, int32_t* flags,
                             void* stream);

/* The cached K and V at n slots as values, into k_out and v_out (exact in
 * bf16 and fp32).  Slots of -1 or outside the cache give zeros.  Errors as
 * lora_rope. */
lora_status_t lora_kv_gather(const lora_kv_cache_t* cache, const int32_t* slots, int32_t n, const lora_heads_t* k_out,
                             const lora_heads_t* v_out, int32_t dtype, void* stream);

/* Attention of the step's rows over the cache, after their own K and V were
 * appended: row t of request i at position p attends to the cached tokens
 * 0 .. min(p, kv_len[i]-1),
 *   o[t][h] = sum_j softmax_j(scale q[t][h] . K[j][h / G]) V[j][h / G]
 * with G = num_q_heads / num_kv_heads.  One new token per request is a
 * decode step; several are a prompt's chunk over its cached context.  A row
 * that sees no token gets zeros; rows that belong to no request are not
 * written.  Tokens in blocks outside the cache, or past the table's width, are
 * not attended (LORA_KV_FLAG_BLOCK_RANGE in the batch's flags).
 * A step with T <= B is planned as a decode step, in items of 16 rows, whatever
 * its requests bring; where several bring long chunks among idle ones, leave
 * the idle ones out or pad T past B.
 * B and T must be those of the batch's lora_kv_build, block_table as that call
 * left it, the cache of the same block_tokens.
 * ws: device, lora_kv_workspace_size(batch) bytes, 16-byte aligned.  The call
 * keeps partial results in ws and arrival counts in the batch's plan, so
 * calls that share either must not run at the same time (issue them on one
 * stream).
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED, WORKSPACE, HIP. */
size_t lora_kv_workspace_size(const lora_kv_batch_t* batch);
lora_status_t lora_kv_attend(const lora_heads_t* q, const lora_heads_t* o, int32_t T, int32_t B, int32_t dtype,
                             const lora_kv_batch_t* batch, const int32_t* block_table, int64_t table_stride,
                             int32_t table_width, const lora_kv_cache_t* cache, float scale, void* ws,
                             size_t ws_bytes, void* stream);

/* Requests that begin with the same cached tokens (a system prompt in front of
 * an adapter's requests, a prompt that a search's beams have in common) attend
 * to them together: what they share is read once for the rows of all of them,
 * in place of once per request.
 *
 * A shared plan is carved from one caller buffer for a batch's capacity and
 * for up to max_groups groups, built by lora_kv_share after each lora_kv_build
 * and read by every layer's lora_kv_attend_shared.
 * It pays where many rows share much: a decode step's attention of 256 requests
 * behind one prompt of 32768 tokens takes 155 us in place of 889, 96 behind 8
 * prompts of up to 4096 49 in place of 123, 64 behind 2000 22 in place of 30.  A few
 * beams over a prompt of 1000, or prompts' chunks of hundreds of rows each, take
 * as long either way or a little longer (11.6 us against 10.4, 246 against 245),
 * and the plan itself, once per step, takes 10 us: these are better left to
 * lora_kv_attend.  No call chooses by itself.
 * Sizes: 0 outside the limits (max_groups in [0, max_seqs]; 2 * max_tokens *
 * query heads per kv head + 2^18 < 2^31, and the work items of
 * lora_kv_batch_size with max_groups more).
 * Errors of init: INVALID_ARG, UNSUPPORTED, ALIGNMENT, WORKSPACE. */
typedef struct {
  int32_t max_groups;
  int32_t* counts; /* [16]: items of the prefixes and of the requests' three classes, rows of partial results, .. */
  int32_t* plan;
} lora_kv_share_t;
size_t lora_kv_share_size(const lora_kv_batch_t* batch, int32_t max_groups);
lora_status_t lora_kv_share_init(void* buf, size_t bytes, const lora_kv_batch_t* batch, int32_t max_groups,
                                 lora_kv_share_t* out);

/* Group g is the requests group_indptr[g] .. group_indptr[g+1]-1 (device,
 * num_groups+1 entries, ascending within 0 .. B; requests before the first and
 * behind the last group are in none), whose first shared_len[g] (device)
 * tokens have the same K and V.  They are read through the table row of the
 * group's first request that brings tokens; whether the other rows name the
 * same blocks or copies of them does not matter.  What is attended to
 * together is cut to a multiple of 16 tokens, and to what every row of the
 * group sees of its own request (ctx_len, the shortest one's); the rest is
 * attended to by each request.  A group that is empty, out of range or of
 * negative length is not shared (LORA_KV_FLAG_GROUPS in the batch's flags for
 * the last two).
 * T, B: those of the batch's lora_kv_build.  No input may reach into the
 * batch's or the plan's buffer.
 * Errors: INVALID_ARG, WORKSPACE (past the capacity), HIP. */
lora_status_t lora_kv_share(const int32_t* group_indptr, const int32_t* shared_len, int32_t num_groups, int32_t T,
                            int32_t B, const lora_kv_batch_t* batch, const lora_kv_share_t* share, void* stream);

/* lora_kv_attend with what groups share attended to together; the same result
 * but for the order of its sums.  num_groups: that of lora_kv_share.
 * ws: device, lora_kv_share_workspace_size(batch, share) bytes, 16-byte
 * aligned, for partial results: calls that share it must not run at the same
 * time.  A plan that was not built for this call's T, B and num_groups, or whose
 * batch was built again since, writes nothing (LORA_KV_FLAG_BATCH).
 * Errors: as lora_kv_attend. */
size_t lora_kv_share_workspace_size(const lora_kv_batch_t* batch, const lora_kv_share_t* share);
lora_status_t lora_kv_attend_shared(const lora_heads_t* q, const lora_heads_t* o, int32_t T, int32_t B,
                                    int32_t num_groups, int32_t dtype, const lora_kv_batch_t* batch,
                                    const lora_kv_share_t* share, const int32_t* block_table, int64_t table_stride,
                                    int32_t table_width, const lora_kv_cache_t* cache, float scale, void* ws,
                                    size_t ws_bytes, void* stream);

/* Causal attention of whole prompts over themselves: B prompts packed into T
 * token rows, prompt i in rows indptr[i] .. indptr[i+1]-1 (device, B+1
 * entries, ascending from 0 or later; entries are cut to [0, T]); row j of a
 * prompt attends to its rows 0..j.  Rows outside every prompt are not
 * written.  Nothing behind a row's own place, infinities and NaN included,
 * changes it.  o may not overlap q, k or v.  Token strides of k and v up to
 * 2^23 elements; (T/64 + B) * heads < 2^23.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED, HIP. */
lora_status_t lora_prompt_attend(const lora_heads_t* q, const lora_heads_t* k, const lora_heads_t* v,
                                 const lora_heads_t* o, const int32_t* indptr, int32_t B, int32_t T, int32_t head_dim,
                                 int32_t dtype, float scale, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_KV_H */
