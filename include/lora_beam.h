/*
 * lora_beam.h -- beam search over the paged 4-bit cache of lora_kv.h: the
 * selection of a step's beams from its logits, the exchange of their block
 * tables, and the copies of blocks that two beams would write to.
 *
 * A step has num_requests requests of `beams` beams each; beam w of request b
 * is row b*beams + w of every array, and of the decode batch (one request of
 * lora_kv_build per beam).  A search's step:
 *   logits -> lora_beam_select -> lora_beam_reorder -> lora_beam_copy
 *   -> lora_kv_build, then per layer lora_kv_append and lora_kv_attend.
 * The beams of a request share its prompt, so lora_kv_attend_shared gives the
 * same; it is faster where beams and prompts are many and long, and slower for a
 * few beams over a thousand tokens (lora_kv.h has the figures).
 *
 * lora_beam_reorder takes its blocks from the front of the free list, and so
 * does lora_kv_build: between the two the list's owner drops its first
 * counts[LORA_BEAM_COUNT_COPIES] ids and may append the
 * counts[LORA_BEAM_COUNT_FREED] of moves->freed.  With the same list for both two
 * rows would write to one block, which no flag shows.  The counts are on the
 * device, so reading them waits for the reorder.
 *
 * The general rules of lora.h hold, as in lora_kv.h: device pointers unless a
 * comment says host, caller-owned buffers, asynchronous enqueue on `stream`,
 * host checks before anything is enqueued, no allocation.  Data-dependent
 * conditions set flags (LORA_BEAM_FLAG_*).
 */
#ifndef LORA_BEAM_H
#define LORA_BEAM_H

#include <stddef.h>
#include <stdint.h>

#include "lora.h"
#include "lora_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_BEAM_MAX 32               /* beams of a request */
#define LORA_BEAM_MAX_VOCAB (1 << 24)
#define LORA_BEAM_MAX_LAYERS 1024      /* caches of one lora_beam_copy */
#define LORA_BEAM_MAX_PENALTY 16       /* powers of length, of either sign */

/* State of the beams, one entry per row. */
typedef struct {
  float* score;    /* sum of the log-probabilities of its tokens; not finite: the row has no beam */
  int32_t* length; /* generated tokens */
  int32_t* done;   /* not 0: the beam has ended */
} lora_beams_t;

#define LORA_BEAM_FLAG_LOGITS 1      /* a logit was NaN or +inf (it counts as -inf) */
#define LORA_BEAM_FLAG_PARENT 2      /* a parent outside its request (the row is left empty) */
#define LORA_BEAM_FLAG_LENGTH 4      /* a negative length, or one past the table's row (cut) */
#define LORA_BEAM_FLAG_FREE_LIST 8   /* the free list ran out (the block's entry is -1) */
#define LORA_BEAM_FLAG_BLOCK_RANGE 16 /* an id outside the cache (of the free list: -1 in its place), an open block missing */

/* The `beams` best continuations of each request.  Row r with logits x (row r
 * of `logits`, row_stride elements apart, any alignment of its type) offers
 * for each token v < vocab
 *   total = score[r] + x[v] - log(sum_u e^x[u]),  length[r] + 1 tokens,
 * and a row that is done offers itself alone: total = score[r], its length,
 * the token eos.  Candidates are ranked by total / max(length, 1)^length_penalty
 * (0: by total), the highest first, equal ones by the lower
 * row, then the higher logit, then the lower token.  Sums and ranks are formed in 64 bits (exponentials in
 * 32), from finite logits of any size, of 16 or 32 bits; totals are rounded once, to fp32.
 * A logit of -inf is never chosen.  Where a request has fewer candidates than
 * beams, the rest of its rows get parent and token -1, score -inf, length 0
 * and done 1.
 * parent: the row that is continued.  out->done: the parent's done, or token
 * == eos (eos -1: no token ends a beam).  `out` may be `in`; other outputs
 * overlap neither each other nor an input.  flags: device, may be NULL; ORed.
 * ws: device, lora_beam_select_workspace bytes, 16-byte aligned; calls that
 * share it must not run at the same time.
 * Limits: beams up to LORA_BEAM_MAX, vocab up to LORA_BEAM_MAX_VOCAB, rows up
 * to LORA_KV_MAX_SEQS.  Errors: INVALID_ARG, UNSUPPORTED, ALIGNMENT,
 * WORKSPACE, HIP. */
size_t lora_beam_select_workspace(int32_t num_requests, int32_t beams, int32_t vocab);
lora_status_t lora_beam_select(const void* logits, int64_t row_stride, int32_t dtype, int32_t num_requests,
                               int32_t beams, int32_t vocab, const lora_beams_t* in, float length_penalty, int32_t eos,
                               int32_t* parent, int32_t* token, const lora_beams_t* out, int32_t* flags, void* ws,
                               size_t ws_bytes, void* stream);

/* What lora_beam_reorder leaves for lora_beam_copy and for the owner of the
 * free list.  Carved from one caller buffer by lora_beam_moves_init for up to
 * max_rows rows and tables of up to table_width entries.
 *   source, target, tokens [max_rows]  copy i: the first tokens[i] tokens of
 *       block source[i] to block target[i]; -1 behind the last one
 *   freed [max_rows * table_width]     blocks that no row holds any longer;
 *       entries behind the last one are left as they are
 *   counts [16]  see LORA_BEAM_COUNT_* */
typedef struct {
  int32_t max_rows;
  int32_t table_width;
  int32_t* source;
  int32_t* target;
  int32_t* tokens;
  int32_t* freed;
  int32_t* counts;
  int32_t* scratch;
} lora_beam_moves_t;
#define LORA_BEAM_COUNT_COPIES 0 /* copies: blocks asked of the free list */
#define LORA_BEAM_COUNT_FREED 1  /* blocks given back */
#define LORA_BEAM_COUNT_FLAGS 8
/* 0 outside the limits: max_rows in [1, LORA_KV_MAX_SEQS], table_width >= 1,
 * their product under 2^30.  Errors of init: INVALID_ARG, UNSUPPORTED,
 * ALIGNMENT, WORKSPACE. */
size_t lora_beam_moves_size(int32_t max_rows, int32_t table_width);
lora_status_t lora_beam_moves_init(void* buf, size_t bytes, int32_t max_rows, int32_t table_width,
                                   lora_beam_moves_t* out);

/* Row c of every request goes on from row parent[c] of the same request (-1:
 * the row is left empty) and takes over its block table: new_table row c is
 * table row parent[c] up to the blocks of its kv_len cached tokens, -1 from
 * there to table_width; new_len[c] = kv_len[parent[c]].
 * Blocks are shared by rows, except a block that is not full and would be
 * written to by several: of the rows whose last block is the same the first
 * keeps it, each other takes the next of free_blocks (in the order of rows) and
 * is listed in moves for lora_beam_copy, beams that have ended among them (the
 * call does not know which).  Where a parent's open block is missing
 * (-1: an earlier step's free list ran out) it is missing in every heir's row
 * too, nothing is taken or listed for it, and LORA_BEAM_FLAG_BLOCK_RANGE is set.
 * Ids of a row outside the cache, other than -1, set it too; they are taken
 * over as they are (the attention leaves such blocks out) and not given back.
 * Blocks of the old rows that no new row of the request holds are listed in
 * moves->freed, each once, in the order of requests, table columns and rows.
 * A block is taken to be shared only among the rows of one request at the same
 * column, as this call and a prompt's common blocks leave it; blocks that
 * other requests hold too must be kept alive by the caller (they are in every
 * row that shares them, so they are listed when the last row goes).
 * The call changes no input.  table and new_table may not overlap.
 * table_width is at most the moves' and the same for both tables.
 * Errors: INVALID_ARG, UNSUPPORTED (beams; block_tokens; num_blocks *
 * block_tokens past 2^31; table_width * block_tokens past 2^30), WORKSPACE
 * (rows or table_width past the moves' capacity), HIP. */
lora_status_t lora_beam_reorder(const int32_t* parent, const int32_t* kv_len, int32_t num_requests, int32_t beams,
                                const int32_t* table, int64_t table_stride, int32_t* new_table,
                                int64_t new_table_stride, int32_t table_width, int32_t* new_len,
                                const int32_t* free_blocks, int32_t num_free, int32_t num_blocks, int32_t block_tokens,
                                const lora_beam_moves_t* moves, void* stream);

/* The copies of lora_beam_reorder in num_layers caches (host array) of one
 * geometry: whole records of 16 tokens, as many as hold the copy's tokens.
 * Copies whose target is -1 or outside a cache are left out; where the source
 * is outside, the target's records are cleared (the values 0), so that nothing
 * of the block's last owner is attended to.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED, HIP. */
lora_status_t lora_beam_copy(const lora_beam_moves_t* moves, const lora_kv_cache_t* caches, int32_t num_layers,
                             void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_BEAM_H */
