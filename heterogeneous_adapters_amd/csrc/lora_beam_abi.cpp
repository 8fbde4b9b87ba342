// C ABI of the beam search operators (lora_beam.h): argument checks, buffer
// carving and launch geometry.  Every check runs before the first HIP call.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "lora_beam_args.h"

using namespace lora::beam;
using namespace lora::kv;

namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool block_tokens_ok(int32_t b) { return b == 16 || b == 32 || b == 64 || b == 128 || b == 256; }
int log2_exact(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

bool rows_ok(int32_t requests, int32_t beams) {
  return beams >= 1 && beams <= LORA_BEAM_MAX && requests >= 0 && (int64_t)requests * beams <= LORA_KV_MAX_SEQS;
}
bool select_ok(int32_t requests, int32_t beams, int32_t vocab) {
  return rows_ok(requests, beams) && vocab >= 1 && vocab <= LORA_BEAM_MAX_VOCAB;
}
struct SelectSizes {
  size_t keys, total;
};
SelectSizes select_sizes(int32_t requests, int32_t beams, int32_t vocab) {
  const size_t rows = (size_t)requests * beams;
  if (rows == 0) return SelectSizes{0, kAlign};
  const size_t waves = (size_t)row_waves(rows, vocab);
  const size_t keys = align_up(rows * waves * beams * sizeof(uint64_t));
  return SelectSizes{keys, keys + align_up(rows * waves * 2 * sizeof(double))};
}

struct MovesSizes {
  size_t list, freed, counts, total;
};
bool moves_ok(int32_t max_rows, int32_t width) {
  return max_rows >= 1 && max_rows <= LORA_KV_MAX_SEQS && width >= 1 && (int64_t)max_rows * width < (1 << 30);
}
MovesSizes moves_sizes(int32_t max_rows, int32_t width) {
  MovesSizes z;
  z.list = align_up(4 * (size_t)max_rows);
  z.freed = align_up(4 * (size_t)max_rows * width);
  z.counts = align_up(64);
  z.total = 3 * z.list + z.freed + z.counts + align_up(8 * (size_t)max_rows);
  return z;
}
lora_status_t check_moves(const lora_beam_moves_t* m) {
  return m && m->source && m->target && m->tokens && m->freed && m->counts && m->scratch &&
                 moves_ok(m->max_rows, m->table_width)
             ? LORA_OK
             : LORA_ERR_INVALID_ARG;
}

bool meet(const void* p, int64_t n, const void* q, int64_t m) {  // n and m bytes
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return n > 0 && m > 0 && a < b + (uint64_t)m && b < a + (uint64_t)n;
}

lora_status_t hip(hipError_t e) { return e == hipSuccess ? LORA_OK : LORA_ERR_HIP; }

}  // namespace

extern "C" {

size_t lora_beam_select_workspace(int32_t num_requests, int32_t beams, int32_t vocab) {
  return select_ok(num_requests, beams, vocab) ? select_sizes(num_requests, beams, vocab).total : 0;
}

lora_status_t lora_beam_select(const void* logits, int64_t row_stride, int32_t dtype, int32_t num_requests,
                               int32_t beams, int32_t vocab, const lora_beams_t* in, float length_penalty, int32_t eos,
                               int32_t* parent, int32_t* token, const lora_beams_t* out, int32_t* flags, void* ws,
                               size_t ws_bytes, void* stream) {
  if (num_requests < 0 || beams < 1 || vocab < 1 || !in || !out || !(fabsf(length_penalty) <= LORA_BEAM_MAX_PENALTY) || eos < -1 || eos >= vocab)
    return LORA_ERR_INVALID_ARG;
  if (dtype != LORA_DTYPE_BF16 && dtype != LORA_DTYPE_F32) return LORA_ERR_UNSUPPORTED;
  if (!select_ok(num_requests, beams, vocab)) return LORA_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)num_requests * beams;
  const int size = dtype == LORA_DTYPE_BF16 ? 2 : 4;
  if (rows > 0) {
    if (!logits || !parent || !token || !in->score || !in->length || !in->done || !out->score || !out->length || !out->done || !ws)
      return LORA_ERR_INVALID_ARG;
    if (rows > 1 && row_stride < vocab) return LORA_ERR_INVALID_ARG;
    if (row_stride > ((int64_t)1 << 40)) return LORA_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(logits) % size || !aligned16(ws)) return LORA_ERR_ALIGNMENT;
    // outputs: `out` may be `in`, entry for entry; nothing else overlaps
    const void* outs[] = {out->score, out->length, out->done, parent, token};
    const void* ins[] = {in->score, in->length, in->done};
    const int64_t logit_bytes = ((rows - 1) * row_stride + vocab) * size;
    for (int i = 0; i < 5; ++i) {
      for (int j = 0; j < i; ++j)
        if (meet(outs[i], 4 * rows, outs[j], 4 * rows)) return LORA_ERR_INVALID_ARG;
      for (int j = 0; j < 3; ++j)
        if (!(i == j && outs[i] == ins[j]) && meet(outs[i], 4 * rows, ins[j], 4 * rows)) return LORA_ERR_INVALID_ARG;
      if (meet(outs[i], 4 * rows, logits, logit_bytes)) return LORA_ERR_INVALID_ARG;
    }
  }
  const SelectSizes z = select_sizes(num_requests, beams, vocab);
  if (ws_bytes < z.total) return LORA_ERR_WORKSPACE;
  if (rows == 0) return LORA_OK;
  SelectArgs A;
  A.logits = logits;
  A.stride = row_stride;
  A.requests = num_requests;
  A.beams = beams;
  A.vocab = vocab;
  A.waves = (int32_t)row_waves(rows, vocab);
  A.chunks = (int32_t)((row_chunks(vocab) + A.waves - 1) / A.waves);
  A.score = in->score;
  A.length = in->length;
  A.done = in->done;
  A.penalty = length_penalty;
  A.eos = eos;
  A.parent = parent;
  A.token = token;
  A.score_out = out->score;
  A.length_out = out->length;
  A.done_out = out->done;
  A.flags = flags;
  A.keys = static_cast<uint64_t*>(ws);
  A.sums = reinterpret_cast<double*>(static_cast<char*>(ws) + z.keys);
  return hip(launch_select(A, dtype, static_cast<hipStream_t>(stream)));
}

size_t lora_beam_moves_size(int32_t max_rows, int32_t table_width) {
  return moves_ok(max_rows, table_width) ? moves_sizes(max_rows, table_width).total : 0;
}

lora_status_t lora_beam_moves_init(void* buf, size_t bytes, int32_t max_rows, int32_t table_width,
                                   lora_beam_moves_t* out) {
  if (!buf || !out || max_rows < 1 || table_width < 1) return LORA_ERR_INVALID_ARG;
  if (!moves_ok(max_rows, table_width)) return LORA_ERR_UNSUPPORTED;
  if (!aligned16(buf)) return LORA_ERR_ALIGNMENT;
  const MovesSizes z = moves_sizes(max_rows, table_width);
  if (bytes < z.total) return LORA_ERR_WORKSPACE;
  char* p = static_cast<char*>(buf);
  auto take = [&p](size_t n) {
    int32_t* r = reinterpret_cast<int32_t*>(p);
    p += n;
    return r;
  };
  out->max_rows = max_rows;
  out->table_width = table_width;
  out->source = take(z.list);
  out->target = take(z.list);
  out->tokens = take(z.list);
  out->freed = take(z.freed);
  out->counts = take(z.counts);
  out->scratch = take(0);
  return LORA_OK;
}

lora_status_t lora_beam_reorder(const int32_t* parent, const int32_t* kv_len, int32_t num_requests, int32_t beams,
                                const int32_t* table, int64_t table_stride, int32_t* new_table,
                                int64_t new_table_stride, int32_t table_width, int32_t* new_len,
                                const int32_t* free_blocks, int32_t num_free, int32_t num_blocks, int32_t block_tokens,
                                const lora_beam_moves_t* moves, void* stream) {
  if (num_requests < 0 || beams < 1 || num_free < 0 || num_blocks < 1 || table_width < 1) return LORA_ERR_INVALID_ARG;
  if (lora_status_t st = check_moves(moves)) return st;
  if (!rows_ok(num_requests, beams) || !block_tokens_ok(block_tokens) || (int64_t)num_blocks * block_tokens > 0x7fffffffll ||
      (int64_t)table_width * block_tokens > (1 << 30))
    return LORA_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)num_requests * beams;
  if (rows > 0 && (!parent || !kv_len || !table || !new_table || !new_len)) return LORA_ERR_INVALID_ARG;
  if (num_free > 0 && !free_blocks) return LORA_ERR_INVALID_ARG;
  if (rows > 1 && (table_stride < table_width || new_table_stride < table_width)) return LORA_ERR_INVALID_ARG;
  if (rows > moves->max_rows || table_width > moves->table_width) return LORA_ERR_WORKSPACE;
  // what the call writes overlaps nothing else of the call
  const MovesSizes z = moves_sizes(moves->max_rows, moves->table_width);
  const int64_t old_bytes = rows ? 4 * ((rows - 1) * table_stride + table_width) : 0;
  const int64_t new_bytes = rows ? 4 * ((rows - 1) * new_table_stride + table_width) : 0;
  const struct {
    const void* p;
    int64_t n;
  } ins[] = {{parent, 4 * rows}, {kv_len, 4 * rows}, {table, old_bytes}, {free_blocks, 4 * (int64_t)num_free}},
    outs[] = {{new_table, new_bytes}, {new_len, 4 * rows}, {moves->source, (int64_t)z.total}};
  for (int i = 0; i < 3; ++i) {
    for (const auto& x : ins)
      if (meet(outs[i].p, outs[i].n, x.p, x.n)) return LORA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (meet(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return LORA_ERR_INVALID_ARG;
  }
  ReorderArgs A;
  A.parent = parent;
  A.kv_len = kv_len;
  A.table = table;
  A.free_blocks = free_blocks;
  A.new_table = new_table;
  A.new_len = new_len;
  A.stride = table_stride;
  A.new_stride = new_table_stride;
  A.requests = num_requests;
  A.beams = beams;
  A.width = table_width;
  A.num_free = num_free;
  A.num_blocks = num_blocks;
  A.bt_log2 = log2_exact(block_tokens);
  A.max_rows = moves->max_rows;
  A.source = moves->source;
  A.target = moves->target;
  A.tokens = moves->tokens;
  A.freed = moves->freed;
  A.counts = moves->counts;
  A.scratch = moves->scratch;
  return hip(launch_reorder(A, static_cast<hipStream_t>(stream)));
}

lora_status_t lora_beam_copy(const lora_beam_moves_t* moves, const lora_kv_cache_t* caches, int32_t num_layers,
                             void* stream) {
  if (lora_status_t st = check_moves(moves)) return st;
  if (num_layers < 0 || (num_layers > 0 && !caches)) return LORA_ERR_INVALID_ARG;
  if (num_layers > LORA_BEAM_MAX_LAYERS) return LORA_ERR_UNSUPPORTED;
  for (int i = 0; i < num_layers; ++i) {
    const lora_kv_cache_t &c = caches[i], &f = caches[0];
    if (!c.base || c.num_blocks < 1 || c.num_kv_heads < 1) return LORA_ERR_INVALID_ARG;
    const size_t bytes = lora_kv_block_bytes(c.block_tokens, c.num_kv_heads, c.head_dim);
    if (bytes == 0) return LORA_ERR_UNSUPPORTED;
    if (c.block_stride < (int64_t)bytes || c.block_stride != f.block_stride || c.num_blocks != f.num_blocks ||
        c.block_tokens != f.block_tokens || c.num_kv_heads != f.num_kv_heads || c.head_dim != f.head_dim)
      return LORA_ERR_INVALID_ARG;
    if (c.block_stride % 16 || !aligned16(c.base)) return LORA_ERR_ALIGNMENT;
  }
  for (int from = 0; from < num_layers; from += kCopyLayers) {
    const lora_kv_cache_t& f = caches[0];
    CopyArgs A;
    A.layers = min_i(num_layers - from, kCopyLayers);
    for (int i = 0; i < A.layers; ++i) A.base[i] = static_cast<uint8_t*>(caches[from + i].base);
    A.stride = f.block_stride;
    A.num_blocks = f.num_blocks;
    A.units = f.block_tokens / kUnit;
    A.heads = f.num_kv_heads;
    A.record = 544 * (f.head_dim / 32);
    A.max_rows = moves->max_rows;
    A.source = moves->source;
    A.target = moves->target;
    A.tokens = moves->tokens;
    A.counts = moves->counts;
    if (hipError_t e = launch_copy(A, static_cast<hipStream_t>(stream))) return hip(e);
  }
  return LORA_OK;
}

}  // extern "C"
