// C ABI of the attention operators (lora_kv.h): argument checks, buffer
// carving and launch geometry.  Every check runs before the first HIP call.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "lora_kv_host.h"

using namespace lora::kv;

namespace {

constexpr size_t kAlign = 256;
// A launch has under 2^32 threads: work-groups of 256, up to four for a work
// item, and a factor of two to spare.
constexpr int64_t kMaxBlocks = (int64_t)1 << 23, kMaxItems = kMaxBlocks / 4;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int esize(int dtype) { return dtype == LORA_DTYPE_BF16 ? 2 : 4; }

lora_status_t check_dtype(int32_t dtype) {
  return dtype == LORA_DTYPE_BF16 || dtype == LORA_DTYPE_F32 ? LORA_OK : LORA_ERR_UNSUPPORTED;
}
bool head_dim_ok(int32_t d) { return d >= 32 && d <= LORA_KV_MAX_HEAD_DIM && d % 32 == 0; }
bool block_tokens_ok(int32_t b) { return b == 16 || b == 32 || b == 64 || b == 128 || b == 256; }
int log2_exact(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

// T rows of heads; head_dim elements each.
lora_status_t check_heads(const lora_heads_t* x, int32_t T, int32_t head_dim, int32_t dtype) {
  if (!x || x->heads < 1 || (!x->data && T > 0)) return LORA_ERR_INVALID_ARG;
  if (x->heads > LORA_KV_MAX_HEADS) return LORA_ERR_UNSUPPORTED;
  const int per = 16 / esize(dtype);
  if (x->head_stride < head_dim && x->heads > 1) return LORA_ERR_INVALID_ARG;
  if (x->token_stride < head_dim && T > 1) return LORA_ERR_INVALID_ARG;
  if (x->token_stride % per || x->head_stride % per || !aligned16(x->data)) return LORA_ERR_ALIGNMENT;
  return LORA_OK;
}
bool has_heads(const lora_heads_t* x) { return x && x->heads > 0; }
Rows rows_of(const lora_heads_t* x) {
  Rows r{nullptr, 0, 0, 0};
  if (x) r = Rows{x->data, x->token_stride, x->head_stride, x->heads};
  return r;
}

lora_status_t check_cache(const lora_kv_cache_t* c) {
  if (!c || !c->base || c->num_blocks < 1 || c->num_kv_heads < 1) return LORA_ERR_INVALID_ARG;
  if (!block_tokens_ok(c->block_tokens) || !head_dim_ok(c->head_dim) || c->num_kv_heads > LORA_KV_MAX_HEADS)
    return LORA_ERR_UNSUPPORTED;
  if (c->block_stride < (int64_t)lora_kv_block_bytes(c->block_tokens, c->num_kv_heads, c->head_dim))
    return LORA_ERR_INVALID_ARG;
  if ((int64_t)c->num_blocks * c->block_tokens > 0x7fffffffll) return LORA_ERR_UNSUPPORTED;
  if (c->block_stride % 16 || !aligned16(c->base)) return LORA_ERR_ALIGNMENT;
  return LORA_OK;
}
Cache cache_of(const lora_kv_cache_t* c) {
  return Cache{static_cast<uint8_t*>(c->base), c->block_stride, c->num_blocks, log2_exact(c->block_tokens),
               c->num_kv_heads, c->head_dim / 32};
}

lora_status_t check_rope(const lora_rope_t* r, int32_t head_dim) {
  if (!r || !r->inv_freq) return LORA_ERR_INVALID_ARG;
  if (r->rot_dim < 2 || r->rot_dim > head_dim || r->rot_dim % 2) return LORA_ERR_INVALID_ARG;
  if (r->layout != LORA_ROPE_HALF && r->layout != LORA_ROPE_INTERLEAVED) return LORA_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(r->inv_freq) & 7u) return LORA_ERR_ALIGNMENT;
  return LORA_OK;
}

// An output that is its input must have its strides.
bool in_place_ok(const lora_heads_t* x, const lora_heads_t* y) {
  return x->data != y->data || (x->token_stride == y->token_stride && x->head_stride == y->head_stride);
}

struct BatchSizes {
  size_t q_indptr, kv_len, row, counts, items, arrive, total;
};
bool batch_ok(int32_t max_tokens, int32_t max_seqs, int32_t hq, int32_t hkv, int32_t head_dim) {
  return max_tokens >= 0 && max_tokens <= LORA_MAX_TOKENS && max_seqs >= 1 && max_seqs <= LORA_KV_MAX_SEQS &&
         hkv >= 1 && hq >= hkv && hq <= LORA_KV_MAX_HEADS && hq % hkv == 0 && head_dim_ok(head_dim) &&
         (int64_t)max_tokens * (hq / hkv) < 0x7fffff00ll &&
         item_cap(max_tokens, max_seqs, hkv, hq / hkv) * hkv < kMaxItems;
}
BatchSizes batch_sizes(int32_t max_tokens, int32_t max_seqs, int32_t hq, int32_t hkv) {
  BatchSizes z;
  z.q_indptr = align_up(4 * ((size_t)max_seqs + 1));
  z.kv_len = align_up(4 * (size_t)max_seqs);
  z.row = align_up(4 * (size_t)std::max(max_tokens, 1));
  z.counts = align_up(4 * kNumCounts);
  z.items = align_up(kClasses * 32 * (size_t)item_cap(max_tokens, max_seqs, hkv, hq / hkv));
  z.arrive = align_up(4 * (size_t)part_cap(hkv) * hkv);
  z.total = z.q_indptr + z.kv_len + 3 * z.row + z.counts + z.items + z.arrive;
  return z;
}

lora_status_t check_batch(const lora_kv_batch_t* b) {
  if (!b || !b->q_indptr || !b->kv_len || !b->token_seq || !b->positions || !b->slots || !b->counts || !b->plan)
    return LORA_ERR_INVALID_ARG;
  return batch_ok(b->max_tokens, b->max_seqs, b->num_q_heads, b->num_kv_heads, b->head_dim) ? LORA_OK
                                                                                            : LORA_ERR_INVALID_ARG;
}

lora_status_t hip(hipError_t e) { return e == hipSuccess ? LORA_OK : LORA_ERR_HIP; }

}  // namespace

extern "C" {

size_t lora_kv_block_bytes(int32_t block_tokens, int32_t num_kv_heads, int32_t head_dim) {
  if (!block_tokens_ok(block_tokens) || !head_dim_ok(head_dim) || num_kv_heads < 1 || num_kv_heads > LORA_KV_MAX_HEADS)
    return 0;
  return (size_t)num_kv_heads * (block_tokens / kUnit) * 544 * (head_dim / 32);
}

size_t lora_kv_batch_size(int32_t max_tokens, int32_t max_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                          int32_t head_dim) {
  if (!batch_ok(max_tokens, max_seqs, num_q_heads, num_kv_heads, head_dim)) return 0;
  return batch_sizes(max_tokens, max_seqs, num_q_heads, num_kv_heads).total;
}

lora_status_t lora_kv_batch_init(void* buf, size_t bytes, int32_t max_tokens, int32_t max_seqs, int32_t num_q_heads,
                                 int32_t num_kv_heads, int32_t head_dim, lora_kv_batch_t* out) {
  if (!buf || !out || max_tokens < 0 || max_seqs < 1 || num_q_heads < 1 || num_kv_heads < 1)
    return LORA_ERR_INVALID_ARG;
  if (!batch_ok(max_tokens, max_seqs, num_q_heads, num_kv_heads, head_dim)) return LORA_ERR_UNSUPPORTED;
  if (!aligned16(buf)) return LORA_ERR_ALIGNMENT;
  const BatchSizes z = batch_sizes(max_tokens, max_seqs, num_q_heads, num_kv_heads);
  if (bytes < z.total) return LORA_ERR_WORKSPACE;
  char* p = static_cast<char*>(buf);
  auto take = [&p](size_t n) {
    int32_t* r = reinterpret_cast<int32_t*>(p);
    p += n;
    return r;
  };
  out->max_tokens = max_tokens;
  out->max_seqs = max_seqs;
  out->num_q_heads = num_q_heads;
  out->num_kv_heads = num_kv_heads;
  out->head_dim = head_dim;
  out->q_indptr = take(z.q_indptr);
  out->kv_len = take(z.kv_len);
  out->token_seq = take(z.row);
  out->positions = take(z.row);
  out->slots = take(z.row);
  out->counts = take(z.counts);
  out->plan = take(z.items + z.arrive);
  return LORA_OK;
}

lora_status_t lora_kv_build(const int32_t* ctx_len, const int32_t* new_len, int32_t B, int32_t T,
                            int32_t* block_table, int64_t table_stride, int32_t table_width,
                            const int32_t* free_blocks, int32_t num_free, int32_t num_blocks, int32_t block_tokens,
                            const lora_kv_batch_t* batch, void* stream) {
  if (B < 0 || T < 0 || num_free < 0 || num_blocks < 1 || table_width < 0) return LORA_ERR_INVALID_ARG;
  if (B > 0 && (!ctx_len || !new_len || !block_table || table_width < 1 || table_stride < table_width))
    return LORA_ERR_INVALID_ARG;
  if (num_free > 0 && !free_blocks) return LORA_ERR_INVALID_ARG;
  if (lora_status_t st = check_batch(batch)) return st;
  if (!block_tokens_ok(block_tokens) || (int64_t)num_blocks * block_tokens > 0x7fffffffll) return LORA_ERR_UNSUPPORTED;
  // a request's tokens, and the attention's steps past its last, stay within 32 bits
  if ((int64_t)table_width * block_tokens > (1 << 30)) return LORA_ERR_UNSUPPORTED;
  if (B > batch->max_seqs || T > batch->max_tokens) return LORA_ERR_WORKSPACE;
  const BatchSizes z = batch_sizes(batch->max_tokens, batch->max_seqs, batch->num_q_heads, batch->num_kv_heads);
  // the call writes the batch while it reads its inputs
  auto meets_batch = [&](const int32_t* p, int64_t n) {
    const uintptr_t from = reinterpret_cast<uintptr_t>(p), own = reinterpret_cast<uintptr_t>(batch->q_indptr);
    return n > 0 && from < own + z.total && from + 4 * (uint64_t)n > own;
  };
  if (meets_batch(ctx_len, B) || meets_batch(new_len, B) || meets_batch(free_blocks, num_free) ||
      meets_batch(block_table, B > 0 ? (B - 1) * table_stride + table_width : 0))
    return LORA_ERR_INVALID_ARG;
  BuildArgs A;
  A.ctx = ctx_len;
  A.add = new_len;
  A.table = block_table;
  A.free_blocks = free_blocks;
  A.tstride = table_stride;
  A.B = B;
  A.T = T;
  A.width = table_width;
  A.nfree = num_free;
  A.blocks = num_blocks;
  A.bt_log2 = log2_exact(block_tokens);
  A.hkv = batch->num_kv_heads;
  A.G = batch->num_q_heads / batch->num_kv_heads;
  A.item_cap = (int32_t)item_cap(batch->max_tokens, batch->max_seqs, A.hkv, A.G);
  A.part_cap = (int32_t)part_cap(A.hkv);
  A.q_indptr = batch->q_indptr;
  A.kv_len = batch->kv_len;
  A.token_seq = batch->token_seq;
  A.positions = batch->positions;
  A.slots = batch->slots;
  A.counts = batch->counts;
  A.items = reinterpret_cast<int4*>(batch->plan);
  A.arrive = batch->plan + z.items / 4;
  return hip(launch_build(A, static_cast<hipStream_t>(stream)));
}

lora_status_t lora_rope_frequencies(int32_t rot_dim, double theta, int32_t scaling, double factor, double original,
                                    double low, double high, double* out, double* scale) {
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > LORA_KV_MAX_HEAD_DIM || !(theta > 1.0) || !out || !scale)
    return LORA_ERR_INVALID_ARG;
  if (scaling < LORA_ROPE_SCALING_NONE || scaling > LORA_ROPE_SCALING_BANDS) return LORA_ERR_INVALID_ARG;
  if (scaling != LORA_ROPE_SCALING_NONE && !(factor >= 1.0 && isfinite(factor))) return LORA_ERR_INVALID_ARG;
  const bool ramps = scaling == LORA_ROPE_SCALING_YARN || scaling == LORA_ROPE_SCALING_BANDS;
  if (low == 0.0) low = 1.0;
  if (high == 0.0) high = scaling == LORA_ROPE_SCALING_YARN ? 32.0 : 4.0;
  if (ramps && (!(original >= 1.0) || !(low > 0.0) || !(high > low))) return LORA_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586477;
  if (scaling == LORA_ROPE_SCALING_NTK) theta *= pow(factor, (double)rot_dim / std::max(rot_dim - 2, 1));
  // the (fractional) pair that turns `turns` times over the original context
  auto pair_of = [&](double turns) { return rot_dim * log(original / (turns * two_pi)) / (2.0 * log(theta)); };
  double from = 0.0, to = 0.0;
  if (scaling == LORA_ROPE_SCALING_YARN) {
    from = std::max(floor(pair_of(high)), 0.0);
    to = std::min(ceil(pair_of(low)), rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = pow(theta, -2.0 * i / rot_dim);
    double keep = 1.0;
    if (scaling == LORA_ROPE_SCALING_LINEAR) keep = 0.0;
    if (scaling == LORA_ROPE_SCALING_YARN)
      keep = 1.0 - std::min(std::max((i - from) / std::max(to - from, 1e-3), 0.0), 1.0);
    if (scaling == LORA_ROPE_SCALING_BANDS)
      keep = std::min(std::max((original * f / two_pi - low) / (high - low), 0.0), 1.0);
    out[i] = scaling == LORA_ROPE_SCALING_NONE || scaling == LORA_ROPE_SCALING_NTK ? f
                                                                                   : f * keep + f / factor * (1.0 - keep);
  }
  *scale = scaling == LORA_ROPE_SCALING_YARN ? 0.1 * log(factor) + 1.0 : 1.0;
  return LORA_OK;
}

// Work-groups of the rotation role for `heads` heads: enough head groups that
// a small batch still spreads over the chip, whole passes of 256 threads else.
static void rotation_geometry(RopeArgs& A, int heads) {
  const int tiles = ceil_div_i(A.T, 4);
  int groups = std::max(1, std::min(heads, ceil_div_i(512, std::max(tiles, 1))));
  A.q_heads_per_group = ceil_div_i(heads, groups);
  A.q_groups = ceil_div_i(heads, A.q_heads_per_group);
  A.rot_blocks = tiles * A.q_groups;
}

// Work-groups of the cache role: 16 rows each, and as many groups of whole
// passes over the heads as spread a small batch over the chip.
static int cache_geometry(RopeArgs& A) {
  const int tiles = ceil_div_i(A.T, 16), at_once = 256 / (16 * A.cache.nc);
  const int passes = ceil_div_i(A.cache.heads, at_once);
  const int groups = std::max(1, std::min(passes, ceil_div_i(512, tiles)));
  A.kv_heads_per_group = ceil_div_i(passes, groups) * at_once;
  A.kv_groups = ceil_div_i(A.cache.heads, A.kv_heads_per_group);
  return tiles * A.kv_groups;
}

lora_status_t lora_rope(const lora_heads_t* q, const lora_heads_t* q_out, const lora_heads_t* k,
                        const lora_heads_t* k_out, const int32_t* positions, int32_t T, int32_t head_dim,
                        int32_t dtype, const lora_rope_t* rope, void* stream) {
  if (T < 0 || T > LORA_MAX_TOKENS || (T > 0 && !positions)) return LORA_ERR_INVALID_ARG;
  if (lora_status_t st = check_dtype(dtype)) return st;
  if (head_dim < 8 || head_dim > LORA_KV_MAX_HEAD_DIM || head_dim % 8) return LORA_ERR_UNSUPPORTED;
  if (lora_status_t st = check_rope(rope, head_dim)) return st;
  if (has_heads(q) != has_heads(q_out) || has_heads(k) != has_heads(k_out)) return LORA_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i) {
    const lora_heads_t *x = i ? k : q, *y = i ? k_out : q_out;
    if (!has_heads(x)) continue;
    if (lora_status_t st = check_heads(x, T, head_dim, dtype)) return st;
    if (lora_status_t st = check_heads(y, T, head_dim, dtype)) return st;
    if (x->heads != y->heads || !in_place_ok(x, y)) return LORA_ERR_INVALID_ARG;
  }
  RopeArgs A;
  memset(&A, 0, sizeof A);
  if (has_heads(q)) A.q = rows_of(q), A.qo = rows_of(q_out);
  if (has_heads(k)) A.k = rows_of(k), A.ko = rows_of(k_out);
  if (T == 0 || A.qo.heads + A.ko.heads == 0) return LORA_OK;
  A.pos = positions;
  A.freq = rope->inv_freq;
  A.fscale = rope->scale;
  A.T = T;
  A.D = head_dim;
  A.rot = rope->rot_dim;
  A.interleaved = rope->layout == LORA_ROPE_INTERLEAVED;
  rotation_geometry(A, A.qo.heads + A.ko.heads);
  return hip(launch_rope(A, dtype, A.rot_blocks, static_cast<hipStream_t>(stream)));
}

lora_status_t lora_kv_append(const lora_heads_t* q, const lora_heads_t* q_out, const lora_heads_t* k,
                             const lora_heads_t* v, const int32_t* positions, const int32_t* slots, int32_t T,
                             int32_t dtype, const lora_rope_t* rope, const lora_kv_cache_t* cache, int32_t* flags,
                             void* stream) {
  if (T < 0 || T > LORA_MAX_TOKENS || (T > 0 && (!slots || (rope && !positions)))) return LORA_ERR_INVALID_ARG;
  if (lora_status_t st = check_dtype(dtype)) return st;
  if (lora_status_t st = check_cache(cache)) return st;
  if (lora_status_t st = check_heads(k, T, cache->head_dim, dtype)) return st;
  if (lora_status_t st = check_heads(v, T, cache->head_dim, dtype)) return st;
  if (k->heads != cache->num_kv_heads || v->heads != cache->num_kv_heads) return LORA_ERR_INVALID_ARG;
  RopeArgs A;
  memset(&A, 0, sizeof A);
  if (rope) {
    if (lora_status_t st = check_rope(rope, cache->head_dim)) return st;
    if (has_heads(q) != has_heads(q_out)) return LORA_ERR_INVALID_ARG;
    if (has_heads(q)) {
      if (lora_status_t st = check_heads(q, T, cache->head_dim, dtype)) return st;
      if (lora_status_t st = check_heads(q_out, T, cache->head_dim, dtype)) return st;
      if (q->heads != q_out->heads || !in_place_ok(q, q_out)) return LORA_ERR_INVALID_ARG;
      A.q = rows_of(q);
      A.qo = rows_of(q_out);
    }
    A.pos = positions;
    A.freq = rope->inv_freq;
    A.fscale = rope->scale;
    A.rot = rope->rot_dim;
    A.interleaved = rope->layout == LORA_ROPE_INTERLEAVED;
  }
  if (T == 0) return LORA_OK;
  A.k = rows_of(k);
  A.v = rows_of(v);
  A.slots = slots;
  A.T = T;
  A.D = cache->head_dim;
  A.cache = cache_of(cache);
  A.flags = flags;
  if (A.qo.heads > 0) rotation_geometry(A, A.qo.heads);
  const int cache_blocks = cache_geometry(A);
  return hip(launch_rope(A, dtype, A.rot_blocks + cache_blocks, static_cast<hipStream_t>(stream)));
}

lora_status_t lora_kv_gather(const lora_kv_cache_t* cache, const int32_t* slots, int32_t n, const lora_heads_t* k_out,
                             const lora_heads_t* v_out, int32_t dtype, void* stream) {
  if (n < 0 || n > LORA_MAX_TOKENS || (n > 0 && !slots)) return LORA_ERR_INVALID_ARG;
  if (lora_status_t st = check_dtype(dtype)) return st;
  if (lora_status_t st = check_cache(cache)) return st;
  if (lora_status_t st = check_heads(k_out, n, cache->head_dim, dtype)) return st;
  if (lora_status_t st = check_heads(v_out, n, cache->head_dim, dtype)) return st;
  if (k_out->heads != cache->num_kv_heads || v_out->heads != cache->num_kv_heads) return LORA_ERR_INVALID_ARG;
  if (n == 0) return LORA_OK;
  RopeArgs A;
  memset(&A, 0, sizeof A);
  A.ko = rows_of(k_out);
  A.v = rows_of(v_out);
  A.slots = slots;
  A.T = n;
  A.D = cache->head_dim;
  A.cache = cache_of(cache);
  return hip(launch_gather(A, dtype, cache_geometry(A), static_cast<hipStream_t>(stream)));
}

size_t lora_kv_workspace_size(const lora_kv_batch_t* b) {
  if (check_batch(b)) return 0;
  return align_up((size_t)part_cap(b->num_kv_heads) * b->num_kv_heads * kUnit * (b->head_dim + 2) * sizeof(float));
}

lora_status_t lora_kv_attend(const lora_heads_t* q, const lora_heads_t* o, int32_t T, int32_t B, int32_t dtype,
                             const lora_kv_batch_t* batch, const int32_t* block_table, int64_t table_stride,
                             int32_t table_width, const lora_kv_cache_t* cache, float scale, void* ws,
                             size_t ws_bytes, void* stream) {
  if (T < 0 || B < 0 || table_width < 0) return LORA_ERR_INVALID_ARG;
  if (B > 0 && (!block_table || table_width < 1 || table_stride < table_width)) return LORA_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || !isfinite(scale)) return LORA_ERR_INVALID_ARG;
  if (lora_status_t st = check_dtype(dtype)) return st;
  if (lora_status_t st = check_batch(batch)) return st;
  if (lora_status_t st = check_cache(cache)) return st;
  if (lora_status_t st = check_heads(q, T, cache->head_dim, dtype)) return st;
  if (lora_status_t st = check_heads(o, T, cache->head_dim, dtype)) return st;
  if (q->heads != batch->num_q_heads || o->heads != batch->num_q_heads || cache->num_kv_heads != batch->num_kv_heads ||
      cache->head_dim != batch->head_dim || (q->data == o->data && T > 0))
    return LORA_ERR_INVALID_ARG;
  if (T > batch->max_tokens || B > batch->max_seqs) return LORA_ERR_WORKSPACE;
  if (!ws) return LORA_ERR_INVALID_ARG;
  if (ws_bytes < lora_kv_workspace_size(batch)) return LORA_ERR_WORKSPACE;
  if (!aligned16(ws)) return LORA_ERR_ALIGNMENT;
  if (T == 0 || B == 0) return LORA_OK;
  const BatchSizes z = batch_sizes(batch->max_tokens, batch->max_seqs, batch->num_q_heads, batch->num_kv_heads);
  AttendArgs A;
  A.q = rows_of(q);
  A.o = rows_of(o);
  A.counts = batch->counts;
  A.items = reinterpret_cast<const int4*>(batch->plan);
  A.arrive = batch->plan + z.items / 4;
  A.table = block_table;
  A.tstride = table_stride;
  A.width = table_width;
  A.T = T;
  A.B = B;
  A.G = batch->num_q_heads / batch->num_kv_heads;
  A.item_cap = (int32_t)item_cap(batch->max_tokens, batch->max_seqs, batch->num_kv_heads, A.G);
  A.cache = cache_of(cache);
  A.scale_log2e = scale * 1.4426950408889634f;
  A.part = static_cast<float*>(ws);
  return hip(launch_attend(A, dtype, many_rows(T, B), static_cast<hipStream_t>(stream)));
}

lora_status_t lora_prompt_attend(const lora_heads_t* q, const lora_heads_t* k, const lora_heads_t* v,
                                 const lora_heads_t* o, const int32_t* indptr, int32_t B, int32_t T, int32_t head_dim,
                                 int32_t dtype, float scale, void* stream) {
  if (B < 0 || T < 0 || T > LORA_MAX_TOKENS || (B > 0 && !indptr)) return LORA_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || !isfinite(scale)) return LORA_ERR_INVALID_ARG;
  if (lora_status_t st = check_dtype(dtype)) return st;
  if (!head_dim_ok(head_dim) || B > LORA_KV_MAX_SEQS) return LORA_ERR_UNSUPPORTED;
  for (const lora_heads_t* x : {q, k, v, o})
    if (lora_status_t st = check_heads(x, T, head_dim, dtype)) return st;
  if (q->heads != o->heads || k->heads != v->heads || q->heads % k->heads) return LORA_ERR_INVALID_ARG;
  if (T > 0 && (o->data == q->data || o->data == k->data || o->data == v->data)) return LORA_ERR_INVALID_ARG;
  // a tile of 64 rows is addressed with 32-bit byte offsets
  if (k->token_stride > (1 << 23) || v->token_stride > (1 << 23)) return LORA_ERR_UNSUPPORTED;
  if (T == 0 || B == 0) return LORA_OK;
  if (((int64_t)T / 64 + B) * q->heads >= kMaxBlocks) return LORA_ERR_UNSUPPORTED;
  PromptArgs A;
  A.q = rows_of(q);
  A.k = rows_of(k);
  A.v = rows_of(v);
  A.o = rows_of(o);
  A.indptr = indptr;
  A.B = B;
  A.T = T;
  A.G = q->heads / k->heads;
  A.scale_log2e = scale * 1.4426950408889634f;
  return hip(launch_prompt(A, dtype, head_dim, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
