// lora_kv_build: block tables, slot maps and the attention's work plan from
// request lengths.
//
// Mathematics: exclusive sums over the requests (new tokens, new blocks, work
// items), then one table lookup per token, new block and item.  Integer work
// on a few kilobytes, bound by latency: one launch, in which every work-group
// sums over all requests by itself (8 bytes per request out of L2) rather
// than waiting for another launch or a grid-wide hand-over, then fills its
// share of the tokens, blocks and items by bisecting the sums in LDS.
#include "lora_kv_dev.h"
#include "lora_kv_host.h"

namespace lora {
namespace kv {

namespace {

constexpr int kThreads = 1024;
constexpr int kWavesB = kThreads / 64;

// Inclusive sum over the work-group; *total gets the sum of all.
template <class V>
__device__ V block_scan(V x, V* scratch, V* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const V y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // scratch may still be read from the call before
  if (lane == 63) scratch[wave] = x;
  __syncthreads();
  V before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWavesB; ++w) {
    const V s = scratch[w];
    before += w < wave ? s : (V)0;
    all += s;
  }
  *total = all;
  return x + before;
}

// Largest i < n with start[i] <= x (start ascending, start[0] <= x).
__device__ __forceinline__ int bisect(const int32_t* start, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// What the call uses of one request's lengths.
struct Request {
  int ctx, add, have, need;  // tokens cached, tokens to come, blocks filled by the first, by both
  bool bad;
};
__device__ __forceinline__ Request request(const BuildArgs& A, int i, int cap) {
  Request r{0, 0, 0, 0, false};
  if (i >= A.B) return r;
  const int c = A.ctx[i], n = A.add[i];
  r.bad = c < 0 || n < 0 || c > cap || (int64_t)max(c, 0) + max(n, 0) > cap;
  r.ctx = min(max(c, 0), cap);
  r.add = max(n, 0);
  const int bt = 1 << A.bt_log2;
  const int end = (int)min((int64_t)r.ctx + r.add, (int64_t)cap);
  r.have = (r.ctx + bt - 1) >> A.bt_log2;
  r.need = (int)(((int64_t)end + bt - 1) >> A.bt_log2);
  return r;
}

__device__ __forceinline__ int64_t tiles_of(int64_t tokens, int G) { return (tokens * G + kUnit - 1) / kUnit; }

__global__ __launch_bounds__(kThreads) void build_kernel(const BuildArgs A) {
  __shared__ int64_t scratch[kWavesB];
  __shared__ int32_t scratch_i[kWavesB];
  __shared__ int32_t s_row[kThreads];    // first token row
  __shared__ int32_t s_fresh[kThreads];  // first new block, counted over the step
  __shared__ int32_t s_item[kThreads];   // first work item
  __shared__ int32_t s_wide[kThreads];   // first work item of 32 rows
  __shared__ int32_t s_ctx[kThreads], s_chunks[kThreads], s_part[kThreads];
  const int tid = threadIdx.x, wg = blockIdx.x, nwg = gridDim.x;
  const int bt = 1 << A.bt_log2;
  const int cap = (int)min((int64_t)A.width << A.bt_log2, (int64_t)0x7fffffff);

  // Tokens per work item, from the cached tokens that all row tiles read.
  int64_t mine = 0;
  for (int i = tid; i < A.B; i += kThreads) {
    const Request r = request(A, i, cap);
    mine += tiles_of(min(r.add, A.T), A.G) * min((int64_t)r.ctx + r.add, (int64_t)cap);
  }
  int64_t read;
  block_scan<int64_t>(mine, scratch, &read);
  const int64_t per = (read * A.hkv + kTargetItems - 1) / kTargetItems;
  const int64_t rounded = max((per + kChunkStep - 1) / kChunkStep * kChunkStep, (int64_t)kMinChunk);
  const int chunk = (int)min(rounded, (int64_t)1 << 30);

  const bool wide_ok = wide_step(A.T, A.B);
  int64_t rows0 = 0, fresh0 = 0;
  int items0 = 0, wide0 = 0, parts0 = 0, flags = 0;
  for (int base = 0; base < A.B; base += kThreads) {
    const int i = base + tid;
    const Request r = request(A, i, cap);
    int64_t rows, fresh;
    const int64_t row_end = rows0 + block_scan<int64_t>(r.add, scratch, &rows);
    const int64_t fresh_end = fresh0 + block_scan<int64_t>(r.need - r.have, scratch, &fresh);
    const int first = (int)min(row_end - r.add, (int64_t)A.T), last = (int)min(row_end, (int64_t)A.T);
    const int64_t fresh_first = fresh_end - (r.need - r.have);
    const int got = (int)max(min((int64_t)A.nfree - fresh_first, (int64_t)(r.need - r.have)), (int64_t)0);
    const int kv = (int)min(min((int64_t)r.ctx + (last - first), (int64_t)cap), (int64_t)(r.have + got) << A.bt_log2);
    const bool wide = wide_ok && (int64_t)(last - first) * A.G > kUnit;
    const int tiles = (int)(((int64_t)(last - first) * A.G + (wide ? 2 * kUnit - 1 : kUnit - 1)) / (wide ? 2 * kUnit : kUnit));
    const int chunks = max((kv + chunk - 1) / chunk, 1);
    int items, wides, parts;
    const int n_all = i < A.B ? tiles * chunks : 0;
    const int n_items = wide ? 0 : n_all, n_wide = wide ? n_all : 0;
    const int n_parts = chunks > 1 ? n_items + 2 * n_wide : 0;
    const int item_end = items0 + block_scan<int32_t>(n_items, scratch_i, &items);
    const int wide_end = wide0 + block_scan<int32_t>(n_wide, scratch_i, &wides);
    const int part_end = parts0 + block_scan<int32_t>(n_parts, scratch_i, &parts);
    s_row[tid] = first;
    s_fresh[tid] = (int)min(fresh_first, (int64_t)0x7fffffff);
    s_item[tid] = item_end - n_items;
    s_wide[tid] = wide_end - n_wide;
    s_ctx[tid] = r.ctx;
    s_chunks[tid] = chunks;
    s_part[tid] = chunks > 1 ? part_end - n_parts : -1;
    if (wg == 0 && i < A.B) {
      A.q_indptr[i] = first;
      A.kv_len[i] = kv;
      if (r.bad) flags |= LORA_KV_FLAG_LENGTH;
      if (row_end > A.T) flags |= LORA_KV_FLAG_TOKENS;
      if (fresh_end > A.nfree) flags |= LORA_KV_FLAG_FREE_LIST;
      // the one cached block that new tokens may lie in
      if (last > first && (r.ctx & (bt - 1)) != 0 &&
          (unsigned)A.table[i * A.tstride + (r.ctx >> A.bt_log2)] >= (unsigned)A.blocks)
        flags |= LORA_KV_FLAG_BLOCK_RANGE;
    }
    __syncthreads();
    const int n = min(kThreads, A.B - base);
    const int row0 = (int)min(rows0, (int64_t)A.T), row1 = (int)min(rows0 + rows, (int64_t)A.T);
    for (int t = row0 + wg * kThreads + tid; t < row1; t += nwg * kThreads) {
      const int k = bisect(s_row, n, t);
      const int64_t pos = (int64_t)s_ctx[k] + (t - s_row[k]);
      int slot = -1;
      if (pos < cap) {
        const int b = (int)(pos >> A.bt_log2), have = (s_ctx[k] + bt - 1) >> A.bt_log2;
        int id = -1;
        if (b < have) {
          id = A.table[(base + k) * A.tstride + b];
        } else {
          const int64_t f = (int64_t)s_fresh[k] + (b - have);
          if (f < A.nfree) id = A.free_blocks[f];
        }
        if ((unsigned)id < (unsigned)A.blocks) slot = (id << A.bt_log2) + (int)(pos & (bt - 1));
      }
      A.token_seq[t] = base + k;
      A.positions[t] = (int)min(pos, (int64_t)0x7fffffff);
      A.slots[t] = slot;
    }
    const int64_t fresh1 = min(fresh0 + fresh, (int64_t)0x7fffffff);
    for (int64_t f = fresh0 + wg * kThreads + tid; f < fresh1; f += nwg * kThreads) {
      const int k = bisect(s_fresh, n, (int)f);
      const int b = ((s_ctx[k] + bt - 1) >> A.bt_log2) + (int)(f - s_fresh[k]);
      int id = f < A.nfree ? A.free_blocks[f] : -1;
      if ((unsigned)id >= (unsigned)A.blocks) id = -1;
      A.table[(base + k) * A.tstride + b] = id;
    }
    if (wg == 0) {
      for (int64_t f = fresh0 + tid; f < min(fresh1, (int64_t)A.nfree); f += kThreads)
        if ((unsigned)A.free_blocks[f] >= (unsigned)A.blocks) flags |= LORA_KV_FLAG_BLOCK_RANGE;
    }
    // One item: its request, tile, chunk and the tile's first part (-1: alone).
    auto fill = [&](const int32_t* start, int w, int units, int4* to) {
      const int k = bisect(start, n, w);
      const int local = w - start[k], tile = local / s_chunks[k], c = local - tile * s_chunks[k];
      int part = -1;
      if (s_part[k] >= 0) {
        part = s_part[k] + tile * s_chunks[k] * units;
        if (part + s_chunks[k] * units > A.part_cap) part = -1;
        if (part >= 0)
          for (int h = 0; c == 0 && h < A.hkv; ++h) A.arrive[(int64_t)part * A.hkv + h] = 0;
      }
      *to = make_int4(base + k, tile, c, part);
    };
    for (int w = items0 + wg * kThreads + tid; w < min(items0 + items, A.item_cap); w += nwg * kThreads)
      fill(s_item, w, 1, A.items + w);
    for (int w = wide0 + wg * kThreads + tid; w < min(wide0 + wides, A.item_cap); w += nwg * kThreads)
      fill(s_wide, w, 2, A.items + A.item_cap + w);
    rows0 += rows;
    fresh0 += fresh;
    items0 += items;
    wide0 += wides;
    parts0 += parts;
    __syncthreads();
  }

  // rows behind the last request's
  const int used = (int)min(rows0, (int64_t)A.T);
  for (int t = used + wg * kThreads + tid; t < A.T; t += nwg * kThreads) {
    A.token_seq[t] = -1;
    A.positions[t] = -1;
    A.slots[t] = -1;
  }
  if (wg == 0) {
#pragma unroll
    for (int d = 32; d; d >>= 1) flags |= __shfl_xor(flags, d);
    __syncthreads();
    if ((tid & 63) == 0) scratch_i[tid >> 6] = flags;
    __syncthreads();
    if (tid < kNumCounts) {
      int all = 0;
      for (int w = 0; w < kWavesB; ++w) all |= scratch_i[w];
      int v = 0;
      if (tid == kCountTokens) v = used;
      if (tid == kCountNewBlocks) v = (int)min(fresh0, (int64_t)0x7fffffff);
      if (tid == kCountItems) v = items0;
      if (tid == kCountParts) v = parts0;
      if (tid == kCountWide) v = wide0;
      if (tid == kCountChunk) v = chunk;
      if (tid == kCountFlags) v = all;
      if (tid == kCountB) v = A.B;
      if (tid == kCountT) v = A.T;
      if (tid == kCountCheck) v = check_word(A.B, A.T, items0, wide0, parts0);
      A.counts[tid] = v;
    }
    if (tid == kThreads - 1) A.q_indptr[A.B] = used;
  }
}

}  // namespace

hipError_t launch_build(const BuildArgs& A, hipStream_t s) {
  // one work-group per 1024 rows or 256 requests, up to 64: each repeats the
  // sums over the requests
  const int want = max_i(ceil_div_i(A.T, kThreads), ceil_div_i(A.B, 256));
  const int grid = min_i(max_i(want, 1), 64);
  build_kernel<<<grid, kThreads, 0, s>>>(A);
  return hipGetLastError();
}

}  // namespace kv
}  // namespace lora
