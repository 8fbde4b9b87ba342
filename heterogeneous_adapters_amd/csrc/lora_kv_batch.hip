// lora_kv_build: block tables, slot maps and the attention's work plan from
// request lengths.
//
// Mathematics: exclusive sums over the requests (new tokens, new blocks, work
// items), then one table lookup per token, new block and item.  Integer work
// on a few kilobytes, bound by latency: one launch, in which every work-group
// sums over all requests by itself (8 bytes per request out of L2) rather
// than waiting for another launch or a grid-wide hand-over, then fills its
// share of the tokens, blocks and items by bisecting the sums in LDS.
// Measured on MI355X: 48 requests 7 us, 1024 decode requests 10.5, 2000
// requests with 133k new tokens 21.5.
#include "lora_kv_dev.h"
#include "lora_kv_host.h"
#include "lora_kv_scan.h"

namespace lora {
namespace kv {

namespace {

// What the call uses of one request's lengths.
struct Request {
  int ctx, add, have, need;  // tokens cached, tokens to come, blocks filled by the first, by both
  bool bad;
};
__device__ __forceinline__ Request request(const BuildArgs& A, int i, int cap) {
  Request r{0, 0, 0, 0, false};
  if (i >= A.B) return r;
  const int c = A.ctx[i], n = A.add[i];
  r.bad = c < 0 || n < 0 || (int64_t)max(c, 0) + max(n, 0) > cap;
  r.ctx = min(max(c, 0), cap);
  r.add = min(max(n, 0), A.T);
  const int bt = 1 << A.bt_log2;
  const int64_t end = min((int64_t)r.ctx + r.add, (int64_t)cap);
  r.have = (int)(((int64_t)r.ctx + bt - 1) >> A.bt_log2);
  r.need = (int)((end + bt - 1) >> A.bt_log2);
  return r;
}

__device__ __forceinline__ int class_of(int rows, bool many) { return rows <= kUnit || !many ? 0 : rows <= kMidMost ? 1 : 2; }
__device__ __forceinline__ int tiles_of(int rows, int cls) {
  const int per = rows_of_class(cls);
  return (rows + per - 1) / per;
}

// kPer: requests per thread and turn.
template <int kThreads, int kPer>
__global__ __launch_bounds__(kThreads) void build_kernel(const BuildArgs A) {
  constexpr int kTurn = kThreads * kPer, kWavesB = kThreads / 64;
  __shared__ uint32_t s_a[kWavesB][8], s_b[kWavesB][8], s_c[kWavesB][8];
  __shared__ int64_t s_read[2][kWavesB];
  __shared__ int32_t s_row[kTurn];    // first token row
  __shared__ int32_t s_fresh[kTurn];  // first new block, counted over the step
  __shared__ int32_t s_item[kClasses][kTurn];  // first work item of its class
  __shared__ int32_t s_ctx[kTurn], s_chunks[kTurn], s_part[kTurn], s_kv[kTurn], s_rows[kTurn];
  const int tid = threadIdx.x, wg = blockIdx.x, nwg = gridDim.x;
  const int bt = 1 << A.bt_log2;
  const int cap = (int)min((int64_t)A.width << A.bt_log2, (int64_t)0x7fffffff);
  const uint32_t builds = wg == 0 && tid == kCountBuild ? (uint32_t)A.counts[kCountBuild] : 0;  // read ahead of its use

  // Tokens per work item, from the cached tokens that all row tiles read.
  const bool many = many_rows(A.T, A.B);
  Request r[kPer];
  int64_t mine = 0, mine_wide = 0;
  for (int base = 0; base < A.B; base += kTurn) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      r[e] = request(A, base + tid * kPer + e, cap);
      const int rows = r[e].add * A.G, cls = class_of(rows, many);
      const int64_t reads = (int64_t)tiles_of(rows, cls) * min((int64_t)r[e].ctx + r[e].add, (int64_t)cap);
      mine += cls == 2 ? 0 : reads;
      mine_wide += cls == 2 ? reads : 0;
    }
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    mine += __shfl_xor(mine, d);
    if (many) mine_wide += __shfl_xor(mine_wide, d);
  }
  if ((tid & 63) == 0) s_read[0][tid >> 6] = mine, s_read[1][tid >> 6] = mine_wide;
  __syncthreads();
  auto chunk_for = [&](const int64_t* reads, int target) {
    int64_t sum = 0;
    for (int w = 0; w < kWavesB; ++w) sum += reads[w];
    const int64_t per = (sum * A.hkv + target - 1) / target;
    const int64_t rounded = max((per + kChunkStep - 1) / kChunkStep * kChunkStep, (int64_t)kMinChunk);
    return (int)min(rounded, (int64_t)1 << 29);
  };
  const int chunk = chunk_for(s_read[0], kTargetItems), chunk_wide = chunk_for(s_read[1], kTargetWide);

  int64_t rows0 = 0, fresh0 = 0, parts0 = 0, items0[kClasses] = {0, 0, 0};
  int flags = 0;
  for (int base = 0; base < A.B; base += kTurn) {
    if (A.B > kTurn) {  // else the first pass left them here
#pragma unroll
      for (int e = 0; e < kPer; ++e) r[e] = request(A, base + tid * kPer + e, cap);
    }
    uint32_t x[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[0] += r[e].add, x[1] += r[e].need - r[e].have;
    int64_t at[2], sum[2];
    block_scan<kWavesB, 2>(x, at, sum, s_a);
    // the one cached block of each request that new tokens may lie in
    int open_block[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int i = base + tid * kPer + e;
      open_block[e] = 0;
      if (wg == 0 && i < A.B && (r[e].ctx & (bt - 1)) != 0) open_block[e] = A.table[i * A.tstride + (r[e].ctx >> A.bt_log2)];
    }
    int first[kPer], last[kPer], kv[kPer], cls[kPer], tiles[kPer], chunks[kPer];
    uint32_t y[1] = {0};
    int64_t row = rows0 + at[0], fresh = fresh0 + at[1];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int i = base + tid * kPer + e, want = r[e].need - r[e].have;
      first[e] = (int)min(row, (int64_t)A.T);
      row += r[e].add;
      last[e] = (int)min(row, (int64_t)A.T);
      const int got = (int)max(min((int64_t)A.nfree - fresh, (int64_t)want), (int64_t)0);
      s_fresh[tid * kPer + e] = (int)min(fresh, (int64_t)0x7fffffff);
      fresh += want;
      kv[e] = (int)min(min((int64_t)r[e].ctx + (last[e] - first[e]), (int64_t)cap), (int64_t)(r[e].have + got) << A.bt_log2);
      const int rows = i < A.B ? (last[e] - first[e]) * A.G : 0;
      cls[e] = class_of(r[e].add * A.G, many);  // as the chunk was chosen
      tiles[e] = tiles_of(rows, cls[e]);
      const int even = even_chunk(kv[e], cls[e] == 2 ? chunk_wide : chunk);
      chunks[e] = max((kv[e] + even - 1) / even, 1);
      if (chunks[e] > 1) y[0] += tiles[e] * chunks[e] * (rows_of_class(cls[e]) / kUnit);
      if (wg == 0 && i < A.B) {
        A.q_indptr[i] = first[e];
        A.kv_len[i] = kv[e];
        if (r[e].bad) flags |= LORA_KV_FLAG_LENGTH;
        if (row > A.T || A.add[i] > A.T) flags |= LORA_KV_FLAG_TOKENS;
        if (want > 0 && fresh > A.nfree) flags |= LORA_KV_FLAG_FREE_LIST;
      }
    }
    int64_t at2[1], sum2[1], at3[3], sum3[3];
    block_scan<kWavesB, 1>(y, at2, sum2, s_b);
    int64_t part = parts0 + at2[0];
    uint32_t z[3] = {0, 0, 0};
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int k = tid * kPer + e;
      s_part[k] = -1;
      if (chunks[e] > 1) {
        const int64_t need = (int64_t)tiles[e] * chunks[e] * (rows_of_class(cls[e]) / kUnit);
        if (part + need <= A.part_cap) s_part[k] = (int)part;
        else chunks[e] = 1;
        part += need;
      }
      z[cls[e]] += tiles[e] * chunks[e];
    }
    block_scan<kWavesB, 3>(z, at3, sum3, s_c);
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int k = tid * kPer + e;
      if (last[e] > first[e] && (unsigned)open_block[e] >= (unsigned)A.blocks) flags |= LORA_KV_FLAG_BLOCK_RANGE;
      s_row[k] = first[e];
      s_ctx[k] = r[e].ctx;
      s_kv[k] = kv[e];
      s_rows[k] = (last[e] - first[e]) * A.G;
      s_chunks[k] = chunks[e];
#pragma unroll
      for (int c = 0; c < kClasses; ++c) {
        s_item[c][k] = (int)(items0[c] + at3[c]);
        at3[c] += cls[e] == c ? tiles[e] * chunks[e] : 0;
      }
    }
    __syncthreads();
    const int n = min(kTurn, A.B - base);
    const int row0 = (int)min(rows0, (int64_t)A.T), row1 = (int)min(rows0 + sum[0], (int64_t)A.T);
    for (int t = row0 + wg * kThreads + tid; t < row1; t += nwg * kThreads) {
      const int k = bisect(s_row, n, t);
      const int64_t pos = (int64_t)s_ctx[k] + (t - s_row[k]);
      int slot = -1;
      if (pos < cap) {
        const int b = (int)(pos >> A.bt_log2), have = (int)(((int64_t)s_ctx[k] + bt - 1) >> A.bt_log2);
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
    const int64_t fresh1 = min(fresh0 + sum[1], (int64_t)0x7fffffff);
    for (int64_t f = fresh0 + wg * kThreads + tid; f < fresh1; f += nwg * kThreads) {
      const int k = bisect(s_fresh, n, (int)f);
      const int b = (int)(((int64_t)s_ctx[k] + bt - 1) >> A.bt_log2) + (int)(f - s_fresh[k]);
      int id = f < A.nfree ? A.free_blocks[f] : -1;
      if ((unsigned)id >= (unsigned)A.blocks) id = -1;
      A.table[(base + k) * A.tstride + b] = id;
    }
    if (wg == 0) {
      for (int64_t f = fresh0 + tid; f < min(fresh1, (int64_t)A.nfree); f += kThreads)
        if ((unsigned)A.free_blocks[f] >= (unsigned)A.blocks) flags |= LORA_KV_FLAG_BLOCK_RANGE;
    }
    for (int c = 0; c < kClasses; ++c) {
      const int units = rows_of_class(c) / kUnit;
      for (int w = (int)items0[c] + wg * kThreads + tid; w < min(items0[c] + sum3[c], (int64_t)A.item_cap); w += nwg * kThreads) {
        const int k = bisect(s_item[c], n, w);
        const int local = w - s_item[c][k], tile = local / s_chunks[k], ci = local - tile * s_chunks[k];
        int part = s_part[k];
        if (part >= 0) {
          part += tile * s_chunks[k] * units;
          if (ci == 0)
            for (int h = 0; h < A.hkv * units; ++h) A.arrive[(int64_t)part * A.hkv + h] = 0;
        }
        int4* to = A.items + 2 * ((int64_t)c * A.item_cap + w);
        to[0] = make_int4(base + k, tile * rows_of_class(c), ci, part);
        to[1] = make_int4(s_row[k], s_rows[k], s_ctx[k], s_kv[k]);
      }
    }
    rows0 += sum[0];
    fresh0 += sum[1];
    parts0 += sum2[0];
    for (int c = 0; c < kClasses; ++c) items0[c] += sum3[c];
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
    if ((tid & 63) == 0) s_a[tid >> 6][0] = (uint32_t)flags;
    __syncthreads();
    if (tid < kNumCounts) {
      int all = 0;
      for (int w = 0; w < kWavesB; ++w) all |= (int)s_a[w][0];
      int v = 0;
      if (tid == kCountTokens) v = used;
      if (tid == kCountNewBlocks) v = (int)min(fresh0, (int64_t)0x7fffffff);
      if (tid == kCountItems) v = (int)items0[0];
      if (tid == kCountParts) v = (int)min(parts0, (int64_t)0x7fffffff);
      if (tid == kCountMid) v = (int)items0[1];
      if (tid == kCountWide) v = (int)items0[2];
      if (tid == kCountChunk) v = chunk;
      if (tid == kCountChunkWide) v = chunk_wide;
      if (tid == kCountFlags) v = all;
      if (tid == kCountB) v = A.B;
      if (tid == kCountT) v = A.T;
      if (tid == kCountCheck) v = check_word(A.B, A.T, (int)items0[0], (int)items0[1], (int)items0[2], (int)min(parts0, (int64_t)0x7fffffff));
      if (tid == kCountBuild) v = (int)(builds + 1);
      A.counts[tid] = v;
    }
    if (tid == kThreads - 1) A.q_indptr[A.B] = used;
  }
}

}  // namespace

hipError_t launch_build(const BuildArgs& A, hipStream_t s) {
  // a work-group per 256 rows or requests, up to 512, each of which repeats
  // the sums over the requests: in one turn of 256, or turns of 1024, two per
  // thread (1024 requests: 10.5 us; 256 threads with four each 11.0, 1024 threads
  // with one each spill, 22)
  const int grid = min_i(max_i(ceil_div_i(max_i(A.T, A.B), 256), 1), 512);
  if (A.B <= 256) build_kernel<256, 1><<<grid, 256, 0, s>>>(A);
  else build_kernel<512, 2><<<ceil_div_i(grid, 2), 512, 0, s>>>(A);
  return hipGetLastError();
}

}  // namespace kv
}  // namespace lora
