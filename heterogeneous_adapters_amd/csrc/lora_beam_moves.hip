// lora_beam_reorder and lora_beam_copy: block tables of a search's next step.
//
// Integer work on the tables of one step (rows x blocks, a few hundred
// kilobytes at most), bound by latency.  A request's beams share blocks at the
// same column only, so what a column still holds is decided within the
// request, without reference counts; two launches, because where a request's
// entries of the lists begin depends on the requests before it (one for one
// request).  The copies are bound by HBM.
//
// Measured on MI355X: one request of 4 beams 6.1 us, and 3.5 for the copies in 4
// layers; 96 requests of 8 beams, up to 2300 tokens in blocks of 64, 5.9 + 10.4, and
// 13.4 for 88 MB of copies (read and written).  With loops over 32 rows whatever
// the request's, 10 and 10 + 13 us.  The loops compare every two rows of a
// request in straight code, whose masks spill to vector registers: 118 scalars
// with 16 beams, 245 with 32 (48 requests of 16 beams 29 us for both launches, 24 of
// 32 70, one of 32 42).
#include "lora_beam_args.h"
#include "lora_kv_dev.h"

namespace lora {
namespace beam {

using namespace lora::kv;

namespace {

constexpr int kMost = LORA_BEAM_MAX;
constexpr int kThreads = 256;

// Sum over the work-group, and what the threads before this one add to it.
__device__ __forceinline__ int block_sum(int x, int& before, int* scratch) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int incl = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(incl, d);
    if (lane >= d) incl += up;
  }
  __syncthreads();
  if (lane == 63) scratch[wave] = incl;
  __syncthreads();
  int all = 0;
  before = incl - x;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    if (w < wave) before += scratch[w];
    all += scratch[w];
  }
  return all;
}

// EMIT: the second launch, which writes; the first counts, where there are
// several requests.  ROWS: at least as many as a request has beams.
template <bool EMIT, int ROWS>
__global__ __launch_bounds__(kThreads) void reorder_kernel(const ReorderArgs A) {
  __shared__ int s_parent[kMost], s_blocks[kMost], s_len[kMost], s_copy[kMost];  // by new row: parent (-1), blocks, copy's place or -1
  __shared__ int s_old[kMost];                                                   // blocks of the old rows
  __shared__ int s_sum[kThreads / 64], s_sum2[kThreads / 64], s_copies, s_flags;
  const int W = A.beams, b = blockIdx.x, row0 = b * W, tid = threadIdx.x, bt = 1 << A.bt_log2;
  int flags = 0;
  if (tid == 0) s_flags = 0;
  if (tid < W) {
    const int64_t cap = (int64_t)A.width << A.bt_log2;
    int p = A.parent[row0 + tid], len = A.kv_len[row0 + tid];
    if (len < 0 || len > cap) flags |= LORA_BEAM_FLAG_LENGTH;
    len = (int)min((int64_t)max(len, 0), cap);
    s_old[tid] = (len + bt - 1) >> A.bt_log2;
    if (p != -1 && (p < row0 || p >= row0 + W)) flags |= LORA_BEAM_FLAG_PARENT, p = -1;
    int n = p < 0 ? 0 : A.kv_len[p];
    n = (int)min((int64_t)max(n, 0), cap);
    s_parent[tid] = p < 0 ? -1 : p - row0;
    s_len[tid] = n;
    s_blocks[tid] = (n + bt - 1) >> A.bt_log2;
  }
  __syncthreads();
  const int32_t* table = A.table + (int64_t)row0 * A.stride;
  // An open block that an earlier row keeps is copied: its parent's, or another
  // row's that holds the same (beams that begin on one prompt's last block).
  // One that is missing (-1) stays missing in every heir's row: a block of the
  // free list in its place would pass its last owner's tokens for the beam's.
  if (tid < 64) {
    const int p = tid < W ? s_parent[tid] : -1;
    const bool open = p >= 0 && (s_len[tid] & (bt - 1)) != 0;
    const int id = open ? table[p * A.stride + s_blocks[tid] - 1] : -1;
    const bool known = (unsigned)id < (unsigned)A.num_blocks, there = open && id != -1;
    if (open && !known) flags |= LORA_BEAM_FLAG_BLOCK_RANGE;
    bool again = false;
    for (int o = 0; o < W; ++o) {
      const int other = __shfl(open ? p : -1, o), other_id = __shfl(id, o);
      again = again || (there && o < tid && (other == p || (known && other_id == id)));
    }
    const uint64_t mask = __ballot(again);
    if (tid < W) s_copy[tid] = again ? __popcll(mask & ((1ull << tid) - 1)) : -1;
    if (tid == 0) s_copies = __popcll(mask);
  }
  __syncthreads();

  // where this request's entries of the lists begin
  int copies0 = 0, freed0 = 0;
  if (EMIT) {
    int x = 0, y = 0, unused;
    for (int i = tid; i < b; i += kThreads) x += A.scratch[2 * i], y += A.scratch[2 * i + 1];
    copies0 = block_sum(x, unused, s_sum);
    freed0 = block_sum(y, unused, s_sum2);
  }

  uint32_t parents = 0;  // old rows that go on
  for (int c = 0; c < W; ++c)
    if (s_parent[c] >= 0) parents |= 1u << s_parent[c];
  int freed = 0;
  for (int j0 = 0; j0 < A.width; j0 += kThreads) {
    const int j = j0 + tid;
    int32_t id[ROWS];
    uint32_t gone = 0;  // rows whose block here nobody holds, the first of those that share it
    if (j < A.width) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) id[r] = r < W && j < s_old[r] ? table[r * A.stride + j] : -1;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (r >= W || j >= s_old[r]) continue;
        if ((unsigned)id[r] >= (unsigned)A.num_blocks) {
          if (id[r] != -1) flags |= LORA_BEAM_FLAG_BLOCK_RANGE;
          continue;
        }
        bool out = true;
#pragma unroll
        for (int o = 0; o < ROWS; ++o) out = out && !(id[o] == id[r] && (o < r || (parents >> o & 1)));
        gone |= out ? 1u << r : 0;
      }
    }
    int before;
    const int all = block_sum(__popc(gone), before, s_sum);
    if (EMIT && j < A.width) {
      int to = freed0 + freed + before;
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
        if (gone >> r & 1) A.freed[to++] = id[r];
    }
    freed += all;
  }
  if (!EMIT) {
    if (tid == 0) A.scratch[2 * b] = s_copies, A.scratch[2 * b + 1] = freed;
    if (b == 0 && tid == 0) A.counts[LORA_BEAM_COUNT_FLAGS] = 0;
    return;
  }

  for (int c = 0; c < W; ++c) {
    const int p = s_parent[c], blocks = s_blocks[c];
    const int32_t* from = table + max(p, 0) * A.stride;
    int32_t* to = A.new_table + (int64_t)(row0 + c) * A.new_stride;
    for (int j = tid; j < A.width; j += kThreads) {
      int id = j < blocks ? from[j] : -1;
      if (s_copy[c] >= 0 && j == blocks - 1) {
        const int at = copies0 + s_copy[c], source = id;
        id = at < A.num_free ? A.free_blocks[at] : -1;
        if (at >= A.num_free) flags |= LORA_BEAM_FLAG_FREE_LIST;
        else if ((unsigned)id >= (unsigned)A.num_blocks) flags |= LORA_BEAM_FLAG_BLOCK_RANGE, id = -1;
        A.source[at] = source;
        A.target[at] = id;
        A.tokens[at] = s_len[c] & (bt - 1);
      }
      to[j] = id;
    }
    if (tid == 0) A.new_len[row0 + c] = s_len[c];
  }
  if (b == A.requests - 1) {  // the lists' ends
    const int copies = copies0 + s_copies;
    for (int i = copies + tid; i < A.max_rows; i += kThreads) A.source[i] = A.target[i] = A.tokens[i] = -1;
    if (tid == 0) A.counts[LORA_BEAM_COUNT_COPIES] = copies, A.counts[LORA_BEAM_COUNT_FREED] = freed0 + freed;
  }
  if (A.requests > 1) {
    if (flags) atomicOr(&A.counts[LORA_BEAM_COUNT_FLAGS], flags);
    return;
  }
  if (flags) atomicOr(&s_flags, flags);  // no launch before this one has cleared them
  __syncthreads();
  if (tid == 0) A.counts[LORA_BEAM_COUNT_FLAGS] = s_flags;
}

// No requests: empty lists.
__global__ __launch_bounds__(kThreads) void no_moves_kernel(const ReorderArgs A) {
  for (int i = threadIdx.x; i < A.max_rows; i += kThreads) A.source[i] = A.target[i] = A.tokens[i] = -1;
  if (threadIdx.x == 0)
    A.counts[LORA_BEAM_COUNT_COPIES] = A.counts[LORA_BEAM_COUNT_FREED] = A.counts[LORA_BEAM_COUNT_FLAGS] = 0;
}

// A wave per (copy, layer, kv head): the head's records of a block lie together.
// What has no source in the cache becomes zeros.
__global__ __launch_bounds__(256) void copy_kernel(const CopyArgs A) {
  const int lane = threadIdx.x & 63;
  const int copies = min(max(A.counts[LORA_BEAM_COUNT_COPIES], 0), A.max_rows);
  const int64_t tasks = (int64_t)copies * A.layers * A.heads, waves = (int64_t)gridDim.x * 4;
  for (int64_t task = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); task < tasks; task += waves) {
    const int h = (int)(task % A.heads), l = (int)(task / A.heads % A.layers), i = (int)(task / A.heads / A.layers);
    const int source = A.source[i], target = A.target[i], units = min((A.tokens[i] + kUnit - 1) / kUnit, A.units);
    if ((unsigned)target >= (unsigned)A.num_blocks) continue;
    const int64_t head = (int64_t)h * A.units * A.record;
    u32x4* to = reinterpret_cast<u32x4*>(A.base[l] + target * A.stride + head);
    const int n = units * A.record / 16;
    if ((unsigned)source >= (unsigned)A.num_blocks) {
      for (int k = lane; k < n; k += 64) to[k] = u32x4{0, 0, 0, 0};
      continue;
    }
    const u32x4* from = reinterpret_cast<const u32x4*>(A.base[l] + source * A.stride + head);
    for (int k = lane; k < n; k += 256) {
      u32x4 x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k + 64 * u < n) x[u] = from[k + 64 * u];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k + 64 * u < n) to[k + 64 * u] = x[u];
    }
  }
}

template <int ROWS>
hipError_t reorder(const ReorderArgs& A, hipStream_t s) {
  if (A.requests > 1) reorder_kernel<false, ROWS><<<A.requests, kThreads, 0, s>>>(A);
  reorder_kernel<true, ROWS><<<A.requests, kThreads, 0, s>>>(A);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_reorder(const ReorderArgs& A, hipStream_t s) {
  if (A.requests == 0) {
    no_moves_kernel<<<1, kThreads, 0, s>>>(A);
    return hipGetLastError();
  }
  if (A.beams <= 4) return reorder<4>(A, s);
  if (A.beams <= 8) return reorder<8>(A, s);
  if (A.beams <= 16) return reorder<16>(A, s);
  return reorder<32>(A, s);
}

hipError_t launch_copy(const CopyArgs& A, hipStream_t s) {
  const int64_t most = ((int64_t)A.max_rows * A.layers * A.heads + 3) / 4;
  copy_kernel<<<(unsigned)(most < 2048 ? most : 2048), 256, 0, s>>>(A);
  return hipGetLastError();
}

}  // namespace beam
}  // namespace lora
