// Sums over a work-group and searches in them, for the plans' builds (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lora {
namespace kv {

// Inclusive sums over a wave: within rows of 16 lanes, then from row to row.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_add(uint32_t x) {
  return x + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
  x = dpp_add<0x111, 0xf>(x);  // row_shr:1
  x = dpp_add<0x112, 0xf>(x);
  x = dpp_add<0x114, 0xf>(x);
  x = dpp_add<0x118, 0xf>(x);
  x = dpp_add<0x142, 0xa>(x);  // lane 15 of rows 0, 2 into rows 1, 3
  return dpp_add<0x143, 0xc>(x);  // lane 31 into rows 2, 3
}

// Exclusive sums of N values over the work-group (32 bits within a wave) and
// their totals.
template <int kWavesB, int N>
__device__ __forceinline__ void block_scan(const uint32_t (&x)[N], int64_t (&before)[N], int64_t (&total)[N],
                                           uint32_t (*scratch)[8]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t incl[N];
#pragma unroll
  for (int v = 0; v < N; ++v) {
    incl[v] = wave_scan(x[v]);
    if (lane == 63) scratch[wave][v] = incl[v];
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < N; ++v) {
    before[v] = incl[v] - x[v];
    total[v] = 0;
#pragma unroll
    for (int w = 0; w < kWavesB; ++w) {
      if (w < wave) before[v] += scratch[w][v];
      total[v] += scratch[w][v];
    }
  }
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

}  // namespace kv
}  // namespace lora
