// Layout of a batch buffer of the attention operators, shared by the host and
// the kernels (internal).
#pragma once

#include <stdint.h>

namespace lora {
namespace kv {

constexpr int kUnit = 16;        // tokens per cache record, rows per attention tile
constexpr int kTile = 32;        // cached tokens per step of a wave
constexpr int kChunkStep = 256;  // chunks are multiples of this: a step of each of 8 waves
constexpr int kMinChunk = 1024;   // smallest chunk of cached tokens per work item
// Work items (over all kv heads) that the plan aims for.
constexpr int kTargetItems = 1024;

constexpr int kCountTokens = 0, kCountNewBlocks = 1, kCountItems = 2, kCountParts = 3, kCountChunk = 4,
              kCountWide = 5, kCountFlags = 8, kCountB = 9, kCountT = 10, kCountCheck = 11, kNumCounts = 16;

#if defined(__HIPCC__)
__host__ __device__
#endif
inline int32_t check_word(int32_t B, int32_t T, int32_t items, int32_t wide, int32_t parts) {
  uint32_t h = 0x4b56u;
  h = (h ^ (uint32_t)B) * 0x9e3779b1u;
  h = (h ^ (uint32_t)T) * 0x85ebca77u;
  h = (h ^ (uint32_t)items) * 0xc2b2ae3du;
  h = (h ^ (uint32_t)wide) * 0x165667b1u;
  h = (h ^ (uint32_t)parts) * 0x27d4eb2fu;
  return (int32_t)(h ^ (h >> 15));
}

// Requests of more than 16 rows (new tokens x query heads per kv head) take
// tiles of 32 rows, in a list of their own, where a step brings more tokens
// than requests (what the host knows of it).
#if defined(__HIPCC__)
__host__ __device__
#endif
inline bool wide_step(int32_t T, int32_t B) { return T > B; }

// Most work items of a step, in either list: sum of tiles_i * ceil(kv_i /
// chunk) <= sum(tiles_i kv_i) / chunk + sum(tiles_i), the first term at most
// kTargetItems / hkv by the choice of the chunk, tiles_i <= new_i G / 16 + 1.
inline int64_t item_cap(int64_t T, int64_t B, int64_t hkv, int64_t G) {
  return kTargetItems / hkv + 1 + T * G / kUnit + 1 + B;
}
// Most parts (16 rows each) of items that share their tile with others:
// ceil(kv / chunk) < 2 kv / chunk of them for each 16 rows, and tiles of 32
// rows have at most half as many 16 rows again as the choice of the chunk
// counts.
inline int64_t part_cap(int64_t hkv) { return 3 * (kTargetItems / hkv + 1); }

}  // namespace kv
}  // namespace lora
