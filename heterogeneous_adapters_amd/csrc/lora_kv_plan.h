// Layout of a batch buffer of the attention operators, shared by the host and
// the kernels (internal).
#pragma once

#include <stdint.h>

namespace lora {
namespace kv {

constexpr int kUnit = 16;        // tokens per cache record, rows per attention tile
constexpr int kTile = 32;        // cached tokens per step of a wave
constexpr int kChunkStep = 256;  // chunks are multiples of this: two steps of each of 4 waves
// Smallest chunk of cached tokens per work item (one request of 32768 tokens:
// 22.5 us with 1024, 25.6 with 512, 24.6 with 2048; other steps within 2 %).
constexpr int kMinChunk = 1024;
// Work items (over all kv heads) that the plan aims for.
constexpr int kTargetItems = 1024;
// The same for items of 128 rows, two of which fill a compute unit and whose
// parts cost 64 KB each to join.
constexpr int kTargetWide = 512;

constexpr int kCountTokens = 0, kCountNewBlocks = 1, kCountItems = 2, kCountParts = 3, kCountChunk = 4,
              kCountMid = 5, kCountWide = 6, kCountChunkWide = 7, kCountFlags = 8, kCountB = 9, kCountT = 10, kCountCheck = 11,
              kNumCounts = 16;

// Work items by class of their request's rows (new tokens x query heads per
// kv head): up to 16 rows, one matrix tile; up to 64, two tiles on the same
// converted keys; more, 128 rows that share the conversion through LDS.  The
// last two only where a step brings more tokens than requests (what the host
// knows of it, so that a decode step, of 12 us or more, launches one kernel; a
// launch without items takes 4.5 us of the mixed step).  Chunks of 512 over 4488 tokens, 32
// heads on 8 of 128, among as many idle requests as tokens: four of them 311 us
// in 16-row items, 201 with T padded past B; one 89 and 99.
constexpr int kClasses = 3;
constexpr int kMidRows = 32, kWideRows = 128, kMidMost = 64;
#if defined(__HIPCC__)
#define LORA_KV_HD __host__ __device__
#else
#define LORA_KV_HD
#endif
LORA_KV_HD inline bool many_rows(int32_t T, int32_t B) { return T > B; }
LORA_KV_HD inline int rows_of_class(int c) { return c == 0 ? kUnit : c == 1 ? kMidRows : kWideRows; }

LORA_KV_HD inline int32_t check_word(int32_t B, int32_t T, int32_t items, int32_t mid, int32_t wide, int32_t parts) {
  uint32_t h = 0x4b56u;
  h = (h ^ (uint32_t)B) * 0x9e3779b1u;
  h = (h ^ (uint32_t)T) * 0x85ebca77u;
  h = (h ^ (uint32_t)items) * 0xc2b2ae3du;
  h = (h ^ (uint32_t)mid) * 0x165667b1u;
  h = (h ^ (uint32_t)wide) * 0x9e3779b1u;
  h = (h ^ (uint32_t)parts) * 0x27d4eb2fu;
  return (int32_t)(h ^ (h >> 15));
}

// Tokens per item of a request with kv cached ones: as many items as the
// step's chunk makes of it, of even length.
LORA_KV_HD inline int even_chunk(int kv, int chunk) {
  if (kv <= chunk) return chunk;
  const int n = (kv + chunk - 1) / chunk, even = (kv + n - 1) / n;
  return (even + kChunkStep - 1) / kChunkStep * kChunkStep;
}

// Most work items of a class: sum of tiles_i * ceil(kv_i / chunk) <=
// sum(tiles_i kv_i) / chunk + sum(tiles_i), the first term at most
// kTargetItems / hkv by the choice of the chunk, tiles_i <= new_i G / 16 + 1.
inline int64_t item_cap(int64_t T, int64_t B, int64_t hkv, int64_t G) {
  return kTargetItems / hkv + 1 + T * G / kUnit + 1 + B;
}
// The same for one class of a step with T tokens and B requests: its launch's
// grid (a work-group without an item costs a launch slot: 9.5 us for 5768), at
// most item_cap of any batch that holds the step.  Requests of class 1 have two
// tiles at most, and more than 16 rows for each but the one that T cuts short.
inline int64_t class_cap(int c, int64_t T, int64_t B, int64_t hkv, int64_t G) {
  const int64_t split = kTargetItems / hkv + 1;
  if (c == 0) return T > B ? split + B : item_cap(T, B, hkv, G);
  if (c == 1) {
    const int64_t by_seqs = (kMidMost / kMidRows) * B, by_rows = T * G / kUnit + 1;
    return split + (by_seqs < by_rows ? by_seqs : by_rows);
  }
  return split + T * G / kWideRows + B;
}
// Room for partial results (16 rows of one chunk each).  A decode step needs
// at most 2 (kTargetItems / hkv + 1) of them; requests of many rows whose
// parts find no room are not split.
inline int64_t part_cap(int64_t hkv) { return 8 * (kTargetItems / hkv + 1); }

// Last of `rows` rows from `first` on, of `len`; -1 where there are none, so that
// `key <= last_row` and `row <= last_row` hold for no key and no row.
LORA_KV_HD inline int last_row(int first, int rows, int len) {
  return first >= len ? -1 : (first + rows < len ? first + rows : len) - 1;
}

// An item is two int4: {request, first row, chunk, first part of the tile or
// -1 (not split)} and {first token row, rows of the request, position of its
// first token, cached tokens}.

}  // namespace kv
}  // namespace lora
