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
              kCountBuild = 12,  // builds of the buffer so far, by which a shared plan knows its own
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
constexpr int kPrefixRows = 256;  // class 3, of shared plans' prefixes only
LORA_KV_HD inline int rows_of_class(int c) { return c == 0 ? kUnit : c == 1 ? kMidRows : c == 2 ? kWideRows : kPrefixRows; }

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

// ---- shared plans: what the requests of a group have in common is attended to
// by all of their rows together, the rest by each request, and both leave
// partial results that a last launch joins.
constexpr int kLists = 4;      // a shared plan's lists: 0 the groups' prefixes, 1 + c the requests' rests of class c
constexpr int kShareItem = 3;  // int4 per item
LORA_KV_HD inline int min_prefix_chunk(int cls) { return cls == 0 ? 512 : 256; }  // smallest chunk of a prefix
// counts of a shared plan: kLists item counts, then
constexpr int kShareRows = 4, kShareGroups = 5, kShareB = 6, kShareT = 7, kShareCheck = 8, kShareBuild = 9, kNumShare = 16;

// Rows of a prefix's item, as a class, by the groups' average (the host's
// arithmetic; sizes of single groups and prefixes are known to the device
// only).  Few rows: items of 16, which go with the requests' rests in one launch
// and read the prefix again from the caches for every 16 rows.  More: class 3, or
// 2 where 256 rows' registers do not suffice.  Attention alone in us, one group,
// 32 query heads on 8, items of 16 rows / else:
//   dims  rows  behind 1000     2000     4000     8000     16384 tokens
//    128   240      17 / 29  20 / 31  26 / 35  31 / 40   44 /  46
//          320      18 / 30  22 / 34  29 / 38  37 / 43   60 /  57
//          512      22 / 34  28 / 38  34 / 42  47 / 48   74 /  62
//         1024      33 / 42  39 / 46  51 / 53  78 / 66  131 /  96
//    256   100      21 / 33           33 / 39            65 /  62
//          200      26 / 36           50 / 45           112 /  89
//          400      41 / 47           71 / 74           160 / 131
// Where it turns depends on the prefix as well, which the rule does not see.  It
// goes by the long ones, behind which the other form costs most: 321 to 1024
// rows behind 4000 tokens or fewer take 1 to 12 us longer than in items of 16.
constexpr int kFewRows = 320, kFewRowsFar = 128;  // up to 128 dims, and past them
LORA_KV_HD inline int prefix_class(int64_t T, int64_t G, int64_t groups, int head_dim) {
  return T * G <= (head_dim > 128 ? kFewRowsFar : kFewRows) * groups ? 0 : head_dim > 128 ? 2 : 3;
}
// Items (over all kv heads) that a plan splits prefixes into: as many
// work-groups as the chip holds of a class's kernel at once.
LORA_KV_HD inline int prefix_items(int cls) { return cls == 0 ? kTargetItems : cls == 2 ? 512 : 256; }
// Most items of the prefix list: sum of tiles_g ceil(prefix_g / chunk) <=
// prefix_items / hkv + sum of tiles_g by the choice of the chunk.
LORA_KV_HD inline int64_t prefix_cap(int cls, int64_t T, int64_t groups, int64_t hkv, int64_t G) {
  return prefix_items(cls) / hkv + 1 + T * G / rows_of_class(cls) + 1 + groups;
}
LORA_KV_HD inline int64_t share_item_cap(int64_t T, int64_t B, int64_t groups, int64_t hkv, int64_t G) {
  return item_cap(T, B, hkv, G) + groups;
}
// Most rows of partial results: a list's rows once, and as many again as the
// rows of the items that its chunks add.
LORA_KV_HD inline int64_t share_row_cap(int64_t T, int64_t hkv, int64_t G) {
  return 2 * T * G + 65536 / hkv + kPrefixRows +  // prefixes of class 2: 128 x 512, of class 3: 256 x 256
         kMidRows * (kTargetItems / hkv + 1) +
         kWideRows * (kTargetWide / hkv + 1);
}
LORA_KV_HD inline int32_t share_word(const int32_t* share) {
  return check_word(share[kShareB], share[kShareT], share[0] + 7 * share[kShareGroups], share[1], share[2] + 5 * share[3], share[kShareRows]);
}

}  // namespace kv
}  // namespace lora
