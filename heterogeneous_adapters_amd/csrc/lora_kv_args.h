// Kernel arguments and launchers of the attention operators (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lora_kv_plan.h"

namespace lora {
namespace kv {

// A list of heads as the kernels see it (strides in elements).
struct Rows {
  void* p;
  int64_t ts, hs;
  int32_t heads;
};

struct Cache {
  uint8_t* base;
  int64_t stride;  // bytes between blocks
  int32_t blocks;
  int32_t bt_log2;  // log2 of a block's tokens
  int32_t heads;
  int32_t nc;  // head_dim / 32
};

struct BuildArgs {
  const int32_t* ctx;
  const int32_t* add;
  int32_t* table;
  const int32_t* free_blocks;
  int64_t tstride;
  int32_t B, T, width, nfree, blocks, bt_log2, hkv, G, item_cap, part_cap;
  int32_t *q_indptr, *kv_len, *token_seq, *positions, *slots, *counts;
  int4* items;
  int32_t* arrive;
};

struct RopeArgs {
  Rows q, qo, k, ko, v;
  const int32_t* pos;
  const int32_t* slots;
  const double* freq;
  double fscale;
  int32_t T, D, rot, interleaved;
  int32_t q_groups;  // work-groups per token tile of the rotation role
  int32_t q_heads_per_group;
  int32_t rot_blocks;  // work-groups of the rotation role, before those of the cache role
  int32_t kv_groups;   // work-groups per token tile of the cache role
  int32_t kv_heads_per_group;
  Cache cache;
  int32_t* flags;
};

struct AttendArgs {
  static constexpr bool kShared = false;
  Rows q, o;
  int32_t* counts;
  const int4* items;
  int32_t* arrive;
  const int32_t* table;
  int64_t tstride;
  int32_t width, T, B, G, item_cap;
  Cache cache;
  float scale_log2e;
  float* part;
};

struct ShareArgs {
  const int32_t *group_indptr, *shared_len;
  int32_t groups, B, T, G, hkv, prefix_class, item_cap, row_cap;
  const int32_t *q_indptr, *kv_len, *positions;
  int32_t *counts, *share, *cut, *first;
  int4 *group_parts, *seq_parts, *items;
};

// Items of one list of a shared plan, or of lists 0 and 1 in one launch; the
// join of their results.
struct SharedArgs : AttendArgs {
  static constexpr bool kShared = true;
  const int32_t* share;
  const int4* seq_parts;
  const int32_t* token_seq;
  float* part_ml;
  int32_t groups, row_cap, list;
  int32_t first_items;  // of list 0 in the launch of list 1
};

struct PromptArgs {
  Rows q, k, v, o;
  const int32_t* indptr;
  int32_t B, T, G;
  float scale_log2e;
};

hipError_t launch_build(const BuildArgs& A, hipStream_t s);
hipError_t launch_rope(const RopeArgs& A, int dtype, int blocks, hipStream_t s);
hipError_t launch_gather(const RopeArgs& A, int dtype, int blocks, hipStream_t s);
hipError_t launch_attend(const AttendArgs& A, int dtype, bool many, hipStream_t s);
hipError_t launch_share(const ShareArgs& A, hipStream_t s);
hipError_t launch_shared(const SharedArgs& A, int dtype, int prefix_class, bool many, hipStream_t s);
hipError_t launch_prompt(const PromptArgs& A, int dtype, int D, hipStream_t s);

}  // namespace kv
}  // namespace lora
