// Kernel arguments and launchers of the beam search operators (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lora_beam.h"
#include "lora_kv_host.h"

namespace lora {
namespace beam {

constexpr int kChunk = 2048;  // logits that a wave holds at once, 32 per lane
// Waves that a selection's rows are cut into, where the vocabulary has as many
// chunks: a wave's first chunk fills its list, so fewer waves insert less, until
// too few are left to hide latency (64 rows x 8 of 128000 bf16 logits and 128 x 16
// of 32000, one form of the kernel: 4096 waves 34 and 40 us, 8192 39 and 46).
constexpr int kTargetWaves = 4096;

// Chunks of a row: its first logit may lie anywhere in a 16-byte vector.
inline int64_t row_chunks(int64_t vocab) { return (vocab + 7 + kChunk - 1) / kChunk; }
inline int64_t row_waves(int64_t rows, int64_t vocab) {
  const int64_t want = (kTargetWaves + rows - 1) / rows, chunks = row_chunks(vocab);
  const int64_t each = (chunks + want - 1) / want;  // chunks of a wave
  return (chunks + each - 1) / each;
}

struct SelectArgs {
  const void* logits;
  int64_t stride;
  int32_t requests, beams, vocab, waves, chunks;  // waves per row, chunks per wave
  const float* score;
  const int32_t *length, *done;
  double penalty;
  int32_t eos;
  int32_t *parent, *token;
  float* score_out;
  int32_t *length_out, *done_out;
  int32_t* flags;
  uint64_t* keys;  // [row][wave][beams]
  double* sums;    // [row][wave] {exponent, sum}
};

struct ReorderArgs {
  const int32_t *parent, *kv_len, *table, *free_blocks;
  int32_t *new_table, *new_len;
  int64_t stride, new_stride;
  int32_t requests, beams, width, num_free, num_blocks, bt_log2, max_rows;
  int32_t *source, *target, *tokens, *freed, *counts, *scratch;  // scratch: [requests] {copies, freed}
};

constexpr int kCopyLayers = 64;  // caches of one launch
struct CopyArgs {
  uint8_t* base[kCopyLayers];
  int64_t stride;
  int32_t layers, num_blocks, units, heads, record, max_rows;  // units of a block, bytes of a unit
  const int32_t *source, *target, *tokens, *counts;
};

hipError_t launch_select(const SelectArgs& A, int dtype, hipStream_t s);
hipError_t launch_reorder(const ReorderArgs& A, hipStream_t s);
hipError_t launch_copy(const CopyArgs& A, hipStream_t s);

}  // namespace beam
}  // namespace lora
