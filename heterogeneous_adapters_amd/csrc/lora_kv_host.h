// Host arithmetic shared by the launchers of the attention operators.
#pragma once

#include <stdint.h>

#include "lora_kv.h"
#include "lora_kv_args.h"

namespace lora {
namespace kv {

inline int ceil_div_i(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
inline int max_i(int a, int b) { return a > b ? a : b; }
inline int min_i(int a, int b) { return a < b ? a : b; }

}  // namespace kv
}  // namespace lora
