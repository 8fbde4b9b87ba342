// Device helpers of the attention operators (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lora {
namespace kv {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ float bf_to_f(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
__device__ __forceinline__ uint16_t f_to_bf(float f) {
  __bf16 h = (__bf16)f;
  return __builtin_bit_cast(uint16_t, h);
}
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
  bf16x2 v;
  v[0] = (__bf16)lo;
  v[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, v);
}

// l plus the eight values of f: two per instruction, summed in fp32 (checked on
// gfx950: within 0.69 units in the last place, nearest in all but 20 of 65536
// draws).
__device__ __forceinline__ float add8(bf16x8 f, float l) {
  const bf16x2 one{(__bf16)1.0f, (__bf16)1.0f};
#pragma unroll
  for (int i = 0; i < 8; i += 2) l = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{f[i], f[i + 1]}, one, l, false);
  return l;
}

// Running maximum before any visible key: the lowest finite number, which no
// score in range is below.
constexpr float kNone = -3.402823466e38f;
// Rows keep their maximum until a score passes it by this much (a factor of
// 2^8 in p, without loss: p is scaled the same in the products and the sum).
constexpr float kSlack = 8.0f;
// p = exp2(s scale - m) is one fma from the exact product, while m is a rounded
// one: a factor common to the row, of up to 2^64 while m is below 2^30.  Past
// that it would leave fp32's range, so there the product is rounded as m was,
// and p of the largest score is 1.
constexpr float kFar = 1073741824.0f;
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) > kFar && m != kNone; }
__device__ __forceinline__ float far_exponent(float s, float scale, float m) {
#pragma clang fp contract(off)
  const float product = s * scale;
  return product - m;
}

// Element types: vectors of 16 bytes to and from fp32.
struct Bf16 {
  typedef uint16_t T;
  static constexpr int kEpv = 8;
};
struct F32 {
  typedef float T;
  static constexpr int kEpv = 4;
};
__device__ __forceinline__ float to_f(uint16_t h) { return bf_to_f(h); }
__device__ __forceinline__ float to_f(float f) { return f; }
__device__ __forceinline__ void from_f(uint16_t* p, float f) { *p = f_to_bf(f); }
__device__ __forceinline__ void from_f(float* p, float f) { *p = f; }
__device__ __forceinline__ float round_to(float f, Bf16) { return bf_to_f(f_to_bf(f)); }
__device__ __forceinline__ float round_to(float f, F32) { return f; }

__device__ __forceinline__ void unpack(u32x4 w, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(w[j] << 16);
    x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(u32x4 w, float (&x)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(w[j]);
}

// N (a multiple of the vector width) consecutive elements at a 16-byte
// aligned address.
template <int N>
__device__ __forceinline__ void load_n(const uint16_t* p, float (&x)[N]) {
  static_assert(N % 8 == 0, "vectors of 8");
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[i + 2 * j] = __uint_as_float(w[j] << 16);
      x[i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}
template <int N>
__device__ __forceinline__ void load_n(const float* p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const f4 w = *reinterpret_cast<const f4*>(p + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[i + j] = w[j];
  }
}
template <int N>
__device__ __forceinline__ void store_n(uint16_t* p, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_bf2(x[i + 2 * j], x[i + 2 * j + 1]);
    *reinterpret_cast<u32x4*>(p + i) = w;
  }
}
template <int N>
__device__ __forceinline__ void store_n(float* p, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    f4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = x[i + j];
    *reinterpret_cast<f4*>(p + i) = w;
  }
}

// s_waitcnt vmcnt(N) with the other counters left alone.
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// The scale of one cached group as the fp32 number whose exponent is scale
// byte `k` of a packed word.  v_cvt_scalef32_* use the exponent field alone
// (checked on gfx950: sign and fraction bits change nothing), so moving the
// byte to bits 30..23 is all that is needed.
template <int K>
__device__ __forceinline__ float scale_of(uint32_t w) {
  return __uint_as_float(K == 3 ? w >> 1 : w << (23 - 8 * K));
}

}  // namespace kv
}  // namespace lora
