// lora_rope, lora_kv_append, lora_kv_gather: rotary positions, K and V into
// the paged 4-bit cache, and back.
//
// Mathematics
//   angle  a = p f / (2 pi) turns, reduced to [-1/2, 1/2] in fp64: 53 bits
//          leave 2^-53 * p f / (2 pi) turns, 1e-10 at a million positions,
//          where fp32 would have lost the angle.  cos and sin of it in fp64,
//          once per (token, pair), shared by the heads of a work-group
//          through LDS.
//   K      rotated in fp64 and rounded once; Q in fp32 from the rounded cos
//          and sin (its 2^-24 disappears in the rounding to bf16).
//   codes  2^e = the smallest power of two with max|x| <= 7 * 2^e, read off
//          the bits of max|x|: fraction above 1.75 moves to the next power.
//          v_cvt_scalef32_pk_fp4_f32 divides by 2^e, rounds to nearest even
//          and saturates (checked on gfx950 at every border).
//
// One launch: work-groups of the rotation role walk (token, head, vector) of
// Q (and of K in lora_rope), those of the cache role (16 tokens, head, group
// of 32).  Both read and write each byte once; the bound is HBM.
#include "lora_kv_dev.h"
#include "lora_kv_host.h"

namespace lora {
namespace kv {

namespace {

constexpr int kThreads = 256;
constexpr int kRotTokens = 4;     // tokens per work-group of the rotation role
constexpr int kCacheTokens = 16;  // tokens per work-group of the cache role
constexpr int kMaxPairs = LORA_KV_MAX_HEAD_DIM / 2;

__device__ __forceinline__ double2 angle(const RopeArgs& A, int pos, int pair) {
  const double turns = (double)pos * A.freq[pair] * 0.15915494309189533577;
  double s, c;
  sincospi(2.0 * (turns - rint(turns)), &s, &c);
  return make_double2(c * A.fscale, s * A.fscale);
}

// ------------------------------------------------------------ rotation role
// V: arithmetic type.  One task = one vector of pairs, or one vector of dims
// behind rot_dim (copied when out of place).
template <class E, class V, class V2>
__device__ __forceinline__ void rotate_heads(const RopeArgs& A, const Rows& in, const Rows& out, int t0, int nt, int h0,
                                             int nh, const V2* cs, int cs_stride) {
  typedef typename E::T T;
  constexpr int EPV = E::kEpv;
  const int half = A.rot >> 1;
  const bool copy = in.p != out.p;
  const bool wide = A.interleaved ? A.rot % EPV == 0 : half % EPV == 0;
  const int pair_tasks = wide ? (A.interleaved ? A.rot / EPV : half / EPV) : half;
  const int tail = copy ? A.D - A.rot : 0;
  const bool tail_wide = A.rot % EPV == 0;
  const int per_head = pair_tasks + (tail_wide ? tail / EPV : tail);
  const int total = nt * nh * per_head;
  for (int idx = threadIdx.x; idx < total; idx += kThreads) {
    const int th = idx / per_head, task = idx - th * per_head;
    const int tl = th / nh, h = h0 + th - tl * nh, t = t0 + tl;
    if (A.pos[t] < 0) continue;
    const T* x = static_cast<const T*>(in.p) + t * in.ts + h * in.hs;
    T* y = static_cast<T*>(out.p) + t * out.ts + h * out.hs;
    const V2* cst = cs + tl * cs_stride;
    if (task >= pair_tasks) {
      if (tail_wide) {
        const int d = A.rot + (task - pair_tasks) * EPV;
        *reinterpret_cast<u32x4*>(y + d) = *reinterpret_cast<const u32x4*>(x + d);
      } else {
        const int d = A.rot + task - pair_tasks;
        y[d] = x[d];
      }
    } else if (!wide) {
      const int d0 = A.interleaved ? 2 * task : task, d1 = A.interleaved ? d0 + 1 : task + half;
      const V a = to_f(x[d0]), b = to_f(x[d1]);
      from_f(y + d0, (float)(a * cst[task].x - b * cst[task].y));
      from_f(y + d1, (float)(b * cst[task].x + a * cst[task].y));
    } else if (A.interleaved) {
      const int d = task * EPV;
      float a[EPV], r[EPV];
      load_n<EPV>(x + d, a);
#pragma unroll
      for (int i = 0; i < EPV / 2; ++i) {
        const V2 w = cst[d / 2 + i];
        const V u = a[2 * i], v = a[2 * i + 1];
        r[2 * i] = (float)(u * w.x - v * w.y);
        r[2 * i + 1] = (float)(v * w.x + u * w.y);
      }
      store_n<EPV>(y + d, r);
    } else {
      const int d = task * EPV;
      float a[EPV], b[EPV], r[EPV], s[EPV];
      load_n<EPV>(x + d, a);
      load_n<EPV>(x + d + half, b);
#pragma unroll
      for (int i = 0; i < EPV; ++i) {
        const V2 w = cst[d + i];
        const V u = a[i], v = b[i];
        r[i] = (float)(u * w.x - v * w.y);
        s[i] = (float)(v * w.x + u * w.y);
      }
      store_n<EPV>(y + d, r);
      store_n<EPV>(y + d + half, s);
    }
  }
}

template <class E>
__device__ __forceinline__ void rotate_role(const RopeArgs& A, int block, double2* lds) {
  float2* lf = reinterpret_cast<float2*>(lds + kRotTokens * kMaxPairs);
  const int half = A.rot >> 1;
  const int t0 = block / A.q_groups * kRotTokens, g = block % A.q_groups;
  const int nt = min(kRotTokens, A.T - t0);
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int tl = i / half, pair = i - tl * half, p = A.pos[t0 + tl];
    if (p < 0) continue;
    const double2 w = angle(A, p, pair);
    lds[tl * half + pair] = w;
    lf[tl * half + pair] = make_float2((float)w.x, (float)w.y);
  }
  __syncthreads();
  // heads of q, then of k
  const int lo = g * A.q_heads_per_group, hi = min(lo + A.q_heads_per_group, A.qo.heads + A.ko.heads);
  const int nq = min(hi, A.qo.heads) - min(lo, A.qo.heads), nk = hi - lo - nq;
  if (nq > 0) rotate_heads<E, float>(A, A.q, A.qo, t0, nt, lo, nq, lf, half);
  if (nk > 0) rotate_heads<E, double>(A, A.k, A.ko, t0, nt, max(lo - A.qo.heads, 0), nk, lds, half);
}

// --------------------------------------------------------------- cache role
// 32 dims of one head as rounded, rotated values.
template <class E, bool ROPE>
__device__ __forceinline__ void load_group(const RopeArgs& A, const typename E::T* x, int c, const double2* cs,
                                           float (&f)[32]) {
  load_n<32>(x + 32 * c, f);
  if constexpr (!ROPE) return;
  const int half = A.rot >> 1, d0 = 32 * c;
  if (d0 >= A.rot) return;
  if (A.interleaved) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (d0 + 2 * i < A.rot) {
        const double2 w = cs[d0 / 2 + i];
        const double u = f[2 * i], v = f[2 * i + 1];
        f[2 * i] = round_to((float)(u * w.x - v * w.y), E{});
        f[2 * i + 1] = round_to((float)(v * w.x + u * w.y), E{});
      }
    }
  } else if (half % 8 == 0) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int d = d0 + 8 * v;
      if (d >= A.rot) continue;
      const bool low = d < half;
      const int pair = low ? d : d - half;
      float o[8];
      load_n<8>(x + (low ? d + half : d - half), o);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double2 w = cs[pair + i];
        const double a = f[8 * v + i], b = o[i];
        f[8 * v + i] = round_to((float)(low ? a * w.x - b * w.y : a * w.x + b * w.y), E{});
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int d = d0 + i;
      if (d >= A.rot) continue;
      const bool low = d < half;
      const double2 w = cs[low ? d : d - half];
      const double a = f[i], b = to_f(x[low ? d + half : d - half]);
      f[i] = round_to((float)(low ? a * w.x - b * w.y : a * w.x + b * w.y), E{});
    }
  }
}

// Scale byte of a group; NaN become 0.  Returns whether all were finite.
__device__ __forceinline__ bool scale_byte(float (&f)[32], int& byte) {
  float most = 0.0f;
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float a = fabsf(f[i]);
    const bool finite = a <= 3.402823466e38f;
    most = fmaxf(most, finite ? a : 0.0f);
    fine = fine && finite;
    if (f[i] != f[i]) f[i] = 0.0f;
  }
  const int e = (int)((__float_as_uint(most) + 0x1fffffu) >> 23) - 2;
  byte = min(max(e, 32), 251);
  return fine;
}

__device__ __forceinline__ uint32_t encode8(float a0, float b0, float a1, float b1, float a2, float b2, float a3,
                                            float b3, float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a0, b0, scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a1, b1, scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a2, b2, scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a3, b3, scale, 3);
  return w;
}

// Value of lane j of each group of four lanes.
template <int J>
__device__ __forceinline__ uint32_t quad(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, J * 0x55, 0xf, 0xf, false);
}

__device__ __forceinline__ uint8_t* record(const Cache& C, int slot, int h) {
  const int block = slot >> C.bt_log2, off = slot & ((1 << C.bt_log2) - 1);
  return C.base + block * C.stride + (((int64_t)h << C.bt_log2 >> 4) + (off >> 4)) * (544 * C.nc);
}

template <class E, bool ROPE>
__device__ __forceinline__ void cache_role(const RopeArgs& A, int block, double2* cs) {
  const Cache& C = A.cache;
  const int nc = C.nc, half = A.rot >> 1;
  const int t0 = block / A.kv_groups * kCacheTokens, g = block % A.kv_groups;
  const int nt = min(kCacheTokens, A.T - t0);
  if constexpr (ROPE) {
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
      const int tl = i / half, p = A.pos[t0 + tl];
      if (p >= 0) cs[i] = angle(A, p, i - tl * half);
    }
    __syncthreads();
  }
  // lane quads hold 4 consecutive tokens of one (head, group): (t/4, c, t%4)
  const int per_head = kCacheTokens * nc, at_once = kThreads / per_head;
  const int hl = threadIdx.x / per_head, r = threadIdx.x - hl * per_head;
  const int j = r & 3, c = (r >> 2) % nc, tl = (r >> 2) / nc * 4 + j, t = t0 + tl;
  const int h_end = min((g + 1) * A.kv_heads_per_group, C.heads);
  int slot = -1;
  if (hl < at_once && tl < nt) {
    slot = A.slots[t];
    if ((unsigned)(slot >> C.bt_log2) >= (unsigned)C.blocks) slot = -1;
    if (ROPE && A.pos[t] < 0) slot = -1;
  }
  // a quad whose tokens fill four neighbouring places of a unit writes V as
  // whole words; else each token writes its bytes
  const int s0 = (int)quad<0>((uint32_t)slot);
  const uint64_t in_row = __ballot(slot >= 0 && (s0 & 3) == 0 && slot == s0 + j);
  const bool whole = ((in_row >> (threadIdx.x & 60)) & 15) == 15;
  bool fine = true;
  for (int h = g * A.kv_heads_per_group + hl; h - hl < h_end; h += at_once) {
    const bool live = slot >= 0 && hl < at_once && h < h_end;
    uint8_t* rec = live ? record(C, slot, h) : nullptr;
    const int u = slot & 15;
    uint32_t q[4] = {0, 0, 0, 0};
    if (live) {
      typedef typename E::T T;
      float f[32];
      int byte;
      load_group<E, ROPE>(A, static_cast<const T*>(A.k.p) + t * A.k.ts + h * A.k.hs, c, cs + tl * half, f);
      fine &= scale_byte(f, byte);
      float scale = __uint_as_float((uint32_t)byte << 23);
#pragma unroll
      for (int gg = 0; gg < 4; ++gg)
        *reinterpret_cast<uint32_t*>(rec + ((u * 4 + gg) * nc + c) * 4) =
            encode8(f[8 * gg], f[8 * gg + 1], f[8 * gg + 2], f[8 * gg + 3], f[8 * gg + 4], f[8 * gg + 5],
                    f[8 * gg + 6], f[8 * gg + 7], scale);
      rec[512 * nc + u * nc + c] = (uint8_t)byte;
      load_n<32>(static_cast<const T*>(A.v.p) + t * A.v.ts + h * A.v.hs + 32 * c, f);
      fine &= scale_byte(f, byte);
      scale = __uint_as_float((uint32_t)byte << 23);
      rec[528 * nc + u * nc + c] = (uint8_t)byte;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        q[i] = encode8(f[4 * i], f[16 + 4 * i], f[4 * i + 1], f[17 + 4 * i], f[4 * i + 2], f[18 + 4 * i],
                       f[4 * i + 3], f[19 + 4 * i], scale);
    }
    // q[i] byte k: dims 4i+k (and 16 more) of this lane's token.  In a whole
    // quad lane j takes dims 4j..4j+3 of all four tokens.
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a0 = quad<0>(q[i]), a1 = quad<1>(q[i]), a2 = quad<2>(q[i]), a3 = quad<3>(q[i]);
      if (i == j) w[0] = a0, w[1] = a1, w[2] = a2, w[3] = a3;
    }
    if (live) {
      uint8_t* vc = rec + 256 * nc + (u >> 2) * 64 * nc + 4 * c;
      if (whole) {
        const uint32_t lo01 = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), hi01 = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
        const uint32_t lo23 = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), hi23 = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
        const uint32_t d[4] = {__builtin_amdgcn_perm(lo23, lo01, 0x05040100u), __builtin_amdgcn_perm(lo23, lo01, 0x07060302u),
                               __builtin_amdgcn_perm(hi23, hi01, 0x05040100u), __builtin_amdgcn_perm(hi23, hi01, 0x07060302u)};
#pragma unroll
        for (int k = 0; k < 4; ++k) *reinterpret_cast<uint32_t*>(vc + (4 * j + k) * 4 * nc) = d[k];
      } else {
#pragma unroll
        for (int d = 0; d < 16; ++d) vc[d * 4 * nc + (u & 3)] = (uint8_t)(q[d >> 2] >> (8 * (d & 3)));
      }
    }
  }
  if (!fine && A.flags) atomicOr(A.flags, LORA_KV_FLAG_NONFINITE);
}

template <class E, bool ROPE>
__global__ __launch_bounds__(kThreads) void rope_kernel(const RopeArgs A) {
  // rotation role: 4 tokens in both precisions; cache role: 16 in fp64
  __shared__ double2 lds[ROPE ? kCacheTokens * kMaxPairs : 1];
  if ((int)blockIdx.x < A.rot_blocks) {
    if constexpr (ROPE) rotate_role<E>(A, blockIdx.x, lds);
  } else {
    cache_role<E, ROPE>(A, blockIdx.x - A.rot_blocks, lds);
  }
}

// ------------------------------------------------------------------- gather
template <class E>
__global__ __launch_bounds__(kThreads) void gather_kernel(const RopeArgs A) {
  const Cache& C = A.cache;
  const int nc = C.nc;
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t th = idx / nc;
  const int c = (int)(idx - th * nc);
  const int64_t t = th / C.heads;
  const int h = (int)(th - t * C.heads);
  if (t >= A.T) return;
  int slot = A.slots[t];
  if ((unsigned)(slot >> C.bt_log2) >= (unsigned)C.blocks) slot = -1;
  float k[32], v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) k[i] = v[i] = 0.0f;
  if (slot >= 0) {
    const uint8_t* rec = record(C, slot, h);
    const int u = slot & 15;
    const float ks = __uint_as_float((uint32_t)rec[512 * nc + u * nc + c] << 23);
    const float vs = __uint_as_float((uint32_t)rec[528 * nc + u * nc + c] << 23);
    auto put = [](float* lo, float* hi, uint32_t byte, float s) {
      const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(byte, s, 0));
      *lo = __uint_as_float(w << 16);
      *hi = __uint_as_float(w & 0xffff0000u);
    };
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + ((u * 4 + g) * nc + c) * 4);
#pragma unroll
      for (int b = 0; b < 4; ++b) put(&k[8 * g + 2 * b], &k[8 * g + 2 * b + 1], w >> (8 * b), ks);
    }
    const uint8_t* vc = rec + 256 * nc + (u >> 2) * 64 * nc + 4 * c + (u & 3);
#pragma unroll
    for (int d = 0; d < 16; ++d) put(&v[d], &v[16 + d], vc[d * 4 * nc], vs);
  }
  typedef typename E::T T;
  store_n<32>(static_cast<T*>(A.ko.p) + t * A.ko.ts + h * A.ko.hs + 32 * c, k);
  store_n<32>(static_cast<T*>(A.v.p) + t * A.v.ts + h * A.v.hs + 32 * c, v);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& A, int dtype, int blocks, hipStream_t s) {
  const bool bf = dtype == LORA_DTYPE_BF16;
  if (A.rot > 0) {
    if (bf) rope_kernel<Bf16, true><<<blocks, kThreads, 0, s>>>(A);
    else rope_kernel<F32, true><<<blocks, kThreads, 0, s>>>(A);
  } else {
    if (bf) rope_kernel<Bf16, false><<<blocks, kThreads, 0, s>>>(A);
    else rope_kernel<F32, false><<<blocks, kThreads, 0, s>>>(A);
  }
  return hipGetLastError();
}

hipError_t launch_gather(const RopeArgs& A, int dtype, hipStream_t s) {
  const int blocks = ceil_div_i((int64_t)A.T * A.cache.heads * A.cache.nc, kThreads);
  if (dtype == LORA_DTYPE_BF16) gather_kernel<Bf16><<<blocks, kThreads, 0, s>>>(A);
  else gather_kernel<F32><<<blocks, kThreads, 0, s>>>(A);
  return hipGetLastError();
}

}  // namespace kv
}  // namespace lora
