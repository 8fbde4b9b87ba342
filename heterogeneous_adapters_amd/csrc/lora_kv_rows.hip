// lora_rope, lora_kv_append, lora_kv_gather: rotary positions, K and V into
// the paged 4-bit cache, and back.
//
// Mathematics
//   angle  a = p f / (2 pi) turns, reduced to [-1/2, 1/2] in fp64: 53 bits
//          leave 2^-53 * p f / (2 pi) turns, 1e-10 at a million positions,
//          where fp32 would have lost the angle.  cos and sin of it in fp64,
//          once per (token, pair), shared by the heads of a work-group
//          through LDS.
//   K      rotated in fp64 and rounded once; Q too where it is fp32, while bf16
//          Q is rotated in fp32 from the rounded cos and sin (2^-24, which
//          disappears in the rounding to bf16).
//   codes  2^e = the smallest power of two with max|x| <= 7 * 2^e, read off
//          the bits of max|x|: fraction above 1.75 moves to the next power.
//          v_cvt_scalef32_pk_fp4_f32 divides by 2^e, rounds to nearest even
//          and saturates (checked on gfx950 at every border).
//
// One launch: work-groups of the rotation role walk (token, head, vector) of
// Q (and of K in lora_rope), those of the cache role (16 tokens, a share of
// the heads).  Both read and write each byte once; the bound is HBM: 38781
// tokens of 32 + 8 heads of 128 take 225 us (3.7 TB/s of the 4.7 that a copy
// reaches), their gather 43 us; 8192 fp32 tokens 82.  A few tokens are bound by the chain position
// -> angle -> product: 9 us for 16, of which a launch alone is 3.
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
// Quotient by a small run-time divisor: n * d < 2^32 here, where m = ceil(2^32
// / d) gives it exactly.
struct Div {
  uint32_t m;
  __device__ explicit Div(int d) : m(d > 1 ? 0xffffffffu / (uint32_t)d + 1 : 0) {}
  __device__ __forceinline__ int operator()(int n) const { return m ? (int)__umulhi((uint32_t)n, m) : n; }
};

// Heads h0 .. h0+nh-1 of `in` into `out` for nt tokens.  V: arithmetic type.
// One task = one vector of pairs, or one vector of dims behind rot_dim (copied
// when out of place).  `angles` fills cs and is called once the first turn's
// loads are on their way.
template <class E, class V, class V2, class F>
__device__ __forceinline__ void rotate_heads(const RopeArgs& A, const Rows& in, const Rows& out, int t0, int nt, int h0,
                                             int nh, const V2* cs, F&& angles) {
  typedef typename E::T T;
  constexpr int EPV = E::kEpv;
  constexpr int U = 4;  // tasks in flight per thread
  const int half = A.rot >> 1;
  const bool copy = in.p != out.p, inter = A.interleaved != 0;
  const bool wide = inter ? A.rot % EPV == 0 : half % EPV == 0;
  const int tail = copy ? A.D - A.rot : 0;
  const bool tail_wide = A.rot % EPV == 0;
  const int pair_tasks = wide ? (inter ? A.rot / EPV : half / EPV) : half;
  const int per_head = pair_tasks + (tail_wide ? tail / EPV : tail);
  const int total = nt * nh * per_head;
  const Div by_head(per_head), by_token(nh);
  if (wide && tail_wide) {
    for (int base = 0; base < total; base += U * kThreads) {
      u32x4 a[U], b[U];
      T* y[U];
      int at[U];  // first dim; -1: nothing to do; + kMaxPairs * 4: a copy
      int tl[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int idx = base + u * kThreads + threadIdx.x;
        at[u] = -1;
        if (idx >= total) continue;
        const int th = by_head(idx), task = idx - th * per_head, h = th - by_token(th) * nh + h0;
        tl[u] = by_token(th);
        const int t = t0 + tl[u];
        if (A.pos[t] < 0) continue;
        const bool pass = task >= pair_tasks;
        const int d = pass ? A.rot + (task - pair_tasks) * EPV : task * EPV;
        const T* x = static_cast<const T*>(in.p) + t * in.ts + h * in.hs + d;
        y[u] = static_cast<T*>(out.p) + t * out.ts + h * out.hs + d;
        at[u] = pass ? d + 4 * kMaxPairs : d;
        a[u] = *reinterpret_cast<const u32x4*>(x);
        if (!inter && !pass) b[u] = *reinterpret_cast<const u32x4*>(x + half);
      }
      if (base == 0) angles();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (at[u] < 0) continue;
        if (at[u] >= 4 * kMaxPairs) {
          *reinterpret_cast<u32x4*>(y[u]) = a[u];
          continue;
        }
        const V2* w = cs + tl[u] * half;
        float xa[EPV], xb[EPV], r[EPV], s[EPV];
        unpack(a[u], xa);
        if (inter) {
          w += at[u] / 2;
#pragma unroll
          for (int i = 0; i < EPV / 2; ++i) {
            const V p = xa[2 * i], q = xa[2 * i + 1];
            r[2 * i] = (float)(p * w[i].x - q * w[i].y);
            r[2 * i + 1] = (float)(q * w[i].x + p * w[i].y);
          }
          store_n<EPV>(y[u], r);
        } else {
          unpack(b[u], xb);
          w += at[u];
#pragma unroll
          for (int i = 0; i < EPV; ++i) {
            const V p = xa[i], q = xb[i];
            r[i] = (float)(p * w[i].x - q * w[i].y);
            s[i] = (float)(q * w[i].x + p * w[i].y);
          }
          store_n<EPV>(y[u], r);
          store_n<EPV>(y[u] + half, s);
        }
      }
    }
    return;
  }
  angles();
  for (int idx = threadIdx.x; idx < total; idx += kThreads) {  // rot_dim not in whole vectors
    const int th = by_head(idx), task = idx - th * per_head;
    const int tl = by_token(th), h = h0 + th - tl * nh, t = t0 + tl;
    if (A.pos[t] < 0) continue;
    const T* x = static_cast<const T*>(in.p) + t * in.ts + h * in.hs;
    T* y = static_cast<T*>(out.p) + t * out.ts + h * out.hs;
    const V2* w = cs + tl * half;
    const int n = task < pair_tasks ? (wide ? EPV : 1) : (tail_wide ? EPV : 1);
    if (task >= pair_tasks) {
      const int d = A.rot + (task - pair_tasks) * n;
      for (int i = 0; i < n; ++i) y[d + i] = x[d + i];
      continue;
    }
    for (int i = 0; i < (wide && inter ? n / 2 : n); ++i) {
      const int pair = wide ? (inter ? task * EPV / 2 : task * EPV) + i : task;
      const int d0 = inter ? 2 * pair : pair, d1 = inter ? d0 + 1 : pair + half;
      const V p = to_f(x[d0]), q = to_f(x[d1]);
      from_f(y + d0, (float)(p * w[pair].x - q * w[pair].y));
      from_f(y + d1, (float)(q * w[pair].x + p * w[pair].y));
    }
  }
}

template <class E>
__device__ __forceinline__ void rotate_role(const RopeArgs& A, int block, double2* lds) {
  constexpr bool kBf16 = sizeof(typename E::T) == 2;
  float2* lf = reinterpret_cast<float2*>(lds + kRotTokens * kMaxPairs);
  const int half = A.rot >> 1;
  const int t0 = block / A.q_groups * kRotTokens, g = block % A.q_groups;
  const int nt = min(kRotTokens, A.T - t0);
  auto angles = [&]() {
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
      const int tl = i / half, p = A.pos[t0 + tl];
      if (p < 0) continue;
      const double2 w = angle(A, p, i - tl * half);
      lds[i] = w;
      if constexpr (kBf16) lf[i] = make_float2((float)w.x, (float)w.y);
    }
    __syncthreads();
  };
  // heads of q, then of k
  const int lo = g * A.q_heads_per_group, hi = min(lo + A.q_heads_per_group, A.qo.heads + A.ko.heads);
  const int nq = min(hi, A.qo.heads) - min(lo, A.qo.heads), nk = hi - lo - nq;
  if constexpr (kBf16) {
    if (nq > 0) rotate_heads<E, float>(A, A.q, A.qo, t0, nt, lo, nq, lf, angles);
  } else {
    if (nq > 0) rotate_heads<E, double>(A, A.q, A.qo, t0, nt, lo, nq, lds, angles);
  }
  if (nk > 0) {
    const int h0 = max(lo - A.qo.heads, 0);
    if (nq > 0) rotate_heads<E, double>(A, A.k, A.ko, t0, nt, h0, nk, lds, [] {});
    else rotate_heads<E, double>(A, A.k, A.ko, t0, nt, h0, nk, lds, angles);
  }
}

// --------------------------------------------------------------- cache role
// Eight dims of one head, from dim d0 on, as rounded, rotated values.
template <class E, bool ROPE>
__device__ __forceinline__ void load_eight(const RopeArgs& A, const typename E::T* x, int d0, const double2* cs,
                                           float (&f)[8]) {
  load_n<8>(x + d0, f);
  if constexpr (!ROPE) return;
  const int half = A.rot >> 1;
  if (d0 >= A.rot) return;
  if (A.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (d0 + 2 * i < A.rot) {
        const double2 w = cs[d0 / 2 + i];
        const double u = f[2 * i], v = f[2 * i + 1];
        f[2 * i] = round_to((float)(u * w.x - v * w.y), E{});
        f[2 * i + 1] = round_to((float)(v * w.x + u * w.y), E{});
      }
    }
  } else if (half % 8 == 0) {
    const bool low = d0 < half;
    const double2* w = cs + (low ? d0 : d0 - half);
    float o[8];
    load_n<8>(x + (low ? d0 + half : d0 - half), o);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double a = f[i], b = low ? -o[i] : o[i];
      f[i] = round_to((float)(a * w[i].x + b * w[i].y), E{});
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = d0 + i;
      if (d >= A.rot) continue;
      const bool low = d < half;
      const double2 w = cs[low ? d : d - half];
      const double a = f[i], b = to_f(x[low ? d + half : d - half]);
      f[i] = round_to((float)(low ? a * w.x - b * w.y : a * w.x + b * w.y), E{});
    }
  }
}

// Largest finite magnitude; NaN become 0.  Clears `fine` unless all are finite.
template <int N>
__device__ __forceinline__ float magnitude(float (&f)[N], bool& fine) {
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float a = fabsf(f[i]);
    const bool finite = a <= 3.402823466e38f;
    most = fmaxf(most, finite ? a : 0.0f);
    fine = fine && finite;
    if (f[i] != f[i]) f[i] = 0.0f;
  }
  return most;
}
// Scale byte of a group: 2^e with the least e with most <= 7 * 2^e.
__device__ __forceinline__ int scale_byte(float most) {
  const int e = (int)((__float_as_uint(most) + 0x1fffffu) >> 23) - 2;
  return min(max(e, 32), 251);
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

// Values of the other lanes of each group of four: CTRL names, for lanes 0 to
// 3, the lane to read (two bits each).
template <int CTRL>
__device__ __forceinline__ uint32_t quad(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, false);
}
template <int J>
__device__ __forceinline__ uint32_t quad_lane(uint32_t x) {
  return quad<J * 0x55>(x);
}

__device__ __forceinline__ uint8_t* record(const Cache& C, int slot, int h) {
  const int block = slot >> C.bt_log2, off = slot & ((1 << C.bt_log2) - 1);
  return C.base + block * C.stride + (((int64_t)h << C.bt_log2 >> 4) + (off >> 4)) * (544 * C.nc);
}

template <class E, bool ROPE>
__device__ __forceinline__ void cache_role(const RopeArgs& A, int block, double2* cs, int* s_slot) {
  typedef typename E::T T;
  const Cache& C = A.cache;
  const int nc = C.nc, half = A.rot >> 1;
  const int t0 = block / A.kv_groups * kCacheTokens, g = block % A.kv_groups;
  const int nt = min(kCacheTokens, A.T - t0);
  const int h_first = g * A.kv_heads_per_group, h_end = min(h_first + A.kv_heads_per_group, C.heads);
  if (threadIdx.x < kCacheTokens) {
    int slot = -1;
    if ((int)threadIdx.x < nt) {
      slot = A.slots[t0 + threadIdx.x];
      if ((unsigned)(slot >> C.bt_log2) >= (unsigned)C.blocks) slot = -1;
      if (ROPE && A.pos[t0 + threadIdx.x] < 0) slot = -1;
    }
    s_slot[threadIdx.x] = slot;
  }
  if constexpr (ROPE) {
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
      const int tl = i / half, p = A.pos[t0 + tl];
      if (p >= 0) cs[i] = angle(A, p, i - tl * half);
    }
  }
  __syncthreads();
  bool fine = true;

  // K: four lanes per group of 32, eight dims and one word of codes each
  {
    const int per_token = 4 * nc, per_head = kCacheTokens * per_token, total = (h_end - h_first) * per_head;
    const Div by_head(per_head), by_token(per_token);
    for (int idx = threadIdx.x; idx < total; idx += kThreads) {
      const int hl = by_head(idx), r = idx - hl * per_head, tl = by_token(r), cv = r - tl * per_token;
      const int slot = s_slot[tl];
      if (slot < 0) continue;  // the same for the four lanes
      const int h = h_first + hl, t = t0 + tl, c = cv >> 2, v = cv & 3, u = slot & 15;
      float f[8];
      load_eight<E, ROPE>(A, static_cast<const T*>(A.k.p) + t * A.k.ts + h * A.k.hs, 8 * cv, cs + tl * half, f);
      float most = magnitude(f, fine);
      most = fmaxf(most, __uint_as_float(quad<0xb1>(__float_as_uint(most))));  // lanes 1 0 3 2
      most = fmaxf(most, __uint_as_float(quad<0x4e>(__float_as_uint(most))));  // lanes 2 3 0 1
      const int byte = scale_byte(most);
      const float scale = __uint_as_float((uint32_t)byte << 23);
      uint8_t* rec = record(C, slot, h);
      *reinterpret_cast<uint32_t*>(rec + ((u * 4 + v) * nc + c) * 4) =
          encode8(f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7], scale);
      if (v == 0) rec[512 * nc + u * nc + c] = (uint8_t)byte;
    }
  }

  // V: four lanes hold 4 consecutive tokens of one (head, group of 32): a word
  // of codes spans them.  Where the tokens fill four neighbouring places of a
  // unit the lanes trade bytes and write whole words; else each token writes
  // its bytes.
  const int per_head = kCacheTokens * nc, at_once = kThreads / per_head;
  const int hl = threadIdx.x / per_head, r = threadIdx.x - hl * per_head;
  const int j = r & 3, c = (r >> 2) % nc, tl = (r >> 2) / nc * 4 + j, t = t0 + tl;
  const int slot = hl < at_once ? s_slot[tl] : -1;
  const int s0 = (int)quad_lane<0>((uint32_t)slot);
  const uint64_t in_row = __ballot(slot >= 0 && (s0 & 3) == 0 && slot == s0 + j);
  const bool whole = ((in_row >> (threadIdx.x & 60)) & 15) == 15;
  for (int h = h_first + hl; h - hl < h_end; h += at_once) {
    const bool live = slot >= 0 && h < h_end;
    uint8_t* rec = live ? record(C, slot, h) : nullptr;
    const int u = slot & 15;
    uint32_t q[4] = {0, 0, 0, 0};
    if (live) {
      float f[32];
      load_n<32>(static_cast<const T*>(A.v.p) + t * A.v.ts + h * A.v.hs + 32 * c, f);
      const int byte = scale_byte(magnitude(f, fine));
      const float scale = __uint_as_float((uint32_t)byte << 23);
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
      const uint32_t a0 = quad_lane<0>(q[i]), a1 = quad_lane<1>(q[i]), a2 = quad_lane<2>(q[i]), a3 = quad_lane<3>(q[i]);
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
__global__ __launch_bounds__(kThreads, 4) void rope_kernel(const RopeArgs A) {
  // rotation role: 4 tokens in both precisions; cache role: 16 in fp64
  __shared__ double2 lds[ROPE ? kCacheTokens * kMaxPairs : 1];
  __shared__ int s_slot[kCacheTokens];
  if ((int)blockIdx.x < A.rot_blocks) {
    if constexpr (ROPE) rotate_role<E>(A, blockIdx.x, lds);
  } else {
    cache_role<E, ROPE>(A, blockIdx.x - A.rot_blocks, lds, s_slot);
  }
}

// ------------------------------------------------------------------- gather
// Eight values of four bytes of codes.
__device__ __forceinline__ void decode8(uint32_t w, float scale, float (&x)[8]) {
  const uint32_t r[4] = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))};
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    x[2 * b] = __uint_as_float(r[b] << 16);
    x[2 * b + 1] = __uint_as_float(r[b] & 0xffff0000u);
  }
}

// The cache role backwards: 16 slots and a share of the heads per work-group.
template <class E>
__global__ __launch_bounds__(kThreads) void gather_kernel(const RopeArgs A) {
  typedef typename E::T T;
  __shared__ int s_slot[kCacheTokens];
  const Cache& C = A.cache;
  const int nc = C.nc;
  const int t0 = blockIdx.x / A.kv_groups * kCacheTokens, g = blockIdx.x % A.kv_groups;
  const int nt = min(kCacheTokens, A.T - t0);
  const int h_first = g * A.kv_heads_per_group, h_end = min(h_first + A.kv_heads_per_group, C.heads);
  if (threadIdx.x < kCacheTokens) {
    int slot = (int)threadIdx.x < nt ? A.slots[t0 + threadIdx.x] : -1;
    if ((unsigned)(slot >> C.bt_log2) >= (unsigned)C.blocks) slot = -1;
    s_slot[threadIdx.x] = slot;
  }
  __syncthreads();

  // K: eight dims per lane
  {
    const int per_token = 4 * nc, per_head = nt * per_token, total = (h_end - h_first) * per_head;
    const Div by_head(per_head), by_token(per_token);
    for (int idx = threadIdx.x; idx < total; idx += kThreads) {
      const int hl = by_head(idx), r = idx - hl * per_head, tl = by_token(r), cv = r - tl * per_token;
      const int slot = s_slot[tl], h = h_first + hl, c = cv >> 2, v = cv & 3, u = slot & 15;
      float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (slot >= 0) {
        const uint8_t* rec = record(C, slot, h);
        const float scale = __uint_as_float((uint32_t)rec[512 * nc + u * nc + c] << 23);
        decode8(*reinterpret_cast<const uint32_t*>(rec + ((u * 4 + v) * nc + c) * 4), scale, x);
      }
      store_n<8>(static_cast<T*>(A.ko.p) + (t0 + tl) * A.ko.ts + h * A.ko.hs + 8 * cv, x);
    }
  }

  // V: four lanes hold 4 consecutive slots of one (head, group of 32)
  const int per_head = kCacheTokens * nc, at_once = kThreads / per_head;
  const int hl = threadIdx.x / per_head, r = threadIdx.x - hl * per_head;
  const int j = r & 3, c = (r >> 2) % nc, tl = (r >> 2) / nc * 4 + j, t = t0 + tl;
  const bool mine = hl < at_once && tl < nt;
  const int slot = mine ? s_slot[tl] : -1;
  const int s0 = (int)quad_lane<0>((uint32_t)slot);
  const uint64_t in_row = __ballot(slot >= 0 && (s0 & 3) == 0 && slot == s0 + j);
  const bool whole = ((in_row >> (threadIdx.x & 60)) & 15) == 15;
  const int u = slot & 15;
  for (int h = h_first + hl; h - hl < h_end; h += at_once) {
    const bool live = slot >= 0 && h < h_end;
    const uint8_t* rec = live ? record(C, slot, h) : nullptr;
    uint32_t q[4] = {0, 0, 0, 0};  // this token's codes: byte k of q[i] is dims 4i+k and 16 more
    uint32_t d[4] = {0, 0, 0, 0};
    if (live) {
      const uint8_t* vc = rec + 256 * nc + (u >> 2) * 64 * nc + 4 * c;
      if (whole) {
#pragma unroll
        for (int k = 0; k < 4; ++k) d[k] = *reinterpret_cast<const uint32_t*>(vc + (4 * j + k) * 4 * nc);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i >> 2] |= (uint32_t)vc[i * 4 * nc + (u & 3)] << (8 * (i & 3));
      }
    }
    // of a whole quad lane j read dims 4j..4j+3 of all four tokens: trade
    const uint32_t lo01 = __builtin_amdgcn_perm(d[1], d[0], 0x05010400u), hi01 = __builtin_amdgcn_perm(d[1], d[0], 0x07030602u);
    const uint32_t lo23 = __builtin_amdgcn_perm(d[3], d[2], 0x05010400u), hi23 = __builtin_amdgcn_perm(d[3], d[2], 0x07030602u);
    const uint32_t of[4] = {__builtin_amdgcn_perm(lo23, lo01, 0x05040100u), __builtin_amdgcn_perm(lo23, lo01, 0x07060302u),
                            __builtin_amdgcn_perm(hi23, hi01, 0x05040100u), __builtin_amdgcn_perm(hi23, hi01, 0x07060302u)};
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // token k's word from each lane, for lane k
      const uint32_t a0 = quad_lane<0>(of[k]), a1 = quad_lane<1>(of[k]), a2 = quad_lane<2>(of[k]), a3 = quad_lane<3>(of[k]);
      if (whole && k == j) q[0] = a0, q[1] = a1, q[2] = a2, q[3] = a3;
    }
    if (mine && h < h_end) {
      float v[32];
      const float scale = live ? __uint_as_float((uint32_t)rec[528 * nc + u * nc + c] << 23) : 1.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[8];
        decode8(q[i], scale, x);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * i + k] = x[2 * k], v[16 + 4 * i + k] = x[2 * k + 1];
      }
      store_n<32>(static_cast<T*>(A.v.p) + t * A.v.ts + h * A.v.hs + 32 * c, v);
    }
  }
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

hipError_t launch_gather(const RopeArgs& A, int dtype, int blocks, hipStream_t s) {
  if (dtype == LORA_DTYPE_BF16) gather_kernel<Bf16><<<blocks, kThreads, 0, s>>>(A);
  else gather_kernel<F32><<<blocks, kThreads, 0, s>>>(A);
  return hipGetLastError();
}

}  // namespace kv
}  // namespace lora
