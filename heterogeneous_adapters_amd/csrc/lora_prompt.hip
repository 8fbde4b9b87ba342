// lora_prompt_attend: causal attention of packed prompts over themselves.
//
// Mathematics: per row one pass over the keys with a running maximum m and
// sum l of exp2(s - m), s = scale log2(e) q.k.  2 * sum L^2 * heads * D
// flops: bound by the issue of products and of the softmax's vector
// instructions (long prompts: 62 % and 49 % of a SIMD's time, beside each other
// for a tenth of it at least); many shorter ones by starts, diagonals and
// barriers too (42 % and 40 %).
//
// bf16: a work-group of 4 waves takes 32 rows per wave of one query head and
// walks the prompt's keys in tiles of 32 or 64, copied straight into LDS
// (buffer loads to LDS, 16 bytes a lane) while the tile before is multiplied.
// v_mfma_f32_32x32x16_bf16 on both products: S^T = K Q^T leaves row lane%32
// with tokens 8(i/4) + 4h + i%4 (h = lane/32) in each lane, which is the B
// operand of O^T = V^T P^T once V^T is read in that token order
// (ds_read_b64_tr_b16: four tokens x sixteen dims per sixteen lanes), so P
// never leaves its registers and the softmax needs no cross-lane step but
// one exchange between the two halves of a row, and that only when a maximum
// moves.
//
// P is rounded to bf16 for the second product (two terms of it would take half
// as many products again, in a kernel bound by their issue), by up to 2^-8 of
// each weight.  l sums the rounded weights, so that they sum to one and what a
// row's visible V share comes out exact; the sums of two per instruction cost
// what those of unrounded weights did (8192 tokens 616 us against 621).
//
// Measured on MI355X: prompts of 8192, 4097 and 1 tokens, 32 query heads of
// 128 on 8 kv heads, 620 us = 1.11 PFLOP/s of causal work (the installed
// library's plain product reaches 1.2); 32 prompts of 128..2048 with 32 kv
// heads 505 us.  Four waves per work-group: three of them share a CU out of
// step (8 waves: 683 against 658).
//
// fp32 (validation): one wave per 16 rows on v_mfma_f32_16x16x4_f32, keys and
// values straight from global memory, a step's all loaded before its products
// (32 prompts of up to 400, 32 heads of 128 on 8: 272 us, 52 TFLOP/s; each value
// loaded where it is used, 748).  Short prompts are bound by the chain of
// products of their last rows, long ones by every wave's reads of the caches.
#include "lora_kv_dev.h"
#include "lora_kv_host.h"

namespace lora {
namespace kv {

namespace {

constexpr int kRowsPerWave = 32;

// Keys per tile.  32 halve the scores in flight, which buys a third wave per
// SIMD at 128 dims and saves registers from spilling to the other bank above
// (8192 keys at 128 dims: 609 us against 624; 4096 at 192: 135 against 141).
// Below 128 registers are no bound and 64 keys per barrier win (64 dims, 8192
// keys: 306 against 326); at 256 so do they (4096 keys: 183 against 458).
constexpr int keys_per_tile(int D) { return D >= 128 && D < 256 ? 32 : 64; }

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef const __attribute__((address_space(3))) bf16x8 lds_bf16x8;

// The prompt and tile of flat tile index w.  Prompt i's tiles start at
// indptr[i] / rows + i, which leaves room for ceil(len / rows) of them.  Each
// wave searches by itself, 64 probes a step, and has the prompt's ends from
// the last step's lanes: one trip to memory for up to 64 prompts and no
// barrier.  Longest tiles come first.
struct Span {
  int begin, len, tile;  // tile < 0: none
};
__device__ __forceinline__ int cut(int x, int T) { return min(max(x, 0), T); }
__device__ __forceinline__ Span find_span(const PromptArgs& A, int w, int rows) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = A.B;  // the prompt is in [lo, hi)
  while (true) {
    const int step = (hi - lo + 63) / 64, p = lo + lane * step;
    int a = 0, b = 0;
    bool at_or_before = false;
    if (p < hi) {
      a = cut(A.indptr[p], A.T);
      b = cut(A.indptr[p + 1], A.T);
      at_or_before = a / rows + p <= w;
    }
    const int n = __popcll(__ballot(at_or_before));
    if (n == 0) return Span{0, 0, -1};
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
    if (step == 1) {
      const int begin = __builtin_amdgcn_readlane(a, n - 1), end = __builtin_amdgcn_readlane(b, n - 1);
      const int local = w - (begin / rows + lo), tiles = (max(end - begin, 0) + rows - 1) / rows;
      return Span{begin, end - begin, local >= 0 && local < tiles ? tiles - 1 - local : -1};
    }
  }
}

// Query head of a launch's b-th work-group among `heads` neighbours.  Work-
// groups go round the 8 XCDs; each XCD gets neighbouring query heads, so that
// the K and V of their kv heads stay in its L2.
__device__ __forceinline__ int head_of(int b, int heads) { return heads % 8 ? b : (b & 7) * (heads >> 3) + (b >> 3); }

// Swizzles of 16-byte pieces within a row of D elements, for 64 banks of 4
// bytes: a K read takes one piece of 16 rows at a time, a V read 4 pieces
// (64 bytes) of 4 rows.  Rows of a multiple of 256 bytes all start in the
// same bank, of 128 bytes alternate between two places, others walk through
// four; the swizzle spreads what the rows' starts do not.  (Spread over 128
// bytes only, half the LDS cycles were conflicts.)
template <int D>
__device__ __forceinline__ int swz_k(int token, int piece) {
  return D % 128 == 0 ? piece ^ (token & 15) : D % 64 == 0 ? piece ^ ((token >> 1) & 7) : piece ^ ((token >> 2) & 3);
}
template <int D>
__device__ __forceinline__ int swz_v(int token, int piece) {
  return D % 128 == 0 ? piece ^ ((token & 3) << 2) : D % 64 == 0 ? piece ^ ((token & 2) << 1) : piece;
}

#if defined(__HIP_DEVICE_COMPILE__)  // the host pass knows no buffer descriptors
// Buffer descriptor of the rest of a head's rows: loads behind the prompt's
// last row return zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const uint16_t* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), 0, (int)min(max(bytes, (int64_t)0), (int64_t)0xfffffff0ll),
                                           0x00020000);
}

#endif

template <int D, int W>
__global__ __launch_bounds__(64 * W, D == 128 ? 3 : 2) void prompt_kernel(const PromptArgs A) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kKeys = keys_per_tile(D), kU = kKeys / 32, kC = kKeys / 16;
  constexpr int kRows = W * kRowsPerWave;
  constexpr int kPieces = D / 8;  // 16-byte pieces per row
  constexpr int kTileBytes = kKeys * D * 2;
  constexpr int kLoads = kTileBytes / 1024;  // 1 KB loads per tensor, dealt to the waves
  constexpr int kSteps = D / 16, kDims = D / 32;
  // one array per buffer and tensor, so that the compiler sees which copy a
  // read depends on
  __shared__ __attribute__((aligned(128))) uint8_t s_k0[kTileBytes], s_v0[kTileBytes], s_k1[kTileBytes], s_v1[kTileBytes];

  const int hq_n = A.q.heads;
  const int flat = blockIdx.x / hq_n, hq = head_of(blockIdx.x - flat * hq_n, hq_n), hk = hq / A.G;
  const Span sp = find_span(A, flat, kRows);
  if (sp.tile < 0) return;

  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 31, h = lane >> 5;
  const int row_first = sp.tile * kRows + wave * kRowsPerWave;
  const int row = row_first + n;
  const int row_last = last_row(row_first, kRowsPerWave, sp.len);  // -1: this wave only copies
  const int n_tiles = (min((sp.tile + 1) * kRows, sp.len) + kKeys - 1) / kKeys;

  bf16x8 qf[kSteps];
  {
    const uint16_t* q = static_cast<const uint16_t*>(A.q.p) + (int64_t)(sp.begin + min(row, sp.len - 1)) * A.q.ts + hq * A.q.hs;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) qf[s] = *reinterpret_cast<const bf16x8*>(q + 16 * s + 8 * h);
  }

  const uint16_t* kbase = static_cast<const uint16_t*>(A.k.p) + (int64_t)sp.begin * A.k.ts + hk * A.k.hs;
  const uint16_t* vbase = static_cast<const uint16_t*>(A.v.p) + (int64_t)sp.begin * A.v.ts + hk * A.v.hs;
  const int64_t kbytes = 2 * ((sp.len - 1) * A.k.ts + D), vbytes = 2 * ((sp.len - 1) * A.v.ts + D);
  // Loads 0..kLoads-1 of a tile fetch K, the others V; wave w takes loads w,
  // w + W, ..  The 16-byte place p of a tile holds piece swz(p) of its row.
  constexpr int kMine = (2 * kLoads + W - 1) / W;
  int off[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int load = wave + i * W, at = (load % kLoads) * 64 + lane;
    const int token = at / kPieces, piece = at - token * kPieces;
    off[i] = load < kLoads ? (int)(token * A.k.ts + swz_k<D>(token, piece) * 8) * 2
                           : (int)(token * A.v.ts + swz_v<D>(token, piece) * 8) * 2;
  }
  auto stage = [&](int tile, uint8_t* sk, uint8_t* sv) {
    const int64_t ko = (int64_t)tile * kKeys * A.k.ts, vo = (int64_t)tile * kKeys * A.v.ts;
    const __amdgpu_buffer_rsrc_t kr = rows_rsrc(kbase + ko, kbytes - 2 * ko), vr = rows_rsrc(vbase + vo, vbytes - 2 * vo);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int load = wave + i * W;
      if (load < kLoads)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(kr, (lds_void*)(sk + load * 1024), 16, off[i], 0, 0, 0);
      else if (load < 2 * kLoads)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(vr, (lds_void*)(sv + (load - kLoads) * 1024), 16, off[i], 0, 0, 0);
    }
  };

  // LDS places of this lane's K pieces (row n of a tile's 32, piece 2c + h)
  // and V pieces (row 4h + i/4, dims 16 sub + 4 (i%4) of 32); the swizzle
  // leaves kKVar and kVVar of them, the rest are constants away
  constexpr int kKVar = D % 128 == 0 ? 8 : D % 64 == 0 ? 4 : 2, kVVar = D % 128 == 0 ? 4 : D % 64 == 0 ? 2 : 1;
  int k_at[kKVar], v_at[kVVar];
#pragma unroll
  for (int c = 0; c < kKVar; ++c) k_at[c] = n * (2 * D) + swz_k<D>(n, 2 * c + h) * 16;
  const int i16 = lane & 15, sub = (lane >> 4) & 1, v_row = 4 * h + (i16 >> 2);
#pragma unroll
  for (int d = 0; d < kVVar; ++d)
    v_at[d] = v_row * (2 * D) + swz_v<D>(v_row, 4 * d + 2 * sub + ((i16 & 3) >> 1)) * 16 + (i16 & 1) * 8;

  f16v o[kDims];
#pragma unroll
  for (int d = 0; d < kDims; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = kNone, l = 0.0f;

  auto compute = [&](int key0, const uint8_t* sk, const uint8_t* sv) {
    f16v s[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        const bf16x8 a = *(lds_bf16x8*)(sk + k_at[c % kKVar] + u * 32 * (2 * D) + (c / kKVar) * (kKVar * 32));
        s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, qf[c], s[u], 0, 0, 0);
      }
#pragma unroll
    for (int i = 0; i < kSteps * kU - 6; ++i) {
      if (i == 0) __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, 6, 0);
    s16x8 vf[kDims];
#pragma unroll
    for (int d = 0; d < kDims; ++d) {
      s16x4 part[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        part[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4*)(sv + v_at[d % kVVar] + 8 * e * (2 * D) + (d / kVVar) * (kVVar * 64)));
      vf[d] = __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7);
    }
    const bool masked = key0 + kKeys - 1 > row_first;
    if (masked) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (key0 + 32 * u + 8 * (i >> 2) + 4 * h + (i & 3) > row) s[u][i] = -INFINITY;
    }
    float most = s[0][0];
#pragma unroll
    for (int i = 1; i < 16 * kU; ++i) most = fmaxf(most, s[i >> 4][i & 15]);
    most *= A.scale_log2e;
    if (__any(most > m + kSlack)) {
      most = fmaxf(most, __shfl_xor(most, 32));
      const float mn = fmaxf(m, most), alpha = exp2_hw(m - mn);
      m = mn;
      l *= alpha;
#pragma unroll
      for (int d = 0; d < kDims; ++d) o[d] *= alpha;
    }
    bf16x8 pf[kC];
#pragma unroll
    for (int i = 0; i < 16 * kU; ++i) pf[i >> 3][i & 7] = (__bf16)exp2_hw(fmaf(s[i >> 4][i & 15], A.scale_log2e, -m));
    // O^T += V^T P^T
    auto v_frag = [&](int c, int d) {
      s16x4 part[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        part[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4*)(sv + v_at[d % kVVar] + (16 * c + 8 * e) * (2 * D) + (d / kVVar) * (kVVar * 64)));
      return __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7);
    };
#pragma unroll
    for (int c = 0; c < kC; ++c)  // 16 tokens each
#pragma unroll
      for (int d = 0; d < kDims; ++d) {
        const s16x8 a = c == 0 ? vf[d] : v_frag(c, d);
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), pf[c], o[d], 0, 0, 0);
        if (d == 0) l = add8(pf[c], l);
      }
  };

  // Two tiles per turn, one per buffer.  Every wave waits for its own copies
  // before the barrier that lets the others read them, whether it computes
  // on the tile or not; past the barrier the other buffer is free.
  stage(0, s_k0, s_v0);
  for (int it = 0; it < n_tiles; it += 2) {
    wait_vm<0>();
    __syncthreads();
    if (it + 1 < n_tiles) stage(it + 1, s_k1, s_v1);
    if (it * kKeys <= row_last) compute(it * kKeys, s_k0, s_v0);
    if (it + 1 >= n_tiles) break;
    wait_vm<0>();
    __syncthreads();
    if (it + 2 < n_tiles) stage(it + 2, s_k0, s_v0);
    if ((it + 1) * kKeys <= row_last) compute((it + 1) * kKeys, s_k1, s_v1);
  }

  // A weight of zero does not hide an infinity or NaN of V from the product:
  // rows that are not finite are computed again, key by key visible or not, and
  // so are rows of far scores, whose form of the weights would cost the loop
  // above registers.
  float odd = 0.0f;  // stays 0 while all is finite
  auto write = [&](float inv, bool check) {
    uint16_t* out = static_cast<uint16_t*>(A.o.p) + (int64_t)(sp.begin + row) * A.o.ts + hq * A.o.hs;
#pragma unroll
    for (int d = 0; d < kDims; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        uint2 w;
        w.x = pack_bf2(o[d][i] * inv, o[d][i + 1] * inv);
        w.y = pack_bf2(o[d][i + 2] * inv, o[d][i + 3] * inv);
        if (check) {
          odd = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w.x), bf16x2{0, 0}, odd, false);
          odd = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w.y), bf16x2{0, 0}, odd, false);
        }
        *reinterpret_cast<uint2*>(out + 32 * d + 2 * i + 4 * h) = w;
      }
  };
  l += __shfl_xor(l, 32);
  if (row <= row_last) write(1.0f / l, true);
  if (row_last < 0 || !__any(odd != odd || is_far(m))) return;

  // The long way, straight from global memory, 32 keys a step: the finite part
  // of V as usual, then, for each sign and for NaN, a product that counts the
  // visible ones.
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
    qf[s] = *reinterpret_cast<const bf16x8*>(static_cast<const uint16_t*>(A.q.p) +
                                             (int64_t)(sp.begin + min(row, sp.len - 1)) * A.q.ts + hq * A.q.hs + 16 * s + 8 * h);
#pragma unroll
  for (int d = 0; d < kDims; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  m = kNone;
  l = 0.0f;
  for (int key0 = 0; key0 <= row_last; key0 += 32) {
    f16v s;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.0f;
    const uint16_t* kr = kbase + (int64_t)min(key0 + n, sp.len - 1) * A.k.ts + 8 * h;
#pragma unroll
    for (int c = 0; c < kSteps; ++c)
      s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<const bf16x8*>(kr + 16 * c), qf[c], s, 0, 0, 0);
    float most = kNone;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (key0 + 8 * (i >> 2) + 4 * h + (i & 3) > row) s[i] = -INFINITY;
      most = fmaxf(most, s[i] * A.scale_log2e);
    }
    most = fmaxf(most, __shfl_xor(most, 32));
    const float mn = fmaxf(m, most), alpha = exp2_hw(m - mn);
    m = mn;
    l *= alpha;
#pragma unroll
    for (int d = 0; d < kDims; ++d) o[d] *= alpha;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      bf16x8 p, sees;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = (__bf16)exp2_hw(far_exponent(s[8 * c + j], A.scale_log2e, m));
        sees[j] = key0 + 16 * c + 8 * (j >> 2) + 4 * h + (j & 3) <= row ? (__bf16)1.0f : (__bf16)0.0f;
      }
      l = add8(p, l);
#pragma unroll
      for (int d = 0; d < kDims; ++d) {
        s16x8 a;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int key = key0 + 16 * c + 8 * (j >> 2) + 4 * h + (j & 3);
          a[j] = key < sp.len ? (short)vbase[(int64_t)key * A.v.ts + 32 * d + n] : (short)0;
          bad = bad || (a[j] & 0x7f80) == 0x7f80;
        }
        if (__any(bad)) {
          const s16x8 raw = a;
#pragma unroll 1
          for (int kind = 1; kind < 4; ++kind) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int bits = (uint16_t)raw[j], mag = bits & 0x7fff;
              const int is = mag < 0x7f80 ? 0 : mag > 0x7f80 ? 3 : bits < 0x8000 ? 1 : 2;  // finite, +inf, -inf, NaN
              a[j] = is == kind ? (short)0x3f80 : (short)0;
            }
            f16v count;
#pragma unroll
            for (int i = 0; i < 16; ++i) count[i] = 0.0f;
            count = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), sees, count, 0, 0, 0);
            const float add = kind == 1 ? INFINITY : kind == 2 ? -INFINITY : NAN;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (count[i] > 0.0f) o[d][i] += add;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) a[j] = (raw[j] & 0x7f80) == 0x7f80 ? (short)0 : raw[j];
        }
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), p, o[d], 0, 0, 0);
      }
    }
  }
  l += __shfl_xor(l, 32);
  if (row <= row_last) write(1.0f / l, false);
#endif
}

// ------------------------------------------------------------------- fp32
constexpr int kRows32 = 64;  // rows per work-group, 16 per wave
constexpr float kMostF32 = 3.402823466e38f;

template <int D>
__global__ __launch_bounds__(256) void prompt_f32_kernel(const PromptArgs A) {
  constexpr int kVecs = D / 16;
  const int hq_n = A.q.heads;
  const int flat = blockIdx.x / hq_n, hq = blockIdx.x - flat * hq_n, hk = hq / A.G;
  const Span sp = find_span(A, flat, kRows32);
  if (sp.tile < 0) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
  const int row_first = sp.tile * kRows32 + wave * 16, row = row_first + n;
  if (row_first >= sp.len) return;
  const int row_last = min(row_first + 16, sp.len) - 1;
  const float* kb = static_cast<const float*>(A.k.p) + (int64_t)sp.begin * A.k.ts + hk * A.k.hs;
  const float* vb = static_cast<const float*>(A.v.p) + (int64_t)sp.begin * A.v.ts + hk * A.v.hs;
  f4 qf[kVecs], o[kVecs];
  const float* q = static_cast<const float*>(A.q.p) + (int64_t)(sp.begin + min(row, sp.len - 1)) * A.q.ts + hq * A.q.hs;
#pragma unroll
  for (int s = 0; s < kVecs; ++s) {
    qf[s] = *reinterpret_cast<const f4*>(q + 16 * s + 4 * g);
    o[s] = f4{0, 0, 0, 0};
  }
  float m = kNone, l = 0.0f;
  bool far = false;  // some row's scores are
  f4 k[kVecs];
  auto load_k = [&](int key0) {
    const float* kr = kb + (int64_t)min(key0 + n, sp.len - 1) * A.k.ts + 4 * g;
#pragma unroll
    for (int c = 0; c < kVecs; ++c) k[c] = *reinterpret_cast<const f4*>(kr + 16 * c);
  };
  load_k(0);
  for (int key0 = 0; key0 <= row_last; key0 += 16) {
    float v[4][kVecs];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float* vr = vb + (int64_t)min(key0 + 4 * g + e, sp.len - 1) * A.v.ts + n;
#pragma unroll
      for (int d = 0; d < kVecs; ++d) v[e][d] = vr[16 * d];
    }
    f4 s{0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < kVecs; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) s = __builtin_amdgcn_mfma_f32_16x16x4f32(k[c][e], qf[c][e], s, 0, 0, 0);
    load_k(key0 + 16);
    const bool masked = key0 + 15 > row_first;
    if (masked) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (key0 + 4 * g + i > row) s[i] = -INFINITY;
    }
    float most = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])) * A.scale_log2e;
    if (__any(most > m + kSlack)) {
      most = fmaxf(most, __shfl_xor(most, 16));
      most = fmaxf(most, __shfl_xor(most, 32));
      const float mn = fmaxf(m, most), alpha = exp2_hw(m - mn);
      m = mn;
      far = far || __any(is_far(mn));
      l *= alpha;
#pragma unroll
      for (int d = 0; d < kVecs; ++d) o[d] *= alpha;
    }
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = exp2_hw(far ? far_exponent(s[i], A.scale_log2e, m) : fmaf(s[i], A.scale_log2e, -m));
      l += p[i];
    }
    if (masked) {
      // a weight of zero does not hide infinities and NaN: they are counted
      // where they are seen
      bool any = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool past = key0 + 4 * g + e >= sp.len;
#pragma unroll
        for (int d = 0; d < kVecs; ++d) {
          if (past) v[e][d] = 0.0f;
          any |= !(fabsf(v[e][d]) <= kMostF32);
        }
      }
      if (__any(any)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float sees = key0 + 4 * g + e <= row ? 1.0f : 0.0f;
          const float adds[3] = {INFINITY, -INFINITY, NAN};
#pragma unroll
          for (int d = 0; d < kVecs; ++d) {
            float& x = v[e][d];
            const bool is[3] = {x > kMostF32, x < -kMostF32, x != x};
            for (int kind = 0; kind < 3; ++kind) {
              const f4 count = __builtin_amdgcn_mfma_f32_16x16x4f32(is[kind] ? 1.0f : 0.0f, sees, f4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (count[i] > 0.0f) o[d][i] += adds[kind];
            }
            if (is[0] || is[1] || is[2]) x = 0.0f;
          }
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int d = 0; d < kVecs; ++d) o[d] = __builtin_amdgcn_mfma_f32_16x16x4f32(v[e][d], p[e], o[d], 0, 0, 0);
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (row < sp.len) {
    const float inv = 1.0f / l;
    float* out = static_cast<float*>(A.o.p) + (int64_t)(sp.begin + row) * A.o.ts + hq * A.o.hs + 4 * g;
#pragma unroll
    for (int d = 0; d < kVecs; ++d) *reinterpret_cast<f4*>(out + 16 * d) = o[d] * inv;
  }
}

template <int D>
hipError_t launch_d(const PromptArgs& A, int dtype, hipStream_t s) {
  if (dtype == LORA_DTYPE_BF16) {
    constexpr int W = 4;
    const int64_t blocks = ((int64_t)A.T / (W * kRowsPerWave) + A.B) * A.q.heads;
    prompt_kernel<D, W><<<(unsigned)blocks, 64 * W, 0, s>>>(A);
  } else {
    const int64_t blocks = ((int64_t)A.T / kRows32 + A.B) * A.q.heads;
    prompt_f32_kernel<D><<<(unsigned)blocks, 256, 0, s>>>(A);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_prompt(const PromptArgs& A, int dtype, int D, hipStream_t s) {
  switch (D) {
    case 32: return launch_d<32>(A, dtype, s);
    case 64: return launch_d<64>(A, dtype, s);
    case 96: return launch_d<96>(A, dtype, s);
    case 128: return launch_d<128>(A, dtype, s);
    case 160: return launch_d<160>(A, dtype, s);
    case 192: return launch_d<192>(A, dtype, s);
    case 224: return launch_d<224>(A, dtype, s);
    default: return launch_d<256>(A, dtype, s);
  }
}

}  // namespace kv
}  // namespace lora
