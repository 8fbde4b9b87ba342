// lora_prompt_attend: causal attention of packed prompts over themselves.
//
// Mathematics: per row one pass over the keys with a running maximum m and
// sum l of exp2(s - m), s = scale log2(e) q.k.  2 * sum L^2 * heads * D
// flops: bound by MFMA and, next to it, by the exponentials and LDS reads.
//
// bf16: a work-group of kWaves waves takes 32 rows per wave of one query
// head and walks the prompt's keys in tiles of 64, copied straight into LDS
// (global_load_lds, 16 bytes a lane) while the tile before is multiplied.
// v_mfma_f32_32x32x16_bf16 on both products: S^T = K Q^T leaves row lane%32
// with tokens 8(i/4) + 4h + i%4 (h = lane/32) in each lane, which is the B
// operand of O^T = V^T P^T once V^T is read in that token order
// (ds_read_b64_tr_b16: four tokens x sixteen dims per sixteen lanes), so P
// never leaves its registers and the softmax needs no cross-lane step but
// one exchange between the two halves of a row, and that only when a maximum
// moves.  LDS rows are XOR-swizzled in 16-byte pieces so neither the K reads
// (eight rows, one piece) nor the V reads (four rows, two pieces) meet in a
// bank.
//
// fp32 (validation): one wave per 16 rows on v_mfma_f32_16x16x4_f32, keys and
// values straight from global memory.
#include "lora_kv_dev.h"
#include "lora_kv_host.h"

namespace lora {
namespace kv {

namespace {

constexpr float kNone = -1e30f;  // running maximum before any key
// Rows keep their maximum until a score passes it by this much (a factor of
// 2^8 in p, without loss: p is scaled the same in the products and the sum).
constexpr float kSlack = 8.0f;

constexpr int kWaves = 4;
constexpr int kRowsPerWave = 32;
constexpr int kRows = kWaves * kRowsPerWave;
constexpr int kKeys = 64;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef const __attribute__((address_space(1))) void global_void;

// The prompt and tile of flat tile index w.  Prompt i's tiles start at
// indptr[i] / rows + i, which leaves room for ceil(len / rows) of them; every
// thread tests its share of the prompts.  Longest tiles come first.
struct Span {
  int begin, len, tile;  // tile < 0: none
};
__device__ __forceinline__ int cut(int x, int T) { return min(max(x, 0), T); }
__device__ __forceinline__ Span find_span(const PromptArgs& A, int w, int rows, int* found) {
  if (threadIdx.x == 0) *found = -1;
  __syncthreads();
  for (int i = threadIdx.x; i < A.B; i += blockDim.x) {
    const int a = cut(A.indptr[i], A.T), b = cut(A.indptr[i + 1], A.T);
    const int local = w - (a / rows + i);
    if (local >= 0 && (int64_t)local * rows < b - a) *found = i;
  }
  __syncthreads();
  const int i = uniform(*found);
  if (i < 0) return Span{0, 0, -1};
  const int a = uniform(cut(A.indptr[i], A.T)), b = uniform(cut(A.indptr[i + 1], A.T));
  const int local = w - (a / rows + i);
  return Span{a, b - a, (b - a + rows - 1) / rows - 1 - local};
}

// Swizzle of 16-byte pieces within a row of D elements: rows of a multiple of
// 128 bytes start in the same bank, others alternate between two halves.
template <int D>
__device__ __forceinline__ int swz_k(int token, int piece) {
  return D % 64 == 0 ? piece ^ (token & 7) : piece ^ ((token >> 1) & 3);
}
template <int D>
__device__ __forceinline__ int swz_v(int token, int piece) {
  return D % 64 == 0 ? piece ^ ((token & 3) << 1) : piece ^ (token & 2);
}

__device__ __forceinline__ bool bf_nonfinite(uint32_t w) {
  return (w & 0x7f800000u) == 0x7f800000u || (w & 0x7f80u) == 0x7f80u;
}

template <int D>
__global__ __launch_bounds__(64 * kWaves) void prompt_kernel(const PromptArgs A) {
  constexpr int kPieces = D / 8;       // 16-byte pieces per row
  constexpr int kTileBytes = kKeys * D * 2;
  constexpr int kLoads = kTileBytes / (64 * kWaves * 16);  // per wave and tensor
  static_assert(kTileBytes % (64 * kWaves * 16) == 0, "whole loads");
  constexpr int kKSteps = D / 16, kDimTiles = D / 32;
  __shared__ __attribute__((aligned(128))) uint8_t s_k[2][kTileBytes];
  __shared__ __attribute__((aligned(128))) uint8_t s_v[2][kTileBytes];
  __shared__ int s_found;

  const int hq_n = A.q.heads;
  const int flat = blockIdx.x / hq_n, hq = blockIdx.x - flat * hq_n, hk = hq / A.G;
  const Span sp = find_span(A, flat, kRows, &s_found);
  if (sp.tile < 0) return;

  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 31, h = lane >> 5;
  const int row_first = sp.tile * kRows + wave * kRowsPerWave;
  const int row = row_first + n;
  const int row_last = min(row_first + kRowsPerWave, sp.len) - 1;  // below row_first: no rows in this wave
  const int n_tiles = (min((sp.tile + 1) * kRows, sp.len) + kKeys - 1) / kKeys;

  bf16x8 qf[kKSteps];
  {
    const uint16_t* q = static_cast<const uint16_t*>(A.q.p) + (int64_t)(sp.begin + min(row, sp.len - 1)) * A.q.ts + hq * A.q.hs;
#pragma unroll
    for (int s = 0; s < kKSteps; ++s) qf[s] = *reinterpret_cast<const bf16x8*>(q + 16 * s + 8 * h);
  }

  const uint16_t* kbase = static_cast<const uint16_t*>(A.k.p) + (int64_t)sp.begin * A.k.ts + hk * A.k.hs;
  const uint16_t* vbase = static_cast<const uint16_t*>(A.v.p) + (int64_t)sp.begin * A.v.ts + hk * A.v.hs;
  // Tokens behind the prompt's last read the last one's row; they are masked.
  auto stage = [&](int tile, int buf) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = (wave * kLoads + i) * 64 + lane;  // 16-byte place in the tile
      const int token = at / kPieces, piece = at - token * kPieces;
      const int64_t t = min(tile * kKeys + token, sp.len - 1);
      __builtin_amdgcn_global_load_lds((global_void*)(kbase + t * A.k.ts + swz_k<D>(token, piece) * 8),
                                       (lds_void*)(s_k[buf] + (wave * kLoads + i) * 1024), 16, 0, 0);
      __builtin_amdgcn_global_load_lds((global_void*)(vbase + t * A.v.ts + swz_v<D>(token, piece) * 8),
                                       (lds_void*)(s_v[buf] + (wave * kLoads + i) * 1024), 16, 0, 0);
    }
  };

  f16v o[kDimTiles];
#pragma unroll
  for (int d = 0; d < kDimTiles; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = kNone, l = 0.0f;

  stage(0, 0);
  for (int it = 0; it < n_tiles; ++it) {
    const int buf = it & 1, key0 = it * kKeys;
    __syncthreads();  // this tile has arrived, and the other buffer is free
    if (it + 1 < n_tiles) stage(it + 1, buf ^ 1);
    if (key0 > row_last) continue;

    f16v s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
      const int token = 32 * u + n;
#pragma unroll
      for (int c = 0; c < kKSteps; ++c) {
        const bf16x8 a = *reinterpret_cast<const bf16x8*>(s_k[buf] + token * (2 * D) + swz_k<D>(token, 2 * c + h) * 16);
        s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, qf[c], s[u], 0, 0, 0);
      }
    }
    const bool masked = key0 + kKeys - 1 > row_first;
    if (masked) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (key0 + 32 * u + 8 * (i >> 2) + 4 * h + (i & 3) > row) s[u][i] = -INFINITY;
    }
    float most = s[0][0];
#pragma unroll
    for (int i = 1; i < 32; ++i) most = fmaxf(most, s[i >> 4][i & 15]);
    most *= A.scale_log2e;
    if (__any(most > m + kSlack)) {
      most = fmaxf(most, __shfl_xor(most, 32));
      const float mn = fmaxf(m, most), alpha = exp2_hw(m - mn);
      m = mn;
      l *= alpha;
#pragma unroll
      for (int d = 0; d < kDimTiles; ++d) o[d] *= alpha;
    }
    bf16x8 pf[4];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float p = exp2_hw(fmaf(s[i >> 4][i & 15], A.scale_log2e, -m));
      l += p;
      pf[i >> 3][i & 7] = (__bf16)p;
    }

    // O^T += V^T P^T: lane i of each sixteen names token i/4, dims 4(i%4)..
    const int i16 = lane & 15, sub = (lane >> 4) & 1;
#pragma unroll
    for (int d = 0; d < kDimTiles; ++d) {
      const int dim = 32 * d + 16 * sub + 4 * (i16 & 3);
#pragma unroll
      for (int c = 0; c < 4; ++c) {  // 16 tokens each
        s16x4 part[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int token = 16 * c + 8 * e + 4 * h + (i16 >> 2);
          part[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4*)(s_v[buf] + token * (2 * D) + swz_v<D>(token, dim >> 3) * 16 + (dim & 4) * 2));
        }
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        const s16x8 a = __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7);
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), pf[c], o[d], 0, 0, 0);
      }
    }
  }

  l += __shfl_xor(l, 32);
  if (row <= row_last) {
    const float inv = 1.0f / l;
    uint16_t* out = static_cast<uint16_t*>(A.o.p) + (int64_t)(sp.begin + row) * A.o.ts + hq * A.o.hs;
#pragma unroll
    for (int d = 0; d < kDimTiles; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        uint2 w;
        w.x = pack_bf2(o[d][i] * inv, o[d][i + 1] * inv);
        w.y = pack_bf2(o[d][i + 2] * inv, o[d][i + 3] * inv);
        *reinterpret_cast<uint2*>(out + 32 * d + 2 * i + 4 * h) = w;
      }
  }
}

// ------------------------------------------------------------------- fp32
constexpr int kRows32 = 64;  // rows per work-group, 16 per wave

template <int D>
__global__ __launch_bounds__(256) void prompt_f32_kernel(const PromptArgs A) {
  constexpr int kVecs = D / 16;
  __shared__ int s_found;
  const int hq_n = A.q.heads;
  const int flat = blockIdx.x / hq_n, hq = blockIdx.x - flat * hq_n, hk = hq / A.G;
  const Span sp = find_span(A, flat, kRows32, &s_found);
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
  for (int key0 = 0; key0 <= row_last; key0 += 16) {
    f4 s{0, 0, 0, 0};
    const float* kr = kb + (int64_t)min(key0 + n, sp.len - 1) * A.k.ts + 4 * g;
#pragma unroll
    for (int c = 0; c < kVecs; ++c) {
      const f4 a = *reinterpret_cast<const f4*>(kr + 16 * c);
#pragma unroll
      for (int e = 0; e < 4; ++e) s = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], qf[c][e], s, 0, 0, 0);
    }
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
      l *= alpha;
#pragma unroll
      for (int d = 0; d < kVecs; ++d) o[d] *= alpha;
    }
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = exp2_hw(fmaf(s[i], A.scale_log2e, -m));
      l += p[i];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float* vr = vb + (int64_t)min(key0 + 4 * g + e, sp.len - 1) * A.v.ts + n;
#pragma unroll
      for (int d = 0; d < kVecs; ++d) o[d] = __builtin_amdgcn_mfma_f32_16x16x4f32(vr[16 * d], p[e], o[d], 0, 0, 0);
    }
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
    const int64_t blocks = ((int64_t)A.T / kRows + A.B) * A.q.heads;
    prompt_kernel<D><<<(unsigned)blocks, 64 * kWaves, 0, s>>>(A);
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
