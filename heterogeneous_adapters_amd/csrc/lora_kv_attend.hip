// lora_kv_attend: attention of a step's rows over the paged 4-bit cache.
//
// Mathematics: per row, one pass over the cached tokens with a running
// maximum m and sum l of exp2((s - m)), s = scale log2(e) q.K.  The keys of a
// request are split into chunks (lora_kv_build's plan); chunks of one row are
// joined by o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
//
// A work item is (16 rows = new tokens x heads that share a kv head, one
// chunk, one kv head), walked by a work-group of 4 waves that take every
// fourth step of 32 tokens and join their results in LDS.  Per step a wave
// reads the 17/16 byte per value pair once, converts the codes to bf16 with
// v_cvt_scalef32_pk_bf16_fp4 (exact), and multiplies on
// v_mfma_f32_16x16x32_bf16: S^T = K Q^T, whose result layout (row = lane%16,
// tokens 4g..4g+3 of each 16) is the B operand that O^T = V^T P^T needs, with
// the record's V order supplying A, so P never leaves its registers.  fp32
// rows are split into three bf16 terms (24 bits), the codes being exact.
#include "lora_kv_dev.h"
#include "lora_kv_host.h"

namespace lora {
namespace kv {

namespace {

constexpr int kThreads = 64 * kAttendWaves;
constexpr float kNone = -1e30f;  // running maximum before any visible key
// Rows keep their maximum until a score passes it by this much (a factor of
// 2^8 in p, without loss: p is scaled the same in the products and the sum).
constexpr float kSlack = 8.0f;

template <int NC>
struct Step {  // one wave's 32 tokens: two units' records
  uint32_t k[2][NC], v[2][NC];
  uint8_t ks[2][NC];
  uint32_t vs[2][NC];
};

template <int NC>
__device__ __forceinline__ void load_unit(const uint8_t* rec, int lane, uint32_t (&k)[NC], uint32_t (&v)[NC],
                                          uint8_t (&ks)[NC], uint32_t (&vs)[NC]) {
  const int m = lane & 15, g = lane >> 4;
  __builtin_memcpy(k, __builtin_assume_aligned(rec + (m * 4 + g) * 4 * NC, 4), 4 * NC);
  __builtin_memcpy(v, __builtin_assume_aligned(rec + 256 * NC + (g * 16 + m) * 4 * NC, 4), 4 * NC);
  __builtin_memcpy(ks, rec + 512 * NC + m * NC, NC);
  __builtin_memcpy(vs, __builtin_assume_aligned(rec + 528 * NC + 4 * g * NC, 4), 4 * NC);
}

__device__ __forceinline__ uint32_t fp4_pair(uint32_t w, float s, int byte) {
  switch (byte) {
    case 0: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    case 1: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    case 2: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    default: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  }
}
__device__ __forceinline__ float byte_scale(uint32_t w, int k) {
  return k == 0 ? scale_of<0>(w) : k == 1 ? scale_of<1>(w) : k == 2 ? scale_of<2>(w) : scale_of<3>(w);
}

__device__ __forceinline__ bf16x8 frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8, u32x4{a, b, c, d});
}

// x as NS bf16 terms: 8 bits each.
template <int NS>
__device__ __forceinline__ void split8(const float (&x)[8], bf16x8 (&f)[NS]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[s][i] = (__bf16)r[i];
      if (s + 1 < NS) r[i] -= (float)f[s][i];
    }
  }
}

template <class E, int NC>
__global__ __launch_bounds__(kThreads) void attend_kernel(const AttendArgs A) {
  constexpr int NS = sizeof(typename E::T) == 2 ? 1 : 3;
  constexpr int D = 32 * NC, LD = D + 4;
  typedef typename E::T T;
  __shared__ float s_o[kAttendWaves][kUnit][LD];
  __shared__ float s_m[kAttendWaves][kUnit], s_l[kAttendWaves][kUnit];

  const int hkv = A.cache.heads;
  const int item = blockIdx.x / hkv, kvh = blockIdx.x - item * hkv;
  const int n_items = A.counts[kCountItems], n_parts = A.counts[kCountParts], chunk = A.counts[kCountChunk];
  if (A.counts[kCountCheck] != check_word(A.counts[kCountB], A.counts[kCountT], n_items, n_parts) ||
      A.counts[kCountB] != A.B || A.counts[kCountT] != A.T || n_items > A.item_cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&A.counts[kCountFlags], LORA_KV_FLAG_BATCH);
    return;
  }
  if (item >= n_items) return;
  const int4 desc = A.items[item];
  const int seq = uniform(desc.x), tile = uniform(desc.y), ci = uniform(desc.z), part = uniform(desc.w);
  const int qs = uniform(A.q_indptr[seq]), qe = uniform(A.q_indptr[seq + 1]), kv = uniform(A.kv_len[seq]);
  const int G = A.G, nrows = (qe - qs) * G, row0 = tile * kUnit;
  const int pos0 = uniform(A.positions[qs]);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
  const int row = row0 + n, rowc = min(row, nrows - 1);
  const int jq = rowc / G, hq = kvh * G + rowc - jq * G;
  const int limit = min(pos0 + jq + 1, kv);  // this lane's row sees tokens below this
  const int limit0 = uniform(min(pos0 + row0 / G + 1, kv));
  const int begin = ci * chunk;
  const int end = min(begin + chunk, uniform(min(pos0 + min(row0 + kUnit - 1, nrows - 1) / G + 1, kv)));

  bf16x8 qf[NC][NS];
  {
    const T* q = static_cast<const T*>(A.q.p) + (int64_t)(qs + jq) * A.q.ts + hq * A.q.hs;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float x[8];
      load_n<8>(q + 32 * c + 8 * g, x);
      split8<NS>(x, qf[c]);
    }
  }

  f4 o[NC][2];
#pragma unroll
  for (int c = 0; c < NC; ++c) o[c][0] = o[c][1] = f4{0, 0, 0, 0};
  float m = kNone, l = 0.0f;

  const int32_t* trow = A.table + (int64_t)seq * A.tstride;
  const uint8_t* head = A.cache.base + ((int64_t)kvh << A.cache.bt_log2 >> 4) * (544 * NC);
  const int unit_mask = (1 << (A.cache.bt_log2 - 4)) - 1;
  const int first = begin / kTile + wave, last = (end + kTile - 1) / kTile;  // steps first, first+4, .. < last
  bool bad_block = false;

  // Block ids of 32 steps, two units each, one per lane; -1 outside the cache.
  auto fetch_ids = [&](int step) {
    const int token = (step + kAttendWaves * (lane >> 1)) * kTile + kUnit * (lane & 1);
    int id = 0;
    if (token < end) {
      id = trow[token >> A.cache.bt_log2];
      if ((unsigned)id >= (unsigned)A.cache.blocks) id = -1, bad_block = true;
    }
    return id;
  };
  auto load_step = [&](Step<NC>& s, int id0, int id1, int step) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int id = u ? id1 : id0, unit = 2 * step + u;
      const uint8_t* rec = head + max(id, 0) * A.cache.stride + (unit & unit_mask) * (544 * NC);
      load_unit<NC>(rec, lane, s.k[u], s.v[u], s.ks[u], s.vs[u]);
    }
  };

  if (first < last) {
    int ids = fetch_ids(first);
    Step<NC> cur, nxt;
    int id0 = __builtin_amdgcn_readlane(ids, 0), id1 = __builtin_amdgcn_readlane(ids, 1);
    load_step(cur, id0, id1, first);
    int k = 0;  // place of the current step among the fetched ids
    for (int step = first; step < last; step += kAttendWaves) {
      const int next = step + kAttendWaves;
      int nid0 = 0, nid1 = 0;
      if (++k == 32) {
        k = 0;
        ids = fetch_ids(next);
      }
      if (next < last) {
        nid0 = __builtin_amdgcn_readlane(ids, 2 * k);
        nid1 = __builtin_amdgcn_readlane(ids, 2 * k + 1);
        load_step(nxt, nid0, nid1, next);
      }

      // S^T = K Q^T
      f4 s[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        s[u] = f4{0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float sc = __uint_as_float((uint32_t)cur.ks[u][c] << 23);
          const uint32_t w = cur.k[u][c];
          const bf16x8 a = frag(fp4_pair(w, sc, 0), fp4_pair(w, sc, 1), fp4_pair(w, sc, 2), fp4_pair(w, sc, 3));
#pragma unroll
          for (int t = 0; t < NS; ++t) s[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, qf[c][t], s[u], 0, 0, 0);
        }
      }
      const int tok = step * kTile;
      if (tok + kTile > limit0 || id0 < 0 || id1 < 0) {  // some row sees less than the whole step
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int id = u ? id1 : id0, t0 = tok + kUnit * u + 4 * g;
          uint32_t keep = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (id < 0 || t0 + i >= limit) s[u][i] = -INFINITY;
            if (id >= 0 && t0 + i < end) keep |= 0xffu << (8 * i);
          }
          // bytes behind the last token may hold anything, a scale of NaN
          // among it: 0 * NaN must not reach the products
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            cur.v[u][c] &= keep;
#pragma unroll
            for (int b = 0; b < 4; ++b)
              if (!((keep >> (8 * ((4 * c + b) / NC))) & 1)) cur.vs[u][c] &= ~(0xffu << (8 * b));
          }
        }
      }

      float most = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                         fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3]))) * A.scale_log2e;
      if (__any(most > m + kSlack)) {
        most = fmaxf(most, __shfl_xor(most, 16));
        most = fmaxf(most, __shfl_xor(most, 32));
        const float mn = fmaxf(m, most), alpha = exp2_hw(m - mn);
        m = mn;
        l *= alpha;
#pragma unroll
        for (int c = 0; c < NC; ++c) o[c][0] *= alpha, o[c][1] *= alpha;
      }
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = exp2_hw(fmaf(s[i >> 2][i & 3], A.scale_log2e, -m));
        l += p[i];
      }
      bf16x8 pf[NS];
      split8<NS>(p, pf);

      // O^T += V^T P^T
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t r[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = j * NC + c;
            r[j] = fp4_pair(cur.v[u][c], byte_scale(cur.vs[u][at >> 2], at & 3), j);
          }
          lo[2 * u] = __builtin_amdgcn_perm(r[1], r[0], 0x05040100u);
          lo[2 * u + 1] = __builtin_amdgcn_perm(r[3], r[2], 0x05040100u);
          hi[2 * u] = __builtin_amdgcn_perm(r[1], r[0], 0x07060302u);
          hi[2 * u + 1] = __builtin_amdgcn_perm(r[3], r[2], 0x07060302u);
        }
        const bf16x8 alo = frag(lo[0], lo[1], lo[2], lo[3]), ahi = frag(hi[0], hi[1], hi[2], hi[3]);
#pragma unroll
        for (int t = 0; t < NS; ++t) {
          o[c][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(alo, pf[t], o[c][0], 0, 0, 0);
          o[c][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ahi, pf[t], o[c][1], 0, 0, 0);
        }
      }
      cur = nxt;
      id0 = nid0;
      id1 = nid1;
    }
  }
  if (__any(bad_block) && lane == 0) atomicOr(&A.counts[kCountFlags], LORA_KV_FLAG_BLOCK_RANGE);

  // join the four waves
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    *reinterpret_cast<f4*>(&s_o[wave][n][32 * c + 4 * g]) = o[c][0];
    *reinterpret_cast<f4*>(&s_o[wave][n][32 * c + 16 + 4 * g]) = o[c][1];
  }
  if (g == 0) {
    s_m[wave][n] = m;
    s_l[wave][n] = l;
  }
  __syncthreads();
  constexpr int kVec = kUnit * D / 4;  // vectors of 4 dims of the tile
  for (int i = threadIdx.x; i < kVec; i += kThreads) {
    const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
    if (row0 + r >= nrows) break;
    float M = s_m[0][r];
#pragma unroll
    for (int w = 1; w < kAttendWaves; ++w) M = fmaxf(M, s_m[w][r]);
    float L = 0.0f;
    f4 acc{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kAttendWaves; ++w) {
      const float a = exp2_hw(s_m[w][r] - M);
      L += a * s_l[w][r];
      acc += a * *reinterpret_cast<const f4*>(&s_o[w][r][d]);
    }
    if (part < 0) {
      const float inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);  // no visible key: zeros; NaN stays
      const int jr = (row0 + r) / G, h = kvh * G + row0 + r - jr * G;
      T* out = static_cast<T*>(A.o.p) + (int64_t)(qs + jr) * A.o.ts + h * A.o.hs + d;
#pragma unroll
      for (int e = 0; e < 4; ++e) from_f(out + e, acc[e] * inv);
    } else {
      float* p = A.part + ((int64_t)(part + ci) * hkv + kvh) * (kUnit * (D + 2));
      if (d == 0) p[r] = M, p[kUnit + r] = L;
      *reinterpret_cast<f4*>(p + 2 * kUnit + r * D + d) = acc;
    }
  }
}

// Joins the chunks of a tile.
template <class E, int NC>
__global__ __launch_bounds__(kThreads) void join_kernel(const AttendArgs A) {
  constexpr int D = 32 * NC;
  typedef typename E::T T;
  const int hkv = A.cache.heads;
  const int item = blockIdx.x / hkv, kvh = blockIdx.x - item * hkv;
  const int n_items = A.counts[kCountItems], n_parts = A.counts[kCountParts], chunk = A.counts[kCountChunk];
  if (A.counts[kCountCheck] != check_word(A.counts[kCountB], A.counts[kCountT], n_items, n_parts) ||
      A.counts[kCountB] != A.B || A.counts[kCountT] != A.T || item >= n_items || n_items > A.item_cap)
    return;
  const int4 desc = A.items[item];
  if (desc.z != 0 || desc.w < 0) return;
  const int seq = desc.x, row0 = desc.y * kUnit, G = A.G;
  const int qs = A.q_indptr[seq], nrows = (A.q_indptr[seq + 1] - qs) * G;
  const int chunks = (A.kv_len[seq] + chunk - 1) / chunk;
  const float* p0 = A.part + ((int64_t)desc.w * hkv + kvh) * (kUnit * (D + 2));
  const int64_t stride = (int64_t)hkv * (kUnit * (D + 2));
  for (int i = threadIdx.x; i < kUnit * D / 4; i += kThreads) {
    const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
    if (row0 + r >= nrows) break;
    float M = kNone;
    for (int c = 0; c < chunks; ++c) M = fmaxf(M, p0[c * stride + r]);
    float L = 0.0f;
    f4 acc{0, 0, 0, 0};
    for (int c = 0; c < chunks; ++c) {
      const float* p = p0 + c * stride;
      const float a = exp2_hw(p[r] - M);
      L += a * p[kUnit + r];
      acc += a * *reinterpret_cast<const f4*>(p + 2 * kUnit + r * D + d);
    }
    const float inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);
    const int jr = (row0 + r) / G, h = kvh * G + row0 + r - jr * G;
    T* out = static_cast<T*>(A.o.p) + (int64_t)(qs + jr) * A.o.ts + h * A.o.hs + d;
#pragma unroll
    for (int e = 0; e < 4; ++e) from_f(out + e, acc[e] * inv);
  }
}

template <class E, int NC>
hipError_t launch(const AttendArgs& A, int blocks, hipStream_t s) {
  attend_kernel<E, NC><<<blocks, kThreads, 0, s>>>(A);
  join_kernel<E, NC><<<blocks, kThreads, 0, s>>>(A);
  return hipGetLastError();
}

template <class E>
hipError_t launch_nc(const AttendArgs& A, int blocks, hipStream_t s) {
  switch (A.cache.nc) {
    case 1: return launch<E, 1>(A, blocks, s);
    case 2: return launch<E, 2>(A, blocks, s);
    case 3: return launch<E, 3>(A, blocks, s);
    case 4: return launch<E, 4>(A, blocks, s);
    case 5: return launch<E, 5>(A, blocks, s);
    case 6: return launch<E, 6>(A, blocks, s);
    case 7: return launch<E, 7>(A, blocks, s);
    default: return launch<E, 8>(A, blocks, s);
  }
}

}  // namespace

hipError_t launch_attend(const AttendArgs& A, int dtype, int blocks, hipStream_t s) {
  return dtype == LORA_DTYPE_BF16 ? launch_nc<Bf16>(A, blocks, s) : launch_nc<F32>(A, blocks, s);
}

}  // namespace kv
}  // namespace lora
