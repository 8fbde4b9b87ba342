// Kernels of attention over the paged 4-bit cache, shared by lora_kv_attend and
// lora_kv_attend_shared (internal).
#pragma once

#include <type_traits>

#include "lora_kv_dev.h"
#include "lora_kv_host.h"

namespace lora {
namespace kv {

namespace {

constexpr int kWaves = 4;  // per work-group of attend_kernel

// Partial results cross XCDs within the launch: agent-scope accesses (write
// through, and past the reader's own L2), 8 bytes each, no cache maintenance.
__device__ __forceinline__ void put2(float* p, float a, float b) {
  const uint64_t u = (uint64_t)__float_as_uint(a) | (uint64_t)__float_as_uint(b) << 32;
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 get2(const float* p) {
  const uint64_t u = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__uint_as_float((uint32_t)u), __uint_as_float((uint32_t)(u >> 32)));
}

template <int NC>
struct Unit {  // a lane's share of a record
  uint32_t k[NC], v[NC], ks[(NC + 3) / 4], vs[NC];
};

// Uniform record, 32-bit lane offsets: scalar base and one offset register.
template <int NC>
__device__ __forceinline__ void load_unit(const uint8_t* rec, int lane, Unit<NC>& x) {
  const uint32_t m = lane & 15, g = lane >> 4;
  __builtin_memcpy(x.k, __builtin_assume_aligned(rec + (m * 4 + g) * 4 * NC, 4), 4 * NC);
  __builtin_memcpy(x.v, __builtin_assume_aligned(rec + 256 * NC + (g * 16 + m) * 4 * NC, 4), 4 * NC);
  __builtin_memcpy(x.ks, rec + 512 * NC + m * NC, NC);
  __builtin_memcpy(x.vs, __builtin_assume_aligned(rec + 528 * NC + 4 * g * NC, 4), 4 * NC);
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

// Whether the batch's plan was built for this call.
__device__ __forceinline__ bool plan_ok(const AttendArgs& A) {
  const int32_t* c = A.counts;
  return c[kCountCheck] == check_word(c[kCountB], c[kCountT], c[kCountItems], c[kCountMid], c[kCountWide], c[kCountParts]) &&
         c[kCountB] == A.B && c[kCountT] == A.T && c[kCountItems] <= A.item_cap && c[kCountMid] <= A.item_cap &&
         c[kCountWide] <= A.item_cap;
}

// Whether the shared plan was built for this call.
__device__ __forceinline__ bool share_ok(const SharedArgs& A) {
  const int32_t* c = A.share;
  return c[kShareCheck] == share_word(c) && c[kShareB] == A.B && c[kShareT] == A.T && c[kShareGroups] == A.groups &&
         c[kShareRows] <= A.row_cap && max(max(c[0], c[1]), max(c[2], c[3])) <= A.item_cap;
}

// A work item: its request, rows and keys.
struct Item {
  int seq, row0, ci, part;    // part: the tile's first partial result, -1 when the tile is not split
  int qs, nrows, pos0, kv;    // first token row, rows, first position, cached tokens
  int begin, end, chunks;     // keys of this item, items of the tile
  int base;                   // cached tokens before those that pos0, kv, begin and end count (a multiple of 16)
};
// The descriptor is read along with the counters it is checked against (the
// grid, class_cap, is at most item_cap), so that one trip to memory serves
// both.  `rows`: rows that the kernel takes of the tile, from row0 + skip on.
__device__ __forceinline__ bool read_item(const AttendArgs& A, int cls, int count_at, int item, int skip, int rows, Item& it) {
  const int4* d = A.items + 2 * ((int64_t)cls * A.item_cap + item);
  const int4 x = d[0], y = d[1];
  if (!plan_ok(A)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&A.counts[kCountFlags], LORA_KV_FLAG_BATCH);
    return false;
  }
  if (item >= A.counts[count_at]) return false;
  it.seq = uniform(x.x), it.row0 = uniform(x.y) + skip, it.ci = uniform(x.z), it.part = uniform(x.w);
  it.qs = uniform(y.x), it.nrows = uniform(y.y), it.pos0 = uniform(y.z), it.kv = uniform(y.w);
  if (it.row0 >= it.nrows) return false;
  const int sees = min(it.pos0 + min(it.row0 + rows - 1, it.nrows - 1) / A.G + 1, it.kv);
  const int chunk = even_chunk(it.kv, A.counts[cls == 2 ? kCountChunkWide : kCountChunk]);
  it.begin = it.part < 0 ? 0 : it.ci * chunk;
  it.end = it.part < 0 ? sees : min(it.begin + chunk, sees);
  it.chunks = it.part < 0 ? 1 : (it.kv + chunk - 1) / chunk;
  it.base = 0;
  return true;
}

// An item of a shared step (lora_kv_share): keys of a group's prefix or of a
// request's rest, always to a partial result.
__device__ __forceinline__ bool read_item(const SharedArgs& A, int, int, int item, int skip, int rows, Item& it) {
  // list 1's launch takes list 0's items of 16 rows along, before its own
  const int list = A.list == 1 && item < A.first_items ? 0 : A.list;
  if (A.list == 1 && list == 1) item -= A.first_items;
  const int4* d = A.items + kShareItem * ((int64_t)list * A.item_cap + item);
  const int4 x = d[0], y = d[1], z = d[2];
  if (!share_ok(A)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&A.counts[kCountFlags], LORA_KV_FLAG_BATCH);
    return false;
  }
  if (item >= A.share[list]) return false;
  it.seq = uniform(x.x), it.row0 = uniform(x.y) + skip, it.part = uniform(x.z), it.base = uniform(x.w);
  it.qs = uniform(y.x), it.nrows = uniform(y.y), it.pos0 = uniform(y.z), it.kv = uniform(y.w);
  if (it.row0 >= it.nrows) return false;
  it.begin = uniform(z.x), it.chunks = 1, it.ci = 0;
  it.end = min(uniform(z.y), min(it.pos0 + min(it.row0 + rows - 1, it.nrows - 1) / A.G + 1, it.kv));
  return true;
}

// Four dims of a row's partial result; it.part is the one of the item's first row.
template <int D>
__device__ __forceinline__ void store_part(const SharedArgs& A, const Item& it, int kvh, int row, int d, f4 acc, float m, float l) {
  const int64_t at = (int64_t)(it.part + row) * A.cache.heads + kvh;
  *reinterpret_cast<f4*>(A.part + at * D + d) = acc;
  if (d == 0) *reinterpret_cast<float2*>(A.part_ml + at * 2) = make_float2(m, l);
}

// Reciprocal of a row's sum: zero for a row that saw no key, NaN kept.
__device__ __forceinline__ float inverse(float l) { return l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l); }

// A part (16 rows of one chunk): rows of D sums, then (m, l) pairs.  A tile's
// parts lie by chunk, then by 16 rows.
template <int D>
__device__ __forceinline__ float* part_at(const AttendArgs& A, int part, int kvh) {
  return A.part + ((int64_t)part * A.cache.heads + kvh) * (kUnit * (D + 2));
}

// Four dims of an output row.
template <class E>
__device__ __forceinline__ void store_out(const AttendArgs& A, const Item& it, int kvh, int row, int d, f4 acc, float inv) {
  typedef typename E::T T;
  const int jr = row / A.G;
  T* out = static_cast<T*>(A.o.p) + (int64_t)(it.qs + jr) * A.o.ts + (kvh * A.G + row - jr * A.G) * A.o.hs + d;
  if constexpr (sizeof(T) == 2) {
    uint2 w;
    w.x = pack_bf2(acc[0] * inv, acc[1] * inv);
    w.y = pack_bf2(acc[2] * inv, acc[3] * inv);
    *reinterpret_cast<uint2*>(out) = w;
  } else {
    *reinterpret_cast<f4*>(out) = acc * inv;
  }
}

// Counts a work-group's arrival at its tile; true in the one that comes last,
// for which every part of the tile is visible.  A wave's wait makes its own
// stores visible before the arrival is counted.
__device__ __forceinline__ bool arrive_last(const AttendArgs& A, const Item& it, int part, int kvh, int* s_last) {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  wait_vm<0>();
  __syncthreads();
  if (threadIdx.x == 0) {
    int32_t* count = A.arrive + (int64_t)part * A.cache.heads + kvh;
    const int before = __hip_atomic_fetch_add(count, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *s_last = before == it.chunks - 1;
    if (*s_last) __hip_atomic_store(count, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // for the next layer
  }
  __syncthreads();
  const bool last = *s_last != 0;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
  return last;
}

// Joins the chunks of `rt` times 16 rows from it.row0 on, whose first parts
// are `part`, part + 1, ..; `units` parts per chunk.  In the order of the
// chunks, whichever work-group does it.  scratch: 6 floats per thread.
template <class E, int D, int kThreads>
__device__ __forceinline__ void join(const AttendArgs& A, const Item& it, int part, int units, int rt, int kvh, float* scratch) {
  constexpr int kVecs = D / 4;
  constexpr int kBatch = 8;  // chunks in flight per thread
  for (int r = 0; r < rt; ++r) {
    const int live = min(it.nrows - it.row0 - r * kUnit, kUnit);
    if (live <= 0) break;
    const int tasks = live * kVecs;
    const int groups = max(1, min(kThreads / tasks, it.chunks));  // threads per task, each every groups-th chunk
    for (int t0 = 0; t0 < tasks; t0 += kThreads) {  // more than one turn only with one group
      const int grp = threadIdx.x / tasks, task = t0 + threadIdx.x - (groups > 1 ? grp * tasks : 0);
      const int row = task / kVecs, d = (task - row * kVecs) * 4;
      const bool work = task < tasks && (groups == 1 || grp < groups);
      float M = kNone, L = 0.0f;
      f4 acc{0, 0, 0, 0};
      if (work) {
        for (int c = groups > 1 ? grp : 0; c < it.chunks; c += kBatch * groups) {
          float2 ml[kBatch], lo[kBatch], hi[kBatch];
#pragma unroll
          for (int e = 0; e < kBatch; ++e) {
            const float* p = part_at<D>(A, part + min(c + e * groups, it.chunks - 1) * units + r, kvh);
            ml[e] = get2(p + kUnit * D + 2 * row);
            lo[e] = get2(p + row * D + d);
            hi[e] = get2(p + row * D + d + 2);
          }
#pragma unroll
          for (int e = 0; e < kBatch; ++e) {
            if (c + e * groups >= it.chunks) break;
            const float mn = fmaxf(M, ml[e].x), a = exp2_hw(M - mn), b = exp2_hw(ml[e].x - mn);
            M = mn;
            L = L * a + ml[e].y * b;
            acc = acc * a + b * f4{lo[e].x, lo[e].y, hi[e].x, hi[e].y};
          }
        }
      }
      if (groups > 1) {
        __syncthreads();
        if (work) {
          float* s = scratch + threadIdx.x * 6;
          s[0] = M, s[1] = L;
          s[2] = acc[0], s[3] = acc[1], s[4] = acc[2], s[5] = acc[3];
        }
        __syncthreads();
        if (work && grp == 0) {
          for (int e = 1; e < groups; ++e) {
            const float* s = scratch + (threadIdx.x + e * tasks) * 6;
            const float mn = fmaxf(M, s[0]), a = exp2_hw(M - mn), b = exp2_hw(s[0] - mn);
            M = mn;
            L = L * a + s[1] * b;
            acc = acc * a + b * f4{s[2], s[3], s[4], s[5]};
          }
        }
      }
      if (work && grp == 0) store_out<E>(A, it, kvh, it.row0 + r * kUnit + row, d, acc, inverse(L));
      if (groups > 1) break;
    }
  }
}

// RT: tiles of 16 rows per work item.  CLS: the items' class; the fp32 kernel
// takes the 128 rows of class 2 in four pieces.  Three waves per SIMD hold two
// steps' records of a decode step in registers (140 of 168).
template <class E, int NC, int RT, int CLS, class Args>
__global__ __launch_bounds__(64 * kWaves, RT == 1 && NC <= 4 && sizeof(typename E::T) == 2 ? 3 : 1) void attend_kernel(const Args A) {
  constexpr int W = kWaves, kThreads = 64 * W;
  constexpr int NS = sizeof(typename E::T) == 2 ? 1 : 3;
  constexpr int D = 32 * NC, LD = D + 4, kVecs = D / 4;
  constexpr int kPieces = CLS >= 2 ? (CLS == 2 ? kWideRows : kPrefixRows) / (kUnit * RT) : 1, kUnits = RT * kPieces;
  typedef typename E::T T;
  __shared__ float s_o[W][kUnit][LD];
  __shared__ float s_m[W][kUnit], s_l[W][kUnit];
  __shared__ int s_last;

  const int hkv = A.cache.heads;
  const int item = blockIdx.x / (hkv * kPieces), piece = blockIdx.x / hkv % kPieces, kvh = blockIdx.x % hkv;
  Item it;
  if (!read_item(A, CLS, CLS == 0 ? kCountItems : CLS == 1 ? kCountMid : kCountWide, item, piece * RT * kUnit, RT * kUnit, it)) return;
  const int part = it.part < 0 ? -1 : it.part + piece * RT;
  const int G = A.G, nrows = it.nrows, row0 = it.row0, qs = it.qs, pos0 = it.pos0, kv = it.kv, begin = it.begin, end = it.end;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
  const int limit0 = uniform(min(pos0 + row0 / G + 1, kv));

  int limit[RT];  // this lane's rows see tokens below these
  bf16x8 qf[RT][NC][NS];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = min(row0 + r * kUnit + n, nrows - 1), jq = row / G;
    limit[r] = min(pos0 + jq + 1, kv);
    const T* q = static_cast<const T*>(A.q.p) + (int64_t)(qs + jq) * A.q.ts + (kvh * G + row - jq * G) * A.q.hs;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float x[8];
      load_n<8>(q + 32 * c + 8 * g, x);
      split8<NS>(x, qf[r][c]);
    }
  }

  f4 o[RT][NC][2];
  float m[RT], l[RT];
  bool far = false;  // some row's scores are
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    m[r] = kNone;
    l[r] = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) o[r][c][0] = o[r][c][1] = f4{0, 0, 0, 0};
  }

  const int32_t* trow = A.table + (int64_t)it.seq * A.tstride;
  const uint8_t* head = A.cache.base + ((int64_t)kvh << A.cache.bt_log2 >> 4) * (544 * NC);
  const int unit_mask = (1 << (A.cache.bt_log2 - 4)) - 1;
  const int first = begin / kTile + wave, last = (end + kTile - 1) / kTile;  // steps first, first+W, .. < last
  bool bad_block = false;

  // Block ids of 32 steps, two units each, one per lane; -1 outside the cache.
  auto fetch_ids = [&](int step) {
    const int token = (step + W * (lane >> 1)) * kTile + kUnit * (lane & 1);
    int id = 0;
    if (token < end) {
      const int at = (it.base + token) >> A.cache.bt_log2;
      id = at < A.width ? trow[at] : -1;  // a table of another call may be narrower
      if ((unsigned)id >= (unsigned)A.cache.blocks) id = -1, bad_block = true;
    }
    return id;
  };
  int ids = 0, ids_at = -32;  // block ids of steps first + W * (ids_at ..  ids_at + 31)
  const int mine = (last - first + W - 1) / W;  // this wave's steps
  // The records of this wave's i-th step.  Past its last step the last one's:
  // loads without a branch, so that no wait counts on their absence.
  auto load_step = [&](Unit<NC> (&x)[2], int (&id)[2], int i) {
    i = min(i, mine - 1);
    if (i >= ids_at + 32) {
      ids_at = i;
      ids = fetch_ids(first + i * W);
      wait_vm<0>();
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      id[u] = __builtin_amdgcn_readlane(ids, 2 * (i - ids_at) + u);
      const int unit = (it.base >> 4) + 2 * (first + i * W) + u;
      load_unit<NC>(head + max(id[u], 0) * A.cache.stride + (unit & unit_mask) * (544 * NC), lane, x[u]);
    }
  };
  auto compute = [&](Unit<NC> (&cur)[2], const int (&ids2)[2], int step) {
    const int id0 = ids2[0], id1 = ids2[1];
    // S^T = K Q^T
    f4 s[RT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int r = 0; r < RT; ++r) s[r][u] = f4{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float sc = byte_scale(cur[u].ks[c >> 2], c & 3);
        const uint32_t w = cur[u].k[c];
        const bf16x8 a = frag(fp4_pair(w, sc, 0), fp4_pair(w, sc, 1), fp4_pair(w, sc, 2), fp4_pair(w, sc, 3));
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int t = 0; t < NS; ++t) s[r][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, qf[r][c][t], s[r][u], 0, 0, 0);
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
#pragma unroll
          for (int r = 0; r < RT; ++r)
            if (id < 0 || t0 + i >= limit[r]) s[r][u][i] = -INFINITY;
          if (id >= 0 && t0 + i < end) keep |= 0xffu << (8 * i);
        }
        // bytes behind the last token may hold anything, a scale of NaN
        // among it: 0 * NaN must not reach the products
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          cur[u].v[c] &= keep;
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (!((keep >> (8 * ((4 * c + b) / NC))) & 1)) cur[u].vs[c] &= ~(0xffu << (8 * b));
        }
      }
    }

    bf16x8 pf[RT][NS];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float most = fmaxf(fmaxf(fmaxf(s[r][0][0], s[r][0][1]), fmaxf(s[r][0][2], s[r][0][3])),
                         fmaxf(fmaxf(s[r][1][0], s[r][1][1]), fmaxf(s[r][1][2], s[r][1][3]))) * A.scale_log2e;
      if (__any(most > m[r] + kSlack)) {
        most = fmaxf(most, __shfl_xor(most, 16));
        most = fmaxf(most, __shfl_xor(most, 32));
        const float mn = fmaxf(m[r], most), alpha = exp2_hw(m[r] - mn);
        m[r] = mn;
        far = far || __any(is_far(mn));
        l[r] *= alpha;
#pragma unroll
        for (int c = 0; c < NC; ++c) o[r][c][0] *= alpha, o[r][c][1] *= alpha;
      }
      float scale = A.scale_log2e, less = m[r];
      if (far) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[r][i >> 2][i & 3] = far_exponent(s[r][i >> 2][i & 3], scale, less);
        scale = 1.0f, less = 0.0f;
      }
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = exp2_hw(fmaf(s[r][i >> 2][i & 3], scale, -less));
        if (NS > 1) l[r] += p[i];
      }
      split8<NS>(p, pf[r]);
      if (NS == 1) l[r] = add8(pf[r][0], l[r]);
    }

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
          r[j] = fp4_pair(cur[u].v[c], byte_scale(cur[u].vs[at >> 2], at & 3), j);
        }
        lo[2 * u] = __builtin_amdgcn_perm(r[1], r[0], 0x05040100u);
        lo[2 * u + 1] = __builtin_amdgcn_perm(r[3], r[2], 0x05040100u);
        hi[2 * u] = __builtin_amdgcn_perm(r[1], r[0], 0x07060302u);
        hi[2 * u + 1] = __builtin_amdgcn_perm(r[3], r[2], 0x07060302u);
      }
      const bf16x8 alo = frag(lo[0], lo[1], lo[2], lo[3]), ahi = frag(hi[0], hi[1], hi[2], hi[3]);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NS; ++t) {
          o[r][c][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(alo, pf[r][t], o[r][c][0], 0, 0, 0);
          o[r][c][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ahi, pf[r][t], o[r][c][1], 0, 0, 0);
        }
    }
  };
  if (mine > 0) {
    Unit<NC> one[2], two[2];
    int id_one[2], id_two[2];
    load_step(one, id_one, 0);
    for (int i = 0; i < mine; i += 2) {
      load_step(two, id_two, i + 1);
      compute(one, id_one, first + i * W);
      if (i + 1 >= mine) break;
      load_step(one, id_one, i + 2);
      compute(two, id_two, first + (i + 1) * W);
    }
  }
  if (__any(bad_block) && lane == 0) atomicOr(&A.counts[kCountFlags], LORA_KV_FLAG_BLOCK_RANGE);

  // join the waves
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    if (r) __syncthreads();
    float lr = l[r];
    lr += __shfl_xor(lr, 16);
    lr += __shfl_xor(lr, 32);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      *reinterpret_cast<f4*>(&s_o[wave][n][32 * c + 4 * g]) = o[r][c][0];
      *reinterpret_cast<f4*>(&s_o[wave][n][32 * c + 16 + 4 * g]) = o[r][c][1];
    }
    if (g == 0) {
      s_m[wave][n] = m[r];
      s_l[wave][n] = lr;
    }
    __syncthreads();
    const int live = min(nrows - row0 - r * kUnit, kUnit);
    for (int i = threadIdx.x; i < live * kVecs; i += kThreads) {
      const int row = i / kVecs, d = (i - row * kVecs) * 4;
      float M = s_m[0][row];
#pragma unroll
      for (int w = 1; w < W; ++w) M = fmaxf(M, s_m[w][row]);
      float L = 0.0f;
      f4 acc{0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float a = exp2_hw(s_m[w][row] - M);
        L += a * s_l[w][row];
        acc += a * *reinterpret_cast<const f4*>(&s_o[w][row][d]);
      }
      if constexpr (Args::kShared) {
        store_part<D>(A, it, kvh, (piece * RT + r) * kUnit + row, d, acc, M, L);
      } else if (part < 0) {
        store_out<E>(A, it, kvh, row0 + r * kUnit + row, d, acc, inverse(L));
      } else {
        float* p = part_at<D>(A, part + it.ci * kUnits + r, kvh);
        put2(p + row * D + d, acc[0], acc[1]);
        put2(p + row * D + d + 2, acc[2], acc[3]);
        if (d == 0) put2(p + kUnit * D + 2 * row, M, L);
      }
    }
  }
  if constexpr (!Args::kShared) {
    if (part < 0 || !arrive_last(A, it, part, kvh, &s_last)) return;
    join<E, D, kThreads>(A, it, part, kUnits, RT, kvh, &s_o[0][0][0]);
  }
}

// ------------------------------------------------------- requests of many rows
// 128 rows on the same keys: tiles of 64 are converted to bf16 once, a unit of
// 16 tokens by each wave, into LDS, while the tile before is multiplied with
// v_mfma_f32_32x32x16_bf16, 32 rows per wave.  K lies by token, V by dim in the
// token order of P's registers, both XOR-swizzled in 16-byte pieces against
// the 64 banks.  Four chunks of 512 tokens over 5000, 32 query heads: 214 to
// 225 us, 670-710 TFLOP/s (32 rows without LDS: 292).  Two waves share a SIMD;
// while a compute unit is busy, conversions and exponentials take 45 % of its
// SIMDs' time and products 41 %, and units are busy for about 70 % of the launch:
// the chunks' work-groups are all resident at once and end at different times.
template <int NC, class Args>
__global__ __launch_bounds__(256, 2) void attend_wide_kernel(const Args A) {
  constexpr int D = 32 * NC, kThreads = 256, kKeys = 64, kUnits = kWideRows / kUnit;
  constexpr int kSteps = D / 16, kDims = D / 32;
  constexpr int kKVar = D % 128 == 0 ? 8 : D % 64 == 0 ? 4 : 2;
  __shared__ __attribute__((aligned(128))) uint8_t s_k[2][kKeys * D * 2], s_v[2][kKeys * D * 2];
  __shared__ __attribute__((aligned(4))) uint8_t s_bad[2][4];  // a tile's units whose block is outside the cache
  __shared__ int s_last;
  auto swz_k = [](int token, int piece) {
    return D % 128 == 0 ? piece ^ (token & 15) : D % 64 == 0 ? piece ^ ((token >> 1) & 7) : piece ^ ((token >> 2) & 3);
  };

  const int hkv = A.cache.heads;
  const int item = blockIdx.x / hkv, kvh = blockIdx.x - item * hkv;
  Item it;
  if (!read_item(A, 2, kCountWide, item, 0, kWideRows, it)) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 31, h = lane >> 5;
  const int m16 = lane & 15, g = lane >> 4;
  const int G = A.G, row_first = it.row0 + wave * 32;
  const int row = min(row_first + n, it.nrows - 1), jq = row / G;
  const bool live = row_first < it.nrows;
  const int limit = min(it.pos0 + jq + 1, it.kv);
  const int limit_first = uniform(min(it.pos0 + min(row_first, it.nrows - 1) / G + 1, it.kv));
  const int limit_last = live ? uniform(min(it.pos0 + min(row_first + 31, it.nrows - 1) / G + 1, it.kv)) : 0;

  bf16x8 qf[kSteps];
  {
    const uint16_t* q = static_cast<const uint16_t*>(A.q.p) + (int64_t)(it.qs + jq) * A.q.ts + (kvh * G + row - jq * G) * A.q.hs;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) qf[s] = *reinterpret_cast<const bf16x8*>(q + 16 * s + 8 * h);
  }

  const int32_t* trow = A.table + (int64_t)it.seq * A.tstride;
  const uint8_t* head = A.cache.base + ((int64_t)kvh << A.cache.bt_log2 >> 4) * (544 * NC);
  const int unit_mask = (1 << (A.cache.bt_log2 - 4)) - 1;
  const int n_tiles = (max(it.end - it.begin, 0) + kKeys - 1) / kKeys;
  bool bad_block = false;

  // Block ids of this wave's unit in 64 tiles, one per lane; -1 outside the cache.
  auto fetch_ids = [&](int tile) {
    const int token = it.begin + (tile + lane) * kKeys + kUnit * wave;
    int id = 0;
    if (token < it.end) {
      const int at = (it.base + token) >> A.cache.bt_log2;
      id = at < A.width ? trow[at] : -1;  // a table of another call may be narrower
      if ((unsigned)id >= (unsigned)A.cache.blocks) id = -1, bad_block = true;
    }
    return id;
  };
  Unit<NC> raw;
  int raw_id = 0;  // its block
  int ids = fetch_ids(0);
  auto load = [&](int tile) {
    if (tile && tile % 64 == 0) ids = fetch_ids(tile);
    raw_id = __builtin_amdgcn_readlane(ids, tile % 64);
    const int token = it.begin + tile * kKeys + kUnit * wave;
    // behind the last token: the id is 0, a block of the cache
    const uint8_t* rec = head + max(raw_id, 0) * A.cache.stride + (((it.base + token) >> 4) & unit_mask) * (544 * NC);
    load_unit<NC>(rec, lane, raw);
  };
  // The unit in registers to bf16 in LDS.
  auto convert = [&](int tile, auto which) {
    constexpr int buf = which;
    const int token = it.begin + tile * kKeys + kUnit * wave;
    if (lane == 0) s_bad[buf][wave] = raw_id < 0;
    if (raw_id < 0 || token + kUnit > it.end) {
      // bytes behind the last token may hold anything, a scale of NaN among it
      uint32_t keep = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (raw_id >= 0 && token + 4 * g + i < it.end) keep |= 0xffu << (8 * i);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        raw.v[c] &= keep;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (!((keep >> (8 * ((4 * c + b) / NC))) & 1)) raw.vs[c] &= ~(0xffu << (8 * b));
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const float sc = byte_scale(raw.ks[c >> 2], c & 3);
      const int t = kUnit * wave + m16;
      *reinterpret_cast<u32x4*>(s_k[buf] + t * (2 * D) + swz_k(t, 4 * c + g) * 16) =
          u32x4{fp4_pair(raw.k[c], sc, 0), fp4_pair(raw.k[c], sc, 1), fp4_pair(raw.k[c], sc, 2), fp4_pair(raw.k[c], sc, 3)};
      uint32_t r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = j * NC + c;
        r[j] = fp4_pair(raw.v[c], byte_scale(raw.vs[at >> 2], at & 3), j);
      }
      // tokens 4g..4g+3 of the unit, one dim: 8 bytes; the two halves of a
      // 16-byte piece are the tokens 8 apart that one lane of P holds
      const int piece = 2 * wave + (g & 1), half = (g >> 1) * 8;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int dim = 32 * c + 16 * e + m16;
        const uint32_t sel = e ? 0x07060302u : 0x05040100u;
        *reinterpret_cast<uint2*>(s_v[buf] + dim * (2 * kKeys) + ((piece ^ ((dim >> 1) & 7)) * 16) + half) =
            make_uint2(__builtin_amdgcn_perm(r[1], r[0], sel), __builtin_amdgcn_perm(r[3], r[2], sel));
      }
    }
  };

  int k_at[kKVar], v_at[4];
#pragma unroll
  for (int c = 0; c < kKVar; ++c) k_at[c] = n * (2 * D) + swz_k(n, 2 * c + h) * 16;
#pragma unroll
  for (int c = 0; c < 4; ++c) v_at[c] = n * (2 * kKeys) + ((2 * c + h) ^ ((n >> 1) & 7)) * 16;

  f16v o[kDims];
#pragma unroll
  for (int d = 0; d < kDims; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = kNone, l = 0.0f;
  bool far = false;  // some row's scores are

  auto compute = [&](int tile, auto which) {
    constexpr int buf = which;
    const int key0 = it.begin + tile * kKeys;
    const uint8_t *sk = s_k[buf], *sv = s_v[buf];
    const uint32_t bad_units = *reinterpret_cast<const uint32_t*>(s_bad[buf]);
    f16v s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        const bf16x8 a = *reinterpret_cast<const bf16x8*>(sk + k_at[c % kKVar] + u * 32 * (2 * D) + (c / kKVar) * (kKVar * 32));
        s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, qf[c], s[u], 0, 0, 0);
      }
    // reads six ahead of their products
    __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
#pragma unroll
    for (int i = 0; i < kSteps * 2 - 6; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, 6, 0);
    const uint32_t bad = (uint32_t)uniform((int)bad_units);
    if (key0 + kKeys > limit_first || bad) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int hide = (bad >> (8 * (2 * u + (i >> 3)))) & 1 ? 0x40000000 : 0;
          if (key0 + 32 * u + 8 * (i >> 2) + 4 * h + (i & 3) + hide >= limit) s[u][i] = -INFINITY;
        }
    }
    float most = s[0][0];
#pragma unroll
    for (int i = 1; i < 32; ++i) most = fmaxf(most, s[i >> 4][i & 15]);
    most *= A.scale_log2e;
    if (__any(most > m + kSlack)) {
      most = fmaxf(most, __shfl_xor(most, 32));
      const float mn = fmaxf(m, most), alpha = exp2_hw(m - mn);
      m = mn;
      far = far || __any(is_far(mn));
      l *= alpha;
#pragma unroll
      for (int d = 0; d < kDims; ++d) o[d] *= alpha;
    }
    float scale = A.scale_log2e, less = m;
    if (far) {
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i >> 4][i & 15] = far_exponent(s[i >> 4][i & 15], scale, less);
      scale = 1.0f, less = 0.0f;
    }
    bf16x8 pf[4];
#pragma unroll
    for (int i = 0; i < 32; ++i) pf[i >> 3][i & 7] = (__bf16)exp2_hw(fmaf(s[i >> 4][i & 15], scale, -less));
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int d = 0; d < kDims; ++d) {
        const bf16x8 a = *reinterpret_cast<const bf16x8*>(sv + v_at[c] + d * (32 * 2 * kKeys));
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, pf[c], o[d], 0, 0, 0);
        if (d == 0) l = add8(pf[c], l);
      }
  };

  if (n_tiles > 0) {
    const std::integral_constant<int, 0> zero;
    const std::integral_constant<int, 1> one;
    auto turn = [&](int t, auto mine, auto other) {
      __syncthreads();  // tile t is in LDS, and tile t-1's buffer is free
      if (t + 1 < n_tiles) {
        convert(t + 1, other);
        if (t + 2 < n_tiles) load(t + 2);
      }
      if (it.begin + t * kKeys < limit_last) compute(t, mine);
    };
    load(0);
    convert(0, zero);
    if (n_tiles > 1) load(1);
    for (int t = 0; t < n_tiles; t += 2) {
      turn(t, zero, one);
      if (t + 1 < n_tiles) turn(t + 1, one, zero);
    }
  }
  if (__any(bad_block) && lane == 0) atomicOr(&A.counts[kCountFlags], LORA_KV_FLAG_BLOCK_RANGE);

  l += __shfl_xor(l, 32);
  if (row_first + n < it.nrows) {
    const float inv = inverse(l);
    float* p = Args::kShared || it.part < 0 ? nullptr : part_at<D>(A, it.part + it.ci * kUnits + 2 * wave + (n >> 4), kvh);
#pragma unroll
    for (int d = 0; d < kDims; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int dim = 32 * d + 2 * i + 4 * h;
        const f4 acc{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
        if constexpr (Args::kShared) {
          store_part<D>(A, it, kvh, wave * 32 + n, dim, acc, m, l);
        } else if (it.part < 0) {
          store_out<Bf16>(A, it, kvh, row, dim, acc, inv);
        } else {
          put2(p + (n & 15) * D + dim, acc[0], acc[1]);
          put2(p + (n & 15) * D + dim + 2, acc[2], acc[3]);
        }
      }
    if (!Args::kShared && it.part >= 0 && h == 0) put2(p + kUnit * D + 2 * (n & 15), m, l);
  }
  if constexpr (!Args::kShared) {
    if (it.part < 0 || !arrive_last(A, it, it.part, kvh, &s_last)) return;
    join<Bf16, D, kThreads>(A, it, it.part, kUnits, kUnits, kvh, reinterpret_cast<float*>(s_k));
  }
}

}  // namespace

}  // namespace kv
}  // namespace lora
