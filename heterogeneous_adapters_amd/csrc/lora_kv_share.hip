// lora_kv_share and lora_kv_attend_shared: attention of requests that begin
// with the same cached tokens.
//
// Mathematics: a row's softmax splits at the prefix's end,
//   o = (2^(m1-M) o1 + 2^(m2-M) o2) / (2^(m1-M) l1 + 2^(m2-M) l2),
// with (m, l, o) the maximum, the sum of weights and the weighted sum of V of
// each part.  The first part is the same keys for every row of a group, so all
// rows of a group are tiled together over them: the prefix is read and
// converted once per tile of rows in place of once per request, and becomes a
// matrix product.  The second is lora_kv_attend's work over what is left.
// Either is cut into chunks that leave partial results; one launch joins them.
#include "lora_kv_scan.h"
#include "lora_kv_tile.h"

namespace lora {
namespace kv {

namespace {

constexpr int kPlanThreads = 512;

// The group of request i, or -1.
__device__ __forceinline__ int group_of(const ShareArgs& A, int i) {
  if (A.groups == 0 || A.group_indptr[0] > i) return -1;
  const int g = bisect(A.group_indptr, A.groups, i);
  return i < A.group_indptr[g + 1] ? g : -1;
}

__device__ __forceinline__ int load_now(const int32_t* p) {  // what atomics left there
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// One entry of a list: rows that attend to the same keys.
struct Entry {
  int list, seq, qs, rows, pos0, kv, base, chunk;
};

// One work-group: integer work on a few kilobytes per step.
__global__ __launch_bounds__(kPlanThreads) void share_kernel(const ShareArgs A) {
  constexpr int kThreads = kPlanThreads, kWavesP = kThreads / 64;
  __shared__ uint32_t s_a[kWavesP][8];
  __shared__ int64_t s_read[3][kWavesP];
  __shared__ int32_t s_item[kLists][kThreads], s_list[kThreads], s_seq[kThreads], s_qs[kThreads], s_rows[kThreads],
      s_pos0[kThreads], s_kv[kThreads], s_base[kThreads], s_chunk[kThreads], s_part[kThreads];
  const int tid = threadIdx.x;
  const int32_t* c = A.counts;
  const bool built = c[kCountCheck] == check_word(c[kCountB], c[kCountT], c[kCountItems], c[kCountMid], c[kCountWide], c[kCountParts]) &&
                     c[kCountB] == A.B && c[kCountT] == A.T;
  if (!built) {  // no lists, and a check word that no call accepts
    if (tid == 0) atomicOr(&A.counts[kCountFlags], LORA_KV_FLAG_BATCH);
    if (tid < kNumShare) A.share[tid] = tid == kShareB ? -1 : 0;
    return;
  }
  const bool many = many_rows(A.T, A.B);

  int flags = 0;
  for (int g = tid; g < A.groups; g += kThreads) {
    const int a = A.group_indptr[g], b = A.group_indptr[g + 1], n = A.shared_len[g];
    const bool bad = a < 0 || b < a || b > A.B || n < 0;
    if (bad) flags |= LORA_KV_FLAG_GROUPS;
    A.cut[g] = bad ? 0 : n;
    A.first[g] = 0x7fffffff;
  }
  __syncthreads();
  // what every row of the group sees, and the first request with rows
  for (int i = tid; i < A.B; i += kThreads) {
    const int at = A.q_indptr[i], g = A.q_indptr[i + 1] > at ? group_of(A, i) : -1;
    if (g < 0) continue;
    atomicMin(&A.cut[g], min(A.positions[at], A.kv_len[i]));
    atomicMin(&A.first[g], i);
  }
  __syncthreads();

  auto prefix_of = [&](int g) {  // tokens that the group's rows attend to together
    return g < 0 || load_now(&A.first[g]) == 0x7fffffff ? 0 : load_now(&A.cut[g]) & ~(kUnit - 1);
  };
  auto group_entry = [&](int g) {
    Entry e{0, 0, 0, 0, 1 << 30, 0, 0, 0};
    if (g >= A.groups) return e;
    e.kv = prefix_of(g);
    if (e.kv == 0) return e;
    e.seq = load_now(&A.first[g]);
    e.qs = A.q_indptr[A.group_indptr[g]];
    e.rows = (A.q_indptr[A.group_indptr[g + 1]] - e.qs) * A.G;
    return e;
  };
  auto request_entry = [&](int i) {
    Entry e{1, i, 0, 0, 0, 0, 0, 0};
    if (i >= A.B) return e;
    e.qs = A.q_indptr[i];
    e.rows = (A.q_indptr[i + 1] - e.qs) * A.G;
    if (e.rows == 0) return e;
    e.list = 1 + (e.rows <= kUnit || !many ? 0 : e.rows <= kMidMost ? 1 : 2);
    e.base = prefix_of(group_of(A, i));
    e.pos0 = A.positions[e.qs] - e.base;
    e.kv = A.kv_len[i] - e.base;
    return e;
  };
  auto class_of_list = [&](int list) { return list == 0 ? A.prefix_class : list - 1; };
  auto tiles_of = [&](const Entry& e) {
    const int per = rows_of_class(class_of_list(e.list));
    return (e.rows + per - 1) / per;
  };

  // Tokens per item, from the keys that all tiles read.
  int64_t reads[3] = {0, 0, 0};
  for (int g = tid; g < A.groups; g += kThreads) {
    const Entry e = group_entry(g);
    reads[0] += (int64_t)tiles_of(e) * e.kv;
  }
  for (int i = tid; i < A.B; i += kThreads) {
    const Entry e = request_entry(i);
    reads[e.list == 3 ? 2 : 1] += (int64_t)tiles_of(e) * e.kv;
  }
#pragma unroll
  for (int v = 0; v < 3; ++v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) reads[v] += __shfl_xor(reads[v], d);
    if ((tid & 63) == 0) s_read[v][tid >> 6] = reads[v];
  }
  __syncthreads();
  auto chunk_for = [&](const int64_t* part, int target, int least) {
    int64_t sum = 0;
    for (int w = 0; w < kWavesP; ++w) sum += part[w];
    const int64_t per = (sum * A.hkv + target - 1) / target;
    return (int)min(max((per + kChunkStep - 1) / kChunkStep * kChunkStep, (int64_t)least), (int64_t)1 << 29);
  };
  const int chunk0 = chunk_for(s_read[0], kTargetPrefix, kMinPrefixChunk), chunk1 = chunk_for(s_read[1], kTargetItems, kMinChunk),
            chunk2 = chunk_for(s_read[2], kTargetWide, kMinChunk);

  int64_t items0[kLists] = {0, 0, 0, 0}, rows0 = 0;
  // Lists the entries of one kind and says where their partial results are.
  auto emit = [&](int count, auto entry, auto note) {
    for (int first = 0; first < count; first += kThreads) {
      Entry e = entry(first + tid);
      if (first + tid >= count) e.rows = 0;
      const int tiles = tiles_of(e);
      e.chunk = even_chunk(e.kv, e.list == 0 ? chunk0 : e.list == 3 ? chunk2 : chunk1);
      const int chunks = e.rows ? max((e.kv + e.chunk - 1) / e.chunk, 1) : 0;
      uint32_t x[kLists + 1];
#pragma unroll
      for (int l = 0; l < kLists; ++l) x[l] = e.list == l ? tiles * chunks : 0;
      x[kLists] = e.rows * chunks;
      int64_t at[kLists + 1], sum[kLists + 1];
      __syncthreads();
      block_scan<kWavesP, kLists + 1>(x, at, sum, s_a);
#pragma unroll
      for (int l = 0; l < kLists; ++l) s_item[l][tid] = (int)(items0[l] + at[l]);
      s_list[tid] = e.list, s_seq[tid] = e.seq, s_qs[tid] = e.qs, s_rows[tid] = e.rows;
      s_pos0[tid] = e.pos0, s_kv[tid] = e.kv, s_base[tid] = e.base, s_chunk[tid] = e.chunk;
      s_part[tid] = (int)(rows0 + at[kLists]);
      note(first + tid, e, (int)(rows0 + at[kLists]), chunks);
      __syncthreads();
      const int n = min(kThreads, count - first);
      for (int l = 0; l < kLists; ++l) {
        const int per = rows_of_class(class_of_list(l));
        for (int w = (int)items0[l] + tid; w < min(items0[l] + sum[l], (int64_t)A.item_cap); w += kThreads) {
          const int k = bisect(s_item[l], n, w);
          const int chunk = s_chunk[k], rows = s_rows[k], kv = s_kv[k], all = max((kv + chunk - 1) / chunk, 1);
          const int local = w - s_item[l][k], tile = local / all, ci = local - tile * all;
          int4* to = A.items + kShareItem * ((int64_t)l * A.item_cap + w);
          to[0] = make_int4(s_seq[k], tile * per, s_part[k] + ci * rows + tile * per, s_base[k]);
          to[1] = make_int4(s_qs[k], rows, s_pos0[k], kv);
          to[2] = make_int4(ci * chunk, min((ci + 1) * chunk, kv), 0, 0);
        }
        items0[l] += sum[l];
      }
      rows0 += sum[kLists];
    }
  };
  // A prefix's partial results: of its first row's first chunk, chunks, first
  // token row, rows.
  emit(A.groups, group_entry, [&](int g, const Entry& e, int part, int chunks) {
    if (g < A.groups) A.group_parts[g] = make_int4(part, chunks, e.qs, e.rows);
  });
  __syncthreads();
  emit(A.B, request_entry, [&](int i, const Entry& e, int part, int chunks) {
    if (i >= A.B) return;
    const int g = e.base > 0 ? group_of(A, i) : -1;
    A.seq_parts[2 * i] = g < 0 ? make_int4(0, 0, 0, 0) : A.group_parts[g];
    A.seq_parts[2 * i + 1] = make_int4(part, chunks, e.qs, e.rows);
  });

  if (flags) atomicOr(&A.counts[kCountFlags], flags);
  if (tid == 0) {
    int32_t s[kNumShare] = {};
    for (int l = 0; l < kLists; ++l) s[l] = (int)items0[l];
    s[kShareRows] = (int)min(rows0, (int64_t)0x7fffffff);
    s[kShareGroups] = A.groups, s[kShareB] = A.B, s[kShareT] = A.T;
    s[kShareCheck] = share_word(s);
    for (int i = 0; i < kNumShare; ++i) A.share[i] = s[i];
  }
}

// Four dims of a row per thread.
template <class E>
__global__ __launch_bounds__(256) void join_kernel(const SharedArgs A, int vecs) {
  typedef typename E::T T;
  if (!share_ok(A)) return;  // the lists' launches have flagged it
  const int D = vecs * 4, hkv = A.cache.heads, hq = hkv * A.G;
  const int64_t task = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int d = (int)(task % vecs) * 4, h = (int)(task / vecs % hq);
  const int64_t t = task / vecs / hq;
  if (t >= A.T) return;
  const int seq = A.token_seq[t];
  if ((unsigned)seq >= (unsigned)A.B) return;
  const int kvh = h / A.G, hg = h - kvh * A.G;
  float M = kNone, L = 0.0f;
  f4 acc{0, 0, 0, 0};
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int4 p = A.seq_parts[2 * seq + side];  // first result's row, chunks, first token row, rows
    const int row = ((int)t - p.z) * A.G + hg;
    // a batch built again after its shared plan
    if (p.y > 0 && ((int)t < p.z || row >= p.w)) {
      if (d == 0 && hg == 0) atomicOr(&A.counts[kCountFlags], LORA_KV_FLAG_BATCH);
      continue;
    }
    for (int c = 0; c < p.y; ++c) {
      const int64_t at = (int64_t)(p.x + c * p.w + row) * hkv + kvh;
      const float2 ml = *reinterpret_cast<const float2*>(A.part_ml + 2 * at);
      const f4 o = *reinterpret_cast<const f4*>(A.part + at * D + d);
      const float mn = fmaxf(M, ml.x), a = exp2_hw(M - mn), b = exp2_hw(ml.x - mn);
      M = mn;
      L = L * a + ml.y * b;
      acc = acc * a + b * o;
    }
  }
  const float inv = inverse(L);
  T* out = static_cast<T*>(A.o.p) + t * A.o.ts + h * A.o.hs + d;
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf2(acc[0] * inv, acc[1] * inv), pack_bf2(acc[2] * inv, acc[3] * inv));
  } else {
    *reinterpret_cast<f4*>(out) = acc * inv;
  }
}

template <class E, int NC>
hipError_t launch(SharedArgs A, int prefix_cls, bool many, hipStream_t s) {
  const int hkv = A.cache.heads;
  auto run = [&](int list, int cls, int64_t items) {
    A.list = list;
    const unsigned n = (unsigned)(items * hkv);
    if (cls == 0) {
      attend_kernel<E, NC, 1, 0, SharedArgs><<<n, 64 * kWaves, 0, s>>>(A);
    } else if (cls == 1) {
      attend_kernel<E, NC, 2, 1, SharedArgs><<<n, 64 * kWaves, 0, s>>>(A);
    } else {
      if constexpr (sizeof(typename E::T) == 2) attend_wide_kernel<NC, SharedArgs><<<n, 256, 0, s>>>(A);
      else attend_kernel<E, NC, 2, 2, SharedArgs><<<n * (kWideRows / kMidRows), 64 * kWaves, 0, s>>>(A);
    }
  };
  if (A.groups > 0) run(0, prefix_cls, prefix_cap(A.T, A.groups, hkv, A.G));
  for (int c = many ? 2 : 0; c >= 0; --c) run(1 + c, c, class_cap(c, A.T, A.B, hkv, A.G));
  const int vecs = 8 * NC;
  const int64_t tasks = (int64_t)A.T * hkv * A.G * vecs;
  join_kernel<E><<<(unsigned)((tasks + 255) / 256), 256, 0, s>>>(A, vecs);
  return hipGetLastError();
}

template <class E>
hipError_t launch_nc(const SharedArgs& A, int prefix_cls, bool many, hipStream_t s) {
  switch (A.cache.nc) {
    case 1: return launch<E, 1>(A, prefix_cls, many, s);
    case 2: return launch<E, 2>(A, prefix_cls, many, s);
    case 3: return launch<E, 3>(A, prefix_cls, many, s);
    case 4: return launch<E, 4>(A, prefix_cls, many, s);
    case 5: return launch<E, 5>(A, prefix_cls, many, s);
    case 6: return launch<E, 6>(A, prefix_cls, many, s);
    case 7: return launch<E, 7>(A, prefix_cls, many, s);
    default: return launch<E, 8>(A, prefix_cls, many, s);
  }
}

}  // namespace

hipError_t launch_share(const ShareArgs& A, hipStream_t s) {
  share_kernel<<<1, kPlanThreads, 0, s>>>(A);
  return hipGetLastError();
}

hipError_t launch_shared(const SharedArgs& A, int dtype, int prefix_cls, bool many, hipStream_t s) {
  return dtype == LORA_DTYPE_BF16 ? launch_nc<Bf16>(A, prefix_cls, many, s) : launch_nc<F32>(A, prefix_cls, many, s);
}

}  // namespace kv
}  // namespace lora
