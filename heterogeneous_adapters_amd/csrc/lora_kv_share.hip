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
// Either is cut into chunks that leave partial results; one launch joins them,
// since the results of a prefix's tile belong to as many requests as it has
// rows (a join by the last work-group of a tile would read 128 results of 16
// chunks in one place).
//
// Measured on MI355X (attention alone, and lora_kv_attend's time for the same):
// 256 requests behind 32768 tokens, 32 heads on 8 of 128, 155 us (889): of the
// three launches' times in a trace, prefix 141, rests 24, join 10.  96 requests
// behind 8 prompts of 256 to 4096, 32/32 heads, 49 us (123), 4.4 TB/s.  48 requests,
// 6 prompts, 15.5 (16.1).  4 beams over 1000 tokens 11.6 (10.4).  Four chunks of 512
// tokens among 32 requests behind 3000 and 6000: 246 (245): rows of one chunk
// share their keys without this.
// 256 requests behind 8192 tokens (floor: products at the library's rate, in
// fp32 three times as many): 76 us (259), floor 25; of 256 dims 179 (630), floor 50;
// fp32 194 (423), floor 74, since its tiles of 32 rows convert the prefix each.
//
// Weights are rounded to bf16 for their product with V, in both parts, and the
// sums are of the rounded weights, as in lora_kv_attend: bf16 results are off by
// 0.0018 to 0.0022 of their size, of which 0.0017 is their own rounding.  fp32 keeps
// 24 bits of queries and weights, and partial results are fp32 in either.
#include <utility>

#include "lora_kv_scan.h"
#include "lora_kv_tile.h"

namespace lora {
namespace kv {

namespace {

constexpr int kPlanThreads = 512;

// f of 0, 1, .. N-1 as constants.
template <int... I, class F>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F f) {
  each_of(std::make_integer_sequence<int, N>(), f);
}

constexpr int kFewTasks = 1 << 16;   // joins of up to as many vectors
constexpr int kLdsGroups = 1024;  // groups whose bounds and cuts lie in LDS

__device__ __forceinline__ int load_now(const int32_t* p) {  // what atomics left there
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// One entry of a list: rows that attend to the same keys.
struct Entry {
  int list, seq, qs, rows, pos0, kv, base, chunk, group;
};

// One work-group: integer work on a few kilobytes per step, 9 to 12 us of
// dependent reads (counters and lengths, positions, results of groups for
// their requests) and sums between barriers. Groups' bounds lie in LDS, and a
// request's numbers in its thread's registers, where there are few enough.
__global__ __launch_bounds__(kPlanThreads) void share_kernel(const ShareArgs A) {
  constexpr int kThreads = kPlanThreads, kWavesP = kThreads / 64;
  __shared__ uint32_t s_a[kWavesP][8];
  __shared__ int64_t s_read[3][kWavesP];
  __shared__ int32_t s_item[kLists][kThreads], s_list[kThreads], s_seq[kThreads], s_qs[kThreads], s_rows[kThreads],
      s_pos0[kThreads], s_kv[kThreads], s_base[kThreads], s_chunk[kThreads], s_part[kThreads];
  __shared__ int32_t s_bounds[kLdsGroups + 1], s_cut[kLdsGroups], s_first[kLdsGroups];
  const int tid = threadIdx.x;
  const int32_t* c = A.counts;
  const bool in_lds = A.groups <= kLdsGroups;
  const int32_t* bounds = in_lds ? s_bounds : A.group_indptr;
  int32_t *cut = in_lds ? s_cut : A.cut, *first_of = in_lds ? s_first : A.first;
  // a request's rows and length: read along with the counters, used after them
  const int at0 = tid < A.B ? A.q_indptr[tid] : 0, at1 = tid < A.B ? A.q_indptr[tid + 1] : 0, kv0 = tid < A.B ? A.kv_len[tid] : 0;
  int flags = 0;
  for (int g = tid; g < A.groups; g += kThreads) {
    const int a = A.group_indptr[g], b = A.group_indptr[g + 1], n = A.shared_len[g];
    const bool bad = a < 0 || b < a || b > A.B || n < 0;
    if (bad) flags |= LORA_KV_FLAG_GROUPS;
    cut[g] = bad ? 0 : n;
    first_of[g] = 0x7fffffff;
    if (in_lds) {
      s_bounds[g] = a;
      if (g == A.groups - 1) s_bounds[g + 1] = b;
    }
  }
  const bool built = c[kCountCheck] == check_word(c[kCountB], c[kCountT], c[kCountItems], c[kCountMid], c[kCountWide], c[kCountParts]) &&
                     c[kCountB] == A.B && c[kCountT] == A.T;
  if (!built) {  // no lists, and a check word that no call accepts
    if (tid == 0) atomicOr(&A.counts[kCountFlags], LORA_KV_FLAG_BATCH);
    if (tid < kNumShare) A.share[tid] = tid == kShareB ? -1 : 0;
    return;
  }
  const bool many = many_rows(A.T, A.B);
  __syncthreads();

  // The group of request i, or -1.
  auto group_of = [&](int i) {
    if (A.groups == 0 || bounds[0] > i) return -1;
    const int g = bisect(bounds, A.groups, i);
    return i < bounds[g + 1] ? g : -1;
  };
  // what every row of the group sees, and the first request with rows
  int group0 = -1, pos0 = 0;  // of request tid
  for (int i = tid; i < A.B; i += kThreads) {
    const bool mine = i == tid;
    const int at = mine ? at0 : A.q_indptr[i], end = mine ? at1 : A.q_indptr[i + 1];
    const int pos = end > at ? A.positions[at] : 0, g = end > at ? group_of(i) : -1;
    if (mine) group0 = g, pos0 = pos;
    if (g < 0) continue;
    atomicMin(&cut[g], min(pos, mine ? kv0 : A.kv_len[i]));
    atomicMin(&first_of[g], i);
  }
  __syncthreads();

  auto prefix_of = [&](int g) {  // tokens that the group's rows attend to together
    return g < 0 || load_now(&first_of[g]) == 0x7fffffff ? 0 : load_now(&cut[g]) & ~(kUnit - 1);
  };
  auto group_entry = [&](int g) {
    Entry e{0, 0, 0, 0, 1 << 30, 0, 0, 0, -1};
    if (g >= A.groups) return e;
    e.kv = prefix_of(g);
    if (e.kv == 0) return e;
    e.seq = load_now(&first_of[g]);
    e.qs = A.q_indptr[bounds[g]];
    e.rows = (A.q_indptr[bounds[g + 1]] - e.qs) * A.G;
    return e;
  };
  auto request_entry = [&](int i) {
    Entry e{1, i, 0, 0, 0, 0, 0, 0, -1};
    if (i >= A.B) return e;
    const bool mine = i == tid;
    e.qs = mine ? at0 : A.q_indptr[i];
    e.rows = ((mine ? at1 : A.q_indptr[i + 1]) - e.qs) * A.G;
    if (e.rows == 0) return e;
    e.list = 1 + (e.rows <= kUnit || !many ? 0 : e.rows <= kMidMost ? 1 : 2);
    e.group = mine ? group0 : group_of(i);
    e.base = prefix_of(e.group);
    e.pos0 = (mine ? pos0 : A.positions[e.qs]) - e.base;
    e.kv = (mine ? kv0 : A.kv_len[i]) - e.base;
    return e;
  };
  auto class_of_list = [&](int list) { return list == 0 ? A.prefix_class : list - 1; };
  auto tiles_of = [&](const Entry& e) {
    const int per = rows_of_class(class_of_list(e.list));
    return (e.rows + per - 1) / per;
  };
  const Entry mine_g = group_entry(tid), mine_r = request_entry(tid);

  // Tokens per item, from the keys that all tiles read.
  int64_t reads[3] = {0, 0, 0};
  for (int g = tid; g < A.groups; g += kThreads) {
    const Entry e = g == tid ? mine_g : group_entry(g);
    reads[0] += (int64_t)tiles_of(e) * e.kv;
  }
  for (int i = tid; i < A.B; i += kThreads) {
    const Entry e = i == tid ? mine_r : request_entry(i);
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
  const int chunk0 = chunk_for(s_read[0], prefix_items(A.prefix_class), min_prefix_chunk(A.prefix_class)), chunk1 = chunk_for(s_read[1], kTargetItems, kMinChunk),
            chunk2 = chunk_for(s_read[2], kTargetWide, kMinChunk);

  int64_t items0[kLists] = {0, 0, 0, 0}, rows0 = 0;
  // Lists the entries of one kind and says where their partial results are.
  auto emit = [&](int count, const Entry& mine, auto entry, auto note) {
    for (int first = 0; first < count; first += kThreads) {
      Entry e = first == 0 ? mine : entry(first + tid);
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
  emit(A.groups, mine_g, group_entry, [&](int g, const Entry& e, int part, int chunks) {
    if (g < A.groups) A.group_parts[g] = make_int4(part, chunks, e.qs, e.rows);
  });
  __syncthreads();
  emit(A.B, mine_r, request_entry, [&](int i, const Entry& e, int part, int chunks) {
    if (i >= A.B) return;
    const int g = e.base > 0 ? e.group : -1;
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
    s[kShareBuild] = c[kCountBuild];
    for (int i = 0; i < kNumShare; ++i) A.share[i] = s[i];
  }
}

// ------------------------------------------------------- prefixes of many rows
// 256 rows on a prefix's keys, which have no limits by row: eight waves of 32
// rows share the conversion of 64 keys at a time to bf16 in LDS (four waves
// convert K, four V, a unit of 16 tokens each). The products of a tile run
// between the softmax of another: while a wave's weights of tile t are formed,
// the matrix unit has the weights of tile t-1 times V and S of tile t+1.
//
// 1024 rows on 32768 keys, 8 kv heads of 128: median of 20 launches 141 us, least
// 137, 977 and 1006 TFLOP/s; the installed library's 8192^3 product reaches 1431 on
// the same card.  No unit is full: matrix units are busy for 47 % of the launch,
// vector units for 44, LDS for 33, and waves wait for 27 % of their cycles.  Issue
// alone (38 cycles a product by a probe of the single instructions: a product
// holds the vector unit for about 10, next to 150 vector instructions of each wave
// and tile, 32 exponentials of about 9 cycles among them) makes 156000 of its 280000
// cycles.  The rest goes to the barrier of every tile: registers leave room for
// one work-group per compute unit, and both waves of a SIMD come out of it in the
// same phase.  Other ways,
// least of 20 launches as the 137 above: four waves that share a conversion 153
// us; four waves of 64 rows, one per SIMD, 223 to 265 (spilled); 32 keys at a time
// with three waves per SIMD 161; every wave converting halves of K and V between
// its products 143; the requests' kernel of 128 rows 156.
template <int NC>
__global__ __launch_bounds__(512, 2) void prefix_kernel(const SharedArgs A) {
  constexpr int D = 32 * NC, kKeys = 64;
  constexpr int kSteps = D / 16, kDims = D / 32;
  // Rows of LDS, 16 bytes longer than their values: 16 lanes reading 16 bytes
  // of a row each meet all 64 banks, and one register addresses them all.
  constexpr int kRowK = 2 * D + 16, kRowV = 2 * kKeys + 16;
  __shared__ __attribute__((aligned(128))) uint8_t s_k[2][kKeys * kRowK], s_v[2][D * kRowV];
  __shared__ __attribute__((aligned(4))) uint8_t s_bad[4][4];  // by tile: its units that no row sees
  const int hkv = A.cache.heads;
  const int item = blockIdx.x / hkv, kvh = blockIdx.x - item * hkv;
  Item it;
  if (!read_item(A, 3, 0, item, 0, kPrefixRows, it)) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 31, h = lane >> 5;
  const int m16 = lane & 15, g = lane >> 4;
  const int G = A.G, row_first = it.row0 + wave * 32;

  bf16x8 qf[kSteps];
  {
    const int row = min(row_first + n, it.nrows - 1), jq = row / G;
    const uint16_t* q = static_cast<const uint16_t*>(A.q.p) + (int64_t)(it.qs + jq) * A.q.ts + (kvh * G + row - jq * G) * A.q.hs;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) qf[s] = *reinterpret_cast<const bf16x8*>(q + 16 * s + 8 * h);
  }

  const int32_t* trow = A.table + (int64_t)it.seq * A.tstride;
  const uint8_t* head = A.cache.base + ((int64_t)kvh << A.cache.bt_log2 >> 4) * (544 * NC);
  const int unit_mask = (1 << (A.cache.bt_log2 - 4)) - 1;
  const int n_tiles = (it.end - it.begin + kKeys - 1) / kKeys;
  bool bad_block = false;

  const bool is_v = wave >= 4;  // this wave converts V of its unit, or K
  const int first = it.begin + kUnit * (wave & 3);  // its unit's first token in tile 0
  // Block ids of this wave's unit in 64 tiles, one per lane; -1 outside the cache.
  auto fetch_ids = [&](int tile) {
    const int token = first + (tile + lane) * kKeys;
    int id = 0;
    if (token < it.end) {
      const int at = token >> A.cache.bt_log2;
      id = at < A.width ? trow[at] : -1;  // a table of another call may be narrower
      if ((unsigned)id >= (unsigned)A.cache.blocks) id = -1, bad_block = true;
    }
    return id;
  };
  uint32_t code[NC], scale[NC];  // a lane's share of the unit's K or V (of K's scales the first bytes)
  int id = 0, ids = fetch_ids(0);
  auto load = [&](int tile) {
    if (tile && tile % 64 == 0) ids = fetch_ids(tile);
    id = __builtin_amdgcn_readlane(ids, tile % 64);
    // behind the last token: the id is 0, a block of the cache
    const uint8_t* rec = head + max(id, 0) * A.cache.stride + (((first + tile * kKeys) >> 4) & unit_mask) * (544 * NC);
    if (is_v) {
      __builtin_memcpy(code, __builtin_assume_aligned(rec + 256 * NC + (g * 16 + m16) * 4 * NC, 4), 4 * NC);
      __builtin_memcpy(scale, __builtin_assume_aligned(rec + 528 * NC + 4 * g * NC, 4), 4 * NC);
    } else {
      __builtin_memcpy(code, __builtin_assume_aligned(rec + (m16 * 4 + g) * 4 * NC, 4), 4 * NC);
      __builtin_memcpy(scale, rec + 512 * NC + m16 * NC, NC);
    }
  };
  const int k_to = (kUnit * (wave & 3) + m16) * kRowK + g * 16;
  // tokens 4g..4g+3 of the unit, one dim: 8 bytes; the two halves of a 16-byte
  // piece are the tokens 8 apart that one lane of P holds
  const int v_to = m16 * kRowV + (2 * (wave & 3) + (g & 1)) * 16 + (g >> 1) * 8;
  // A unit outside the cache, or behind the last token: its bytes may hold
  // anything, a scale of NaN among it.
  auto convert_k = [&](int tile, int buf) {
    if (lane == 0) s_bad[tile & 3][wave] = id < 0 || first + tile * kKeys >= it.end;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const float sc = byte_scale(scale[c >> 2], c & 3);
      *reinterpret_cast<u32x4*>(s_k[buf] + k_to + 64 * c) =
          u32x4{fp4_pair(code[c], sc, 0), fp4_pair(code[c], sc, 1), fp4_pair(code[c], sc, 2), fp4_pair(code[c], sc, 3)};
    }
  };
  auto convert_v = [&](int tile, int buf) {
    if (id < 0 || first + tile * kKeys >= it.end) {
#pragma unroll
      for (int c = 0; c < NC; ++c) code[c] = scale[c] = 0;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      uint32_t r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = j * NC + c;
        r[j] = fp4_pair(code[c], byte_scale(scale[at >> 2], at & 3), j);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t sel = e ? 0x07060302u : 0x05040100u;
        *reinterpret_cast<uint2*>(s_v[buf] + v_to + (32 * c + 16 * e) * kRowV) =
            make_uint2(__builtin_amdgcn_perm(r[1], r[0], sel), __builtin_amdgcn_perm(r[3], r[2], sel));
      }
    }
  };

  // The x-th piece of a turn's products: V's first, whose weights' registers
  // then are free for this turn's, K's when half of this turn's scores are.
  constexpr int kHalf = 4 * NC;
  auto piece_of = [&](int x, int buf) {
    if (x < kHalf) {
      const int c = x / kDims, d = x % kDims;
      return *reinterpret_cast<const bf16x8*>(s_v[buf] + (n + 32 * d) * kRowV + (2 * c + h) * 16);
    }
    const int u = (x - kHalf) / kSteps, c = (x - kHalf) % kSteps;
    return *reinterpret_cast<const bf16x8*>(s_k[buf] + (n + 32 * u) * kRowK + (2 * c + h) * 16);
  };

  f16v o[kDims], s[2];
  float m = kNone, l = 0.0f, most;
  bool far = false;  // some row's scores are
  bf16x8 pf[4];      // the weights of the tile before
#pragma unroll
  for (int d = 0; d < kDims; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  auto highest = [&](int u) {  // .. of the first 32 tokens' scores, and of the others
    if (u == 0) most = s[0][0];
#pragma unroll
    for (int i = 0; i < 16; ++i) most = fmaxf(most, s[u][i]);
  };

  // Tile t's weights, next to the products of its neighbours; t's parity is
  // `which`.  `most` holds the highest of its first 32 tokens' scores.
  auto turn = [&](int t, auto which, auto first) {
    constexpr int buf = which;
    constexpr bool kFirst = first;
    constexpr int kFrom = kFirst ? kHalf : 0, kSlots = 2 * kHalf - kFrom, kAhead = 4;
    bf16x8 ahead[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) ahead[x] = piece_of(kFrom + x, 1 - buf);
    const uint32_t bad = (uint32_t)uniform((int)*reinterpret_cast<const uint32_t*>(s_bad[t & 3]));
    if (bad) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if ((bad >> (8 * (2 * u + (i >> 3)))) & 1) s[u][i] = -INFINITY;
      highest(0);
    }
    highest(1);
    float alpha = 1.0f;
    const bool moved = __any(most * A.scale_log2e > m + kSlack);
    if (moved) {
      const float mn = fmaxf(m, fmaxf(most, __shfl_xor(most, 32)) * A.scale_log2e);
      alpha = exp2_hw(m - mn);
      m = mn;
      far = far || __any(is_far(mn));
      l *= alpha;
    }
    float by = A.scale_log2e, less = m;
    if (far) {
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i >> 4][i & 15] = far_exponent(s[i >> 4][i & 15], by, less);
      by = 1.0f, less = 0.0f;
    }
    if (is_v) {
      convert_v(t, buf);
      load(t + 1);
    } else {
      convert_k(t + 2, buf);
      load(t + 3);
    }

    f16v next[2];
    bf16x8 now[4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) next[u][i] = 0.0f;
    constexpr int kMaxFrom = kSlots - 2 * NC + 1, kPer = 2 * NC - 1;
    // one product a slot, in this order
    each<kSlots>([&](auto slot) {
      constexpr int y = slot, x = kFrom + y;
      __builtin_amdgcn_sched_barrier(0);
      const bf16x8 a = ahead[y % kAhead];
      if constexpr (x < kHalf) {
        o[x % kDims] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, pf[x / kDims], o[x % kDims], 0, 0, 0);
      } else {
        constexpr int u = (x - kHalf) / kSteps, c = (x - kHalf) % kSteps;
        next[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, qf[c], next[u], 0, 0, 0);
      }
      if constexpr (y + kAhead < kSlots) ahead[y % kAhead] = piece_of(x + kAhead, 1 - buf);
      // this tile's weights
      constexpr int from = y * 32 / kSlots, to = (y + 1) * 32 / kSlots;
      each<to - from>([&](auto at) {
        constexpr int i = from + at;
        now[i >> 3][i & 7] = (__bf16)exp2_hw(fmaf(s[i >> 4][i & 15], by, -less));
        if constexpr ((i & 7) == 7) l = add8(now[i >> 3], l);
      });
      if constexpr (y >= kMaxFrom) {  // the next tile's first scores
        constexpr int a0 = (y - kMaxFrom) * 16 / kPer, a1 = (y - kMaxFrom + 1) * 16 / kPer;
        each<a1 - a0>([&](auto at) {
          constexpr int i = a0 + at;
          most = i ? fmaxf(most, next[0][i]) : next[0][0];
        });
      }
    });
    __builtin_amdgcn_sched_barrier(0);
    // formed here, not where they are used
#pragma unroll
    for (int c = 0; c < 4; ++c) asm volatile("" : "+v"(now[c]));
    asm volatile("" : "+v"(most));
#pragma unroll
    for (int u = 0; u < 2; ++u) s[u] = next[u];
#pragma unroll
    for (int c = 0; c < 4; ++c) pf[c] = now[c];
    if (moved) {
#pragma unroll
      for (int d = 0; d < kDims; ++d) o[d] *= alpha;
    }
    __syncthreads();  // K of t+2 and V of t are in LDS, and what this turn read is free
  };

  const std::integral_constant<int, 0> zero;
  const std::integral_constant<int, 1> one;
  const std::integral_constant<bool, true> yes;
  const std::integral_constant<bool, false> no;
  load(0);
  if (!is_v) {
    convert_k(0, 0);
    load(1);
    convert_k(1, 1);
    load(2);
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
#pragma unroll
    for (int c = 0; c < kSteps; ++c) s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(piece_of(kHalf + u * kSteps + c, 0), qf[c], s[u], 0, 0, 0);
  }
  highest(0);
  __syncthreads();  // turn 0 writes K of tile 2 there
  turn(0, zero, yes);
  int t = 1;
  for (; t + 1 < n_tiles; t += 2) {
    turn(t, one, no);
    turn(t + 1, zero, no);
  }
  auto finish = [&](auto which) {  // O of the last tile
    constexpr int buf = which;
#pragma unroll
    for (int x = 0; x < kHalf; ++x)
      o[x % kDims] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(piece_of(x, buf), pf[x / kDims], o[x % kDims], 0, 0, 0);
  };
  if (t < n_tiles) {
    turn(t, one, no);
    finish(one);
  } else {
    finish(zero);
  }
  if (__any(bad_block) && lane == 0) atomicOr(&A.counts[kCountFlags], LORA_KV_FLAG_BLOCK_RANGE);

  l += __shfl_xor(l, 32);
  if (row_first + n < it.nrows) {
#pragma unroll
    for (int d = 0; d < kDims; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        store_part<D>(A, it, kvh, wave * 32 + n, 32 * d + 2 * i + 4 * h, f4{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]}, m, l);
  }
}

// Four dims of a row by kGroups threads of a work-group, each every kGroups-th
// result, joined in a fixed order.
template <class E, int kGroups>
__global__ __launch_bounds__(256) void join_kernel(const SharedArgs A, int vecs) {
  typedef typename E::T T;
  constexpr int kBatch = 4, kTasks = 256 / kGroups;  // results in flight; tasks of a work-group
  __shared__ float s_part[kGroups > 1 ? 256 : 1][6];
  const bool ok = share_ok(A), last_build = A.share[kShareBuild] == A.counts[kCountBuild];
  // Another call's plan, which the lists' launches have flagged; or one of an
  // earlier build, whose results lie within the workspace all the same: asked
  // here alone, of the batch's buffer that this launch reads anyway.
  if (!ok || !last_build) {
    if (ok && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&A.counts[kCountFlags], LORA_KV_FLAG_BATCH);
    return;
  }
  const int D = vecs * 4, hkv = A.cache.heads, hq = hkv * A.G;
  const int grp = threadIdx.x / kTasks;
  const int64_t task = (int64_t)blockIdx.x * kTasks + threadIdx.x % kTasks;
  const int d = (int)(task % vecs) * 4, h = (int)(task / vecs % hq);
  const int64_t t = task / vecs / hq;
  const int seq = t < A.T ? A.token_seq[t] : -1;
  const bool live = (unsigned)seq < (unsigned)A.B;
  const int kvh = h / A.G, hg = h - kvh * A.G;
  float M = kNone, L = 0.0f;
  f4 acc{0, 0, 0, 0};
  auto add = [&](float m, float l, f4 o) {
    const float mn = fmaxf(M, m), a = exp2_hw(M - mn), b = exp2_hw(m - mn);
    M = mn;
    L = L * a + l * b;
    acc = acc * a + b * o;
  };
  if (live) {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int4 p = A.seq_parts[2 * seq + side];  // first result's row, chunks, first token row, rows
      const int row = ((int)t - p.z) * A.G + hg;  // one of p.w: rows and plan are of one build
      for (int c0 = grp; c0 < p.y; c0 += kBatch * kGroups) {
        float2 ml[kBatch];
        f4 o[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const int64_t at = (int64_t)(p.x + min(c0 + e * kGroups, p.y - 1) * p.w + row) * hkv + kvh;
          ml[e] = *reinterpret_cast<const float2*>(A.part_ml + 2 * at);
          o[e] = *reinterpret_cast<const f4*>(A.part + at * D + d);
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          if (c0 + e * kGroups >= p.y) break;
          add(ml[e].x, ml[e].y, o[e]);
        }
      }
    }
  }
  if constexpr (kGroups > 1) {
    float* s = s_part[threadIdx.x];
    s[0] = M, s[1] = L, s[2] = acc[0], s[3] = acc[1], s[4] = acc[2], s[5] = acc[3];
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int e = 1; e < kGroups; ++e) {
      const float* o = s_part[threadIdx.x + e * kTasks];
      add(o[0], o[1], f4{o[2], o[3], o[4], o[5]});
    }
  }
  if (!live) return;
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
  auto blocks = [&](int list, int64_t items) {
    A.list = list;
    return (unsigned)(items * hkv);
  };
  constexpr bool kBf16 = sizeof(typename E::T) == 2;
  A.first_items = 0;
  if (A.groups > 0) {
    const int64_t items = prefix_cap(prefix_cls, A.T, A.groups, hkv, A.G);
    if (prefix_cls == 0) {
      A.first_items = (int32_t)items;
    } else if (prefix_cls == 2) {
      const unsigned n = blocks(0, items);
      if constexpr (kBf16 && NC > 4) attend_wide_kernel<NC, SharedArgs><<<n, 256, 0, s>>>(A);
      if constexpr (!kBf16 && NC > 4) attend_kernel<E, NC, 2, 2, SharedArgs><<<n * (kWideRows / kMidRows), 64 * kWaves, 0, s>>>(A);
    } else {
      const unsigned n = blocks(0, items);
      if constexpr (kBf16 && NC <= 4) prefix_kernel<NC><<<n, 512, 0, s>>>(A);
      if constexpr (!kBf16 && NC <= 4) attend_kernel<E, NC, 2, 3, SharedArgs><<<n * (kPrefixRows / kMidRows), 64 * kWaves, 0, s>>>(A);
    }
  }
  if (many) {
    const unsigned wide = blocks(3, class_cap(2, A.T, A.B, hkv, A.G));
    if constexpr (kBf16) attend_wide_kernel<NC, SharedArgs><<<wide, 256, 0, s>>>(A);
    else attend_kernel<E, NC, 2, 2, SharedArgs><<<wide * (kWideRows / kMidRows), 64 * kWaves, 0, s>>>(A);
    attend_kernel<E, NC, 2, 1, SharedArgs><<<blocks(2, class_cap(1, A.T, A.B, hkv, A.G)), 64 * kWaves, 0, s>>>(A);
  }
  attend_kernel<E, NC, 1, 0, SharedArgs><<<blocks(1, A.first_items + class_cap(0, A.T, A.B, hkv, A.G)), 64 * kWaves, 0, s>>>(A);
  const int vecs = 8 * NC;
  const int64_t tasks = (int64_t)A.T * hkv * A.G * vecs;
  // few rows have many results each: eight threads for one
  if (tasks <= kFewTasks) join_kernel<E, 8><<<(unsigned)((tasks + 31) / 32), 256, 0, s>>>(A, vecs);
  else join_kernel<E, 1><<<(unsigned)((tasks + 255) / 256), 256, 0, s>>>(A, vecs);
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
