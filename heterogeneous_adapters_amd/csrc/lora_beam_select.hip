// lora_beam_select: the best continuations of every request's beams.
//
// Mathematics: a row's candidates are ordered as its logits are, so a row needs
// its `beams` highest logits and log(sum e^x), both from one pass: a wave
// holds 2048 logits in registers, sums e^(x - r) against a logit r that none has
// passed by more than 8 (each chunk's sum in fp32 per lane, the chunks' in fp64)
// and keeps the highest logits so far, one per lane in descending order, as keys (the logit
// as an ordered integer, then the token's complement, so that equal logits go
// by the lower token).  A chunk whose highest logit is below the last of these
// is done with its sum.  A second launch joins the waves of each row and ranks
// the request's beams * beams candidates in 64 bits.
//
// Measured on MI355X (rows, then picks): 64 requests of 8 beams, 128000 bf16
// logits, 32 + 8 us, 4.1 TB/s of logits; without looking for candidates the
// rows' launch takes 23, 5.6 TB/s (the read rate is 6.1), so what bounds it is the
// comparisons and insertions of the chunks that follow a wave's first. Fewer,
// longer waves look less (kTargetWaves); waves that tell one another
// their lowest kept logit gain nothing, as they keep pace. 128 x 16 of 32000 38 + 8 us;
// 32 x 5 of 50257 fp32 11 + 11; 1 x 4 of 32000 6.7 + 5.5, latency.  A vocabulary masked
// with one finite number takes long, as a chunk's equal logits are looked at one
// after the other: 64 x 8 of 128000 with 300 tokens left 376 us at -1e4 or -1e9; 42 at
// -inf, which is no candidate.
#include <type_traits>

#include "lora_beam_args.h"
#include "lora_kv_dev.h"

namespace lora {
namespace beam {

using namespace lora::kv;

namespace {

constexpr float kLog2eHi = 1.44269502162933349609375f;  // log2(e) to 24 bits, and the rest
constexpr float kLog2eLo = 1.92596299112661746887e-08f;

constexpr double kLog2e = 1.44269504088896340736, kLn2 = 0.693147180559945309417;
constexpr float kSlackLogit = 8.0f;

// Around references past this the difference to the reference comes first, then
// its product with log2(e).  Below it r log2(e) rounded to fp32 is off by at
// most 2^-8, so e^off, which takes that back, by less than 2^-27 after its second
// power; farther out the three terms do not hold, and from about 2e9 on the
// weights themselves leave fp32's range.  Every finite logit is right by the
// difference; ordinary rows never take that way.
constexpr float kFarLogit = 65536.0f;

// Floats as integers of the same order; 0 is below every one that stands for a logit.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t kMinusInf = 0x007fffffu;  // ordered(-inf)

// The lane before's, 0 in the first.
__device__ __forceinline__ uint64_t shift64(uint64_t x) {
  const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)x, 0x138, 0xf, 0xf, true);  // wave_shr:1
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(x >> 32), 0x138, 0xf, 0xf, true);
  return (uint64_t)(uint32_t)lo | (uint64_t)(uint32_t)hi << 32;
}
__device__ __forceinline__ uint64_t lane64(uint64_t x, int lane) {  // a uniform lane
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, lane) |
         (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), lane) << 32;
}

// A value sent to lane `to` of each lane; 0 where none is sent.
__device__ __forceinline__ uint64_t send64(uint64_t x, int to) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_ds_permute(4 * to, (int)(uint32_t)x) |
         (uint64_t)(uint32_t)__builtin_amdgcn_ds_permute(4 * to, (int)(x >> 32)) << 32;
}

// The highest n keys seen so far, lane i the i-th; 0 where there are none.
struct Best {
  uint64_t list = 0, least = 0;  // least: the n-th, uniform
  __device__ __forceinline__ void put(uint64_t key, int n) {  // a uniform key above `least`
    const int lane = threadIdx.x & 63;
    const int at = __popcll(__ballot(list > key));
    const uint64_t up = shift64(list);
    list = lane < at ? list : lane == at ? key : up;
    least = lane64(list, n - 1);
  }
  // The keys of the first `count` lanes (of others 0), all different: each
  // finds its place by counting those above it.
  __device__ __forceinline__ void merge(uint64_t keys, int count, int n) {
    const int lane = threadIdx.x & 63;
    int mine = lane, place = 0;  // of `list`, of `keys`
    for (int j = 0; j < count; ++j) {
      const uint64_t k = lane64(keys, j);
      mine += k > list;
      place += k > keys;
    }
    if (lane64(list, 0)) {
      for (int j = 0; j < n; ++j) place += lane64(list, j) > keys;
    }
    // no list has a 64th entry: what has no place goes there
    const uint64_t a = send64(list, list && mine < n ? mine : 63), b = send64(keys, keys && place < n ? place : 63);
    list = lane < n ? a | b : 0;
    least = lane64(list, n - 1);
  }
};

// The n-th highest of the lanes' values, or a little less: its upper 16 bits.
__device__ __forceinline__ uint32_t nth_highest(uint32_t x, int n) {
  uint32_t t = 0;
  for (int b = 31; b >= 16; --b) {
    const uint32_t up = t | 1u << b;
    if (__popcll(__ballot(x >= up)) >= n) t = up;
  }
  return t;
}

template <class E>
__global__ __launch_bounds__(256) void rows_kernel(const SelectArgs A) {
  typedef typename E::T T;
  constexpr int kEpv = E::kEpv, kVecs = 32 / kEpv;
  __shared__ uint64_t s_cand[4][64];
  const int lane = threadIdx.x & 63;
  uint64_t* cand = s_cand[threadIdx.x >> 6];
  const int64_t job = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int row = uniform((int)(job / A.waves)), wave = uniform((int)(job - (int64_t)row * A.waves));
  if (row >= A.requests * A.beams) return;
  const float score = A.score[row];
  if (A.done[row] != 0 || !(fabsf(score) < INFINITY)) return;  // not continued

  const T* x = static_cast<const T*>(A.logits) + row * A.stride;
  // vectors start before the row where its first logit is not aligned
  const int skew = (int)((reinterpret_cast<uintptr_t>(x) / sizeof(T)) % kEpv);
  const int first = wave * A.chunks, last = min(first + A.chunks, (A.vocab + skew + kChunk - 1) / kChunk);

  Best best;
  float ref = -INFINITY;  // a logit that the others pass by 8 at most
  float less = 0.0f;      // ref log2(e)
  double by = 0.0;        // what its rounding makes of each weight
  double sum = 0.0;       // of e^(x - ref), this lane's share
  float bound = -INFINITY;  // logits below this are not among the highest
  bool odd = false;
  u32x4 raw[kVecs] = {};
  auto vec_at = [&](int chunk, int v) { return chunk * kChunk + (v * 64 + lane) * kEpv - skew; };
  auto load = [&](int chunk) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int at = vec_at(chunk, v);
      if (at >= 0 && at + kEpv <= A.vocab) raw[v] = *reinterpret_cast<const u32x4*>(x + at);
    }
  };
  if (first < last) load(first);
  for (int chunk = first; chunk < last; ++chunk) {
    float y[32];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      float part[kEpv];
      unpack(raw[v], part);
#pragma unroll
      for (int i = 0; i < kEpv; ++i) y[v * kEpv + i] = part[i];
    }
    if (chunk + 1 < last) load(chunk + 1);
    if (chunk * kChunk < skew || (chunk + 1) * kChunk - skew > A.vocab) {  // an end of the row: vectors that are not whole
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        const int at = vec_at(chunk, v);
        if (at >= 0 && at + kEpv <= A.vocab) continue;
#pragma unroll
        for (int i = 0; i < kEpv; ++i) y[v * kEpv + i] = at + i >= 0 && at + i < A.vocab ? to_f(x[at + i]) : -INFINITY;
      }
    }

    float most, s, high[4];  // of eight each
    auto weigh = [&](auto rare) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        high[j] = y[8 * j];
#pragma unroll
        for (int i = 1; i < 8; ++i) high[j] = fmaxf(high[j], y[8 * j + i]);
      }
      most = fmaxf(fmaxf(high[0], high[1]), fmaxf(high[2], high[3]));
      if (__any(most > ref + kSlackLogit)) {
        float top = most;
#pragma unroll
        for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
        if (ref > -INFINITY) sum *= exp((double)ref - (double)top);
        ref = top;
        less = ref * kLog2eHi;
        const double off = ((double)less - (double)ref * kLog2e) * kLn2;  // see kFarLogit: e^off by its first terms
        by = 1.0 + off * (1.0 + 0.5 * off);
      }
      s = 0.0f;
      if (rare) {
        if (ref == -INFINITY) return;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += exp2_hw(fmaf(y[i] - ref, kLog2eLo, (y[i] - ref) * kLog2eHi));
        sum += (double)s;
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) s += exp2_hw(fmaf(y[i], kLog2eLo, fmaf(y[i], kLog2eHi, -less)));
      }
    };
    const double sum0 = sum, by0 = by;
    const float ref0 = ref, less0 = less;
    weigh(std::false_type());
    // A NaN or an infinity shows in the sum or the highest, what is far in the reference.
    if (__any(!(s == s)) || !(fabsf(ref) < kFarLogit)) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (!(y[i] < INFINITY)) odd = true, y[i] = -INFINITY;
      sum = sum0, by = by0, ref = ref0, less = less0;
      weigh(std::true_type());
    } else {
      sum += (double)s * by;
    }

    // candidates
    if (!__any(most >= bound) || !__any(most > -INFINITY)) continue;
    // token and key of this lane's i-th logit, for any lane's bits
    auto key_of = [&](int i, uint32_t bits, int from) {
      const int token = chunk * kChunk + ((i / kEpv) * 64 + from) * kEpv + i % kEpv - skew;
      return (uint64_t)ordered(__uint_as_float(bits) + 0.0f) << 32 | (uint32_t)~token;  // one zero
    };
    if (best.least == 0) {  // the first chunk: sorted together
      const uint32_t nth = nth_highest(ordered(most), A.beams);
      bound = fmaxf(bound, nth > kMinusInf ? from_ordered(nth) : -3.402823466e38f);
      int count = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const uint64_t mask = __ballot(y[i] >= bound);
        const int at = count + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
        if (y[i] >= bound && at < 64) cand[at] = key_of(i, __float_as_uint(y[i]), lane);
        count += __popcll(mask);
      }
      if (count <= 64) {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        best.merge(lane < count ? cand[lane] : 0, count, A.beams);
        if (best.least) bound = fmaxf(bound, from_ordered((uint32_t)(best.least >> 32)));
        continue;
      }
    }
    // few, or many equal ones: one after the other
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!__any(high[j] >= bound)) continue;
#pragma unroll
      for (int i = 8 * j; i < 8 * j + 8; ++i) {
        uint64_t mask = __ballot(y[i] >= bound);
        while (mask) {
          const int from = __ffsll((long long)mask) - 1;
          mask &= mask - 1;
          const uint64_t key = key_of(i, (uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(y[i]), from), from);
          if (key > best.least) best.put(key, A.beams);
        }
      }
      if (best.least) bound = fmaxf(bound, from_ordered((uint32_t)(best.least >> 32)));
    }
  }
  if (__any(odd) && lane == 0 && A.flags) atomicOr(A.flags, LORA_BEAM_FLAG_LOGITS);
#pragma unroll
  for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  const int64_t at = (int64_t)row * A.waves + wave;
  if (lane < A.beams) A.keys[at * A.beams + lane] = best.list;
  if (lane == 0) A.sums[2 * at] = ref, A.sums[2 * at + 1] = sum;
}

// One work-group per request, a wave per row where there are as many.
__global__ __launch_bounds__(1024) void pick_kernel(const SelectArgs A) {
  constexpr int kMost = LORA_BEAM_MAX;
  __shared__ double s_rank[kMost * kMost], s_total[kMost * kMost];
  __shared__ int32_t s_token[kMost * kMost];
  __shared__ int32_t s_length[kMost], s_done[kMost], s_chosen;
  const int W = A.beams, row0 = blockIdx.x * W, keys = A.waves * W;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  if (threadIdx.x == 0) s_chosen = 0;
  for (int w = wave; w < W; w += waves) {
    const int64_t at = (int64_t)(row0 + w) * A.waves;
    // one trip to memory: what a row that is not continued left there is not used
    const float score = A.score[row0 + w];
    const int32_t length = A.length[row0 + w];
    const bool live = fabsf(score) < INFINITY, done = A.done[row0 + w] != 0;
    uint64_t key = lane < keys ? A.keys[at * W + lane] : 0;
    double ref = lane < A.waves ? A.sums[2 * (at + lane)] : -INFINITY, sum = lane < A.waves ? A.sums[2 * (at + lane) + 1] : 0.0;
    double total = -INFINITY;
    int token = -1;
    if (live && done) {
      if (lane == 0) total = score, token = A.eos;
    } else if (live) {
      const double mine = ref;
      for (int i = lane + 64; i < A.waves; i += 64) ref = fmax(ref, A.sums[2 * (at + i)]);
#pragma unroll
      for (int d = 32; d; d >>= 1) ref = fmax(ref, __shfl_xor(ref, d));
      sum = mine > -INFINITY ? sum * exp(mine - ref) : 0.0;
      for (int i = lane + 64; i < A.waves; i += 64) {
        const double r = A.sums[2 * (at + i)];
        if (r > -INFINITY) sum += A.sums[2 * (at + i) + 1] * exp(r - ref);
      }
#pragma unroll
      for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
      Best best;
      best.merge(key, min(keys, 64), W);
      for (int i0 = 64; i0 < keys; i0 += 64) {
        key = i0 + lane < keys ? A.keys[at * W + i0 + lane] : 0;
        best.merge(key, min(keys - i0, 64), W);
      }
      if (lane < W && best.list) {
        total = (double)score + ((double)from_ordered((uint32_t)(best.list >> 32)) - ref - log(sum));
        token = (int)~(uint32_t)best.list;
      }
    }
    if (lane < W) {
      double rank = total;
      if (A.penalty != 0.0) rank = total / pow((double)max(length + (done ? 0 : 1), 1), A.penalty);
      s_rank[w * W + lane] = rank, s_total[w * W + lane] = total, s_token[w * W + lane] = token;
    }
    if (lane == 0) s_length[w] = length, s_done[w] = done;
  }
  __syncthreads();
  // each candidate's place: a row's lie in their order, so of another row's the
  // better ones are counted by halving; four threads count for one
  const int all = W * W, part = threadIdx.x & 3;
  for (int i = threadIdx.x >> 2; i < all; i += blockDim.x >> 2) {
    const double rank = s_rank[i];
    const int w = i / W;
    int before = part ? 0 : i - w * W;
    for (int o = part; o < W && before < W; o += 4) {
      if (o == w) continue;
      int lo = 0, hi = W;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        const double other = s_rank[o * W + mid];
        if (other > rank || (other == rank && o < w)) lo = mid + 1; else hi = mid;
      }
      before += lo;
    }
    before += __shfl_xor(before, 1);
    before += __shfl_xor(before, 2);
    if (part || before >= W || !(s_total[i] > -INFINITY)) continue;
    atomicAdd(&s_chosen, 1);
    const int to = row0 + before, token = s_token[i];
    const bool done = s_done[w] != 0;
    A.parent[to] = row0 + w;
    A.token[to] = token;
    A.score_out[to] = (float)s_total[i];
    A.length_out[to] = s_length[w] + (done ? 0 : 1);
    A.done_out[to] = done || (token == A.eos && A.eos >= 0);
  }
  __syncthreads();
  if (threadIdx.x >= s_chosen && threadIdx.x < W) {
    const int to = row0 + threadIdx.x;
    A.parent[to] = -1;
    A.token[to] = -1;
    A.score_out[to] = -INFINITY;
    A.length_out[to] = 0;
    A.done_out[to] = 1;
  }
}

}  // namespace

hipError_t launch_select(const SelectArgs& A, int dtype, hipStream_t s) {
  const int64_t jobs = (int64_t)A.requests * A.beams * A.waves;
  const unsigned blocks = (unsigned)((jobs + 3) / 4);
  if (dtype == LORA_DTYPE_BF16) rows_kernel<Bf16><<<blocks, 256, 0, s>>>(A);
  else rows_kernel<F32><<<blocks, 256, 0, s>>>(A);
  pick_kernel<<<A.requests, 64 * max_i(4, min_i(A.beams, 16)), 0, s>>>(A);
  return hipGetLastError();
}

}  // namespace beam
}  // namespace lora
