// lora_kv_attend: attention of a step's rows over the paged 4-bit cache.
//
// Mathematics: per row, one pass over the cached tokens with a running
// maximum m and sum l of exp2((s - m)), s = scale log2(e) q.K.  The keys of a
// request are split into chunks (lora_kv_build's plan); chunks of one row are
// joined by o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
//
// A work item is (16 or 32 rows = new tokens x heads that share a kv head, one
// chunk, one kv head), walked by a work-group whose waves take turns at steps
// of 32 tokens and join their results in LDS; the work-group that finishes a
// row's last chunk joins the chunks.  Per step a wave
// reads the 17/16 byte per value pair once, converts the codes to bf16 with
// v_cvt_scalef32_pk_bf16_fp4 (exact), and multiplies on
// v_mfma_f32_16x16x32_bf16: S^T = K Q^T, whose result layout (row = lane%16,
// tokens 4g..4g+3 of each 16) is the B operand that O^T = V^T P^T needs, with
// the record's V order supplying A, so P never leaves its registers.  It is
// rounded to bf16 there, by up to 2^-8 of each weight (with a second term the
// large decode step below takes 231 us against 222, and its error against 64
// bits, of which rounding the result makes 0.0017, 0.0017 against 0.0020); l
// sums the rounded weights, so that they sum to one (no change in time).  fp32 rows and weights are split into three bf16
// terms (24 bits), the codes being exact.
//
// Measured on MI355X: 128 requests of up to 4097 tokens, 32 kv heads of 128,
// 213 us = 5.5 TB/s of codes and scales (a read of 1 GiB reaches 6.1, a copy
// 4.7): HBM is the bound, with the vector units about half busy converting.
// The loads of a wave's next step go out, without a branch, before the current
// one's arithmetic; loads behind a condition, or spilled registers between
// them (4 waves per SIMD leave 128), cost waits for those just sent: 257 us.
// Small steps are bound by latency (one request of 32768 tokens 16 us, 48 of
// up to 2049 12 us: item, block ids, keys and the join follow one another).
// Work-groups of 4 waves take what those of 8 do, in half the LDS.
#include "lora_kv_tile.h"

namespace lora {
namespace kv {

namespace {

template <class E, int NC>
hipError_t launch(const AttendArgs& A, bool many, hipStream_t s) {
  auto blocks = [&](int c) { return (unsigned)(class_cap(c, A.T, A.B, A.cache.heads, A.G) * A.cache.heads); };
  if (many) {
    if constexpr (sizeof(typename E::T) == 2) attend_wide_kernel<NC, AttendArgs><<<blocks(2), 256, 0, s>>>(A);
    else attend_kernel<E, NC, 2, 2, AttendArgs><<<blocks(2) * (kWideRows / kMidRows), 64 * kWaves, 0, s>>>(A);
    attend_kernel<E, NC, 2, 1, AttendArgs><<<blocks(1), 64 * kWaves, 0, s>>>(A);
  }
  attend_kernel<E, NC, 1, 0, AttendArgs><<<blocks(0), 64 * kWaves, 0, s>>>(A);
  return hipGetLastError();
}

template <class E>
hipError_t launch_nc(const AttendArgs& A, bool many, hipStream_t s) {
  switch (A.cache.nc) {
    case 1: return launch<E, 1>(A, many, s);
    case 2: return launch<E, 2>(A, many, s);
    case 3: return launch<E, 3>(A, many, s);
    case 4: return launch<E, 4>(A, many, s);
    case 5: return launch<E, 5>(A, many, s);
    case 6: return launch<E, 6>(A, many, s);
    case 7: return launch<E, 7>(A, many, s);
    default: return launch<E, 8>(A, many, s);
  }
}

}  // namespace

hipError_t launch_attend(const AttendArgs& A, int dtype, bool many, hipStream_t s) {
  return dtype == LORA_DTYPE_BF16 ? launch_nc<Bf16>(A, many, s) : launch_nc<F32>(A, many, s);
}

}  // namespace kv
}  // namespace lora
