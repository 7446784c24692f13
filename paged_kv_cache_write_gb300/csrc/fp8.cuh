// Device helpers of the 8-bit cache: e4m3 values, their conversions and the
// power-of-two scale of a (block, KV head).
//
// An element of an 8-bit pool stands for (e4m3 value) * (scale of its block
// and KV head).  Scales are powers of two 2^e, kFp8MinExp <= e <= kFp8MaxExp:
// e4m3 is a floating format, so a finer scale would not make its relative
// error smaller, and with a power of two
//   - x * 2^-e is exact, so e4m3's rounding is the only one of a write,
//   - moving a block to a larger scale is exact but for values that become
//     subnormal (below 2^-6 of the scale),
//   - every value of the cache has 4 significand bits and an exponent far
//     inside bf16's range: it is a bf16 number.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "device.cuh"

namespace pkv {

constexpr int kFp8MinExp = -60;
constexpr int kFp8MaxExp = 60;

// 2^e for an exponent of the normal range.
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// Scale for values of magnitude at most a (a >= 0, not NaN): 2^e with the
// smallest e in range such that a <= 448 * 2^e.  a = m * 2^E with 1 <= m < 2
// needs e = E - 8 if m <= 1.75, else E - 7; zero, subnormals and infinity
// are settled by the clamp.
__device__ __forceinline__ float fp8_scale_for(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int E = static_cast<int>(bits >> 23) - 127;
  int e = E - ((bits & 0x7fffffu) <= 0x600000u ? 8 : 7);
  e = max(kFp8MinExp, min(kFp8MaxExp, e));
  return pow2f(e);
}

// Two e4m3 bytes (lo in the low byte), round to nearest even; magnitudes
// past 448 become 448, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The two e4m3 bytes of `b` as f16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t b) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(b));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t b) {
  const uint32_t h = e4m3x2_to_f16x2(b);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// What a prefill reports of one sequence's chunk, query rows q0 .. end - 1 of
// total_q, at the end of L tokens (last: the batch's last sequence).  The kernels
// compute no chunk that reaches outside the rows or has more queries than tokens,
// and not more than max_q_len rows of a longer one for certain.
struct ChunkLimits {
  int total_q, max_q_len, max_len;
  int64_t table_tokens;  // that a table row has blocks for
};

__device__ __forceinline__ void report_bad_chunk(int32_t* err, const ChunkLimits& m, int q0,
                                                 int end, int L, bool last) {
  const int64_t c = int64_t(end) - q0;
  if (q0 < 0 || c < 0 || c > m.max_q_len || end > m.total_q || (last && end != m.total_q))
    report(err, PKV_DEVERR_LENGTH);
  if (c <= 0) return;  // (nothing of the sequence is read)
  if (L < c) report(err, PKV_DEVERR_LENGTH);
  else if (L > m.max_len)
    report(err, L > m.table_tokens ? PKV_DEVERR_TABLE_WIDTH : PKV_DEVERR_LENGTH);
}

// True in one lane of a converged warp.  Unlike a test of the lane id this
// lets the compiler keep what the lane issues asynchronous operations with
// (descriptors, shared-memory addresses) in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Waits of the 8-bit kernels: the hardware parks the thread until the phase is
// complete or, for a poll that fails, for up to kParkNs; after kFp8Polls of
// those (2 s) the wait gives up.
constexpr uint32_t kParkNs = 100000;
constexpr uint32_t kFp8Polls = 20000;

__device__ __forceinline__ bool mbar_park(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity), "r"(kParkNs)
      : "memory");
  return done != 0;
}

// Bounded wait that also ends once some thread of the CTA has given up.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity,
                                              volatile int* abort_flag,
                                              uint32_t polls = kFp8Polls) {
  if (mbar_park(bar, parity)) return true;
  for (uint32_t i = 0; i < polls; ++i) {
    if (mbar_park(bar, parity)) return true;
    if (*abort_flag) return false;
  }
  return false;
}

// The same by a whole warp, whose lanes then agree: each lane looks for itself,
// and one may see the flag where another sees the phase complete, but what
// follows (shuffles, matrix products) is the whole warp's.
__device__ __forceinline__ bool warp_wait_or_abort(uint64_t* bar, uint32_t parity,
                                                   volatile int* abort_flag,
                                                   uint32_t polls = kFp8Polls) {
  return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, polls)) != 0;
}

// The same without a vote for each wait (one costs a consumer of narrow heads 3 to
// 8%): a lane that gives up sets the flag and goes on with its warp.  The warp looks
// at the flag, by vote, before it stores what it computed.
__device__ __forceinline__ void wait_or_flag(uint64_t* bar, uint32_t parity,
                                             volatile int* abort_flag, int32_t* err,
                                             uint32_t polls = kFp8Polls) {
  if (!wait_or_abort(bar, parity, abort_flag, polls)) {
    // (the one that gives up first reports: the others see its flag)
    if (!*abort_flag) report(err, PKV_DEVERR_TIMEOUT);
    *abort_flag = 1;
  }
}

}  // namespace pkv
