// Shared parts of the attention kernels over the paged NVFP4 key/value cache.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace moe {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A running maximum is raised only when a score passes it by this much (in powers of two):
// the weights then stay below 2^8, far inside float16, and most tiles rescale nothing.
constexpr float kRaise = 8.0f;
constexpr float kNoMax = -3.402823466e38f;  // no key seen yet

MOE_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

MOE_DEV uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// two E4M3 bytes (low, high) -> f16x2, exact
MOE_DEV uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}

MOE_DEV uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// mbar_wait with the limit read once per block: short in code (the roles of a block share the
// instruction caches) and without a load from global memory in every wait.
struct Patience {
  volatile int abort;
  unsigned long long limit;
};
MOE_DEV bool wait_soon(uint64_t* bar, uint32_t parity, Patience* w, int32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (w->abort) return false;
    if (globaltimer_ns() - t0 > w->limit) {
      w->abort = 1;
      atomicExch(status, kStatusTimeout);
      return false;
    }
  }
  return true;
}

// A sequence of the batch, clamped so that no index made from it leaves its array.
struct SeqSpan {
  int q0, n_q, ctx;
};

MOE_DEV SeqSpan load_seq(const KvAttnArgs& a, int b) {
  SeqSpan s;
  const int lo = a.cu_q[b], hi = a.cu_q[b + 1];
  s.q0 = min(max(lo, 0), a.T);
  s.n_q = max(min(hi, a.T) - s.q0, 0);
  s.ctx = (int)min((int64_t)max(a.ctx_lens[b], 0), (int64_t)a.max_pages * a.cache.page_size);
  return s;
}

}  // namespace moe
