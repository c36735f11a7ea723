// What the linear-attention kernels share: decays, packed fp32 and bf16 arithmetic, bounded waits, operand images.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace kda {
namespace {

// lam^n; 1 at n = 0 whatever the decay.  Only whole n >= 0 occur, so nothing overflows however fast a head forgets;
// the fp32 error of n log lam, at most 2^-24 |n log lam|, is largest beside e^-1.
__device__ __forceinline__ float decay_pow(float log_decay, int64_t n) {
  return n == 0 ? 1.f : expf((float)n * log_decay);
}
__device__ __forceinline__ int64_t item_tokens(const int32_t* lengths, int b, int64_t N) {
  if (!lengths) return N;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : (n > N ? N : n);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return reinterpret_cast<const uint32_t&>(v);
}
// Two fp32 in one register pair, multiplied by one instruction.
__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("{\n\t.reg .b64 m;\n\tmov.b64 m, 0xbf800000bf800000;\n\tfma.rn.f32x2 %0, %2, m, %1;\n\t}" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// A bf16 pair as two fp32.
__device__ __forceinline__ uint64_t wide2(uint32_t v) {
  return pair2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(uint64_t ab) {
  float a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(ab));
  return pack2(a, b);
}
// ab = bf16 pair + the rest.  A value above the largest bf16 one takes that one (rounded to nearest it would be infinite,
// and the rest with it): the rest is below 2^-8 of it either way.
__device__ __forceinline__ uint32_t take2(uint64_t& ab) {
  float a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(ab));
  uint32_t v;
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(b), "f"(a));
  ab = sub2(ab, wide2(v));
  return v;
}
// Bounded wait; a wait that gives up sets the CTA's flag, and every later wait returns at once.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = tc::globaltimer_ns();
  while (!tc::mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (tc::globaltimer_ns() - t0 > kWaitNs) { *abort_flag = 1; return false; }
  }
  return true;
}
// The same for a whole warp: one answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag));
}

// Byte offset of 16-byte chunk c8 of row r in an image of rows x (64 columns per panel).
__device__ __forceinline__ uint32_t image_off(int rows, int r, int c8) {
  return (uint32_t)((c8 >> 3) * rows * 128 + r * 128 + (((c8 ^ r) & 7) << 4));
}

// The decay of a whole segment multiplies a state again and again, so its fp32 rounding would add up; it is kept
// in two fp32 terms of the fp64 power.
struct Factor { float hi, lo; };
__device__ __forceinline__ Factor segment_factor(float log_decay, int64_t n) {
  const double f = n == 0 ? 1.0 : exp((double)n * (double)log_decay);
  const float hi = (float)f;
  return {hi, (float)(f - (double)hi)};
}

}  // namespace
}  // namespace kda
