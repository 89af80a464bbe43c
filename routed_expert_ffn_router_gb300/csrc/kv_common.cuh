// Device helpers shared by the paged cache's kernels.
#pragma once

#include "kv_internal.h"

namespace moe {
namespace kv {

__device__ __forceinline__ int add_acq_rel_gpu(int* p, int v) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two values of the cache's type, x in the low half.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&v));
  else return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// log2 of the factor that the matrix kernels' probabilities carry, and with them
// their sums l and o. fp16 has a fixed step below 2^-14: lifted by 2^7 (to 2^15 at
// most, the running maximum being at most 2^8 low), half of that step is 2^-32 of
// the largest probability.
template <bool F16>
__host__ __device__ constexpr float lift() { return F16 ? 7.f : 0.f; }

// The sequence that row t of a call belongs to.
__device__ __forceinline__ int seq_of_row(const Rows& r, int t) {
  if (!r.row_start) return t / r.n_q;
  int lo = 0, hi = r.B - 1;  // the last sequence that starts at or before it
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (r.row_start[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

}  // namespace kv
}  // namespace moe
