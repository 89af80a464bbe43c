// Device helpers shared by the linear attention kernels.
#pragma once

#include "block_internal.h"

namespace moe {
namespace block {

// The rows of one sequence of a call.
struct Span {
  int slot;     // -1: out of range
  int row0, n;
};
__device__ __forceinline__ Span load_span(const Linear& a, const kv::Rows& r, int b) {
  Span s;
  s.row0 = r.row_start ? r.row_start[b] : b * r.n_q;
  const int row1 = r.row_start ? r.row_start[b + 1] : s.row0 + r.n_q;
  s.row0 = max(0, min(s.row0, r.n_rows));
  s.n = max(0, min(row1, r.n_rows) - s.row0);
  s.slot = r.slots ? r.slots[b] : b;
  if (s.slot < 0 || s.slot >= a.n_slots) s.slot = -1;
  return s;
}

// Whether sequence b may use its slot: it is in range and no earlier sequence of
// the call has it (two of them would write one state). By all threads of the CTA.
__device__ __forceinline__ bool span_allowed(const Linear& a, const kv::Rows& r, int b, const Span& s, bool report) {
  int bad = s.slot < 0 ? DEV_BAD_SLOT : 0;
  if (s.slot >= 0 && r.slots)
    for (int i = threadIdx.x; i < b; i += blockDim.x)
      if (r.slots[i] == s.slot) bad = kv::DEV_REFUSED;
  const bool any = __syncthreads_or(bad);
  if (bad && report && a.status) atomicOr(a.status, bad);
  return !any;
}

// The logarithm of a decay: at most 0, at least -1e4 (its exponential is 0 in fp32
// long before, and sums of many stay finite: no -inf - -inf). NaN stays.
__device__ __forceinline__ float bounded_g(float g) { return g < 0.f ? fmaxf(g, -1e4f) : g == g ? 0.f : g; }

// S -> e^g S as fma(S, x, S y): with y = 1 and x = e^g - 1 near 1, where e^g in fp32
// is off by up to 2^-24 the same way for every token of a constant decay (after
// 4,000 tokens that was 3e-4 of the state); with y = 0 and x = e^g else, where the
// difference of S and S (1 - e^g) would be off by 2^-24 of S.
__device__ __forceinline__ float2 decay_of(float g) {
  const bool near = !(g < -0.5f);
  return near ? make_float2(expm1f(g), 1.f) : make_float2(expf(g), 0.f);
}

}  // namespace block
}  // namespace moe
