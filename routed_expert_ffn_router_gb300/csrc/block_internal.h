// Internal declarations of the decoder-block operators (include/moe_block.h).
#pragma once

#include "kinds.h"
#include "kv_internal.h"
#include "moe_block.h"

namespace moe {
namespace block {

using kv::launch_pdl;

constexpr int kMostNormH = 16384;

// vec: rows can be read and written 8 values at a time (see moe_norm_args).
cudaError_t launch_rms_norm(const moe_norm_args& a, bool vec, cudaStream_t st);

cudaError_t launch_token_logprobs(const moe_logprobs_args& a, cudaStream_t st);

struct Linear {
  int n_slots, Hk, Hv, Dk, Dv;
  float *state;
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  const float *g;
  long long g_stride;
  float scale;
  uint16_t *o;
  int32_t *status;
};
// The recurrence, row by row (any shape).
cudaError_t launch_linear_rows(const Linear& a, const kv::Rows& r, bool f16, bool step, cudaStream_t st);

// Prompt chunks on the tensor cores: Dk and Dv of 64 or 128.
bool linear_chunk_supported(const Linear& a);
cudaError_t launch_linear_chunk(const Linear& a, const kv::Rows& r, bool f16, cudaStream_t st);

}  // namespace block
}  // namespace moe
