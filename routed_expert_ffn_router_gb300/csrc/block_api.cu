// C ABI of the decoder-block operators (include/moe_block.h): argument
// validation and choice of kernel.
#include <climits>

#include "block_internal.h"

using namespace moe;
using namespace moe::block;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
bool is_input(int t) { return t == MOE_T_F32 || t == MOE_T_BF16 || t == MOE_T_F16; }
int size_of(int t) { return t == MOE_T_F32 ? 4 : t == MOE_T_E4M3 ? 1 : 2; }

moe_status linear(const moe_linear_desc* d, const moe_kv_rows* r, const moe_linear_args* a, void* stream, bool step) {
  launch_count_reset();
  if (!d || !r || !a) return MOE_ERR_INVALID;
  if (d->dtype != MOE_KV_BF16 && d->dtype != MOE_KV_F16) return MOE_ERR_INVALID;
  if (d->n_slots < 1 || d->Hk < 1 || d->Hv < 1 || d->Hv % d->Hk || d->Dk < 1 || d->Dv < 1) return MOE_ERR_INVALID;
  if (!d->state || !aligned(d->state, 16)) return MOE_ERR_INVALID;
  if (d->Dk % 8 || d->Dk > 256 || d->Dv % 8 || d->Dv > 256 || d->Hv > 65535 || d->n_slots > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  if (r->B < 0 || r->n_rows < 0 || !aligned(r->slots, 4) || !aligned(r->row_start, 4)) return MOE_ERR_INVALID;
  if ((r->n_rows > 0 && r->B < 1) || (r->B > 0 && !r->row_start && r->n_rows % r->B)) return MOE_ERR_INVALID;
  if (step && r->row_start) return MOE_ERR_INVALID;
  if (step && r->B > 0 && r->n_rows / r->B > 16) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)r->B * d->Hv * ((d->Dv + 31) / 32) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (!(a->scale > -3.0e38f && a->scale < 3.0e38f) || !aligned(a->status, 4)) return MOE_ERR_INVALID;
  if (r->n_rows == 0) return MOE_OK;
  if (!a->q || !a->k || !a->v || !a->g || !a->o) return MOE_ERR_INVALID;
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->o, 16) || !aligned(a->g, 4))
    return MOE_ERR_INVALID;
  const int64_t qk = (int64_t)d->Hk * d->Dk, vo = (int64_t)d->Hv * d->Dv;
  if (a->q_stride % 8 || a->k_stride % 8 || a->v_stride % 8 || a->q_stride < qk || a->k_stride < qk || a->v_stride < vo)
    return MOE_ERR_INVALID;
  if (a->g_stride != 0 && a->g_stride < d->Hv) return MOE_ERR_INVALID;
  Linear l;
  l.n_slots = d->n_slots; l.Hk = d->Hk; l.Hv = d->Hv; l.Dk = d->Dk; l.Dv = d->Dv; l.state = d->state;
  l.q = static_cast<const uint16_t*>(a->q); l.k = static_cast<const uint16_t*>(a->k); l.v = static_cast<const uint16_t*>(a->v);
  l.q_stride = a->q_stride; l.k_stride = a->k_stride; l.v_stride = a->v_stride;
  l.g = a->g; l.g_stride = a->g_stride; l.scale = a->scale; l.o = static_cast<uint16_t*>(a->o); l.status = a->status;
  kv::Rows rw;
  rw.B = r->B; rw.n_rows = r->n_rows; rw.n_q = r->row_start ? 0 : r->n_rows / r->B;
  rw.slots = r->slots; rw.row_start = r->row_start;
  // A chunk of few rows goes row by row, as a decode window: 32 heads of 128, 8
  // sequences of 8 rows 15 us row by row and 22 on the tensor cores, of 16 rows 26 and
  // 22; heads of 64, 16 rows 10 and 17. With rows given by row_start a sequence may
  // have all of them.
  const int rows_each = r->row_start ? r->n_rows : rw.n_q;
  if (!step && rows_each > (d->Dk > 64 || d->Dv > 64 ? 12 : 24) && linear_chunk_supported(l))
    return cuda_status(launch_linear_chunk(l, rw, d->dtype == MOE_KV_F16, static_cast<cudaStream_t>(stream)));
  return cuda_status(launch_linear_rows(l, rw, d->dtype == MOE_KV_F16, step, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

moe_status moe_rms_norm(const moe_norm_args* a, void* stream) {
  launch_count_reset();
  if (!a || a->T < 0 || a->H < 1) return MOE_ERR_INVALID;
  if (!is_input(a->x_type) || (a->res && !is_input(a->res_type)) || (a->w && !is_input(a->w_type))) return MOE_ERR_INVALID;
  if (!is_input(a->y_type) && a->y_type != MOE_T_E4M3) return MOE_ERR_INVALID;
  if (!(a->eps >= 0.f && a->eps < 3.0e38f) || !(a->w_offset > -3.0e38f && a->w_offset < 3.0e38f)) return MOE_ERR_INVALID;
  const bool fp8 = a->y_type == MOE_T_E4M3;
  if (a->group && (!fp8 || a->group < 16 || (a->group & (a->group - 1)) || a->H % a->group)) return MOE_ERR_INVALID;
  if (a->H > kMostNormH || a->T > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  if (a->T == 0) return MOE_OK;
  if (!a->x || !a->y || (fp8 && !a->scales) || a->x == a->res || a->y == a->res) return MOE_ERR_INVALID;
  if (a->x_stride < a->H || a->y_stride < a->H || (a->res && a->res_stride < a->H)) return MOE_ERR_INVALID;
  if (a->x == a->y && (a->x_type != a->y_type || a->x_stride != a->y_stride)) return MOE_ERR_INVALID;
  if (!aligned(a->x, size_of(a->x_type)) || !aligned(a->y, size_of(a->y_type)) || !aligned(a->scales, 4) ||
      (a->res && !aligned(a->res, size_of(a->res_type))) || (a->w && !aligned(a->w, size_of(a->w_type))))
    return MOE_ERR_INVALID;
  const bool vec = a->H % 8 == 0 && a->x_stride % 8 == 0 && a->y_stride % 8 == 0 && aligned(a->x, 16) &&
                   aligned(a->y, fp8 ? 8 : 16) && aligned(a->w, 16) && (!a->res || (a->res_stride % 8 == 0 && aligned(a->res, 16)));
  return cuda_status(launch_rms_norm(*a, vec, static_cast<cudaStream_t>(stream)));
}

moe_status moe_token_logprobs(const moe_logprobs_args* a, void* stream) {
  launch_count_reset();
  if (!a || a->T < 0 || a->V < 1 || a->top < 0 || !is_input(a->type)) return MOE_ERR_INVALID;
  if (!(a->temperature >= 1e-30f && a->temperature < 3.0e38f)) return MOE_ERR_INVALID;
  if (a->top > a->V || a->top > 32 || a->V > (1 << 28)) return MOE_ERR_UNSUPPORTED;
  if (a->T == 0) return MOE_OK;
  if (!a->logits || !aligned(a->logits, size_of(a->type)) || a->stride < a->V) return MOE_ERR_INVALID;
  if ((a->logprob || a->rank) && !a->tokens) return MOE_ERR_INVALID;
  if (a->top ? !a->top_ids || !a->top_logprobs : a->top_ids || a->top_logprobs) return MOE_ERR_INVALID;
  if (!aligned(a->tokens, 4) || !aligned(a->logprob, 4) || !aligned(a->rank, 4) || !aligned(a->entropy, 4) ||
      !aligned(a->top_ids, 4) || !aligned(a->top_logprobs, 4))
    return MOE_ERR_INVALID;
  return cuda_status(launch_token_logprobs(*a, static_cast<cudaStream_t>(stream)));
}

moe_status moe_linear_step(const moe_linear_desc* d, const moe_kv_rows* r, const moe_linear_args* a, void* stream) {
  return linear(d, r, a, stream, true);
}

moe_status moe_linear_chunk(const moe_linear_desc* d, const moe_kv_rows* r, const moe_linear_args* a, void* stream) {
  return linear(d, r, a, stream, false);
}

}  // extern "C"
