/*
 * moe_block.h - C ABI of what a decoder layer has around its attention
 * (moe_kv.h) and its routed experts (moe.h), for sm_103a: the norm with the
 * residual's addition, linear attention with a decay, and the log
 * probabilities of tokens. Rotary positions are a part of the cache's append
 * (moe_kv_append_rope in moe_kv.h).
 *
 * Conventions are those of moe.h: every pointer is a DEVICE pointer unless its
 * comment says host, the caller owns every buffer, calls are asynchronous on
 * `stream` and never synchronise, may be captured into a CUDA graph after one
 * warm-up call per kind, and report host-detected errors before anything is
 * launched. These calls need no workspace, so any number of them may be under
 * way at once; buffers that a call writes must not overlap others of the call,
 * but where a comment says so. Results are deterministic: the same call gives
 * the same bits.
 */
#ifndef MOE_BLOCK_GB300_H
#define MOE_BLOCK_GB300_H

#include "moe_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_T_F32 = 0, MOE_T_BF16 = 1, MOE_T_F16 = 2, MOE_T_E4M3 = 3 } moe_type;

/* The residual's addition and the root-mean-square norm of T rows of H values:
 *   r    <- x + r                                 rounded to r's type, in place
 *   y[i]  = r[i] (w[i] + w_offset) / sqrt(mean(r^2) + eps)
 * The norm is of what r then holds. res NULL: y is the norm of x; w NULL: ones.
 * Sums in fp32, one rounding to y's type. y in e4m3: for each group of `group`
 * columns (0: the whole row; else a power of two from 16 that divides H)
 *   scales[t][g] = max |y| / 448,   y[t][i] = e4m3(y / scales[t][g])
 * (a group of zeros has scale 0), saturating, NaN kept. Squares beyond fp32
 * make a row's mean infinite and its y 0 or NaN.
 *
 * H up to 16,384, T up to 2^30; strides are elements from row to row, at least H. Rows whose
 * pointers and strides keep 8 values on a 16-byte boundary (8 bytes for e4m3)
 * and H a multiple of 8 are read 8 values at a time, others one by one. y may
 * be x where type and stride are the same. x, res: F32, BF16 or F16; w: the
 * same; y: any; scales [T][H / group] fp32 (e4m3 only). A HOST struct. */
typedef struct {
  int32_t T, H;
  moe_type x_type, res_type, w_type, y_type;
  int32_t group;
  float eps, w_offset;
  const void *x;
  int64_t x_stride;
  void *res;
  int64_t res_stride;
  const void *w;
  void *y;
  int64_t y_stride;
  float *scales;
} moe_norm_args;

moe_status moe_rms_norm(const moe_norm_args *a, void *stream);

/* Log probabilities over T rows of V logits z, at a temperature:
 *   p_i = exp(z_i / temperature) / sum_j exp(z_j / temperature)
 *   logprob[t] = ln p_token          rank[t] = how many tokens come before it
 *   entropy[t] = -sum_i p_i ln p_i   top_ids[t][0..top), top_logprobs[t][0..top)
 * in the order of the logits, ties to the lower id. One pass over the logits,
 * sums in fp32. Each output may be NULL (top_ids and top_logprobs go together);
 * tokens [T] int32 is needed for logprob and rank. A token outside [0, V) (a
 * padded row) has logprob 0 and rank -1. Logits of -inf have p = 0; in a row of
 * nothing else every logprob is -inf and the entropy 0. With a NaN or +inf in a
 * row its logprobs and entropy are NaN; in the order a NaN stands with -inf.
 * How a row is split depends on T, so its last bits may differ in another call.
 *
 * logits: F32, BF16 or F16, `stride` elements from row to row (at least V), of
 * the type's own alignment; V up to 2^28, top up to min(V, 32), temperature
 * from 1e-30. A HOST struct. */
typedef struct {
  int32_t T, V, top;
  moe_type type;
  float temperature;
  const void *logits;
  int64_t stride;
  const int32_t *tokens;
  float *logprob;
  int32_t *rank;
  float *entropy;
  int32_t *top_ids;
  float *top_logprobs;
} moe_logprobs_args;

moe_status moe_token_logprobs(const moe_logprobs_args *a, void *stream);

/* Linear attention with a decay. Each slot holds a state S [Hv][Dk][Dv] in
 * fp32; for the rows of a sequence in their order, v head h reading q and k
 * head h / (Hv / Hk),
 *   S   <- exp(g[t][h]) S + k_t^T v_t        o[t][h] = scale q_t S
 * g is the logarithm of the decay: above 0 counts as 0, -inf forgets all finite values
 * before the token (0 times an infinity or a NaN is NaN: a state that holds one is emptied by
 * writing zeros); g_stride 0: one row of g for all tokens. The rows are
 * those of moe_kv_rows: sequence b is slot slots[b] (NULL: slot b), the slots
 * of a call distinct; a sequence without rows leaves its state as it was. A
 * slot out of range (2) or one that an earlier sequence of the call has (64)
 * ORs that bit into *status (nullable): its rows' o is 0 and no state changes. 4: a
 * bounded wait expired, the call's results are incomplete.
 * Rows behind the last sequence are left as they were.
 *
 * q, k [n_rows][Hk][Dk] and v [n_rows][Hv][Dv] in `dtype`, 16-byte aligned, the
 * heads of a row contiguous, strides (elements from row to row) a multiple of
 * 8, so that they may be parts of one projection; o [n_rows][Hv][Dv]
 * contiguous, 16-byte aligned; state 16-byte aligned. Dk, Dv multiples of 8 up
 * to 256, Hv a multiple of Hk up to 65,535. HOST structs. */
typedef struct {
  int32_t n_slots, Hk, Hv, Dk, Dv;
  moe_kv_dtype dtype;
  float *state; /* [n_slots][Hv][Dk][Dv] */
} moe_linear_desc;

typedef struct {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const float *g;
  int64_t g_stride;
  float scale;
  void *o;
  int32_t *status;
} moe_linear_args;

/* Decode windows: the same number of rows (1 .. 16) for every sequence,
 * row_start NULL. The state is read and written once; products in fp32. */
moe_status moe_linear_step(const moe_linear_desc *d, const moe_kv_rows *rows, const moe_linear_args *a, void *stream);

/* Prompt chunks: any number of rows per sequence. With Dk and Dv of 64 or 128, and
 * more than a few rows, on the tensor cores: a state and a score enter their products
 * rounded once to `dtype`. The state itself stays within fp32's roundings in bf16; in
 * fp16 each decayed key is besides off by up to 2^-38 of the largest |k| of its head among
 * the 128 tokens around it, which shows where larger keys have all but decayed. How a
 * long sequence is split depends on the call, so a row's last bits may differ in
 * another call. There a state and values that a sequence's rows see must be finite: a NaN or an
 * infinity may reach rows before it. Other sequences' rows and heads, and rows behind
 * the last sequence, reach nothing. */
moe_status moe_linear_chunk(const moe_linear_desc *d, const moe_kv_rows *rows, const moe_linear_args *a, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_GB300_H */
