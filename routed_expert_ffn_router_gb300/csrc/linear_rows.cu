// Linear attention with a decay, row by row (include/moe_block.h): decode windows
// of any shape, and the prompt chunks that the matrix kernel does not take.
//
// The columns of a state are independent: a CTA owns 32 columns of one head's
// [Dk][Dv] and keeps them in registers (a thread has 4 columns of every 16th row)
// from one read to one write, whatever the number of rows, so a decode window
// costs a read and a write of the state. Rows come through shared memory up to 16 at a
// time; a row's products q S are summed over Dk within a warp by shuffles and over
// the four warps once per 16 rows.
//
// What bounds it: the state, read and written once; a token's arithmetic is 6 Dk Dv
// flops per head and small beside it. Measured, back to back in a graph: 64 sequences
// of one token, 32 heads of [128][128], 43 us for 270 MB (6.2 TB/s, 0.92 of a copy's
// rate). CTAs of 64 columns were no faster. A one-row window's q, k and v fetched beside the
// state took 42 to 44 us, and longer windows a fifth more.
#include "block_internal.h"
#include "kv_common.cuh"
#include "linear_common.cuh"

namespace moe {
namespace block {

namespace {

constexpr int kCols = 32;   // of Dv per CTA
constexpr int kThreads = 4 * kCols, kWarps = kThreads / 32;
constexpr int kRows = 16;   // tokens staged at a time, at most

template <bool F16>
__device__ __forceinline__ float one(const uint16_t* p) {
  return kv::unpack2<F16>((uint32_t)*p).x;
}

// DK: 64, 128 or 256, at least the head size. staged: tokens at a time.
template <bool F16, int DK>
__global__ void __launch_bounds__(kThreads, DK <= 128 ? 8 : 4) linear_rows_kernel(Linear a, kv::Rows r, int staged) {
  constexpr int NI = DK / 16, kLanes = kCols / 4;  // lanes of a row
  extern __shared__ __align__(16) float smem_rows[];
  float (*qs)[DK] = reinterpret_cast<float (*)[DK]>(smem_rows);
  float (*ks)[DK] = qs + staged;
  float (*vs)[kCols] = reinterpret_cast<float (*)[kCols]>(ks + staged);
  float (*po)[kWarps][kCols] = reinterpret_cast<float (*)[kWarps][kCols]>(vs + staged);
  __shared__ float2 decay[kRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, col = (tid % kLanes) * 4, row = tid / kLanes;
  griddep_wait();
  griddep_launch_dependents();
  const int tiles = (a.Dv + kCols - 1) / kCols;
  const int tile = blockIdx.x % tiles, h = blockIdx.x / tiles % a.Hv, b = blockIdx.x / tiles / a.Hv;
  const int c0 = tile * kCols, hk = h / (a.Hv / a.Hk);
  const Span s = load_span(a, r, b);
  if (s.n == 0) return;
  float4* state = reinterpret_cast<float4*>(a.state + ((long long)max(s.slot, 0) * a.Hv + h) * a.Dk * a.Dv + c0 + col);
  const bool mine = c0 + col < a.Dv && s.slot >= 0;
  float4 S[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int d = row + 16 * i;
    // (evict first, here and below: 64 sequences 48.4 -> 43.3 us, of three rows 69 -> 57; states
    // that stay in the L2, as those of a model of many layers do not, 12.6 -> 13.9)
    S[i] = mine && d < a.Dk ? __ldcs(&state[(long long)d * a.Dv / 4]) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const bool ok = span_allowed(a, r, b, s, tile == 0 && h == 0);
  for (int t0 = 0; t0 < s.n; t0 += staged) {
    const int m = min(staged, s.n - t0);
    __syncthreads();  // the last rows have been used
    for (int i = tid; i < m * a.Dk; i += kThreads) {
      const int j = i / a.Dk, d = i - j * a.Dk;
      const long long t = s.row0 + t0 + j;
      qs[j][d] = one<F16>(a.q + t * a.q_stride + (long long)hk * a.Dk + d) * a.scale;
      ks[j][d] = one<F16>(a.k + t * a.k_stride + (long long)hk * a.Dk + d);
    }
    for (int i = tid; i < m * kCols; i += kThreads) {
      const int j = i / kCols, c = i % kCols;
      vs[j][c] = c0 + c < a.Dv ? one<F16>(a.v + (s.row0 + t0 + j) * a.v_stride + (long long)h * a.Dv + c0 + c) : 0.f;
    }
    if (tid < m) decay[tid] = decay_of(bounded_g(a.g[(s.row0 + t0 + tid) * a.g_stride + h]));
    __syncthreads();
    for (int j = 0; j < m; ++j) {
      const float2 e = decay[j];
      const float4 v = *reinterpret_cast<const float4*>(&vs[j][col]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int d = row + 16 * i;
        if (DK == 256 && d >= a.Dk) break;
        const float k = d < a.Dk ? ks[j][d] : 0.f, q = d < a.Dk ? qs[j][d] : 0.f;
        S[i].x = fmaf(k, v.x, fmaf(S[i].x, e.x, S[i].x * e.y)); S[i].y = fmaf(k, v.y, fmaf(S[i].y, e.x, S[i].y * e.y));
        S[i].z = fmaf(k, v.z, fmaf(S[i].z, e.x, S[i].z * e.y)); S[i].w = fmaf(k, v.w, fmaf(S[i].w, e.x, S[i].w * e.y));
        o.x = fmaf(q, S[i].x, o.x); o.y = fmaf(q, S[i].y, o.y);
        o.z = fmaf(q, S[i].z, o.z); o.w = fmaf(q, S[i].w, o.w);
      }
#pragma unroll
      for (int x = kLanes; x < 32; x <<= 1) {
        o.x += __shfl_xor_sync(0xffffffffu, o.x, x); o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, x); o.w += __shfl_xor_sync(0xffffffffu, o.w, x);
      }
      if (lane < kLanes) *reinterpret_cast<float4*>(&po[j][warp][col]) = o;
    }
    __syncthreads();
    for (int i = tid; i < m * kCols / 2; i += kThreads) {
      const int j = i / (kCols / 2), c = i % (kCols / 2) * 2;
      if (c0 + c >= a.Dv) continue;
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 f = *reinterpret_cast<const float2*>(&po[j][w][c]);
        x += f.x;
        y += f.y;
      }
      *reinterpret_cast<uint32_t*>(a.o + ((s.row0 + t0 + j) * (long long)a.Hv + h) * a.Dv + c0 + c) = ok ? kv::pack2<F16>(x, y) : 0u;
    }
  }
  if (!ok || !mine) return;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int d = row + 16 * i;
    if (d < a.Dk) __stcs(&state[(long long)d * a.Dv / 4], S[i]);
  }
}

template <bool F16, int DK>
cudaError_t launch_rows(const Linear& a, const kv::Rows& r, bool step, cudaStream_t st) {
  // no more shared memory than a window's rows need: 16 rows' of it (27 KB) left six
  // CTAs on an SM and a window of one row at 52 us instead of 47
  const int staged = step && r.n_q < kRows ? r.n_q : kRows;
  const size_t smem = (size_t)staged * (2 * DK + kCols + kWarps * kCols) * 4;
  const unsigned grid = (unsigned)((long long)r.B * a.Hv * ((a.Dv + kCols - 1) / kCols));
  return launch_pdl(step ? K_LINEAR_STEP : K_LINEAR_CHUNK, linear_rows_kernel<F16, DK>, dim3(grid), kThreads, smem, st, a, r, staged);
}

}  // namespace

cudaError_t launch_linear_rows(const Linear& a, const kv::Rows& r, bool f16, bool step, cudaStream_t st) {
  if (f16) return a.Dk <= 64 ? launch_rows<true, 64>(a, r, step, st) : a.Dk <= 128 ? launch_rows<true, 128>(a, r, step, st) : launch_rows<true, 256>(a, r, step, st);
  return a.Dk <= 64 ? launch_rows<false, 64>(a, r, step, st) : a.Dk <= 128 ? launch_rows<false, 128>(a, r, step, st) : launch_rows<false, 256>(a, r, step, st);
}

}  // namespace block
}  // namespace moe
