// Attention over a paged cache for any head size and page size: one warp per
// (row, query head). The online softmax keeps the running maximum m, the sum l
// = sum 2^(s - m) and o = sum 2^(s - m) v in fp32 registers,
//   m' = max(m, s),  l' = l 2^(m - m') + 2^(s - m'),  o' = o 2^(m - m') + 2^(s - m') v,
// s in base-2 units (scale * log2 e folded into the product). A group of lanes
// holds one key (8 elements of D per lane), the groups of a warp take keys in
// turn and are joined at the end in a fixed order.
#include "kv_internal.h"

namespace moe {
namespace kv {

namespace {

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F16) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    } else {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// LPK lanes per key: the smallest of 8, 16, 32 with 8 * LPK >= D.
template <bool F16, int LPK>
__global__ void __launch_bounds__(128) attn_rows_kernel(Cache c, Rows r, Attn a, int32_t* status) {
  constexpr int NG = 32 / LPK;
  const int lane = threadIdx.x & 31, g = lane / LPK, gl = lane % LPK;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= (long long)r.n_rows * a.Hq) return;
  const int t = (int)(w / a.Hq), hq = (int)(w - (long long)t * a.Hq), hk = hq / a.G;
  int b;
  if (r.row_start) {
    int lo = 0, hi = r.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (r.row_start[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
  } else {
    b = t / r.n_q;
  }
  const Seq s = load_seq(c, r, b, lane == 0 ? status : nullptr);
  const int tok = s.len - s.n + (t - s.row0);
  const bool act = gl * 8 < c.D;
  float q[8], o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = o[i] = 0.f;
  if (act) unpack8<F16>(*reinterpret_cast<const uint4*>(a.q + (long long)t * a.q_stride + hq * c.D + gl * 8), q);
  float m = -INFINITY, l = 0.f;
  if (s.slot >= 0 && tok >= 0 && t >= s.row0 && t < s.row0 + s.n) {
    const float sc = a.scale * 1.4426950408889634f;
    const int32_t* tab = c.table + (long long)s.slot * c.max_pages;
    // the visible tokens: [0, first) and [from, tok]
    const int from = a.window > 0 ? max(0, tok - a.window + 1) : 0;
    const int first = min(a.n_sink, from);
    const int count = first + (tok + 1 - from);
    for (int i0 = 0; i0 < count; i0 += NG) {
      const int i = i0 + g;
      const int j = i < first ? i : i - first + from;
      int pg = -1;
      if (i < count) {
        pg = tab[j / c.page];
        if (pg < 0 || pg >= c.n_pages) {
          atomicOr(status, DEV_BAD_SLOT);
          pg = -1;
        }
      }
      const long long at = (((long long)pg * c.Hkv + hk) * c.page + j % c.page) * c.D + gl * 8;
      float x = 0.f, kv[8];
      if (pg >= 0 && act) {
        unpack8<F16>(*reinterpret_cast<const uint4*>(c.k + at), kv);
#pragma unroll
        for (int e = 0; e < 8; ++e) x = fmaf(q[e], kv[e], x);
      }
#pragma unroll
      for (int d = LPK / 2; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      if (pg < 0) continue;
      x *= sc;
      const float m2 = fmaxf(m, x);
      const float al = m2 == -INFINITY ? 1.f : exp2f(m - m2), p = m2 == -INFINITY ? 0.f : exp2f(x - m2);
      m = m2;
      l = fmaf(l, al, p);
      if (act) {
        unpack8<F16>(*reinterpret_cast<const uint4*>(c.v + at), kv);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(p, kv[e], o[e] * al);
      }
    }
  }
#pragma unroll
  for (int d = LPK; d < 32; d <<= 1) {  // join the groups
    const float m1 = __shfl_xor_sync(0xffffffffu, m, d), l1 = __shfl_xor_sync(0xffffffffu, l, d);
    const float m2 = fmaxf(m, m1);
    const float x0 = m2 == -INFINITY ? 0.f : exp2f(m - m2), x1 = m2 == -INFINITY ? 0.f : exp2f(m1 - m2);
    m = m2;
    l = l * x0 + l1 * x1;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = o[e] * x0 + __shfl_xor_sync(0xffffffffu, o[e], d) * x1;
  }
  if (g == 0 && act) {
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float y0 = o[2 * i] * inv, y1 = o[2 * i + 1] * inv;
      if constexpr (F16) {
        const __half2 h = __floats2half2_rn(y0, y1);
        out[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(y0, y1);
        out[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(a.o + ((long long)t * a.Hq + hq) * c.D + gl * 8) = make_uint4(out[0], out[1], out[2], out[3]);
    if (gl == 0 && a.lse)
      a.lse[(long long)t * a.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
}

}  // namespace

cudaError_t launch_attn_rows(const Cache& c, const Rows& r, const Attn& a, bool f16, int32_t* status, cudaStream_t st) {
  const long long warps = (long long)r.n_rows * a.Hq;
  const unsigned grid = (unsigned)((warps + 3) / 4);
  launch_begin(K_ATTN_ROWS, st);
#define MOE_KV_ROWS(F, L) attn_rows_kernel<F, L><<<grid, 128, 0, st>>>(c, r, a, status)
  if (c.D <= 64) {
    if (f16) MOE_KV_ROWS(true, 8);
    else MOE_KV_ROWS(false, 8);
  } else if (c.D <= 128) {
    if (f16) MOE_KV_ROWS(true, 16);
    else MOE_KV_ROWS(false, 16);
  } else {
    if (f16) MOE_KV_ROWS(true, 32);
    else MOE_KV_ROWS(false, 32);
  }
#undef MOE_KV_ROWS
  launch_end(st);
  return cudaGetLastError();
}

}  // namespace kv
}  // namespace moe
