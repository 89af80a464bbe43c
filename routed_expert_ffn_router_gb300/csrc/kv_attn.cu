// Attention over a paged cache for any head size and page size: warps for each
// (row, query head). The online softmax keeps the running maximum m, the sum l
// = sum 2^(s - m) and o = sum 2^(s - m) v in fp32 registers,
//   m' = max(m, s),  l' = l 2^(m - m') + 2^(s - m'),  o' = o 2^(m - m') + 2^(s - m') v,
// s in base-2 units (scale * log2 e folded into the product). A group of lanes
// holds a key (8 elements of D per lane) and takes kAhead of them at a time, so
// that their loads are under way together; groups and warps are joined at the
// end in a fixed order.
//
// Every query head reads its keys by itself (from L2), and a key costs a chain of
// page number, key and value: bound by those latencies. Measured: 8 sequences of
// up to 4,093 tokens, 16 / 2 heads of 80, 86 us (one warp per row and one key at
// a time: 1,580); 64 sequences, 32 / 8 heads, 790 us; a 512-token prompt, 16 / 4
// heads of 80, 287 us.
#include "kv_common.cuh"

namespace moe {
namespace kv {

namespace {

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<F16>(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

// (row, head) pairs of a chunk below which warps share a row: over 3,000 tokens,
// 1,600 pairs 673 us against 832 with a warp each, 3,200 1,311 against 1,572, 6,400
// the same, a 512-token prompt (8,192 pairs) 461 against 294.
constexpr int kFewRows = 4096;
constexpr int kAhead = 4;  // keys of a group whose loads are under way together

// LPK lanes per key: the smallest of 8, 16, 32 with 8 * LPK >= D. SP warps share
// a row's keys (1: a warp has a row to itself, four rows a CTA).
template <bool F16, int LPK, int SP>
__global__ void __launch_bounds__(SP == 1 ? 128 : 32 * SP) attn_rows_kernel(Cache c, Rows r, Attn a, int32_t* status) {
  constexpr int NG = 32 / LPK;
  __shared__ float s_part[SP == 1 ? 1 : SP][2 + 8 * LPK];
  const int lane = threadIdx.x & 31, g = lane / LPK, gl = lane % LPK, part = SP == 1 ? 0 : threadIdx.x >> 5;
  const long long w = SP == 1 ? (long long)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  if (w >= (long long)r.n_rows * a.Hq) return;
  const int t = (int)(w / a.Hq), hq = (int)(w - (long long)t * a.Hq), hk = hq / a.G;
  const Seq s = load_seq(c, r, seq_of_row(r, t), lane == 0 && part == 0 ? status : nullptr);
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
    for (int i0 = part * NG * kAhead; i0 < count; i0 += SP * NG * kAhead) {
      uint4 kk[kAhead], vv[kAhead];
      float x[kAhead];
      bool in[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * NG + g, j = i < first ? i : i - first + from;
        int pg = -1;
        if (i < count) {
          pg = tab[j / c.page];
          if (pg < 0 || pg >= c.n_pages) {
            atomicOr(status, DEV_BAD_SLOT);
            pg = -1;
          }
        }
        in[u] = pg >= 0;
        if (in[u] && act) {
          const long long at = (((long long)pg * c.Hkv + hk) * c.page + j % c.page) * c.D + gl * 8;
          kk[u] = *reinterpret_cast<const uint4*>(c.k + at);
          vv[u] = *reinterpret_cast<const uint4*>(c.v + at);
        }
      }
      float m2 = m;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        x[u] = 0.f;
        if (in[u] && act) {
          float kv[8];
          unpack8<F16>(kk[u], kv);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[u] = fmaf(q[e], kv[e], x[u]);
        }
#pragma unroll
        for (int d = LPK / 2; d > 0; d >>= 1) x[u] += __shfl_xor_sync(0xffffffffu, x[u], d);
        x[u] = in[u] ? x[u] * sc : -INFINITY;
        m2 = fmaxf(m2, x[u]);
      }
      const float al = m2 == -INFINITY ? 1.f : exp2f(m - m2);
      m = m2;
      l *= al;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] *= al;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (!in[u]) continue;  // what lies there reaches nothing
        const float p = m2 == -INFINITY ? 0.f : exp2f(x[u] - m2);
        l += p;
        if (act) {
          float kv[8];
          unpack8<F16>(vv[u], kv);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = fmaf(p, kv[e], o[e]);
        }
      }
      __syncwarp();
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
  uint16_t* out = a.o + ((long long)t * a.Hq + hq) * c.D;
  float* lse = a.lse ? a.lse + (long long)t * a.Hq + hq : nullptr;
  if constexpr (SP > 1) {  // the warps' parts, in warp order
    if (g == 0) {
      if (gl == 0) {
        s_part[part][0] = m;
        s_part[part][1] = l;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s_part[part][2 + gl * 8 + e] = o[e];
    }
    __syncthreads();
    if (threadIdx.x >= LPK) return;
    m = -INFINITY;
    for (int i = 0; i < SP; ++i) m = fmaxf(m, s_part[i][0]);
    l = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.f;
    for (int i = 0; i < SP; ++i) {
      const float x = m == -INFINITY ? 0.f : exp2f(s_part[i][0] - m);
      l = fmaf(s_part[i][1], x, l);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(s_part[i][2 + gl * 8 + e], x, o[e]);
    }
  }
  if (g == 0 && act) {
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = pack2<F16>(o[2 * i] * inv, o[2 * i + 1] * inv);
    *reinterpret_cast<uint4*>(out + gl * 8) = make_uint4(y[0], y[1], y[2], y[3]);
    if (gl == 0 && lse) *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
}

}  // namespace

cudaError_t launch_attn_rows(const Cache& c, const Rows& r, const Attn& a, bool f16, bool decode, int32_t* status,
                             cudaStream_t st) {
  const long long rows = (long long)r.n_rows * a.Hq;
  // Sixteen warps share a row of a decode window (always, so that a row's bits do
  // not depend on the rest of the call) and of a chunk too small to fill the GPU.
  constexpr int kShare = 16;
  const bool share = decode || rows < kFewRows;
  const unsigned grid = (unsigned)(share ? rows : (rows + 3) / 4);
  launch_begin(K_ATTN_ROWS, st);
#define MOE_KV_ROWS(F, L)                                                                    \
  if (share) attn_rows_kernel<F, L, kShare><<<grid, 32 * kShare, 0, st>>>(c, r, a, status);  \
  else attn_rows_kernel<F, L, 1><<<grid, 128, 0, st>>>(c, r, a, status)
  if (c.D <= 64) {
    if (f16) { MOE_KV_ROWS(true, 8); } else { MOE_KV_ROWS(false, 8); }
  } else if (c.D <= 128) {
    if (f16) { MOE_KV_ROWS(true, 16); } else { MOE_KV_ROWS(false, 16); }
  } else {
    if (f16) { MOE_KV_ROWS(true, 32); } else { MOE_KV_ROWS(false, 32); }
  }
#undef MOE_KV_ROWS
  launch_end(st);
  return cudaGetLastError();
}

}  // namespace kv
}  // namespace moe
