// moe_kv_append_rope: new queries and keys turned by their positions, keys and
// values written into the cache's pages (include/moe_kv.h).
//
// Angles. Pair i of a token at position p stands at p freq[i] / 2^64 of a turn:
// freq is an integer, so the product modulo 2^64 is the exact angle modulo a
// turn at any position, in one 64-bit multiplication. Its upper 32 bits, as a
// signed number of half turns / 2^31, go to sincospif: an error of 2^-25 half
// turns, 2e-7 radians, wherever the token lies. (In fp32, p times a frequency is
// off by 2^-24 p: 0.008 radians at 131,072.) A row's rot / 2 sines and cosines
// are computed once and serve all its heads.
//
// One CTA per row. A thread turns 8 pairs of a head (two 16-byte loads, two
// stores) and reads both halves before it writes them, so q_out may be q. The
// first loads are under way while the row's sequence, length and page are looked
// up, which is a chain of loads that a short call's time consists of.
#include "kv_common.cuh"

namespace moe {
namespace kv {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 2;  // items of a thread that are fetched before the row is looked up

struct Rope {
  int rot, interleaved;
  float gain;
  const unsigned long long* freq;
  const int32_t* positions;
  int Hq;
  const uint16_t* q;
  uint16_t* q_out;
  long long q_stride, q_out_stride;
};

template <bool F16>
__device__ __forceinline__ void turn8(uint4& x, uint4& y, const float2* cs) {  // pairs (x[i], y[i])
  uint32_t* a = reinterpret_cast<uint32_t*>(&x);
  uint32_t* b = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = unpack2<F16>(a[i]), v = unpack2<F16>(b[i]), c0 = cs[2 * i], c1 = cs[2 * i + 1];
    a[i] = pack2<F16>(u.x * c0.x - v.x * c0.y, u.y * c1.x - v.y * c1.y);
    b[i] = pack2<F16>(v.x * c0.x + u.x * c0.y, v.y * c1.x + u.y * c1.y);
  }
}
template <bool F16>
__device__ __forceinline__ void turn4(uint4& x, const float2* cs) {  // pairs (x[2 i], x[2 i + 1])
  uint32_t* a = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = unpack2<F16>(a[i]), c = cs[i];
    a[i] = pack2<F16>(u.x * c.x - u.y * c.y, u.y * c.x + u.x * c.y);
  }
}

// MODE 0: halves, 16-byte pieces of 8 pairs (rot a multiple of 16). 1:
// interleaved, 16-byte pieces of 4 pairs (rot a multiple of 8). 2: single values
// (any rot, either layout).
template <bool F16, int MODE>
__global__ void __launch_bounds__(kThreads) append_rope_kernel(Cache c, Rows r, Rope p, const uint16_t* k, const uint16_t* v,
                                                               long long stride, int32_t* status) {
  __shared__ __align__(16) float2 cs[128];
  const int t = blockIdx.x, tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const int half = p.rot >> 1;
  // pieces of a turned head and of a copied one
  const int vd = c.D >> 3, pieces = MODE == 0 ? vd - (p.rot >> 4) : MODE == 1 ? vd : c.D - half;
  const int n_q = p.Hq * pieces, n_k = n_q + c.Hkv * pieces, n_all = n_k + c.Hkv * vd;
  // Item i of the row: a piece of a head of q (kind 0), k (1) or v (2): the values
  // from d0 on, and their partners from d1 on (-1: there are none).
  struct Item {
    int kind, h, d0, d1;
    const uint16_t* src;
  };
  const auto item = [&](int i) {
    Item x;
    if (i >= n_k) {
      x.kind = 2;
      x.h = (i - n_k) / vd;
      x.d0 = (i - n_k - x.h * vd) * 8;
      x.d1 = -1;
      x.src = v + (long long)t * stride + (long long)x.h * c.D;
      return x;
    }
    x.kind = i >= n_q;
    const int j = x.kind ? i - n_q : i;
    x.h = j / pieces;
    const int e = j - x.h * pieces;
    x.src = x.kind ? k + (long long)t * stride + (long long)x.h * c.D : p.q + (long long)t * p.q_stride + (long long)x.h * c.D;
    if (MODE == 0) {
      const int n8 = p.rot >> 4;
      x.d0 = e < n8 ? e * 8 : p.rot + (e - n8) * 8;
      x.d1 = e < n8 ? half + e * 8 : -1;
    } else if (MODE == 1) {
      x.d0 = e * 8;
      x.d1 = -1;
    } else {
      x.d0 = e >= half ? p.rot + e - half : p.interleaved ? 2 * e : e;
      x.d1 = e >= half ? -1 : p.interleaved ? 2 * e + 1 : e + half;
    }
    return x;
  };
  // the thread's first items: on their way while the row is looked up
  uint4 first[kAhead][2];
  if constexpr (MODE != 2) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = tid + u * kThreads;
      if (i < n_all) {
        const Item x = item(i);
        first[u][0] = *reinterpret_cast<const uint4*>(x.src + x.d0);
        if (MODE == 0 && x.d1 >= 0) first[u][1] = *reinterpret_cast<const uint4*>(x.src + x.d1);
      }
    }
  }
  const Seq s = load_seq(c, r, seq_of_row(r, t), tid == 0 ? status : nullptr);
  const bool inside = t >= s.row0 && t < s.row0 + s.n;
  if (!inside) return;  // behind the last sequence
  const int tok = s.slot < 0 ? -1 : s.len - s.n + (t - s.row0);
  int pg = -1;
  if (tok >= 0) {
    pg = c.table[(long long)s.slot * c.max_pages + tok / c.page];
    if (pg < 0 || pg >= c.n_pages) {
      if (tid == 0) atomicOr(status, DEV_BAD_SLOT);
      pg = -1;
    }
    const long long pos = p.positions ? p.positions[t] : tok;
    for (int i = tid; i < half; i += kThreads) {
      const unsigned long long turns = (unsigned long long)pos * p.freq[i];
      float sn, cn;
      sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &sn, &cn);
      cs[i] = make_float2(cn * p.gain, sn * p.gain);
    }
  }
  __syncthreads();
  const long long base = (long long)(pg < 0 ? 0 : pg) * c.Hkv * c.page + (tok < 0 ? 0 : tok % c.page);
  const int last = tok < 0 ? n_q : pg < 0 ? n_q : n_all;  // without a page keys and values go nowhere
  const auto work = [&](int i, int u) {  // u: which of `first` holds it, -1 none
    const Item x = item(i);
    uint16_t* dst = x.kind == 0 ? p.q_out + (long long)t * p.q_out_stride + (long long)x.h * c.D
                                : (x.kind == 1 ? c.k : c.v) + (base + (long long)x.h * c.page) * c.D;
    if constexpr (MODE != 2) {
      uint4 v0 = u >= 0 ? first[u < 0 ? 0 : u][0] : *reinterpret_cast<const uint4*>(x.src + x.d0), v1;
      if (MODE == 0 && x.d1 >= 0) {
        v1 = u >= 0 ? first[u < 0 ? 0 : u][1] : *reinterpret_cast<const uint4*>(x.src + x.d1);
        if (tok >= 0) turn8<F16>(v0, v1, cs + x.d0);
        *reinterpret_cast<uint4*>(dst + x.d1) = v1;
      }
      if (MODE == 1 && x.kind < 2 && tok >= 0 && x.d0 < p.rot) turn4<F16>(v0, cs + (x.d0 >> 1));
      *reinterpret_cast<uint4*>(dst + x.d0) = v0;
    } else if (x.kind == 2) {
      *reinterpret_cast<uint4*>(dst + x.d0) = *reinterpret_cast<const uint4*>(x.src + x.d0);
    } else if (x.d1 >= 0) {
      uint32_t xy = (uint32_t)x.src[x.d0] | (uint32_t)x.src[x.d1] << 16;
      if (tok >= 0) {
        const float2 f = unpack2<F16>(xy), w = cs[p.interleaved ? x.d0 >> 1 : x.d0];
        xy = pack2<F16>(f.x * w.x - f.y * w.y, f.y * w.x + f.x * w.y);
      }
      dst[x.d0] = (uint16_t)xy;
      dst[x.d1] = (uint16_t)(xy >> 16);
    } else {
      dst[x.d0] = x.src[x.d0];
    }
  };
  if constexpr (MODE != 2) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (tid + u * kThreads < last) work(tid + u * kThreads, u);
    for (int i = tid + kAhead * kThreads; i < last; i += kThreads) work(i, -1);
  } else {
    for (int i = tid; i < last; i += kThreads) work(i, -1);
  }
}

}  // namespace

cudaError_t launch_append_rope(const Cache& c, const Rows& r, const moe_rope_desc& d, const int32_t* positions, int Hq,
                               const uint16_t* q, long long q_stride, uint16_t* q_out, long long q_out_stride, const uint16_t* k,
                               const uint16_t* v, long long stride, bool f16, int32_t* status, cudaStream_t st) {
  Rope p;
  p.rot = d.rot; p.interleaved = d.layout == MOE_ROPE_INTERLEAVED; p.gain = d.gain;
  p.freq = reinterpret_cast<const unsigned long long*>(d.freq);
  p.positions = positions;
  p.Hq = Hq; p.q = q; p.q_out = q_out; p.q_stride = q_stride; p.q_out_stride = q_out_stride;
  const int mode = p.interleaved ? (d.rot % 8 ? 2 : 1) : (d.rot % 16 ? 2 : 0);
  const auto go = [&](auto kernel) {
    return launch_pdl(K_KV_APPEND, kernel, dim3(r.n_rows), kThreads, 0, st, c, r, p, k, v, stride, status);
  };
  if (f16) return mode == 0 ? go(append_rope_kernel<true, 0>) : mode == 1 ? go(append_rope_kernel<true, 1>) : go(append_rope_kernel<true, 2>);
  return mode == 0 ? go(append_rope_kernel<false, 0>) : mode == 1 ? go(append_rope_kernel<false, 1>) : go(append_rope_kernel<false, 2>);
}

}  // namespace kv
}  // namespace moe
