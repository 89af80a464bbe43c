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
// One CTA per row. What a short call's time consists of is the chain of loads that
// finds the row's sequence, length and page: three of them, by a warp whose lanes look
// at all sequences at once; each thread's first pieces are under way meanwhile. A
// thread turns 8 pairs of a head at a time (two 16-byte loads, two stores) and reads
// both halves before it writes them, so q_out may be q. Four rows per CTA, which go
// through the chain together, were slower (11.4 us for 2,048 rows of 32 / 8 heads
// against 11.0): their larger CTAs fill the GPU less evenly.
//
// Measured, back to back in a graph: 8 rows of 16 / 2 heads 2.9 us, the chain and a
// launch; 2,048 rows of 32 / 8 heads, pages of 64, 9.3 us for 50 MB (5.4 TB/s, 0.79 of a
// copy's rate); five ragged chunks of up to 901 rows, 28 / 4 heads, 64 of 128 values
// turned in interleaved pairs, fp16, 13.6 us (0.64). A CTA's life is the chain (three
// latencies of memory) and then few bytes, so that waves of CTAs and not bandwidth
// bound the long calls. With the values' first pieces fetched behind the chain: 10.8 and
// 14.3. In halves three pieces at a time and seven CTAs per SM were the best for 16 to 64
// query heads (32 / 8: four and eight 10.4, four and seven 10.0, two and eight 10.2);
// interleaved pairs gain and lose with the shape (32 / 8 11.3 with four and eight, 11.7
// with two and eleven; the ragged case 13.6 and 12.9).
#include <climits>

#include "kv_common.cuh"

namespace moe {
namespace kv {

namespace {

constexpr int kThreads = 128;

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

// Sines and cosines lie in shared memory by pairs of pairs: those of pairs 2 j and
// 2 j + 1 of all pieces side by side, so that a warp's 16-byte reads meet no bank
// twice (piece after piece they took four times as long as all the rest).
// cs: the piece's first two pairs, n: pieces of a head.
template <bool F16>
__device__ __forceinline__ void turn8(uint4& x, uint4& y, const float4* cs, int n) {  // pairs (x[i], y[i])
  uint32_t* a = reinterpret_cast<uint32_t*>(&x);
  uint32_t* b = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = unpack2<F16>(a[i]), v = unpack2<F16>(b[i]);
    const float4 w = cs[i * n];  // cos, sin, cos, sin
    a[i] = pack2<F16>(u.x * w.x - v.x * w.y, u.y * w.z - v.y * w.w);
    b[i] = pack2<F16>(v.x * w.x + u.x * w.y, v.y * w.z + u.y * w.w);
  }
}
template <bool F16>
__device__ __forceinline__ void turn4(uint4& x, const float4* cs, int n) {  // pairs (x[2 i], x[2 i + 1])
  uint32_t* a = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 u = unpack2<F16>(a[2 * i]), v = unpack2<F16>(a[2 * i + 1]);
    const float4 w = cs[i * n];
    a[2 * i] = pack2<F16>(u.x * w.x - u.y * w.y, u.y * w.x + u.x * w.y);
    a[2 * i + 1] = pack2<F16>(v.x * w.z - v.y * w.w, v.y * w.z + v.x * w.w);
  }
}

// A thread's way through the pieces of its row's heads: piece e of head h, then the
// piece `step` further.
struct Cursor {
  int h, e, dh, de, per;
  __device__ Cursor(int at, int step, int per_head) : h(at / per_head), dh(step / per_head), per(per_head) {
    e = at - h * per_head;
    de = step - dh * per_head;
  }
  __device__ void next() {
    h += dh;
    e += de;
    if (e >= per) {
      e -= per;
      ++h;
    }
  }
};

// The sequence of row t, by a whole warp. Up to 32 sequences: every lane looks at one.
__device__ __forceinline__ Seq find_seq(const Cache& c, const Rows& r, int t, int32_t* status) {
  const int lane = threadIdx.x & 31;
  if (!r.row_start || r.B > 32) return load_seq(c, r, seq_of_row(r, t), lane == 0 ? status : nullptr);
  const Seq mine = load_seq(c, r, min(lane, r.B - 1), nullptr);
  const int first = lane < r.B ? r.row_start[lane] : INT_MAX;
  // the last sequence that starts at or before the row
  const int b = max(0, __popc(__ballot_sync(0xffffffffu, first <= t)) - 1);
  Seq s;
  s.slot = __shfl_sync(0xffffffffu, mine.slot, b);
  s.len = __shfl_sync(0xffffffffu, mine.len, b);
  s.row0 = __shfl_sync(0xffffffffu, mine.row0, b);
  s.n = __shfl_sync(0xffffffffu, mine.n, b);
  if (lane == b && (mine.slot < 0 || c.lens[mine.slot] > (long long)c.max_pages * c.page)) atomicOr(status, DEV_BAD_SLOT);
  return s;
}

// MODE 0: halves, 16-byte pieces of 8 pairs (rot a multiple of 16). 1:
// interleaved, 16-byte pieces of 4 pairs (rot a multiple of 8). 2: single values
// (any rot, either layout).
template <bool F16, int MODE>
__global__ void __launch_bounds__(kThreads, MODE == 0 ? 7 : 8) append_rope_kernel(Cache c, Rows r, Rope p, const uint16_t* k, const uint16_t* v,
                                                               long long stride, int32_t* status) {
  __shared__ __align__(16) float2 cs[kThreads];
  __shared__ int s_tok, s_page, s_pos;  // token (-1: none, -2: no row), page (-1: none), position
  constexpr int kBatch = MODE == 0 ? 3 : 4;  // pieces of a thread under way together
  const int at = threadIdx.x;
  const long long t = blockIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const int half = p.rot >> 1, vd = c.D >> 3;
  // pieces of a turned head (q's heads, then k's) and of a copied one
  const int pieces = MODE == 0 ? vd - (p.rot >> 4) : MODE == 1 ? vd : c.D - half;
  const int n_turn = (p.Hq + c.Hkv) * pieces, n_copy = c.Hkv * vd;
  const uint16_t* q_row = p.q + t * p.q_stride;
  const uint16_t* k_row = k + t * stride;
  const auto source = [&](const Cursor& x) { return x.h < p.Hq ? q_row + x.h * c.D : k_row + (x.h - p.Hq) * c.D; };
  // where a piece begins, and its partners (-1: it has none and is copied)
  const auto begin = [&](int e) { return MODE == 0 ? (e < (p.rot >> 4) ? e * 8 : half + e * 8) : e * 8; };
  const auto partner = [&](int e) { return MODE == 0 && e < (p.rot >> 4) ? half + e * 8 : -1; };
  uint4 x[kBatch], y[kBatch];
  const auto fetch = [&](Cursor cur, int i) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (i + u * kThreads < n_turn) {
        const uint16_t* src = source(cur);
        x[u] = *reinterpret_cast<const uint4*>(src + begin(cur.e));
        if (MODE == 0 && partner(cur.e) >= 0) y[u] = *reinterpret_cast<const uint4*>(src + partner(cur.e));
      }
      cur.next();
    }
  };
  Cursor cur(at, kThreads, pieces);
  if (MODE != 2) fetch(cur, at);
  const uint16_t* v_row = v + t * stride;
  Cursor copy(at, kThreads, vd);
  uint4 first_v;
  if (at < n_copy) first_v = *reinterpret_cast<const uint4*>(v_row + copy.h * c.D + copy.e * 8);
  const unsigned long long freq = at < half ? p.freq[at] : 0;

  if (at < 32) {
    const Seq s = find_seq(c, r, (int)t, status);
    if (at == 0) {
      int tok = -2, pg = -1, pos = 0;
      if (t >= s.row0 && t < s.row0 + s.n) {
        tok = s.slot < 0 ? -1 : max(-1, s.len - s.n + ((int)t - s.row0));
        if (tok >= 0) {
          pg = c.table[(long long)s.slot * c.max_pages + tok / c.page];
          if (pg < 0 || pg >= c.n_pages) {
            atomicOr(status, DEV_BAD_SLOT);
            pg = -1;
          }
          pos = p.positions ? p.positions[t] : tok;
        }
      }
      s_tok = tok;
      s_page = pg;
      s_pos = pos;
    }
  }
  __syncthreads();
  const int tok = s_tok, pg = s_page;
  if (tok >= 0 && at < half) {
    const unsigned long long turns = (unsigned long long)(long long)s_pos * freq;
    float sn, cn;
    sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &sn, &cn);
    const int per = MODE == 0 ? 8 : 4;  // pairs of a piece
    const int to = MODE == 2 ? at : (((at % per) >> 1) * (half / per) + at / per) * 2 + (at & 1);
    cs[to] = make_float2(cn * p.gain, sn * p.gain);
  }
  __syncthreads();
  if (tok == -2) return;  // behind the last sequence
  const float4* cs4 = reinterpret_cast<const float4*>(cs);
  const long long base = (long long)max(pg, 0) * c.Hkv * c.page + (tok < 0 ? 0 : tok % c.page);
  const auto target = [&](int h) {
    return h < p.Hq ? p.q_out + t * p.q_out_stride + h * c.D : c.k + (base + (long long)(h - p.Hq) * c.page) * c.D;
  };
  const int last = pg < 0 ? p.Hq * pieces : n_turn;  // without a page keys and values go nowhere
  if constexpr (MODE != 2) {
    for (int i = at; i < last; i += kBatch * kThreads) {
      if (i != at) fetch(cur, i);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (i + u * kThreads < last) {
          uint16_t* dst = target(cur.h);
          const int d0 = begin(cur.e), d1 = partner(cur.e);
          if (MODE == 0 && d1 >= 0) {
            if (tok >= 0) turn8<F16>(x[u], y[u], cs4 + cur.e, half >> 3);
            *reinterpret_cast<uint4*>(dst + d1) = y[u];
          }
          if (MODE == 1 && tok >= 0 && d0 < p.rot) turn4<F16>(x[u], cs4 + cur.e, half >> 2);
          *reinterpret_cast<uint4*>(dst + d0) = x[u];
        }
        cur.next();
      }
    }
  } else {
    for (int i = at; i < last; i += kThreads, cur.next()) {
      const uint16_t* src = source(cur);
      uint16_t* dst = target(cur.h);
      if (cur.e < half) {
        const int d0 = p.interleaved ? 2 * cur.e : cur.e, d1 = p.interleaved ? 2 * cur.e + 1 : cur.e + half;
        uint32_t xy = (uint32_t)src[d0] | (uint32_t)src[d1] << 16;
        if (tok >= 0) {
          const float2 f = unpack2<F16>(xy), w = cs[cur.e];
          xy = pack2<F16>(f.x * w.x - f.y * w.y, f.y * w.x + f.x * w.y);
        }
        dst[d0] = (uint16_t)xy;
        dst[d1] = (uint16_t)(xy >> 16);
      } else {
        const int d = half + cur.e;
        dst[d] = src[d];
      }
    }
  }
  if (pg < 0) return;
  for (int i = at; i < n_copy; i += kThreads, copy.next())
    *reinterpret_cast<uint4*>(c.v + (base + (long long)copy.h * c.page) * c.D + copy.e * 8) =
        i == at ? first_v : *reinterpret_cast<const uint4*>(v_row + copy.h * c.D + copy.e * 8);
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
