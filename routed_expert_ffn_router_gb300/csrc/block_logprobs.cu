// Log probabilities of given tokens, ranks, entropies and top alternatives over
// rows of logits (include/moe_block.h).
//
// One pass. With a running maximum m (scores in units of log2, c = log2 e /
// temperature, d_i = (z_i - m) c):
//   l = sum 2^d_i,  s = sum 2^d_i d_i      a larger maximum m': a = (m - m') c,
//   s' = 2^a (s + l a),  l' = 2^a l
// and at the end ln p_i = (z_i - m) / temperature - ln l, entropy = ln l - ln 2 s / l.
// z - m is taken before the product: c m, rounded, would be off by 2^-24 of itself in
// all terms alike. Two forms of the sums: where m is so far above the lowest values
// that those vanish, logits below kLow (-inf, the type's lowest value) count as kLow;
// else d is bounded by -200, where 2^d is 0 in fp32 already (a row of the type's
// lowest value is uniform, and -inf - -inf no NaN).
//
// One value of the maximum is left out of l, which ln(1 + l) puts back: where one token
// has nearly all of the probability, its logarithm and the entropy are as exact
// relative to themselves as elsewhere.
//
// A row is read by a cluster of 1 to 8 CTAs, each by 8 warps that take chunks of 32
// lanes x 64 bytes in turn, through shared memory, the next chunk's copies under way; rows
// start anywhere, so the pieces of a row go by 16-byte boundaries of memory and the
// first and the last by single values. The parts meet through shared memory, then
// through the cluster's: few rows use many SMs without a workspace or a second launch.
//
// Top alternatives: each warp keeps its best 32 as sorted keys (order of the logit,
// then lower id: all distinct), one per lane. A chunk is looked through only if its
// maximum, which the sum needs anyway, reaches the k-th best so far of any warp of
// the CTA; at first a bound from the lanes' maxima of the first chunks stands in for
// that. Ruled out tokens (-inf) never enter; a row with fewer than k others is
// filled up at the end. The rank likewise counts only in chunks whose maximum
// reaches the token's logit.
//
// Measured, back to back in a graph: a row of 32,000 fp32 logits 7.2 us (latency: first
// loads, joins); 64 rows of 50,257, nine tenths ruled out, 20 alternatives, 17.1 us (five
// alternatives 13.7, none 8.6; nothing ruled out 16.2; without tokens 16.0); 2,048
// rows of 131,072 bf16, one alternative, 109 us for 537 MB (4.9 TB/s, 0.73 of a copy's
// rate). What binds there is the way through a chunk (maximum, vote, sums) and the
// ends of rows, not the copies: three or four chunks under way take as long, chunks of 16,
// 32, 48, 80 and 96 bytes a lane 157, 123, 115, 108 and 109 us (the larger ones cost the
// short calls), five and six CTAs per SM 112 and 117. Chunks in registers, which
// spilled, took 126; two CTAs a row then 146, CTAs of 512 threads 137.
#include "block_internal.h"
#include "kv_common.cuh"
#include "packed.cuh"

namespace moe {
namespace block {

namespace {

typedef unsigned long long Key;

constexpr int kThreads = 256;
constexpr int kWarpsPerCta = kThreads / 32;
constexpr int kVecs = 4;  // 16-byte pieces of a lane's chunk
constexpr int kStages = 2;  // chunks of a warp: one is worked on, the others under way
constexpr int kMostParts = 8;  // CTAs of a row
static_assert(kWarpsPerCta >= kMostParts, "a warp fetches each part's result, and they meet in the warps' places");

// Over some values with the maximum m: one value of m is left out of l (and its share of
// s is 0), so that ln(1 + l) is right where the maximum is nearly all.
struct Part {
  float m, l, s;
  int rank;
};
struct Shared {
  Part part[kWarpsPerCta];
  Key key[kWarpsPerCta][32];
  float mth[kWarpsPerCta];
  float floor;  // some warp's k-th best logit: no smaller one is among the k best
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_max_nan(float x) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
// NaN becomes -200
__device__ __forceinline__ float bounded(float d) { return fmaxf(d, -200.f); }

__device__ __forceinline__ void join(Part& a, const Part& b, float c) {
  const float m = max_nan(a.m, b.m);
  const float da = bounded((a.m - m) * c), db = bounded((b.m - m) * c);
  const float ea = kv::ex2(da), eb = kv::ex2(db);
  const bool first = a.m >= b.m;  // whose value is left out; the other's joins
  const float e = first ? eb : ea, d = first ? db : da;
  a.s = ea * (a.s + a.l * da) + eb * (b.s + b.l * db) + e * d;
  a.l = ea * a.l + eb * b.l + e;
  a.m = m;
  a.rank += b.rank;
}

__device__ __forceinline__ Key shfl_key(Key k, int src) { return __shfl_sync(0xffffffffu, k, src); }

// The 32 best of two sorted lists (lane i holds the i-th best of each).
__device__ __forceinline__ Key merge32(Key a, Key b) {
  const int lane = threadIdx.x & 31;
  b = shfl_key(b, 31 - lane);
  a = a > b ? a : b;  // the 32 best, bitonic
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Key x = __shfl_xor_sync(0xffffffffu, a, o);
    const bool upper = lane & o;
    a = (a > x) == !upper ? a : x;
  }
  return a;
}

// The lists and sums of the CTA's warps [0, n) (n a power of two) meet in warp 0.
__device__ void join_warps(Shared& sh, int n, bool top, float c) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  for (int h = n >> 1; h > 0; h >>= 1) {
    if (warp < h) {
      if (lane == 0) join(sh.part[warp], sh.part[warp + h], c);
      if (top) sh.key[warp][lane] = merge32(sh.key[warp][lane], sh.key[warp + h][lane]);
    }
    __syncthreads();
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// An address of this CTA's shared memory, in the CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t peer_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ Key peer_u64(uint32_t a) {
  Key v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
template <int N>
__device__ __forceinline__ void copies_but() {  // all but the last N groups are there
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// How a type's values lie in the 32-bit words of a piece.
template <int TYPE>
struct Words {
  static constexpr bool kWide = TYPE == MOE_T_F32, kHalf = TYPE == MOE_T_F16;
  static constexpr int kSize = kWide ? 4 : 2, kPer = 16 / kSize;  // values per piece
  static constexpr uint32_t kNone = kWide ? 0xff800000u : kHalf ? 0xfc00fc00u : 0xff80ff80u;  // -inf
  // where the fast sums count everything lower as this much
  static constexpr uint32_t kLowBits = kWide ? 0xf147edcdu : kHalf ? 0xfbfffbffu : 0xf149f149u;
  static constexpr float kLow = kHalf ? -65504.f : -9.9e29f;  // (that or lower)
  __device__ static float at(const uint4& v, int e) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (kWide) return __uint_as_float(w[e]);
    const float2 f = kv::unpack2<kHalf>(w[e >> 1]);
    return e & 1 ? f.y : f.x;
  }
  __device__ static __half2 half2_of(uint32_t a) { return *reinterpret_cast<__half2*>(&a); }
  __device__ static __nv_bfloat162 bf162_of(uint32_t a) { return *reinterpret_cast<__nv_bfloat162*>(&a); }
  template <typename T2>
  __device__ static uint32_t word(T2 a) { return *reinterpret_cast<const uint32_t*>(&a); }
  // the larger, NaN if one is NaN
  __device__ static uint32_t max_word(uint32_t a, uint32_t b) {
    if constexpr (kWide) return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
    if constexpr (kHalf) return word(__hmax2_nan(half2_of(a), half2_of(b)));
    return word(__hmax2_nan(bf162_of(a), bf162_of(b)));
  }
  // the bits of a value of w that is m; 0: none
  __device__ static uint32_t half_at(uint32_t w, float m) {
    if constexpr (kWide) return __uint_as_float(w) == m ? ~0u : 0u;
    const float2 f = kv::unpack2<kHalf>(w);
    return f.x == m ? 0xffffu : f.y == m ? 0xffff0000u : 0u;
  }
  // per 16-bit value: the sum; 1 where a >= b or a > b, else 0 (and with a NaN)
  __device__ static uint32_t add_word(uint32_t a, uint32_t b) {
    if constexpr (kHalf) return word(__hadd2(half2_of(a), half2_of(b)));
    return word(__hadd2(bf162_of(a), bf162_of(b)));
  }
  __device__ static uint32_t ge_word(uint32_t a, uint32_t b) {
    if constexpr (kHalf) return word(__hge2(half2_of(a), half2_of(b)));
    return word(__hge2(bf162_of(a), bf162_of(b)));
  }
  __device__ static uint32_t gt_word(uint32_t a, uint32_t b) {
    if constexpr (kHalf) return word(__hgt2(half2_of(a), half2_of(b)));
    return word(__hgt2(bf162_of(a), bf162_of(b)));
  }
  __device__ static float max_of(uint32_t w) {
    if constexpr (kWide) return __uint_as_float(w);
    const float2 f = kv::unpack2<kHalf>(w);
    return max_nan(f.x, f.y);
  }
};

// The row's values as the kernel reads them.
template <int TYPE>
struct Row {
  using W = Words<TYPE>;
  const char* row;
  const char* base;  // the 16-byte boundary at or before the row
  int V, lead, n_vec;
  __device__ Row(const moe_logprobs_args& a, int t) {
    row = static_cast<const char*>(a.logits) + (long long)t * a.stride * W::kSize;
    V = a.V;
    lead = (int)(reinterpret_cast<uintptr_t>(row) & 15) / W::kSize;
    base = row - lead * W::kSize;
    n_vec = (lead + V + W::kPer - 1) / W::kPer;
  }
  __device__ uint32_t bits(int id) const {
    return W::kWide ? *reinterpret_cast<const uint32_t*>(row + (long long)id * 4) : *reinterpret_cast<const uint16_t*>(row + (long long)id * 2);
  }
  __device__ float one(int id) const {
    return W::kWide ? __uint_as_float(bits(id)) : kv::unpack2<W::kHalf>(bits(id)).x;
  }
  __device__ int id_of(int j, int e) const { return j * W::kPer + e - lead; }
  // Piece j: whole ones at once; the first and the last, and what lies behind, with
  // -inf in the other places.
  __device__ uint4 piece(int j) const {
    uint4 v = make_uint4(W::kNone, W::kNone, W::kNone, W::kNone);
    if (j * W::kPer >= lead && (j + 1) * W::kPer <= lead + V) {
      v = __ldcs(reinterpret_cast<const uint4*>(base + (long long)j * 16));
    } else if (j < n_vec) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = W::kNone;
        if constexpr (W::kWide) {
          if ((unsigned)id_of(j, i) < (unsigned)V) w[i] = bits(id_of(j, i));
        } else {
          if ((unsigned)id_of(j, 2 * i) < (unsigned)V) w[i] = (w[i] & 0xffff0000u) | bits(id_of(j, 2 * i));
          if ((unsigned)id_of(j, 2 * i + 1) < (unsigned)V) w[i] = (w[i] & 0xffffu) | bits(id_of(j, 2 * i + 1)) << 16;
        }
      }
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
  }
};

// The lanes' values (none is NaN) in descending order.
__device__ __forceinline__ float sorted_lanes(float x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 2; w <= 32; w <<= 1)
#pragma unroll
    for (int o = w >> 1; o > 0; o >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, x, o);
      const bool larger = ((lane & w) == 0) == ((lane & o) == 0);
      x = larger ? fmaxf(x, y) : fminf(x, y);
    }
  return x;
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const __grid_constant__ moe_logprobs_args a, int parts) {
  using W = Words<TYPE>;
  constexpr int E = W::kPer;
  __shared__ Shared sh;
  __shared__ uint4 ring[kStages * kWarpsPerCta * kVecs * 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x / parts, rank = parts > 1 ? (int)cluster_rank() : 0;
  const Row<TYPE> row(a, t);
  const float kNone = -__int_as_float(0x7f800000), kBig = __int_as_float(0x7f800000);
  const int step = parts * kWarpsPerCta * 32 * kVecs;
  int v0 = (rank * kWarpsPerCta + warp) * 32 * kVecs;
  // chunks that hold whole pieces only
  const int whole0 = row.lead ? 1 : 0, whole1 = (row.lead + a.V) / E;
  // Chunk v on its way into a stage, where a lane finds the pieces that it has fetched
  // itself (no other reads them, so its own waits are all there is).
  const auto place = [&](int stage) { return ring + (stage * kWarpsPerCta + warp) * kVecs * 32 + lane; };
  const auto fetch = [&](int stage, int v) {
    uint4* to = place(stage);
    if (v >= whole0 && v + 32 * kVecs <= whole1) {
      const uint4* from = reinterpret_cast<const uint4*>(row.base) + v + lane;
#pragma unroll
      for (int u = 0; u < kVecs; ++u) copy16(to + u * 32, from + u * 32);
    } else if (v < row.n_vec) {
#pragma unroll
      for (int u = 0; u < kVecs; ++u) to[u * 32] = row.piece(v + u * 32 + lane);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i, v0 + i * step);
  const float c = 1.4426950408889634f / a.temperature;
  const int token = a.tokens ? a.tokens[t] : -1;
  const bool has = token >= 0 && token < a.V;
  const float mine_raw = has ? row.one(token) : 0.f;
  // what the rank counts from: with no token, nothing; NaN stands with -inf
  const float mine = !has ? kBig : mine_raw == mine_raw ? mine_raw : kNone;
  // a logit above this one is at or above `mine` (for ids before the token's)
  const float below = mine == 0.f ? -1e-45f : __int_as_float(__float_as_int(mine) + (mine > 0.f ? -1 : 1));
  const auto largest = [&](const uint4* at) {
    uint32_t mw = W::kNone;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const uint4 v = at[u * 32];
      mw = W::max_word(W::max_word(mw, W::max_word(v.x, v.y)), W::max_word(v.z, v.w));
    }
    return W::max_of(mw);
  };
  // What the k best are not below, from the first chunks: the k-th largest of the
  // warp's lane maxima; and with m = k / warps (rounded up) the smallest of the warps'
  // m-th largest, since m of each are not below it.
  float floor = kNone;
  if (a.top) {
    const int warps = min(max((row.n_vec - rank * kWarpsPerCta * 32 * kVecs + 32 * kVecs - 1) / (32 * kVecs), 0), kWarpsPerCta);
    if (warp < warps) {
      copies_but<kStages - 2>();
      const float mx = largest(place(0)), x = sorted_lanes(mx == mx ? mx : kNone);
      floor = __shfl_sync(0xffffffffu, x, a.top - 1);
      if (lane == (a.top + warps - 1) / warps - 1) sh.mth[warp] = x;
    }
    __syncthreads();
    float low = kBig;
    for (int w = 0; w < warps; ++w) low = fminf(low, sh.mth[w]);
    if (warps) floor = fmaxf(floor, low);
    if (tid == 0) sh.floor = floor;
    __syncthreads();
  }

  float m = kNone;  // the warp's
  float2 l2 = make_float2(0.f, 0.f), s2 = l2;  // the lane's, but for one value of m
  int count = 0;
  Key best = 0;
  const uint32_t mine_word = has && !W::kWide ? row.bits(token) * 0x10001u : 0;
  // (Each pass over a chunk reads it from shared memory again: held in registers, it could
  // not be as large.)
  const auto chunk = [&](uint4* at, int v0) {
    const float mx = largest(at), top = warp_max_nan(mx);
    if (top == kNone && mine != kNone) return;  // nothing in it
    const bool rose = top > m || top != top;
    bool out = false;  // whether the lane leaves one of its values out
    if (rose) {
      const float up = max_nan(m, top), d = bounded((m - up) * c), e = kv::ex2(d);
      s2 = fma2(l2, make_float2(d, d), s2);
      s2.x *= e; s2.y *= e;
      l2.x *= e; l2.y *= e;
      if (lane == 0) {  // the value that had been left out
        l2.x += e;
        s2.x = fmaf(e, d, s2.x);
      }
      m = up;
      out = lane == __ffs(__ballot_sync(0xffffffffu, mx == top)) - 1;
    }
    asm volatile("" ::: "memory");
    if (m < 1e29f && (m - W::kLow) * c > 200.f && c < 1e6f) {  // (the products stay finite)
      // The value that is left out gives way to one that adds nothing, for the time of the sums.
      uint32_t *gone = nullptr, was = 0;
      if (out) {
#pragma unroll 1
        for (int u = 0; u < kVecs && !gone; ++u) {
          const uint4 v = at[u * 32];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t half = W::half_at(w[i], m);
            if (!gone && half) {
              gone = reinterpret_cast<uint32_t*>(at + u * 32) + i;
              was = w[i];
              *gone = (was & ~half) | (W::kLowBits & half);
            }
          }
        }
      }
      const float2 c2 = make_float2(c, c), m2 = make_float2(-m, -m);
      float2 l = make_float2(0.f, 0.f), s = l;
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        const uint4 v = at[u * 32];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          float2 f;
          if constexpr (W::kWide)
            f = make_float2(fmaxf(__uint_as_float(w[2 * i]), W::kLow), fmaxf(__uint_as_float(w[2 * i + 1]), W::kLow));
          else
            f = kv::unpack2<W::kHalf>(W::max_word(w[i], W::kLowBits));
          const float2 d = mul2(add2(f, m2), c2), e = make_float2(kv::ex2(d.x), kv::ex2(d.y));
          l = add2(l, e);
          s = fma2(e, d, s);
        }
      }
      l2 = add2(l2, l);
      s2 = add2(s2, s);
      if (gone) *gone = was;
    } else {
#pragma unroll 1
      for (int u = 0; u < kVecs; ++u) {
        const uint4 v = at[u * 32];
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float x = W::at(v, i), d = bounded((x - m) * c), e = kv::ex2(d);
          if (out && x == m) {
            out = false;
          } else {
            l2.x += e;
            s2.x = fmaf(e, d, s2.x);
          }
        }
      }
    }
    if (!(mx < mine)) {
      const bool before = row.id_of(v0 + 32 * kVecs, 0) <= token, after = row.id_of(v0, 0) > token;
      if (!W::kWide && mine != kNone && (before || after)) {
        // two at a time: ones, summed up in the type (16 at most)
        uint32_t n = 0;
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
          const uint4 v = at[u * 32];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) n = W::add_word(n, before ? W::ge_word(w[i], mine_word) : W::gt_word(w[i], mine_word));
        }
        const float2 two = kv::unpack2<W::kHalf>(n);
        count += (int)(two.x + two.y);
      } else if (mine != kNone) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {  // (those beside the token in its piece: below)
          const uint4 v = at[u * 32];
          const float limit = row.id_of(v0 + u * 32 + lane, E - 1) < token ? below : mine;
#pragma unroll
          for (int i = 0; i < E; ++i) count += W::at(v, i) > limit ? 1 : 0;
        }
      } else {
#pragma unroll 1
        for (int u = 0; u < kVecs; ++u) {
          const uint4 v = at[u * 32];
#pragma unroll
          for (int i = 0; i < E; ++i)
            count += W::at(v, i) > kNone || (unsigned)row.id_of(v0 + u * 32 + lane, i) < (unsigned)token ? 1 : 0;
        }
      }
    }
    if (a.top) {
      floor = fmaxf(floor, *const_cast<volatile float*>(&sh.floor));
      const float reach = mx == mx ? mx : kBig;  // a lane with a NaN is looked through
      if (top != top || top >= floor) {
        if (__any_sync(0xffffffffu, reach >= floor)) {
#pragma unroll
          for (int u = 0; u < kVecs; ++u) {
            const uint4 v = at[u * 32];
            uint32_t mask = 0;  // of this lane's values
#pragma unroll
            for (int i = 0; i < E; ++i) mask |= W::at(v, i) >= floor && W::at(v, i) > kNone ? 1u << i : 0u;
            unsigned todo = __ballot_sync(0xffffffffu, mask != 0);
            while (todo) {
              const int src = __ffs(todo) - 1, e = __ffs(mask) - 1;
              const uint32_t w = (e >> (W::kWide ? 0 : 1)) == 0 ? v.x : (e >> (W::kWide ? 0 : 1)) == 1 ? v.y
                                 : (e >> (W::kWide ? 0 : 1)) == 2 ? v.z : v.w;
              const float x = W::kWide ? __uint_as_float(w) : (e & 1 ? kv::unpack2<W::kHalf>(w).y : kv::unpack2<W::kHalf>(w).x);
              const Key k = shfl_key((Key)order_key(x) << 32 | (uint32_t)~row.id_of(v0 + u * 32 + lane, e), src);
              if (lane == src) mask &= mask - 1;
              todo = __ballot_sync(0xffffffffu, mask != 0);
              const int at = __popc(__ballot_sync(0xffffffffu, best > k));  // its place in the list
              if (at < a.top) {
                const Key up = __shfl_up_sync(0xffffffffu, best, 1);
                best = lane < at ? best : lane == at ? k : up;
                const Key last = shfl_key(best, a.top - 1);
                if (last) floor = fmaxf(floor, key_value((uint32_t)(last >> 32)));
              }
            }
          }
          if (lane == 0 && floor > *const_cast<volatile float*>(&sh.floor)) *const_cast<volatile float*>(&sh.floor) = floor;
        }
      }
    }
  };
  for (int stage = 0; v0 < row.n_vec; v0 += step) {
    copies_but<kStages - 2>();
    // into the stage that was worked on last
    fetch(stage == 0 ? kStages - 1 : stage - 1, v0 + (kStages - 1) * step);
    chunk(place(stage), v0);
    stage = stage == kStages - 1 ? 0 : stage + 1;
  }
  // equal logits before the token in its own piece
  if (rank == 0 && warp == 0 && has && mine != kNone) {
    const int id = token - 1 - lane;
    if (lane < (token + row.lead) % E && id >= 0) count += row.one(id) == mine ? 1 : 0;
  }
  Part p = {m, l2.x + l2.y, s2.x + s2.y, count};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {  // (one maximum for the warp)
    p.l += __shfl_xor_sync(0xffffffffu, p.l, o);
    p.s += __shfl_xor_sync(0xffffffffu, p.s, o);
  }
  p.rank = __reduce_add_sync(0xffffffffu, p.rank);
  if (lane == 0) sh.part[warp] = p;
  sh.key[warp][lane] = best;
  join_warps(sh, kWarpsPerCta, a.top > 0, c);
  if (parts > 1) {
    cluster_sync();
    if (rank == 0) {  // warp w fetches part w's result; its own stays
      Part q = {kNone, 0.f, 0.f, 0};
      Key k = 0;
      if (warp > 0 && warp < parts) {
        const uint32_t ps = peer(&sh.part[0], warp);
        q = {__uint_as_float(peer_u32(ps)), __uint_as_float(peer_u32(ps + 4)), __uint_as_float(peer_u32(ps + 8)), (int)peer_u32(ps + 12)};
        k = peer_u64(peer(&sh.key[0][lane], warp));
      }
      __syncthreads();
      if (warp > 0 && warp < parts) {
        if (lane == 0) sh.part[warp] = q;
        sh.key[warp][lane] = k;
      }
      join_warps(sh, parts, a.top > 0, c);
    }
    cluster_sync();  // the peers' shared memory has been read
    if (rank != 0) return;
  }
  if (warp != 0) return;
  p = sh.part[0];
  const float nan = __int_as_float(0x7fffffff);
  const bool broken = !(p.m < __int_as_float(0x7f800000)), empty = p.m == kNone;
  const float ln_l = log1pf(p.l);
  const auto log_p = [&](float z) { return broken ? nan : empty ? kNone : (z - p.m) / a.temperature - ln_l; };
  if (lane == 0) {
    if (a.logprob) a.logprob[t] = has ? log_p(mine_raw) : 0.f;
    if (a.rank) a.rank[t] = has ? p.rank : -1;
    if (a.entropy) a.entropy[t] = broken ? nan : empty ? 0.f : fmaxf(ln_l - 0.6931471805599453f * (p.s / (1.f + p.l)), 0.f);
  }
  if (a.top) {
    Key k = sh.key[0][lane];
    const int got = __popc(__ballot_sync(0xffffffffu, k != 0));
    if (got < a.top) {  // fewer than that are not ruled out: the lowest ids of those that are
      int place = got;
      for (int id0 = 0; id0 < a.V && place < a.top; id0 += 32) {
        const int id = id0 + lane;
        const float z = id < a.V ? row.one(id) : 0.f;
        const unsigned out = __ballot_sync(0xffffffffu, z == kNone || z != z);
        const int n = lane - place;  // this lane's place is the n-th of them
        if (n >= 0 && n < __popc(out)) {
          const int src = __fns(out, 0, n + 1);
          k = (Key)order_key(kNone) << 32 | (uint32_t)~(id0 + src);
        }
        place += __popc(out);
      }
    }
    if (lane >= a.top) return;
    a.top_ids[(long long)t * a.top + lane] = (int)~(uint32_t)k;
    a.top_logprobs[(long long)t * a.top + lane] = log_p(key_value((uint32_t)(k >> 32)));
  }
}

template <int TYPE>
cudaError_t launch_type(const moe_logprobs_args& a, int parts, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.T * parts);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = parts;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  launch_begin(K_LOGPROBS, st);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, logprobs_kernel<TYPE>, moe_logprobs_args(a), int(parts));
  launch_end(st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_token_logprobs(const moe_logprobs_args& a, cudaStream_t st) {
  // CTAs per row: while all fit on the GPU (four per SM, 608) and a part is more than a
  // chunk for each warp. (2,048 rows of 131,072 by two CTAs each, when one took 126 us: 146;
  // the last third of them by two, in a launch of its own: no change.)
  int parts = 1;
  const long long chunk = (long long)kThreads * kVecs * (a.type == MOE_T_F32 ? 4 : 8);
  while (parts < kMostParts && (long long)a.T * parts * 2 <= 608 && a.V > chunk * parts) parts *= 2;
  if (a.type == MOE_T_F32) return launch_type<MOE_T_F32>(a, parts, st);
  return a.type == MOE_T_F16 ? launch_type<MOE_T_F16>(a, parts, st) : launch_type<MOE_T_BF16>(a, parts, st);
}

}  // namespace block
}  // namespace moe
