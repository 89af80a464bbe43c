// Attention of a decode window over the paged cache: one launch, bound by the
// HBM read of the visible keys and values.
//
// Items and spans. An item is (sequence, tile of 16 query rows, KV head): the
// rows are the window's new tokens times the query heads of the KV head, and
// the item's keys and values are read once for all of them. An item's visible
// tiles (first tokens that stay visible, then the window) are cut into spans
// (span_log). Every span is computed by itself and the spans are folded in
// order,
//   M' = max(M, m),  L' = L 2^(M - M') + l 2^(m - M'),  O' = O 2^(M - M') + o 2^(m - M'),
// so a row's result depends on its own sequence only, not on the other
// sequences nor on how the spans fall on the CTAs.
//
// CTAs. A producer warp and, for each 8 query rows of a tile, a group of four
// consumer warps around a ring of tiles (K and V of 64 or 128 tokens, TMA boxes
// of a page's rows, 128-byte swizzle): items of up to 8 rows run two CTAs per SM
// with 96 KB of tiles each, items of 16 rows one CTA with 192 KB. The list of
// all items' tiles is divided evenly; a CTA takes the spans that start in its
// part. It folds consecutive spans of an item in registers; an item that lies
// in several CTAs is joined, through partials in the workspace, by the CTA that
// finishes last. (Three CTAs per SM with 64 KB each: a window of 1,024 tokens
// 17.9 us instead of 20.7, but the long cases lose, 64 conversations 210 us
// instead of 202, 131,057 tokens 98 instead of 93.)
//
// A tile. A warp has a quarter of its keys, in blocks of 16, to itself: S^T =
// K Q^T (mma m16n8k16 with its group's 8 query rows as N, so no half of the
// product is padding), the softmax of its 16 x 8 scores in registers, P^T turned
// into the B operand by movmatrix, O^T += V^T P^T over all of D. The warps meet
// only at a span's end, where their (m, l, o) are added up through shared memory
// in warp order. (With the keys shared by all warps, which exchange maxima and
// probabilities per tile: 64 conversations 224 us instead of 208.) A probability
// enters the product with V as a sum of two values of the cache's type (rounding
// 2^-17 for bf16 instead of 2^-8; the second product costs nothing next to the
// HBM read). fp16 has a fixed step below 2^-14, where the second value is lost too:
// its probabilities are lifted by 2^7 (to 2^15 at most), so that half of that step
// is 2^-32 of the largest one. The running maximum is raised only by more than 2^8 (sums are in
// fp32), so O is seldom rescaled. Keys that only some rows see are added with
// scalar products, keys that no row sees get a zero value row: nothing that lies
// in a masked place reaches a result, NaN and infinities included.
//
// Measured (head size 128, bf16, append included; of 6.78 TB/s copied): 64
// conversations of up to 8,191 tokens, 32 / 8 heads: 199 us, 6.2 TB/s (0.92);
// one of 131,057 tokens: 90 us, 5.9 TB/s (0.87). Short calls are a chain of
// latencies (division of the list, page table, first tile, the joins): 517
// tokens 9.7 us, 8 sequences of up to 4,093 tokens 17 us.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "kv_common.cuh"
#include "kv_tma.h"

namespace moe {
namespace kv {

namespace {

// Tokens of a tile for RG groups of rows: a warp has 16 or 32 keys of it. With 32
// its chain of products and reductions is paid half as often (what one CTA per
// SM, or 16 KB of keys and values per 64 tokens, needs to keep up with the HBM).
__host__ __device__ constexpr int tile_of(int D, int RG) { return D == 128 && RG == 1 ? 64 : 128; }
// RG groups of four consumer warps and the producer.
template <int RG>
__host__ __device__ constexpr int dec_threads() { return 32 * (4 * RG + 1); }
template <int RG>
__host__ __device__ constexpr int dec_ring() { return RG * 96 * 1024; }
template <int RG>
__host__ __device__ constexpr int dec_ctas() { return 3 - RG; }  // per SM
constexpr int kAllBar = 3;              // named barrier of all consumer warps (1, 2: a group's)
constexpr int kOPitch = 64 + 4;         // floats per row of the buffer in which the warps' O meet
constexpr uint32_t kTries = 1u << 24;   // of a wait, up to 128 ns long each
constexpr int kSeqCap = 128;            // sequences per launch
constexpr int kCntBase = 2048;          // this kernel's counters in the workspace head

struct DecArgs {
  CUtensorMap tm_k, tm_v;
  Cache c;
  Rows r;
  Attn a;
  int b0;             // first sequence of this launch; r.B the sequences in it
  int RT;             // row tiles per sequence
  int logP;           // log2 of a box's rows: min(page, tile)
  int logpage;
  int max_span;       // spans of an item at most
  int span_c, most_spans;  // the rule for their length
  float* part;        // [keys][max_span][RG] partials
  int32_t *status, *cnt;
};

// log2 of a span's tiles, by the item's own length and the call's heads: the
// smallest k with at most c 2^k spans (their number and their length both grow
// as the square root of the length) and at most most_spans.
__host__ __device__ inline int span_log(int nvis, int c, int most_spans) {
  int k = 0;
  while (nvis > ((long long)c << (2 * k)) || nvis > ((long long)most_spans << k)) ++k;
  return k;
}

// (m, l, o) of a span folded into (M, L, O): written with explicit rounding so
// that the fold in registers and the join give the same bits.
__device__ __forceinline__ void fold_ml(float& M, float& L, float m, float l, float& a, float& b) {
  const float n = fmaxf(M, m), z = n == -INFINITY ? 0.f : n;
  a = ex2(M - z);
  b = ex2(m - z);
  L = __fmaf_rn(l, b, __fmul_rn(L, a));
  M = n;
}
__device__ __forceinline__ float fold_o(float O, float o, float a, float b) { return __fmaf_rn(o, b, __fmul_rn(O, a)); }

__device__ __forceinline__ float4 fold_o4(const float4& O, const float4& o, float a, float b) {
  return make_float4(fold_o(O.x, o.x, a, b), fold_o(O.y, o.y, a, b), fold_o(O.z, o.z, a, b), fold_o(O.w, o.w, a, b));
}

// One item as every role sees it.
struct Item {
  int slot, len;
  int pf, pl;        // tokens of its first and last row (pl < 0: nothing is seen)
  int ns, wt, nvis;  // tiles of first tokens, first window tile, visible tiles
  int ks, nspan;     // spans of 2^ks tiles
  __device__ int tile(int v) const { return v < ns ? v : v - ns + wt; }
};

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (F16) mma_f16_16816(d, a0, a1, a2, a3, b0, b1);
  else mma_bf16_16816(d, a0, a1, a2, a3, b0, b1);
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

template <bool F16>
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : (m + (log2f(l) - lift<F16>())) * 0.6931471805599453f;
}

// A row's result: columns 64 h .. + 3 of o.
template <bool F16, int D>
__device__ __forceinline__ void put_row(float m, float l, const float4 (&O)[D / 64], uint16_t* o, float* lse) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int h = 0; h < D / 64; ++h)
    *reinterpret_cast<uint2*>(o + 64 * h) =
        make_uint2(pack2<F16>(O[h].x * inv, O[h].y * inv), pack2<F16>(O[h].z * inv, O[h].w * inv));
  if (lse) *lse = lse_of<F16>(m, l);
}

// A split item whose spans are all there.
struct Join {
  int b, rt, hk, n;   // n partials
  const float* p;
};

// A group's part of a span's partial: m and l of its 8 rows, o [8][D].
template <int D>
__host__ __device__ constexpr int part_floats() { return 16 + 8 * D; }

// The fold of n partials of a group's rows (from p on, pstride floats apart) in
// order, for row `row` and the columns col + 64 h .. + 3, by the group's 128
// threads. The partials come through shared memory (BUF bytes from buf), U at a
// time while U are folded: a join reads some 100 KB that other SMs wrote, and
// what it waits for is the latency of those reads.
template <bool F16, int D, int BUF>
__device__ __forceinline__ void join_rows(const float* p, long long pstride, int n, uint32_t buf, int bar_id, int row, int col,
                                          uint16_t* o, float* lse) {
  constexpr int NH = D / 64, kVecs = part_floats<D>() / 4, kBytes = part_floats<D>() * 4;
  constexpr int kFit = BUF / (2 * kBytes), U = kFit < 8 ? kFit : 8;
  static_assert(U >= 4);
  const int t = threadIdx.x & 127;
  auto fetch = [&](int s0) {  // partials s0 .. s0 + U - 1 into their half of the buffer
    for (int u = 0; u < U && s0 + u < n; ++u) {
      const float* q = p + (s0 + u) * pstride;
      const uint32_t d = buf + ((s0 / U & 1) * U + u) * kBytes;
      for (int i = t; i < kVecs; i += 128)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + 16 * i), "l"(q + 4 * i) : "memory");
    }
    cp_async_commit();
  };
  float M = -INFINITY, L = 0.f;
  float4 O[NH];
#pragma unroll
  for (int h = 0; h < NH; ++h) O[h] = make_float4(0.f, 0.f, 0.f, 0.f);
  fetch(0);
  for (int s0 = 0; s0 < n; s0 += U) {
    fetch(s0 + U);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    named_bar_sync(bar_id, 128);
    // past the last partial: m = -inf and zeros, which the fold leaves as it is
    float m[U], l[U];
    float4 w[U][NH];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t d = buf + ((s0 / U & 1) * U + u) * kBytes;
      const bool in = s0 + u < n;
      m[u] = in ? __uint_as_float(ld_s32(d + row * 4)) : -INFINITY;
      l[u] = in ? __uint_as_float(ld_s32(d + 32 + row * 4)) : 0.f;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const uint4 v = ld_s128(d + 64 + (row * D + col + 64 * h) * 4);
        w[u][h] = in ? make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w))
                     : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float a, b;
      fold_ml(M, L, m[u], l[u], a, b);
#pragma unroll
      for (int h = 0; h < NH; ++h) O[h] = fold_o4(O[h], w[u][h], a, b);
    }
    named_bar_sync(bar_id, 128);  // before this half is filled again
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (o) put_row<F16, D>(M, L, O, o + col, lse);
}

template <bool F16, int D, int RG>
__global__ void __launch_bounds__(dec_threads<RG>(), dec_ctas<RG>()) decode_kernel(const __grid_constant__ DecArgs g) {
  constexpr int kDecThreads = dec_threads<RG>();
  constexpr int kTile = tile_of(D, RG), KB = kTile / 64;  // KB blocks of 16 keys per warp
  constexpr int kStage = kTile * D * 4;      // K and V of a tile
  constexpr int kStages = dec_ring<RG>() / kStage;
  constexpr int KK = D / 16, NH = D / 64;
  extern __shared__ __align__(1024) uint8_t smem_dec[];
  __shared__ __align__(8) uint64_t s_bar[2 * kStages + 4];
  __shared__ uint32_t s_badbox[kStages];
  __shared__ int s_off[kSeqCap + 1], s_len[kSeqCap], s_slot[kSeqCap];
  __shared__ __align__(16) float s_o[RG][4][8][kOPitch];  // the warps' O: 8 rows, 64 columns at a time
  __shared__ float s_ml[RG][2][4][8];                     // the warps' maxima and sums
  __shared__ int s_scan[4 * RG + 1];
  __shared__ Join s_join[RG][2];  // split items that this CTA completes: its first and its last at most
  __shared__ int s_njoin[RG];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = g.r.B, G = g.a.G, n_q = g.r.n_q, W = g.a.window, S = g.a.n_sink, Hkv = g.c.Hkv;
  const uint32_t ring = smem_u32(smem_dec);  // aligned as declared: a swizzled box starts on 1 KB
  const uint32_t full = smem_u32(s_bar), empty = full + 8 * kStages;
  const uint32_t pair = empty + 8 * kStages;  // [4]: the warps of two groups with the same keys
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 4 * RG);
    }
    for (int i = 0; i < 4; ++i) mbar_init(pair + 8 * i, 2);
    fence_barrier_init();
    for (int i = 0; i < RG; ++i) s_njoin[i] = 0;
  }
  griddep_wait();  // the rows' keys and values of an append before this launch
  griddep_launch_dependents();

  auto item_of = [&](int slot, int len, int rt) {
    Item it;
    it.slot = slot;
    it.len = len;
    const int r1 = min(n_q * G, rt * 16 + 16);
    it.pf = len - n_q + (rt ? rt * 16 / G : 0);
    it.pl = slot < 0 ? -1 : len - n_q + (r1 == n_q * G ? n_q - 1 : (r1 - 1) / G);
    it.ns = it.wt = it.nvis = 0;
    if (it.pl >= 0) {
      const int from = W > 0 ? max(0, max(0, it.pf) - W + 1) : 0;
      it.ns = (min(S, from) + kTile - 1) / kTile;
      it.wt = max(from / kTile, it.ns);
      it.nvis = it.ns + it.pl / kTile - it.wt + 1;
    }
    it.ks = span_log(it.nvis, g.span_c, g.most_spans);
    it.nspan = max(1, (it.nvis + (1 << it.ks) - 1) >> it.ks);
    return it;
  };

  // the sequences' lengths and where their tiles start in the list of all tiles
  int base = 0;
  for (int b0 = 0; b0 < B; b0 += kDecThreads) {
    const int b = b0 + tid;
    int w = 0;
    if (b < B) {
      const Seq s = load_seq(g.c, g.r, b, g.status);
      s_len[b] = s.len;
      s_slot[b] = s.slot;
      for (int rt = 0; rt < g.RT; ++rt) w += max(1, item_of(s.slot, s.len, rt).nvis);
      w *= Hkv;
    }
    int x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < kDecThreads / 32; ++i) {
      before += i < warp ? s_scan[i] : 0;
      sum += s_scan[i];
    }
    if (b < B) s_off[b] = base + before + x - w;
    base += sum;
    __syncthreads();
  }
  const int total = base;
  if (tid == 0) s_off[B] = total;
  __syncthreads();

  // the list's division: CTA i takes the spans that start in [lo(i), lo(i + 1))
  const int nc = gridDim.x, tq = total / nc, tr = total - tq * nc;
  auto lo_of = [&](int i) { return i * tq + min(i, tr); };
  auto cta_of = [&](int off) { return off < tr * (tq + 1) ? off / (tq + 1) : tr + (off - tr * (tq + 1)) / tq; };
  const int lo = lo_of(blockIdx.x), hi = lo_of(blockIdx.x + 1);

  // the walk over this CTA's spans, the same in every role
  int b = 0, rt = 0, hk = 0, span = 0, ioff = 0;
  Item it;
  {
    int l = 0, h = B - 1;
    while (l < h) {
      const int m = (l + h + 1) >> 1;
      if (s_off[m] <= lo) l = m;
      else h = m - 1;
    }
    b = l;
    ioff = s_off[b];
    it = item_of(s_slot[b], s_len[b], 0);
    while (true) {
      const int w = max(1, it.nvis);
      if (lo - ioff < w * Hkv || rt + 1 == g.RT) {
        hk = min(Hkv - 1, (lo - ioff) / w);
        ioff += hk * w;
        span = (lo - ioff + (1 << it.ks) - 1) >> it.ks;
        break;
      }
      ioff += w * Hkv;
      it = item_of(s_slot[b], s_len[b], ++rt);
    }
  }
  auto next_item = [&] {  // -> false past the last item
    ioff += max(1, it.nvis);
    span = 0;
    if (++hk < Hkv) return true;
    hk = 0;
    if (++rt == g.RT) {
      rt = 0;
      if (++b == B) return false;
    }
    it = item_of(s_slot[b], s_len[b], rt);
    return true;
  };
  bool more = lo < hi;
  if (more && span >= it.nspan) more = next_item();
  // A wait on the ring, a few instructions long. After an expired one (the status
  // word says that the results are incomplete) a warp goes on without waiting,
  // so that all meet at every barrier.
  bool dead = false;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    uint32_t n = dead ? 1u : kTries;
    while (!mbar_try_wait_ns(bar, parity, 128) && --n) {
    }
    dead |= n == 0;
    __syncwarp();
  };

  if (warp == 4 * RG) {
    // ================= producer =================
    const int P = 1 << g.logP, nbox = kTile >> g.logP, box = P * D * 2;
    int st = 0, ph = 1;
    while (more && !dead && ioff + (span << it.ks) < hi) {
      const int v0 = span << it.ks, v1 = min(it.nvis, v0 + (1 << it.ks));
      const int from = W > 0 ? max(0, max(0, it.pf) - W + 1) : 0, first = min(S, from);
      const int32_t* tab = g.c.table + (long long)it.slot * g.c.max_pages;
      // page numbers of 32 boxes at a time, one per lane
      const int per = 32 / nbox;  // tiles whose boxes fill the lanes
      for (int vb = v0; vb < v1 && !dead; vb += per) {
        int row = -1;       // the box's first row in the pool; -1 not needed, -2 bad page
        {
          const int v = vb + lane / nbox;
          if (v < v1) {
            const int j = it.tile(v) * kTile + (lane & (nbox - 1)) * P;
            if (j <= it.pl && (j + P > from || j < first)) {
              const int pg = tab[j >> g.logpage];
              if (pg >= 0 && pg < g.c.n_pages) {
                row = ((pg * Hkv + hk) << g.logpage) + (j & (g.c.page - 1));
              } else {
                row = -2;
                atomicOr(g.status, DEV_BAD_SLOT);
              }
            }
          }
        }
        for (int t = 0; t < per && vb + t < v1; ++t) {
          wait(empty + 8 * st, ph);
          if ((dead = __any_sync(0xffffffffu, dead))) break;
          const int mine = __shfl_sync(0xffffffffu, row, t * nbox + (lane & (nbox - 1)));
          const unsigned load = __ballot_sync(0xffffffffu, lane < nbox && mine >= 0);
          const unsigned bad = __ballot_sync(0xffffffffu, lane < nbox && mine == -2);
          if (lane == 0) {
            s_badbox[st] = bad;
            mbar_expect_tx(full + 8 * st, 2 * __popc(load) * box);
          }
          __syncwarp();
          if (load >> lane & 1) {
            const uint32_t dst = ring + st * kStage + lane * box;
            tma_load_3d(dst, &g.tm_k, 0, mine, 0, full + 8 * st);
            tma_load_3d(dst + kStage / 2, &g.tm_v, 0, mine, 0, full + 8 * st);
          }
          if (++st == kStages) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      if (++span >= it.nspan) more = next_item();
    }
    if (dead) atomicOr(g.status, DEV_TIMEOUT);
    return;
  }

  // ================= consumers =================
  const int grp = warp >> 2, wg = warp & 3, bar_id = 1 + grp;  // the group's rows: 8 grp .. of the item
  const int P = 1 << g.logP, boxb = P * D * 2, halfb = P * 128;
  // score product: this lane's ldmatrix row of the warp's keys; value product: the same
  uint32_t koff[KB], voff[KB];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const int k0 = (wg * KB + kb) * 16, kr = k0 + (lane & 15), vr = k0 + (lane & 7) + ((lane >> 4) << 3);
    koff[kb] = (kr >> g.logP) * boxb + (kr & (P - 1)) * 128;
    voff[kb] = (vr >> g.logP) * boxb + (vr & (P - 1)) * 128;
  }
  const uint32_t kx = (uint32_t)((lane >> 4) ^ (lane & 7)) << 4, vx = (uint32_t)(((lane >> 3) & 1) ^ (lane & 7)) << 4;
  const int ra = 2 * (lane & 3);
  const int mrow = lane >> 2, mcol = wg * 16 + 4 * (lane & 3);  // merged: row mrow, columns 64 h + mcol .. + 3
  const float sc = g.a.scale * 1.4426950408889634f;
  int st = 0, ph = 0, pph = 0;

  uint32_t q[KK][2];
  int pos[2];                    // tokens of this lane's score rows ra, ra + 1 (-1: no row, or before the first token)
  float M = -INFINITY, L = 0.f;
  float4 O[NH];
  int run0 = -1;                 // first span of the current run of spans of one item

  const int items = B * Hkv * g.RT;
  // the group's partials of an item split over CTAs
  constexpr long long pstride = RG * part_floats<D>();
  auto part_of = [&](int key, int s) {
    return g.part + ((long long)key * g.max_span + s) * pstride + grp * part_floats<D>();
  };
  // an item's place among the partials
  auto key_of = [&] { return items <= nc ? (b * g.RT + rt) * Hkv + hk : cta_of(ioff); };
  auto put = [&](float* p, float m, float l, const float4 (&o)[NH]) {
    if (wg == 0 && (lane & 3) == 0) {
      p[mrow] = m;
      p[8 + mrow] = l;
    }
#pragma unroll
    for (int h = 0; h < NH; ++h) *reinterpret_cast<float4*>(p + 16 + mrow * D + 64 * h + mcol) = o[h];
  };
  // token of a sequence's row, and the row's place in a tensor [row][Hq]
  auto token_of = [&](int rr) { return n_q == 1 ? 0 : rr / G; };
  auto place_of = [&](int b, int hk, int rr) {
    const int i = token_of(rr);
    return ((long long)b * n_q + i) * g.a.Hq + hk * G + rr - i * G;
  };
  // index of the group's row r among the sequence's rows, -1 if there is none
  auto row_of = [&](int r) {
    const int rr = rt * 16 + 8 * grp + r;
    return rr < n_q * G ? rr : -1;
  };

  while (more && ioff + (span << it.ks) < hi) {
    if (run0 < 0) {  // a new item: its query rows as B operands
      run0 = span;
      const int rr = row_of(lane >> 2), qi = token_of(rr);
      const uint16_t* qp = g.a.q + ((long long)b * n_q + qi) * g.a.q_stride + (hk * G + rr - qi * G) * D + ra;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          q[kk][e] = rr >= 0 ? *reinterpret_cast<const uint32_t*>(qp + kk * 16 + e * 8) : 0u;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = row_of(ra + e);
        pos[e] = r >= 0 && it.slot >= 0 ? it.len - n_q + token_of(r) : -1;
      }
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[KK][4];
#pragma unroll
    for (int i = 0; i < KK; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    const int v1 = min(it.nvis, (span + 1) << it.ks);
    for (int v = span << it.ks; v < v1; ++v) {
      const int j0 = it.tile(v) * kTile + wg * 16 * KB;  // the warp's first key
      wait(full + 8 * st, ph);
      const uint32_t bad = *(volatile uint32_t*)&s_badbox[st];
      const uint32_t sk = ring + st * kStage, sv = sk + kStage / 2;
      // ---- scores: keys 16 kb + lane / 4, + 8; rows ra, ra + 1
      float s[KB][4];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        float x[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          uint32_t kf[4];
          ldsm4(sk + koff[kb] + (kk >> 2) * halfb + (((kk & 3) << 5) ^ kx), kf);
          mma<F16>(x[kk & 1], kf[0], kf[1], kf[2], kf[3], q[kk][0], q[kk][1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[kb][e] = (x[0][e] + x[1][e]) * sc;
      }
      const bool plain =
          bad == 0 && it.pf >= 0 && j0 + 16 * KB - 1 <= it.pf && (W == 0 || j0 > it.pl - W || j0 + 16 * KB <= S);
      if (!plain) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = 16 * kb + 8 * (e >> 1) + (lane >> 2), j = j0 + k, p = pos[e & 1];
            if (!(j <= p && (W == 0 || j > p - W || j < S)) || (bad >> ((wg * 16 * KB + k) >> g.logP) & 1))
              s[kb][e] = -INFINITY;
          }
      }
      // ---- running maximum, probabilities
      float top[2];
      bool up[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = fmaxf(s[0][e], s[0][e + 2]);
#pragma unroll
        for (int kb = 1; kb < KB; ++kb) y = fmaxf(y, fmaxf(s[kb][e], s[kb][e + 2]));
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
        top[e] = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
        up[e] = top[e] > m[e] + 8.f || (m[e] == -INFINITY && top[e] > m[e]);
      }
      if (__any_sync(0xffffffffu, up[0] || up[1])) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f[e] = up[e] ? ex2(m[e] - top[e]) : 1.f;
          m[e] = up[e] ? top[e] : m[e];
          l[e] *= f[e];
        }
#pragma unroll
        for (int i = 0; i < KK; ++i) {
          o[i][0] *= f[0];
          o[i][1] *= f[1];
          o[i][2] *= f[0];
          o[i][3] *= f[1];
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float z = m[e & 1] == -INFINITY ? 0.f : m[e & 1] - lift<F16>();
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          s[kb][e] = ex2(s[kb][e] - z);
          l[e & 1] += s[kb][e];
        }
      }
      if (!plain) {
        // which keys no row of the item sees, and which only some see (bit = key of the warp)
        const int pf = max(0, it.pf), kl = lane & (16 * KB - 1), j = j0 + kl;
        const bool good = !(bad >> ((wg * 16 * KB + kl) >> g.logP) & 1);
        const bool any = good && j <= it.pl && (W == 0 || j > pf - W || j < S);
        // (a first row before token 0 sees nothing: then no key is seen by all)
        const bool all = good && j <= it.pf && (W == 0 || j > it.pl - W || j < S);
        constexpr unsigned kKeys = KB == 2 ? 0xffffffffu : 0xffffu;
        const unsigned cut = __ballot_sync(0xffffffffu, !all) & kKeys, some = __ballot_sync(0xffffffffu, any && !all) & kKeys;
        auto vptr = [&](int k, int c) {  // address of 16 bytes: columns 8 c .. of V of the warp's key k
          const int key = wg * 16 * KB + k, r = key & (P - 1);
          return sv + (key >> g.logP) * boxb + (c >> 3) * halfb + r * 128 + ((uint32_t)((c & 7) ^ (r & 7)) << 4);
        };
        for (unsigned ms = some; ms; ms &= ms - 1) {
          const int i = __ffs(ms) - 1, jj = j0 + i, src = (i & 7) * 4 + (lane & 3);
          float pa = 0.f, pb = 0.f;
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (i >> 3 == 2 * kb + e) {
                pa = s[kb][2 * e];
                pb = s[kb][2 * e + 1];
              }
          pa = __shfl_sync(0xffffffffu, pa, src);
          pb = __shfl_sync(0xffffffffu, pb, src);
          const bool va = jj <= pos[0] && (W == 0 || jj > pos[0] - W || jj < S);
          const bool vb = jj <= pos[1] && (W == 0 || jj > pos[1] - W || jj < S);
#pragma unroll
          for (int d = 0; d < KK; ++d)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint16_t bits;
              asm volatile("ld.shared.b16 %0, [%1];" : "=h"(bits) : "r"(vptr(i, 2 * d + e) + 2 * (lane >> 2)));
              const float vv = unpack2<F16>(bits).x;
              if (va) o[d][2 * e] = fmaf(pa, vv, o[d][2 * e]);
              if (vb) o[d][2 * e + 1] = fmaf(pb, vv, o[d][2 * e + 1]);
            }
        }
        // The other group's warp of these keys has added them too. It comes here for the
        // same tiles, but after an expired wait the two may read different `bad`: so a
        // bounded wait, where a named barrier could wait for ever.
        __syncwarp();
        if constexpr (RG > 1) {
          if (lane == 0) mbar_arrive(pair + 8 * wg);
          wait(pair + 8 * wg, pph);
          pph ^= 1;
        }
        for (int i = lane; i < 16 * KB * (D / 8); i += 32) {
          const int k = i / (D / 8);
          if (cut >> k & 1)
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(vptr(k, i % (D / 8))), "r"(0) : "memory");
        }
        __syncwarp();
      }
      // ---- O^T += V^T P^T, P as a sum of two values of the type
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        uint32_t ph2[2], pl2[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t h = pack2<F16>(s[kb][2 * e], s[kb][2 * e + 1]);
          const float2 f = unpack2<F16>(h);
          ph2[e] = transpose8x8(h);
          pl2[e] = transpose8x8(pack2<F16>(s[kb][2 * e] - f.x, s[kb][2 * e + 1] - f.y));
        }
#pragma unroll
        for (int d = 0; d < KK; ++d) {
          uint32_t vf[4];
          ldsm4t(sv + voff[kb] + (d >> 2) * halfb + (((d & 3) << 5) ^ vx), vf);
          mma<F16>(o[d], vf[0], vf[1], vf[2], vf[3], ph2[0], ph2[1]);
          mma<F16>(o[d], vf[0], vf[1], vf[2], vf[3], pl2[0], pl2[1]);
        }
      }
      if (!plain) fence_proxy_async_shared();  // the zeros before the next TMA box
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * st);
      if (++st == kStages) {
        st = 0;
        ph ^= 1;
      }
    }
    // ---- the span's end: the group's sums added up in warp order
    float ms = -INFINITY, ls = 0.f, f[4];
    float4 os[NH];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
      if (lane < 4) {
        s_ml[grp][0][wg][ra + e] = m[e];
        s_ml[grp][1][wg][ra + e] = l[e];
      }
    }
#pragma unroll
    for (int h = 0; h < NH; ++h) {
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) s_o[grp][wg][ra + (e & 1)][16 * d + 8 * (e >> 1) + (lane >> 2)] = o[4 * h + d][e];
      named_bar_sync(bar_id, 128);
      if (h == 0) {
#pragma unroll
        for (int w = 0; w < 4; ++w) ms = fmaxf(ms, s_ml[grp][0][w][mrow]);
        const float z = ms == -INFINITY ? 0.f : ms;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          f[w] = ex2(s_ml[grp][0][w][mrow] - z);
          ls = __fmaf_rn(s_ml[grp][1][w][mrow], f[w], ls);
        }
      }
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float4 u = *reinterpret_cast<const float4*>(&s_o[grp][w][mrow][mcol]);
        y = make_float4(__fmaf_rn(u.x, f[w], y.x), __fmaf_rn(u.y, f[w], y.y), __fmaf_rn(u.z, f[w], y.z),
                        __fmaf_rn(u.w, f[w], y.w));
      }
      os[h] = y;
      named_bar_sync(bar_id, 128);  // before the buffer is written again
    }
    // ---- folded onto the spans before it
    if (run0 != 0) {
      put(part_of(key_of(), span), ms, ls, os);
    } else {
      if (span == 0) {
        M = -INFINITY;
        L = 0.f;
#pragma unroll
        for (int h = 0; h < NH; ++h) O[h] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float fa, fb;
      fold_ml(M, L, ms, ls, fa, fb);
#pragma unroll
      for (int h = 0; h < NH; ++h) O[h] = fold_o4(O[h], os[h], fa, fb);
    }
    const bool item_end = span + 1 == it.nspan, run_end = item_end || ioff + ((span + 1) << it.ks) >= hi;
    if (run_end && run0 == 0 && item_end) {
      const int rr = row_of(mrow);
      if (rr >= 0) {
        const long long at = place_of(b, hk, rr);
        put_row<F16, D>(M, L, O, g.a.o + at * D + mcol, g.a.lse && wg == 0 && (lane & 3) == 0 ? g.a.lse + at : nullptr);
      }
    } else if (run_end) {
      if (run0 == 0) put(part_of(key_of(), span), M, L, O);
      named_bar_sync(bar_id, 128);  // the group's partials before the count, which releases them
      if ((tid & 127) == 0) {
        const int c0 = cta_of(ioff), mine = span - run0 + 1;
        int32_t* cnt = g.cnt + 2 * c0 + grp;
        if (add_acq_rel_gpu(cnt, mine) + mine == it.nspan) {
          *cnt = 0;  // ready for the next call
          // the first run's last span holds the fold of the spans before it
          const int n0 = min(it.nspan, (lo_of(c0 + 1) - ioff + (1 << it.ks) - 1) >> it.ks) - 1;
          s_join[grp][s_njoin[grp]++] = {b, rt, hk, it.nspan - n0, part_of(key_of(), n0)};
        }
      }
    }
    if (item_end) {
      run0 = -1;
      more = next_item();
    } else {
      ++span;
    }
  }
  if (__any_sync(0xffffffffu, dead)) {
    // No copy is under way when the CTA ends: what this warp did not wait for, with a
    // limit of its own, is every slot's last fill.
    atomicOr(g.status, DEV_TIMEOUT);
    dead = false;
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) wait(full + 8 * i, i < st ? ph : ph ^ 1);
  }
  // ---- joins, after the loop over tiles: they would take registers from it,
  // and the ring is free once every group is here
  named_bar_sync(kAllBar, 128 * RG);
  for (int i = 0; i < s_njoin[grp]; ++i) {
    const Join jn = s_join[grp][i];
    const int rr = jn.rt * 16 + 8 * grp + mrow;
    const bool real = rr < n_q * G;
    const long long at = real ? place_of(jn.b, jn.hk, rr) : 0;
    join_rows<F16, D, dec_ring<RG>() / RG>(jn.p, pstride, jn.n, ring + grp * (dec_ring<RG>() / RG), bar_id, mrow, mcol,
                      real ? g.a.o + at * D : nullptr, g.a.lse && wg == 0 && (lane & 3) == 0 ? g.a.lse + at : nullptr);
  }
}

int log2_of(int v) {
  int k = 0;
  while ((1 << k) < v) ++k;
  return k;
}

int sm_count(int* dev_out) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  *dev_out = dev;
  return sms > 0 ? sms : 1;
}

constexpr int kMaxCtas = 2 * 304;  // counters and partials of the largest grid

template <bool F16, int D, int RG>
cudaError_t launch_rg(DecArgs& g, int sms, int dev, cudaStream_t st) {
  constexpr int smem = dec_ring<RG>();
  static std::mutex mu;
  static bool configured[64] = {};
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!configured[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(decode_kernel<F16, D, RG>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) {
        cudaGetLastError();
        return e;
      }
      configured[dev] = true;
    }
  }
  const int ctas = dec_ctas<RG>() * sms;
  return launch_pdl(K_ATTN_DECODE, decode_kernel<F16, D, RG>, dim3(ctas < kMaxCtas ? ctas : kMaxCtas), dec_threads<RG>(),
                    smem, st, g);
}

template <bool F16, int D>
cudaError_t launch_one(DecArgs& g, int sms, int dev, cudaStream_t st) {
  return g.r.n_q * g.a.G > 8 ? launch_rg<F16, D, 2>(g, sms, dev, st) : launch_rg<F16, D, 1>(g, sms, dev, st);
}

}  // namespace

bool decode_supported(int D, int page, int Hkv, int G, int n_q, int max_pages) {
  if (D != 64 && D != 128) return false;
  if (page < 8 || (page & (page - 1))) return false;
  if (!encode_fn()) return false;
  // the tiles of one sequence count in int32
  const long long RT = (n_q * (long long)G + 15) / 16, tiles = ((long long)max_pages * page + 63) / 64;
  return Hkv * RT * (tiles + 1) < (1LL << 30);
}

// The rule for the spans of an item: with few items per sequence more spans, so
// that one sequence fills the GPU; with many only as many as that takes, since
// every span costs its end and the join.
int span_c_of(int Hkv, int RT) {
  const int c = 32 / (Hkv * RT);
  return c < 4 ? 4 : c;
}
int most_spans_of(int Hkv, int RT) {
  const int n = 256 / (Hkv * RT);
  return n > 8 ? n : 8;
}

// Spans of an item at most, for tables of max_pages pages.
int max_span_of(int page, int max_pages, int tile, int span_c, int most_spans) {
  const int tiles = (int)(((long long)max_pages * page + tile - 1) / tile);
  int most = 1;
  for (int k = 0;; ++k) {  // the longest item with spans of 2^k tiles
    long long t = (long long)span_c << (2 * k);
    if (t > ((long long)most_spans << k)) t = (long long)most_spans << k;
    if (t > tiles) t = tiles;
    const long long n = (t + (1LL << k) - 1) >> k;
    if (n > most) most = (int)n;
    if (t == tiles) return most;
  }
}

size_t decode_ws_bytes(int page, int max_pages, int Hkv, int G, int D, int max_rows) {
  // an item split over CTAs has its partials at its own place when there are
  // no more items than CTAs, else at the place of its first CTA
  const long long rows = max_rows < 16 ? max_rows : 16;
  size_t most = 0;
  for (int n_q = 1; n_q <= rows; ++n_q) {
    const int RT = (n_q * G + 15) / 16;
    const int seqs = max_rows / n_q < kSeqCap ? max_rows / n_q : kSeqCap;  // of one launch; the next one starts over
    const long long items = seqs * (long long)RT * Hkv, keys = items < kMaxCtas ? items : kMaxCtas;
    const int RG = n_q * G > 8 ? 2 : 1;
    const size_t n = (size_t)keys * RG *
                     max_span_of(page, max_pages, tile_of(D, RG), span_c_of(Hkv, RT), most_spans_of(Hkv, RT));
    most = n > most ? n : most;
  }
  return align256(most * (D == 128 ? part_floats<128>() : part_floats<64>()) * 4);
}

cudaError_t launch_attn_decode(const Cache& c, const Rows& r, const Attn& a, bool f16, int32_t* status, int32_t* sync,
                               void* scratch, cudaStream_t st) {
  int dev = 0;
  const int sms = sm_count(&dev);
  if (!sms) return cudaErrorInvalidDevice;
  const int tile = tile_of(c.D, r.n_q * a.G > 8 ? 2 : 1);
  DecArgs g;
  if (!pool_maps(c, &g.tm_k, &g.tm_v, c.page < tile ? c.page : tile)) return cudaErrorInvalidValue;
  g.c = c;
  g.a = a;
  g.RT = (r.n_q * a.G + 15) / 16;
  g.logpage = log2_of(c.page);
  g.logP = log2_of(tile);
  if (g.logpage < g.logP) g.logP = g.logpage;
  g.span_c = span_c_of(c.Hkv, g.RT);
  g.most_spans = most_spans_of(c.Hkv, g.RT);
  g.max_span = max_span_of(c.page, c.max_pages, tile, g.span_c, g.most_spans);
  g.part = static_cast<float*>(scratch);
  g.status = status;
  g.cnt = sync + kCntBase;
  const long long tiles = ((long long)c.max_pages * c.page + tile - 1) / tile + 1;
  long long per = ((1LL << 30)) / (c.Hkv * (long long)g.RT * tiles);  // sequences whose tiles count in int32
  per = per < 1 ? 1 : per > kSeqCap ? kSeqCap : per;
  for (int b0 = 0; b0 < r.B; b0 += (int)per) {
    g.r = r;
    g.r.B = (int)(r.B - b0 < per ? r.B - b0 : per);
    if (r.slots) {
      g.r.slots = r.slots + b0;
    } else if (b0) {  // sequence b is slot b: shift the slots' arrays
      g.c.table = c.table + (long long)b0 * c.max_pages;
      g.c.lens = c.lens + b0;
      g.c.n_slots = c.n_slots - b0;
    }
    const long long row0 = (long long)b0 * r.n_q;
    g.r.n_rows = g.r.B * r.n_q;
    g.a.q = a.q + row0 * a.q_stride;
    g.a.o = a.o + row0 * a.Hq * c.D;
    g.a.lse = a.lse ? a.lse + row0 * a.Hq : nullptr;
    cudaError_t e;
    if (c.D == 128) e = f16 ? launch_one<true, 128>(g, sms, dev, st) : launch_one<false, 128>(g, sms, dev, st);
    else e = f16 ? launch_one<true, 64>(g, sms, dev, st) : launch_one<false, 64>(g, sms, dev, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace kv
}  // namespace moe
