// Attention of prompt chunks over the paged cache on the 5th-generation tensor
// cores: S = Q K^T and O += P V as tcgen05 products with S, P and O in tensor
// memory, the online softmax between them in registers. Bound by the tensor
// cores at D = 128 (two products of 128 x 128 x 128 per tile and block of 128
// keys, 1,024 cycles) and by the softmax at D = 64.
//
// Units and blocks. A tile is 128 query rows: 128 / G tokens (rounded down)
// times the G query heads of one KV head, so the heads of a group share one
// read of their keys. A unit is two tiles in a row of one sequence and KV head;
// its blocks are 128 keys each, packed from the TMA boxes (a page, or 128 rows of
// one) that some row sees: first tokens that stay visible, then the window.
// (With blocks of 128 tokens in a row, a window of 512 and 4 first tokens was
// seven blocks a unit instead of five, 55 us instead of 48 for the five chunks
// below.) The list of all units' blocks is
// divided evenly over one CTA per SM: a causal chunk's later tiles see more
// keys than its early ones, and few rows over a long context are work for all
// SMs. A unit that lies in several CTAs leaves partial sums (m, l, o in fp32),
// which the last of them to end joins in the order of the keys, or, of units in
// many CTAs, combine_kernel.
//
// Warps. 0-3 and 4-7: the softmax of tile 0 and of tile 1 (a thread is a row);
// 8: issues the products; 9: TMA of Q, K and V; 10: zeroes the value rows that
// no row sees (whatever lies there must not meet a zero probability); 11:
// divides the list and hands out this CTA's segments (a unit, a range of its
// blocks) through a small ring, ahead of the others. While a softmax group
// works on its scores, the tensor cores run the other tile's products:
//   S0 S1 | PV0 S0' | PV1 S1' | PV0' ...
//
// The running maximum is only raised when a row's scores pass it by more than
// 2^8 (probabilities up to 256 are rounded no worse than those up to 1), so the
// accumulators in tensor memory are seldom rescaled. Probabilities are rounded to
// the cache's type for the product (half a step, 2^-8 for bf16 and 2^-11 for fp16,
// independent per key); their sum is kept in fp32 before that rounding. fp16 has a
// fixed step below 2^-14: its probabilities are lifted by 2^7 (to 2^15 at most), so
// that half of that step is 2^-32 of the largest one. Without the lift, keys 2^-25
// below it vanished from the product and stayed in the sum.
//
// Measured (head size 128, bf16, append included; of 1,917 TFLOP/s): 2,048 tokens
// after 30,693, 32 / 8 heads, 660 to 680 us, 1,590 TFLOP/s (0.83), and 740 to 760
// called back to back for long, when the power limit lowers the clock (0.74; of the
// 1,720 TFLOP/s that a long loop of products keeps up, 0.83); a 2,048-token prompt,
// 16 / 4 heads, 33 us; five chunks of up to 901 tokens with a window of 512 and 4
// first tokens, 28 / 4 heads, 47 us. A pair of tiles takes about 3,000 cycles per
// block, 2,048 of them products; a tile's chain is its softmax (1,700), its two
// products (1,024) and the barriers between. Steps of 64 keys with two buffers of
// scores break that chain, but a product of 64 keys takes 51 cycles instead of
// 32 (both operands come from shared memory): 886 us. So were probabilities
// taken with the maximum so far while the block's own is found (+8 %), two
// threads per row (813 us). A short prompt is bound by what stands around its
// blocks: 10,000 cycles until the first scores (the list's division 5,000), 5,000
// to 9,000 at a segment's end, 2,000 to 4,000 more where it is joined, most of
// them instruction fetches of code that runs once.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "kv_common.cuh"
#include "kv_tma.h"
#include "moe_tc.cuh"

namespace moe {
namespace kv {

using namespace tc;

namespace {

constexpr int kBlk = 128;               // keys per block
constexpr int kChunkThreads = 384;
constexpr int kLaunchRegs = 168;        // registers per thread at launch; the groups share 3 x 168
constexpr int kSoftRegs = 224, kRestRegs = 56;
constexpr int kChunkSeqs = 256;         // sequences per launch
constexpr int kMaxGrid = 304;
constexpr int kUnitCost = 3;            // a unit's start and end, in blocks, for the division among the CTAs
constexpr int kSnap = 1;                // a piece of so many blocks or fewer is not cut off (2 is as good)
constexpr int kBadRing = 8;
constexpr int kJoinMost = 3;            // parts that a unit's last CTA joins where combine_kernel follows for the others
constexpr int kFewBlocks = 17;          // a unit of no more blocks: its last CTA joins it
constexpr uint32_t kTries = 1u << 22;   // of a wait, each up to a microsecond long
constexpr int kSegRing = 4;
constexpr int kSegReaders = 11;         // warps 0 .. 10
constexpr int kOutPitch = 80;           // bytes per row of a warp's output buffer (64 and a pad)

// A unit for combine_kernel, in CTAs c0 .. c1, kept at CTA c0 + 1's place (else c0 = -1).
struct Split {
  int c0, c1;
  int row0, rows;     // its first row (token) and how many
  int hk;
};

struct ChunkArgs {
  CUtensorMap tm_q, tm_k, tm_v;
  Cache c;
  Rows r;
  Attn a;
  int b0, nseq;       // sequences of this launch
  int tq;             // tokens per tile
  int logP, logpage;  // rows of a TMA box: min(page, 128)
  int combine;        // whether combine_kernel follows
  int32_t* cnt;       // [grid][2 tiles][4 warps]: parts of the unit that starts in a CTA, zero between calls
  float* part;        // [2 grid][2 tiles][D / 4][128][4]
  float* pml;         // [2 grid][2 tiles][m, l][128]
  Split* split;       // [grid]
  int32_t* status;
};

// The two tiles of a unit and the blocks they see.
struct Unit {
  int b, qb, hk;
  int slot, row0, nt;      // first row (token) of the call and tokens
  int pf, pl;              // positions of the first and the last token; pl = -1 if nothing is seen
  int from, first;         // the window's first token; first tokens below it that stay visible
  // Its keys are the TMA boxes that some row sees, in order: position i of them is
  // token i below ns (the boxes of the first tokens), token i + gap from there on
  // (the window's). Block u is positions 128 u .. 128 u + 127.
  int ns, gap, nb;
  int u0, u1;              // this CTA's blocks of it
  int c0, c1;              // the CTAs that share it
  int more;                // 0: no unit, the end of the list
  // tokens' positions of tile t: [tf, tl], tl < tf if it has none
  __device__ void tile(int t, int tq, int& tf, int& tl) const {
    tf = pf + t * tq;
    tl = pf + min(nt, (t + 1) * tq) - 1;
  }
};

// The sequences of a launch and the division of their blocks, in shared memory.
struct Plan {
  int off[kChunkSeqs + 1];         // list positions before each sequence
  int nq[kChunkSeqs];              // units of one KV head
  int slot[kChunkSeqs], len[kChunkSeqs], n[kChunkSeqs], row0[kChunkSeqs];
};

// A unit's positions in the list, and the block at which a CTA boundary that
// falls `at` positions into it cuts it: at its start or its end where the piece
// would be small (a cut costs both sides a start, an end and the join).
__device__ __forceinline__ int weight(int nb) { return max(1, nb) + kUnitCost; }
__device__ __forceinline__ int cut_at(int nb, int at) {
  if (at <= 0) return 0;
  if (nb < 2) return max(1, nb);  // one piece (an empty unit counts as one block): where it starts
  const int x = at - kUnitCost;
  return x <= min(kSnap, nb / 2) ? 0 : x >= nb - kSnap ? nb : x;
}

__device__ __forceinline__ Unit unit_at(const Plan& p, const ChunkArgs& g, int b, int qb, int hk) {
  Unit x;
  const int W = g.a.window, i0 = qb * 2 * g.tq;
  x.b = b; x.qb = qb; x.hk = hk;
  x.slot = p.slot[b];
  x.row0 = p.row0[b] + i0;
  x.nt = min(p.n[b] - i0, 2 * g.tq);
  x.pf = p.len[b] - p.n[b] + i0;
  x.pl = x.slot < 0 ? -1 : x.pf + x.nt - 1;
  x.from = x.first = x.ns = x.gap = x.nb = 0;
  if (x.pl >= 0) {
    x.from = W > 0 ? max(0, max(0, x.pf) - W + 1) : 0;
    x.first = min(g.a.n_sink, x.from);
    const int P = 1 << g.logP;
    x.ns = (x.first + P - 1) & -P;
    x.gap = max(x.from & -P, x.ns) - x.ns;
    x.nb = ((x.pl & -P) + P - x.gap + kBlk - 1) / kBlk;
  }
  return x;
}

// CTA i's part of `total` positions among nc CTAs starts at lo(i); cta(at) is
// the last i with lo(i) <= at.
struct Division {
  int q, r;
  __device__ Division(int total, int nc) : q(total / nc), r(total - total / nc * nc) {}
  __device__ int lo(int i) const { return i * q + min(i, r); }
  __device__ int cta(int at) const { return at < r * (q + 1) ? at / (q + 1) : r + (at - r * (q + 1)) / q; }
};

__device__ __forceinline__ int warp_scan(int v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// The whole of warp 11: the division, then this CTA's segments into the ring.
__device__ __forceinline__ void schedule(Plan& p, const ChunkArgs& g, Unit* ring, uint32_t full, uint32_t empty,
                                         uint32_t shared) {
  const int lane = threadIdx.x & 31, Hkv = g.c.Hkv;
  // the sequences, and the list positions of the units of each
  int total = 0, units = 0;
  for (int b0 = 0; b0 < g.nseq; b0 += 32) {
    const int b = b0 + lane;
    int nq = 0;
    if (b < g.nseq) {
      const Seq s = load_seq(g.c, g.r, g.b0 + b, blockIdx.x == 0 ? g.status : nullptr);
      nq = (s.n + 2 * g.tq - 1) / (2 * g.tq);
      p.slot[b] = s.slot; p.len[b] = s.len; p.n[b] = s.n; p.row0[b] = s.row0; p.nq[b] = nq;
    }
    __syncwarp();
    // a lane per sequence, or for few sequences a lane per unit
    int w = 0;
    if (g.nseq >= 8) {
      for (int q = 0; q < nq; ++q) w += weight(unit_at(p, g, b, q, 0).nb);
    } else {
      for (int k = 0; k < g.nseq; ++k) {
        int part = 0;
        for (int q = lane; q < p.nq[k]; q += 32) part += weight(unit_at(p, g, k, q, 0).nb);
        part = __reduce_add_sync(0xffffffffu, part);
        if (lane == k) w = part;
      }
    }
    const int x = warp_scan(w * Hkv, lane);
    if (b < g.nseq) p.off[b] = total + x - w * Hkv;
    total += __shfl_sync(0xffffffffu, x, 31);
    units += __reduce_add_sync(0xffffffffu, nq) * Hkv;
  }
  if (lane == 0) p.off[g.nseq] = total;
  __syncwarp();
  // a CTA per unit, or per two blocks where units are longer than that (512 tokens
  // 19 us, 20 with four)
  const int nc = min(max((total + 1 + kUnitCost) / (2 + kUnitCost), units), (int)gridDim.x);
  const bool work = (int)blockIdx.x < nc;
  const Division dv(total, max(nc, 1));
  const int lo = work ? dv.lo(blockIdx.x) : 0, hi = work ? dv.lo(blockIdx.x + 1) : 0;
  Unit x;
  int start = 0;
  if (lo < hi) {
    // the unit that holds position lo
    int b = 0, h = g.nseq - 1;  // the last sequence that starts at or before it
    while (b < h) {
      const int m = (b + h + 1) >> 1;
      if (p.off[m] <= lo) b = m;
      else h = m - 1;
    }
    start = p.off[b];
    int qb = 0;
    for (int q0 = 0;; q0 += 32) {
      const int q = q0 + lane;
      const int w = q < p.nq[b] ? weight(unit_at(p, g, b, q, 0).nb) * Hkv : 0;
      const int s = warp_scan(w, lane);
      const unsigned in = __ballot_sync(0xffffffffu, lo < start + s);
      if (in || q0 + 32 >= p.nq[b]) {
        const int src = in ? __ffs(in) - 1 : 31;
        qb = q0 + src;
        start += __shfl_sync(0xffffffffu, s - w, src);
        break;
      }
      start += __shfl_sync(0xffffffffu, s, 31);
    }
    x = unit_at(p, g, b, qb, 0);
    x.hk = (lo - start) / weight(x.nb);
    start += x.hk * weight(x.nb);
  }
  int i = 0, ph = 1;
  auto put = [&](int more) {
    if (!__all_sync(0xffffffffu, mbar_wait_sleep(empty + 8 * i, ph, g.status))) return false;
    x.more = more;
    if (lane == 0) {
      ring[i] = x;
      mbar_arrive(full + 8 * i);
    }
    __syncwarp();
    return true;
  };
  // the CTAs that share the segment's unit follow: its readers need them at its end only
  auto put_shared = [&] {
    if (lane == 0) {
      ring[i].c0 = x.c0;
      ring[i].c1 = x.c1;
      mbar_arrive(shared + 8 * i);
    }
    __syncwarp();
    if (++i == kSegRing) {
      i = 0;
      ph ^= 1;
    }
  };
  Split sp;
  sp.c0 = -1;
  bool ok = true;
  while (ok && start < hi) {
    const int a = cut_at(x.nb, lo - start), e = cut_at(x.nb, hi - start);
    if (a < e) {  // this CTA has a part of it
      x.u0 = min(a, x.nb);
      x.u1 = min(e, x.nb);
      x.c0 = x.c1 = blockIdx.x;
      ok = put(1);
      if (x.u0 > 0 || x.u1 < x.nb) {  // a split unit: the CTAs of its first and its last block
        if (x.u0 > 0) {
          x.c0 = dv.cta(start + kUnitCost);
          while (cut_at(x.nb, dv.lo(x.c0 + 1) - start) <= 0) ++x.c0;
        }
        if (x.u1 < x.nb) {
          x.c1 = dv.cta(start + kUnitCost + x.nb - 1);
          while (cut_at(x.nb, dv.lo(x.c1) - start) >= x.nb) --x.c1;
        }
        if (g.combine && x.c1 - x.c0 >= kJoinMost && x.c0 + 1 == (int)blockIdx.x)
          sp = {x.c0, x.c1, x.row0, x.nt, x.hk};
      }
      if (ok) put_shared();
    }
    start += weight(x.nb);
    if (start >= hi) break;
    if (++x.hk == Hkv) {
      int b = x.b, qb = x.qb + 1;
      while (qb >= p.nq[b]) {
        ++b;
        qb = 0;
      }
      x = unit_at(p, g, b, qb, 0);
    }
  }
  if (ok) put(0);
  if (lane == 0 && g.combine) g.split[blockIdx.x] = sp;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 w, x, y;\n"
      " mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// The n lowest bits (none below 0, all from 32 on).
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }
// Scores I .. I + 63 of keys that the row does not see become -inf.
template <int I>
__device__ __forceinline__ void cut(uint32_t (&s)[kBlk], const uint32_t (&vis)[4]) {
#pragma unroll
  for (int i = I; i < I + 64; ++i) s[i] = vis[i / 32] & (1u << (i % 32)) ? s[i] : 0xff800000u;
}

template <int D>
__host__ __device__ constexpr int stages() { return D == 128 ? 4 : 8; }
template <int D>
__host__ __device__ constexpr int chunk_smem() {
  return 1024 + 2 * kBlk * D * 2 + stages<D>() * kBlk * D * 2 + 8 * 32 * kOutPitch;
}

template <bool F16, int D>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_kernel(const __grid_constant__ ChunkArgs g) {
  constexpr int NH = D / 64;               // halves of 64 columns
  constexpr int kTileB = kBlk * D * 2;     // bytes of a Q tile, or of a K or V block
  constexpr int kHalf = kBlk * 128;
  constexpr int NST = stages<D>();
  extern __shared__ __align__(1024) uint8_t smem_chunk[];
  __shared__ Plan s_plan;
  __shared__ __align__(8) uint64_t s_bar[3 * NST + 3 * kSegRing + 13];
  __shared__ uint32_t s_bad[kBadRing];
  __shared__ __align__(16) Unit s_seg[kSegRing];
  __shared__ uint32_t s_tmem;
  __shared__ int s_tok[kBlk];      // token of each row of a tile

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int W = g.a.window, S = g.a.n_sink, G = g.a.G, tq = g.tq;
  const uint32_t sq = (smem_u32(smem_chunk) + 1023u) & ~1023u, ring = sq + 2 * kTileB;
  const uint32_t kv_full = smem_u32(s_bar), kv_empty = kv_full + 8 * NST, v_ready = kv_empty + 8 * NST;
  const uint32_t q_full = v_ready + 8 * NST, q_empty = q_full + 8;
  const uint32_t s_full = q_empty + 8, p_full = s_full + 16, pv_done = p_full + 32, o_free = pv_done + 16;
  const uint32_t drained = o_free + 16, seg_full = drained + 8, seg_empty = seg_full + 8 * kSegRing;
  const uint32_t seg_shared = seg_empty + 8 * kSegRing;
  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(kv_full + 8 * i, 1);
      mbar_init(kv_empty + 8 * i, 1);
      mbar_init(v_ready + 8 * i, 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full + 8 * t, 1);
      mbar_init(p_full + 16 * t, 4);
      mbar_init(p_full + 16 * t + 8, 4);
      mbar_init(pv_done + 8 * t, 1);
      mbar_init(o_free + 8 * t, 4);
    }
    mbar_init(drained, 1);
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(seg_full + 8 * i, 1);
      mbar_init(seg_shared + 8 * i, 1);
      mbar_init(seg_empty + 8 * i, kSegReaders);
    }
    fence_barrier_init();
  }
  if (tid < kBlk) s_tok[tid] = tid / G;
  if (tid == 32 * 9) {
    prefetch_tensormap(&g.tm_q);
    prefetch_tensormap(&g.tm_k);
    prefetch_tensormap(&g.tm_v);
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  griddep_wait();  // an append's rows, and the workspace of the launch before

  // The blocks of a unit of which tile t sees something: those below `end` that
  // are below `early` (first tokens) or not below `win` (the tile's own window).
  struct Taken {
    int end, early, win;
    __device__ bool operator()(int u) const { return u < end && (u < early || u >= win); }
  };
  auto taken = [&](const Unit& x, int t) {
    int tf, tl;
    x.tile(t, tq, tf, tl);
    const int last = tl < x.ns ? tl : max(x.ns - 1, tl - x.gap);  // its last token's position
    Taken k;
    k.end = tl >= max(tf, 0) ? last / kBlk + 1 : 0;
    k.early = W > 0 ? (max(x.ns, S - x.gap) + kBlk - 1) / kBlk : 0;
    k.win = W > 0 ? max(x.ns, max(tf, 0) - W + 1 - x.gap) / kBlk : 0;
    return k;
  };
  // A wait is a few instructions: the warp that issues the products runs from a
  // cold instruction cache between the softmax warps' loops, and a wait that
  // found its phase complete cost it 270 cycles with the time taken inside.
  bool dead = false;  // an expired wait: go on without waiting (the status word says so)
  auto wait = [&](uint32_t bar, uint32_t parity) {
    uint32_t n = dead ? 1u : kTries;
    while (!mbar_try_wait_ns(bar, parity, 1000) && --n) {
    }
    dead |= n == 0;
    __syncwarp();
  };
  auto wait2 = [&](uint32_t bar, uint32_t parity, uint32_t bar2, uint32_t parity2) {  // for both
    uint32_t n = dead ? 1u : kTries;
    while (true) {
      const bool a = mbar_try_wait_ns(bar, parity, 1000), b = mbar_try_wait_ns(bar2, parity2, 1000);
      if ((a && b) || !--n) break;
    }
    dead |= n == 0;
    __syncwarp();
  };
  // this CTA's segments: next_seg() waits for one (false: there are no more),
  // done_seg() gives its place back
  int seg_i = 0, seg_ph = 0;
  auto next_seg = [&] {
    wait(seg_full + 8 * seg_i, seg_ph);
    dead = __any_sync(0xffffffffu, dead);
    return !dead && s_seg[seg_i].more != 0;
  };
  auto done_seg = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(seg_empty + 8 * seg_i);
    if (++seg_i == kSegRing) {
      seg_i = 0;
      seg_ph ^= 1;
    }
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
    if (warp == 9) {
      // ================= TMA producer =================
      const int P = 1 << g.logP, nbox = kBlk >> g.logP;
      int st = 0, ph = 1, bad_at = 0, qph = 1;
      bool opening = true;
      while (next_seg()) {
        const Unit x = s_seg[seg_i];
        done_seg();
        if (x.u0 == x.u1) continue;
        const int nt = x.nt > tq ? 2 : 1;
        const int32_t* tab = g.c.table + (long long)x.slot * g.c.max_pages;
        // lane's box of block u: its first row in the pool; for a box that no row
        // sees, or of a bad page, the row past the pool's end, from where TMA
        // fills in zeros
        const int past = g.c.n_pages * g.c.Hkv << g.logpage;
        // (page() only reads the table: its result is first needed in row_of())
        auto token = [&](int u) {  // of lane's box, -1 if there is none
          const int i = u * kBlk + lane * P, j = i < x.ns ? i : i + x.gap;
          return lane < nbox && j <= x.pl ? j : -1;
        };
        auto page = [&](int u) {
          const int j = token(u);
          return j >= 0 ? tab[j >> g.logpage] : 0;
        };
        auto row_of = [&](int u, int pg) {
          const int j = token(u);
          if (j < 0) return past;
          if (pg >= 0 && pg < g.c.n_pages) return ((pg * g.c.Hkv + x.hk) << g.logpage) + (j & (g.c.page - 1));
          atomicOr(g.status, DEV_BAD_SLOT);
          return past + 1;
        };
        auto queries = [&] {
          wait(q_empty, qph);
          if (!dead) qph ^= 1;
          if (lane == 0 && !dead) {
            mbar_expect_tx(q_full, (uint32_t)(nt * NH * tq * G * 128));
            for (int t = 0; t < nt; ++t)
              for (int h = 0; h < NH; ++h)
                tma_load_3d(sq + t * kTileB + h * kHalf, &g.tm_q, h * 64, x.hk * G, x.row0 + t * tq, q_full);
          }
          __syncwarp();
        };
        int pg = page(x.u0);
        if (opening) queries();  // the CTA's first segment: the queries first
        for (int u = x.u0; u < x.u1 && !dead; ++u) {
          const int row = row_of(u, pg);
          pg = u + 1 < x.u1 ? page(u + 1) : 0;
          const unsigned bad = __ballot_sync(0xffffffffu, row == past + 1);
          for (int kv = 0; kv < 2; ++kv) {
            wait(kv_empty + 8 * st, ph);
            if ((dead = __any_sync(0xffffffffu, dead))) break;
            if (lane == 0) {
              if (kv == 0) s_bad[bad_at] = bad;
              mbar_expect_tx(kv_full + 8 * st, kTileB);
            }
            __syncwarp();
            if (lane < nbox)
#pragma unroll
              for (int h = 0; h < NH; ++h)
                tma_load_2d(ring + st * kTileB + h * kHalf + lane * P * 128, kv ? &g.tm_v : &g.tm_k, h * 64, row,
                            kv_full + 8 * st);
            if (++st == NST) {
              st = 0;
              ph ^= 1;
            }
            // later ones after the first keys, which need not wait for the last segment's products
            if (u == x.u0 && kv == 0 && !opening) queries();
          }
          bad_at = (bad_at + 1) % kBadRing;
        }
        opening = false;
      }
      // No copy is under way when the CTA ends, also where a warp went on without
      // waiting: a wait, with a limit of its own, for every slot's last fill (a slot
      // never filled is in the phase before its first).
      const bool gave_up = dead;
      dead = false;
#pragma unroll 1
      for (int i = 0; i < NST; ++i) wait(kv_full + 8 * i, i < st ? ph ^ 1 : ph);
      wait(q_full, qph);
      dead |= gave_up;
    } else if (warp == 10) {
      // ================= values that no row sees become zeros =================
      const int P = 1 << g.logP;
      int st = 1, ph = 0;
      while (next_seg()) {
        const Unit x = s_seg[seg_i];
        done_seg();
        for (int u = x.u0; u < x.u1; ++u) {
          const int i0 = u * kBlk;
          wait(kv_full + 8 * st, ph);
          // positions [a, e) of the boxes that some row sees and some rows of which
          // none does: past the last token, after the first tokens, before the window
          auto zero = [&](int a, int e) {
            a = max(a - i0, 0);
            e = min(e - i0, kBlk);
            for (int r = a + (lane >> 3); r < e; r += 4)  // eight lanes a row of 128 bytes
#pragma unroll
              for (int h = 0; h < NH; ++h) st_s128(ring + st * kTileB + h * kHalf + r * 128 + (lane & 7) * 16, 0u, 0u, 0u, 0u);
            return a < e;
          };
          const int end = (x.pl < x.ns ? x.pl : x.pl - x.gap) + 1;
          bool any = zero(end, (end + P - 1) & -P);
          any |= zero(x.first, min(x.ns, x.from));
          any |= zero(x.ns, x.from - x.gap);
          if (any) fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(v_ready + 8 * st);
          st += 2;
          if (st >= NST) {
            st = 1;
            ph ^= 1;
          }
        }
      }
    } else if (warp == 8) {
      // ================= tensor-core products =================
      const uint32_t lead = elect_lane();
      const uint32_t id_s = idesc_16(F16, 128, kBlk, false), id_o = idesc_16(F16, 128, D, true);
      // descriptors of the first tiles; the others differ by their address / 16
      // in the low field (no carry: shared addresses < 256 KB)
      const uint64_t qd0 = sdesc_sw128(sq), kd0 = sdesc_sw128(ring), vd0 = sdesc_sw128_n(ring, kHalf);
      int kst = 0, kph = 0;        // ring slot and phase of the next K block (its V block is the slot after)
      uint32_t np = 0, nseg = 3;   // bit t: parity of tile t's products so far; of its segments (for o_free)
      int nq = 0;
      while (next_seg()) {
        const Unit x = s_seg[seg_i];
        done_seg();
        if (x.u0 == x.u1) continue;
        wait(q_full, nq & 1);
        ++nq;
        tc_fence_after();
        bool started[2] = {false, false};
        auto score = [&](int t, int st) {
          const uint64_t qd = qd0 + (uint32_t)(t * kTileB >> 4), kd = kd0 + (uint32_t)(st * kTileB >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
            tc_mma_el(tmem + t * kBlk, qd + o, kd + o, id_s, kk > 0, lead);
          }
          tc_commit_el(s_full + 8 * t, lead);
        };
        auto product = [&](int t, int st) {
          if (!started[t]) {  // the tile's accumulator has been read by the segment before
            wait(o_free + 8 * t, nseg >> t & 1);
            nseg ^= 1u << t;
          }
          const uint64_t vd = vd0 + (uint32_t)(st * kTileB >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // the block's first 64 keys, while the others' probabilities are made
            wait(p_full + 16 * t + 8 * h, np >> t & 1);
            tc_fence_after();
#pragma unroll
            for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
              tc_mma_ts_el(tmem + 256 + t * 128, tmem + t * kBlk + kk * 8, vd + kk * (2048 >> 4), id_o,
                           started[t] || kk > 0, lead);
          }
          np ^= 1u << t;
          started[t] = true;
          tc_commit_el(pv_done + 8 * t, lead);
        };
        const Taken k0 = taken(x, 0), k1 = taken(x, 1);
        bool t0 = k0(x.u0), t1 = k1(x.u0);
        wait(kv_full + 8 * kst, kph);
        tc_fence_after();
        if (t0) score(0, kst);
        if (t1) score(1, kst);
        tc_commit_el(kv_empty + 8 * kst, lead);
        if (x.u0 + 1 == x.u1) tc_commit_el(q_empty, lead);
        for (int u = x.u0; u < x.u1; ++u) {
          const int vst = kst + 1, vph = kph;
          kst += 2;
          if (kst == NST) {
            kst = 0;
            kph ^= 1;
          }
          const bool nx = u + 1 < x.u1;
          const bool n0 = nx && k0(u + 1), n1 = nx && k1(u + 1);
          if (nx) wait2(v_ready + 8 * vst, vph, kv_full + 8 * kst, kph);
          else wait(v_ready + 8 * vst, vph);
          tc_fence_after();
          if (t0) product(0, vst);
          if (n0) score(0, kst);
          if (t1) product(1, vst);
          tc_commit_el(kv_empty + 8 * vst, lead);
          if (n1) score(1, kst);
          if (nx) {
            tc_commit_el(kv_empty + 8 * kst, lead);
            if (u + 2 == x.u1) tc_commit_el(q_empty, lead);  // the segment's last product with Q
          }
          t0 = n0;
          t1 = n1;
        }
      }
      // every product has ended before tensor memory is given back
      tc_commit_el(drained, lead);
      mbar_wait_short(drained, 0, g.status);
    }
    else {
      // ================= the division and this CTA's segments =================
      schedule(s_plan, g, s_seg, seg_full, seg_empty, seg_shared);
    }
  } else {
    // ================= softmax (a thread is a row of its tile) =================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + t * kBlk, to = tmem + lanes + 256 + t * 128;
    const float sc = g.a.scale * 1.4426950408889634f;
    const uint32_t sout = ring + NST * kTileB + warp * 32 * kOutPitch;
    uint32_t nsc = 0;   // score blocks of this tile so far
    int bad_at = 0;
    while (next_seg()) {
      const Unit& x = s_seg[seg_i];  // read again at the segment's end: few registers are left in the loop
      int tf, tl;
      x.tile(t, tq, tf, tl);
      const int tok = s_tok[r];
      const int pos = tok < tq && tf + tok <= tl && x.slot >= 0 ? tf + tok : -1;
      float m = -INFINITY, l = 0.f;
      bool any = false;     // the accumulator holds a product of this segment
      const int ns = x.ns, gap = x.gap, u1 = x.u1;
      const Taken mine = taken(x, t);
      for (int u = x.u0; u < u1; ++u) {
        if (!mine(u)) {
          bad_at = (bad_at + 1) % kBadRing;
          continue;
        }
        // keys below `cut_k` are the tokens from u * kBlk on, the others those from jw on
        const int cut_k = ns - u * kBlk, jw = u * kBlk + (cut_k < kBlk ? gap : 0);
        const bool all = (cut_k <= 0 || cut_k >= kBlk) && jw + kBlk - 1 <= tf && (W == 0 || jw > tl - W || jw + kBlk <= S);
        wait(s_full + 8 * t, nsc & 1);
        tc_fence_after();
        const uint32_t bad = *(volatile uint32_t*)&s_bad[bad_at];
        bad_at = (bad_at + 1) % kBadRing;
        uint32_t s[kBlk];
        float mx[4];
        tc_ld32(ts, s);
        tc_ld32(ts + 32, s + 32);
        tc_ld_wait();
        tc_ld32(ts + 64, s + 64);
        tc_ld32(ts + 96, s + 96);
        const bool edge = bad || !all;
        uint32_t vis[4];
        if (edge) {  // bit i: the row sees key i of the block
          auto seen = [&](int j0, int w) {
            const int last = pos - j0, low = W > 0 ? pos - W - j0 : -1, keep = W > 0 ? S - j0 : 0;
            return below(last + 1 - 32 * w) & (~below(low + 1 - 32 * w) | below(keep - 32 * w));
          };
#pragma unroll
          for (int w = 0; w < 4; ++w) vis[w] = seen(jw, w);
          if (cut_k > 0 && cut_k < kBlk)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t early = below(cut_k - 32 * w);
              vis[w] = (vis[w] & ~early) | (seen(u * kBlk, w) & early);
            }
          if (bad)
#pragma unroll
            for (int w = 0; w < 4; ++w)
              for (int i = 0; i < 32; i += 8)
                if (bad >> ((32 * w + i) >> g.logP) & 1) vis[w] &= ~(0xffu << i);
          cut<0>(s, vis);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(s[i]);
#pragma unroll
        for (int i = 4; i < 64; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i]));
        tc_ld_wait();
        if (edge) cut<64>(s, vis);
#pragma unroll
        for (int i = 64; i < kBlk; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
        const bool raise = top > m + 8.f || (m == -INFINITY && top > m);
        if (__any_sync(0xffffffffu, raise)) {
          const float m2 = raise ? top : m;
          const float f = m == m2 ? 1.f : ex2(m - m2);
          m = m2;
          l *= f;
          if (any) {  // the product before is still running, maybe
            wait(pv_done + 8 * t, (nsc & 1) ^ 1);
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
              uint32_t o[32];
              tc_ld32(to + i, o);
              tc_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tc_st32(to + i, o);
            }
          }
        }
        const float z = m == -INFINITY ? 0.f : m - lift<F16>();
        const float2 sc2 = make_float2(sc, sc), z2 = make_float2(-z, -z);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < kBlk / 64; ++c) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float2 e = fma2(make_float2(__uint_as_float(s[64 * c + 2 * i]), __uint_as_float(s[64 * c + 2 * i + 1])), sc2, z2);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            sum[i & 1] = add2(sum[i & 1], e);
            pk[i] = pack2<F16>(e.x, e.y);
          }
          tc_st32(ts + 32 * c, pk);
          tc_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + 16 * t + 8 * c);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        ++nsc;
        any = true;
      }
      // ---- the segment's end: the tile's rows out. Its loops are kept small: the
      // code runs once per segment, mostly cold, and its fetches are what it
      // waits for (unrolled over 64 columns the ends took twice as long).
      const bool whole = x.u0 == 0 && x.u1 == x.nb;
      // A unit in several CTAs: all but the last to end leave their part (place
      // 2 c + 1 if it holds the unit's first block, else 2 c); the last one adds
      // the parts up in the order of the keys, its own from tensor memory.
      wait(seg_shared + 8 * seg_i, seg_ph);
      const int c0 = x.c0, c1 = x.c1, me = blockIdx.x;
      auto place = [&](int c) { return (2 * c + (c == c0 ? 1 : 0)) * 2 + t; };
      const bool here = !(g.combine && c1 - c0 >= kJoinMost);
      int32_t* cnt = g.cnt + c0 * 8 + (warp & 7);
      bool last = whole;
      if (!whole && here) {  // while the last product runs
        last = __shfl_sync(0xffffffffu, lane == 0 ? ld_acquire_gpu(cnt) : 0, 0) == c1 - c0;
        __syncwarp();
      }
      if (any) {
        wait(pv_done + 8 * t, (nsc & 1) ^ 1);
        tc_fence_after();
      }
      if (!last) {
        float* pm = g.pml + place(me) * 256;
        pm[r] = m;
        pm[128 + r] = l;
        if (any) {
          float* pp = g.part + (long long)place(me) * D * 128 + r * 4;
#pragma unroll 1
          for (int i = 0; i < D; i += 32) {
            uint32_t o[32];
            tc_ld32(to + i, o);
            tc_ld_wait();
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(pp + (long long)(i / 4 + e) * 512) =
                  make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        if (here) {
          __syncwarp();
          last = __shfl_sync(0xffffffffu, lane == 0 ? add_acq_rel_gpu(cnt, 1) : 0, 0) == c1 - c0;
          __syncwarp();
        }
      }
      if (last) {
        // the first part of another CTA, 32 columns ahead of their use
        const int cf = c0 == me ? c0 + 1 : c0;
        float4 ahead[8];
        auto fetch = [&](int i) {
          const float* pp = g.part + (long long)place(cf) * D * 128 + i * 128 + r * 4;
#pragma unroll
          for (int e = 0; e < 8; ++e) ahead[e] = __ldcg(reinterpret_cast<const float4*>(pp + e * 512));
        };
        float mt = m, lt = l, mf = -INFINITY, lf = 0.f;
        if (!whole) {
          fetch(0);
          mt = -INFINITY;
          lt = 0.f;
#pragma unroll 1
          for (int c = c0; c <= c1; ++c) {
            const float* pm = g.pml + place(c) * 256 + r;
            const float mc = c == me ? m : __ldcg(pm), lc = c == me ? l : __ldcg(pm + 128);
            const float n = fmaxf(mt, mc), z = n == -INFINITY ? 0.f : n;
            lt = fmaf(lc, ex2(mc - z), lt * ex2(mt - z));
            mt = n;
            if (c == cf) {
              mf = mc;
              lf = lc;
            }
          }
        }
        const float zt = mt == -INFINITY ? 0.f : mt, inv = lt == 0.f ? 0.f : 1.f / lt;
        // factors; 0 for a row that saw nothing in a part (which may have left no accumulator)
        const float f_me = l != 0.f ? ex2(m - zt) : 0.f, f_cf = lf != 0.f ? ex2(mf - zt) : 0.f;
        // a thread holds a row; 32 columns at a time through the warp's own
        // buffer, from which four lanes write 64 bytes of a row
        const int nt = min(tq, tl - tf + 1);  // tokens of the tile
        uint16_t* po = g.a.o + (((long long)x.row0 + t * tq) * g.a.Hq + x.hk * G) * D + (lane & 3) * 8;
        int off[4];  // -1: a row of no token
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = (warp & 3) * 32 + k * 8 + (lane >> 2), tk = s_tok[rr];
          off[k] = tk < nt ? (tk * (g.a.Hq - G) + rr) * D : -1;
        }
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          float y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = 0.f;
#pragma unroll 1
          for (int c = c0; c <= c1; ++c) {
            if (c == me || whole) {
              if (!any) continue;
              uint32_t o[32];
              tc_ld32(to + i, o);
              tc_ld_wait();
              if (f_me != 0.f) {
#pragma unroll
                for (int k = 0; k < 32; ++k) y[k] = fmaf(__uint_as_float(o[k]), f_me, y[k]);
              }
            } else {
              float f = f_cf;
              float4 v[8];
              if (c == cf) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = ahead[e];
                if (i + 32 < D) fetch(i + 32);
              } else {
                const float* pm = g.pml + place(c) * 256 + r;
                const float lc = __ldcg(pm + 128), mc = __ldcg(pm);
                const float* pp = g.part + (long long)place(c) * D * 128 + i * 128 + r * 4;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __ldcg(reinterpret_cast<const float4*>(pp + e * 512));
                f = lc != 0.f ? ex2(mc - zt) : 0.f;
              }
              if (f != 0.f) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  y[4 * e] = fmaf(v[e].x, f, y[4 * e]);
                  y[4 * e + 1] = fmaf(v[e].y, f, y[4 * e + 1]);
                  y[4 * e + 2] = fmaf(v[e].z, f, y[4 * e + 2]);
                  y[4 * e + 3] = fmaf(v[e].w, f, y[4 * e + 3]);
                }
              }
              __syncwarp();
            }
          }
          const bool none = lt == 0.f;  // the row sees nothing
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = none ? 0u : pack2<F16>(y[8 * e + 2 * k] * inv, y[8 * e + 2 * k + 1] * inv);
            st_s128(sout + lane * kOutPitch + e * 16, w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (off[k] >= 0)
              *reinterpret_cast<uint4*>(po + off[k] + i) = ld_s128(sout + (k * 8 + (lane >> 2)) * kOutPitch + (lane & 3) * 16);
          __syncwarp();
        }
        if (g.a.lse && tok < nt)
          g.a.lse[((long long)x.row0 + t * tq + tok) * g.a.Hq + x.hk * G + r - tok * G] =
              lt == 0.f ? -INFINITY : (mt + (log2f(lt) - lift<F16>())) * 0.6931471805599453f;
        if (!whole && lane == 0) *cnt = 0;  // ready for the next call
      }
      if (any) {  // the accumulator may be written again
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free + 8 * t);
      }
      done_seg();
    }
  }
  if (dead) atomicOr(g.status, DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();
  if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Units that lie in many CTAs: their parts folded in the order of the keys. A
// job is eight columns of a tile of such a unit, a thread per row; the parts
// come kFold at a time, so that a few reads' latency covers them all (one by one
// 38 parts took 40 us).
constexpr int kFold = 8;
template <bool F16, int D>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ ChunkArgs g, int grid) {
  __shared__ int s_list[kMaxGrid], s_n;
  griddep_wait();
  griddep_launch_dependents();
  const int r = threadIdx.x;
  if (r < 32) {  // the units
    int n = 0;
    for (int i0 = 1; i0 < grid; i0 += 32) {
      const bool is = i0 + r < grid && __ldcg(&g.split[i0 + r].c0) >= 0;
      const unsigned all = __ballot_sync(0xffffffffu, is);
      if (is) s_list[n + __popc(all & ((1u << r) - 1u))] = i0 + r;
      n += __popc(all);
    }
    if (r == 0) s_n = n;
  }
  __syncthreads();
  constexpr int kCols = D / 8;
  for (int job = blockIdx.x; job < s_n * 2 * kCols; job += gridDim.x) {
    const Split sp = g.split[s_list[job / (2 * kCols)]];
    const int t = job / kCols & 1, q = job % kCols;
    const int tok = r / g.a.G, local = t * g.tq + tok;
    if (tok >= g.tq || local >= sp.rows) continue;
    float m = -INFINITY, l = 0.f, o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = 0.f;
#pragma unroll 1
    for (int b = sp.c0; b <= sp.c1; b += kFold) {
      float mc[kFold], lc[kFold];
      float4 v[kFold][2];
#pragma unroll
      for (int i = 0; i < kFold; ++i) {
        const int c = min(b + i, sp.c1);
        const long long place = (2 * c + (c == sp.c0 ? 1 : 0)) * 2 + t;
        const float* pp = g.part + place * D * 128 + q * 1024 + r * 4;
        mc[i] = __ldcg(g.pml + place * 256 + r);
        lc[i] = b + i <= sp.c1 ? __ldcg(g.pml + place * 256 + 128 + r) : 0.f;
        v[i][0] = __ldcg(reinterpret_cast<const float4*>(pp));
        v[i][1] = __ldcg(reinterpret_cast<const float4*>(pp + 512));
      }
#pragma unroll
      for (int i = 0; i < kFold; ++i) {
        if (lc[i] == 0.f) continue;  // the row saw nothing here (its accumulator may not have been written)
        const float n = fmaxf(m, mc[i]), f = ex2(m - n), e = ex2(mc[i] - n);  // mc is finite
        m = n;
        l = fmaf(lc[i], e, l * f);
        const float w[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = fmaf(w[k], e, o[k] * f);
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const long long at_row = (long long)(sp.row0 + local) * g.a.Hq + sp.hk * g.a.G + r - tok * g.a.G;
    *reinterpret_cast<uint4*>(g.a.o + at_row * D + q * 8) =
        make_uint4(pack2<F16>(o[0] * inv, o[1] * inv), pack2<F16>(o[2] * inv, o[3] * inv),
                   pack2<F16>(o[4] * inv, o[5] * inv), pack2<F16>(o[6] * inv, o[7] * inv));
    if (q == 0 && g.a.lse) g.a.lse[at_row] = l == 0.f ? -INFINITY : (m + (log2f(l) - lift<F16>())) * 0.6931471805599453f;
  }
}

template <bool F16, int D>
cudaError_t launch_one(ChunkArgs& g, int grid, int dev, cudaStream_t st) {
  constexpr int smem = chunk_smem<D>();
  static std::mutex mu;
  static bool configured[64] = {};
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!configured[dev]) {
      cudaError_t e = cudaFuncSetAttribute(chunk_kernel<F16, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      cudaFuncAttributes fa;
      if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, chunk_kernel<F16, D>);
      // the register shares add up to what the block is launched with
      if (e == cudaSuccess && fa.numRegs < kLaunchRegs) e = cudaErrorInvalidConfiguration;
      if (e != cudaSuccess) {
        cudaGetLastError();
        return e;
      }
      configured[dev] = true;
    }
  }
  const cudaError_t e = launch_pdl(K_ATTN_CHUNK, chunk_kernel<F16, D>, dim3(grid), kChunkThreads, smem, st, g);
  if (e != cudaSuccess || !g.combine) return e;
  return launch_pdl(K_ATTN_COMBINE, combine_kernel<F16, D>, dim3(2 * grid), 128, 0, st, g, grid);
}

int chunk_grid(int* dev) {
  int sms = 0;
  if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, *dev);
  return sms < 1 ? 1 : sms < kMaxGrid ? sms : kMaxGrid;
}

}  // namespace

bool chunk_supported(int D, int page, int Hkv, int G, int B, int n_rows, int max_pages, float scale) {
  if (G < 1 || G > 128) return false;
  // the list of all units' blocks counts in int32
  const long long units = (n_rows / (2 * (128 / G)) + (long long)B) * Hkv, blocks = (long long)max_pages * page / kBlk + 2;
  if (units * blocks >= (1LL << 31)) return false;
  // a scale above zero: the largest product is then the largest score
  return (D == 64 || D == 128) && page >= 8 && (page & (page - 1)) == 0 && scale > 0.f && encode_fn();
}

size_t chunk_ws_bytes(int D) {
  return align256((size_t)2 * kMaxGrid * 2 * 128 * (D + 2) * 4 + kMaxGrid * sizeof(Split));
}

cudaError_t launch_attn_chunk(const Cache& c, const Rows& r, const Attn& a, bool f16, int32_t* status, int32_t* sync,
                              void* scratch, cudaStream_t st) {
  int dev = 0;
  const int grid = chunk_grid(&dev);
  if (!grid) return cudaErrorInvalidDevice;
  ChunkArgs g;
  g.c = c;
  g.r = r;
  g.a = a;
  g.tq = 128 / a.G;
  g.logpage = 0;
  while ((1 << g.logpage) < c.page) ++g.logpage;
  g.logP = g.logpage < 7 ? g.logpage : 7;
  g.cnt = sync;
  g.part = static_cast<float*>(scratch);
  g.pml = g.part + (size_t)2 * kMaxGrid * 2 * 128 * c.D;
  g.split = reinterpret_cast<Split*>(g.pml + (size_t)2 * kMaxGrid * 2 * 256);
  g.status = status;
  if (!pool_maps_2d(c, &g.tm_k, &g.tm_v, 1 << g.logP) || !query_map(a, c.D, r.n_rows, g.tq, &g.tm_q))
    return cudaErrorInvalidValue;
  for (g.b0 = 0; g.b0 < r.B; g.b0 += kChunkSeqs) {
    g.nseq = r.B - g.b0 < kChunkSeqs ? r.B - g.b0 : kChunkSeqs;
    // The kernel that joins many parts follows only where a unit can lie in many
    // CTAs (either way is right). Not where one sequence's units fill the GPU:
    // the longest is at most about twice the mean. And not where the table or the
    // window leaves a unit few blocks: a launch less is 2 us of 15 for 40 rows.
    // Joined there, 38 parts of 40 rows over 30,000 tokens are 31 us; 8 parts of
    // 4,000 tokens 23 us (35 by the last CTA), 256 rows over 16,000 69 (79). The host
    // knows the table's width and not the lengths: 40 rows of a short sequence take
    // 9.7 us with a table for 64 tokens and 11.8 with one for 32,768.
    const bool full_gpu = r.B == 1 && 3LL * ((r.n_rows + 2 * g.tq - 1) / (2 * g.tq)) * c.Hkv >= 2LL * grid;
    long long seen = (long long)c.max_pages * c.page;
    const long long win = (long long)a.window + 2 * g.tq - 1;
    if (a.window > 0 && win + a.n_sink + kBlk < seen) seen = win + a.n_sink + kBlk;  // both ends inside blocks
    g.combine = !full_gpu && (seen + kBlk - 1) / kBlk + 1 > kFewBlocks;
    cudaError_t e;
    if (c.D == 128) e = f16 ? launch_one<true, 128>(g, grid, dev, st) : launch_one<false, 128>(g, grid, dev, st);
    else e = f16 ? launch_one<true, 64>(g, grid, dev, st) : launch_one<false, 64>(g, grid, dev, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace kv
}  // namespace moe
