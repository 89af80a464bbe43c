// Linear attention of prompt chunks on the 5th-generation tensor cores
// (include/moe_block.h), head sizes 64 and 128.
//
// Blocks of 128 tokens. With G_i the sum of the logarithms of the decays of a
// block's tokens up to i, G the sum of all of them, and S the state before it:
//   o_i = scale (e^G_i q_i S + sum_{j <= i} e^(G_i - G_j) (q_i . k_j) v_j)
//   S'  = e^G S + sum_j (e^(G - G_j) k_j) v_j^T
// Three products, accumulators in tensor memory:
//   A = Q K^T      U = K'^T V      O = [A o D | Q'] [V ; S]
// K' = e^(G - G_j) k_j, Q' = e^G_i q_i, D_ij = e^(G_i - G_j) for j <= i, else 0. Where
// e^-G is no more than 2^32 (2^8 in fp16), Q' is q itself, D_ij is e^-G_j and the
// factor e^G_i is left to the output: Q' is then exact where the state matters most.
// K'^T, A o D and Q' are first operands in tensor memory, which leaves shared memory to the
// tiles that TMA brings, two of K and of V. U does not depend on S, so the blocks of a
// sequence wait for one another only in S' = e^G S + U, in registers.
//
// Rounding. The state is fp32 throughout: in bf16 K' enters U as three values that
// add up to its fp32 exactly, in fp16 as two (its rounding and the rest, 2^-22 of
// it), and U is a fresh sum each block. (Two values of bf16 left the state off by
// 2.4e-6.) S, A o D and a scaled Q', which only o sees, are rounded once to the type (half a
// step each, as o itself is). In fp16, whose range is narrow and whose step is fixed
// below 2^-14, K' and S are scaled by a power of two per block and a row of A o D and
// Q' by one of its own, which bring the largest magnitude to 2^13 and are undone in
// fp32: the smallest values are then off by up to 2^-38 of the largest. (Of the largest
// |k|, not the largest decayed one: a head that forgets within a few tokens keeps fewer bits
// of a key that has decayed to 2^-14 or less when the block ends.) Sums of
// logarithms are pairs of fp32 values, so that G_i - G_j is right next to large |G|
// (in fp64 a block's sums took 5,000 cycles).
//
// Work. An item is a sequence and a v head, by a cluster of 1 to 8 CTAs that have
// consecutive parts of its blocks. With more than one, each first sums up its own
// part's state (K and V only), the parts meet through the cluster's shared memory
// (S at a part's start: the initial state and the parts before it), and each then
// goes through its part. So a long prompt of few heads fills the GPU in one launch
// and without a workspace. Items are started longest first.
//
// Warps. 0-3: A o D and Q' (a thread is a token); 4-7: the state (a thread is a row of
// it); 8-11: the output; 12-15 and 16-19: K', each group 32 tokens of every 64;
// 20 and 23: issue the products, those of A and O and those of U (a product takes a
// warp 20 instructions, more time than the tensor cores need for it); 21: TMA; 22:
// decays, two blocks ahead.
//
// Measured, back to back in a graph, 16 k heads and 32 v heads of [128][128], bf16: a
// prompt of 2,048 tokens 40 us (floor 8.1 us of bytes: the time is latency, start,
// two passes over a part's four blocks, the exchange); eight ragged prompts of
// up to 4,001 tokens 161 us (532 MB, floor 78.3 us; tensor pipe 34 % busy, a
// block of 128 tokens 7,500 cycles of products, conversions and the waits that tie
// them). An item's fixed cost is about 11 us, which is why few rows go row by row; a
// short sequence of a call that comes here beside long ones pays it too (64 sequences of
// one row 194 us, where a decode window of them takes 44). The roles share 80 registers a
// thread: 112 bytes are spilled by stores and 336 by loads of the code of 128 x 128 in bf16
// (up to 156 / 468 in the others), by which role is not known. The
// chain of a block: A, its conversion by the warp with the last 32 tokens (which has
// four pieces of A, the first warp one), O, the next A, which takes the place that O reads. Tried on
// the eight prompts (159 us that time): the output's warps converting half of A 189 (they
// come late from the output), Q' taken from shared memory where it is q itself 174 (Q's tile
// is free later), V before Q 162.
#include <cuda.h>

#include <atomic>

#include "block_internal.h"
#include "kv_common.cuh"
#include "kv_tma.h"
#include "linear_common.cuh"
#include "moe_tc.cuh"
#include "packed.cuh"

namespace moe {
namespace block {

using namespace tc;

namespace {

constexpr int kBlk = 128;               // tokens per block
constexpr int kThreads = 768;
constexpr int kRegsScore = 72, kRegsState = 168, kRegsOut = 64, kRegsKey = 64, kRegsRest = 48;  // (KEY twice) at most 6 x 80 together
constexpr uint32_t kTries = 1u << 22;   // of a wait, each up to a microsecond long
constexpr int kHalf = kBlk * 128;       // bytes of 128 rows of 64 values
constexpr int kTile = 2 * kHalf;
constexpr int kPitch = 144;             // bytes per row of a warp's output buffer (64 values and a pad)
constexpr int kSmem = 1024 + 6 * kTile + 4 * 32 * kPitch;  // Q, two of K and of V, S; outputs
constexpr int kSortB = 512;             // sequences that are put in order of their length
constexpr int kKeyCols = 48;            // tensor memory of a group of K's warps: three values of 32 tokens
constexpr int kMostParts = 8;
constexpr int kAhead = 2;               // blocks that are fetched into L2 ahead

struct ChunkArgs {
  CUtensorMap tm_q, tm_k, tm_v;
  Linear a;
  kv::Rows r;
  int parts;  // CTAs of a cluster
};

// What the decays of a block come to.
struct alignas(16) Decays {
  float gh[kBlk], gl[kBlk];  // -G_j / ln 2 as two values
  float k[kBlk];      // e^(G - G_j)
  float q[kBlk];      // e^G_i
  float col[kBlk];    // weak: e^-G_j; else e^(G_p - G_j), p the last of j's 32 tokens
  bool weak;          // whether e^-G is within reach (kWeak)
  float2 all;         // e^G (decay_of)
};

__device__ __forceinline__ void ldmatrix4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
// 16 lanes x 16 columns: r[2 i] column 4 i + t % 4 of lane t / 4, r[2 i + 1] of lane 8 + t / 4.
__device__ __forceinline__ void tc_st_16x16(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ uint4 ld_s128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer(uint32_t a, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 peer_f128(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float peer_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void prefetch_3d(const void* tmap, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(tmap), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
// Up to which sum of a block's decays (in powers of two) its tokens are weighted by
// e^-G_j alone.
template <bool F16>
__device__ constexpr float kWeak() { return F16 ? 8.f : 32.f; }
// 2^e as a float, e in the normal range
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// The exponent that brings a largest magnitude m (>= 0) to [2^13, 2^14); bounded so
// that it and its negative are normal numbers.
__device__ __forceinline__ int lift_of(float m) {
  const int e = 13 - ((__float_as_int(m) >> 23) - 127);
  return max(-100, min(100, e));
}

template <bool F16, int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1) linear_chunk_kernel(const __grid_constant__ ChunkArgs p) {
  constexpr int HK = DK / 64, HV = DV / 64;
  constexpr int kTerms = F16 ? 2 : 3;  // values that stand for a K'
  extern __shared__ __align__(1024) uint8_t smem_linear[];
  __shared__ __align__(16) Decays s_dec[2];
  __shared__ __align__(8) uint64_t s_bar[40];
  __shared__ float s_row[2][kBlk];           // by block: what makes a row of O the output
  __shared__ int s_state_up[2];              // log2 of what S is scaled by
  __shared__ float s_key_down[2];            // what undoes the scale of K'
  __shared__ float s_max[4];
  __shared__ uint32_t s_kmax[8];
  __shared__ float s_part;                   // e^(sum of the part's logarithms)
  __shared__ uint32_t s_tmem;
  __shared__ int s_b;

  const Linear& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sq = (smem_u32(smem_linear) + 1023u) & ~1023u;
  const uint32_t sk = sq + kTile, sv = sk + 2 * kTile, ss = sv + 2 * kTile, so = ss + kTile;
  const uint32_t sums = sk, start = sv;  // between the passes: this part's sum, the state at its start (K's tiles, V's)
  const uint32_t bar = smem_u32(s_bar);
  // (by block parity where there are two)
  const uint32_t q_full = bar, q_empty = bar + 8, k_full = bar + 16, k_empty = bar + 32, v_full = bar + 48, v_ready = bar + 64;
  const uint32_t v_empty = bar + 80, a_full = bar + 96, p_ready = bar + 112;
  const uint32_t s_ready = bar + 128, kt_full = bar + 256, kt_empty = bar + 288, u_full = bar + 168, u_free = bar + 176;
  const uint32_t o_full = bar + 184, o_free = bar + 192, g_full = bar + 200, g_empty = bar + 216;
  const uint32_t drained = bar + 240, u_drained = bar + 248;
  if (tid == 0) {
    mbar_init(q_full, 1); mbar_init(q_empty, 5);
#pragma unroll 1
    for (int i = 0; i < 16; i += 8) {
      mbar_init(k_full + i, 1); mbar_init(k_empty + i, 9);
      mbar_init(v_full + i, 1); mbar_init(v_empty + i, 2);
      mbar_init(kt_full + i, 4); mbar_init(kt_empty + i, 1);
      mbar_init(g_full + i, 1); mbar_init(g_empty + i, 16);
    }
    mbar_init(v_ready, 4); mbar_init(a_full, 1); mbar_init(p_ready, 4);
    mbar_init(s_ready, 4); mbar_init(u_full, 1); mbar_init(u_free, 4);
    mbar_init(o_full, 1); mbar_init(o_free, 4);
    mbar_init(drained, 1); mbar_init(u_drained, 1);
    fence_barrier_init();
  }
  if (tid == 32 * 21) {
    prefetch_tensormap(&p.tm_q);
    prefetch_tensormap(&p.tm_k);
    prefetch_tensormap(&p.tm_v);
  }
  griddep_wait();
  griddep_launch_dependents();

  // ---- the item: its sequence (the longest ones first) and head
  const int parts = p.parts, part = parts > 1 ? (int)cluster_rank() : 0;
  const int item = blockIdx.x / parts, h = item % a.Hv, hk = h / (a.Hv / a.Hk);
  if (p.r.row_start && p.r.B > 1 && p.r.B <= kSortB) {
    int* len = reinterpret_cast<int*>(s_dec);
    const int n = tid < p.r.B ? load_span(a, p.r, tid).n : -1;
    if (tid < kSortB) len[tid] = n;
    __syncthreads();
    if (tid < p.r.B) {
      int place = 0;
#pragma unroll 1
      for (int i = 0; i < p.r.B; ++i) place += len[i] > n || (len[i] == n && i < tid) ? 1 : 0;
      if (place == item / a.Hv) s_b = tid;
    }
  } else if (tid == 0) {
    s_b = item / a.Hv;
  }
  __syncthreads();
  const int b = s_b;
  const Span s = load_span(a, p.r, b);
  if (s.n == 0) return;  // (as the other CTAs of the cluster)
  if (!span_allowed(a, p.r, b, s, h == 0 && part == 0)) {
#pragma unroll 1
    for (int i = part * kThreads + tid; i < s.n * (DV / 8); i += parts * kThreads)
      *reinterpret_cast<uint4*>(a.o + ((long long)(s.row0 + i / (DV / 8)) * a.Hv + h) * DV + i % (DV / 8) * 8) =
          make_uint4(0, 0, 0, 0);
    return;
  }
  const int blocks = (s.n + kBlk - 1) / kBlk, per = (blocks + parts - 1) / parts;
  const int first = min(part * per, blocks), n2 = min(blocks - first, per);   // this CTA's blocks
  const bool last = n2 > 0 && first + n2 == blocks;                           // with the sequence's last one
  const int n1 = parts > 1 && !last ? n2 : 0;                                 // summed up before
  // step i: block first + i of the part's own sum for i < n1, then of the pass proper

  if (warp == 20) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t ta = 0, to = ta + 128, tu = ta + 256, tk = ta + 384;  // (all 512 columns are allocated) A, then A o D and Q'; O; U; K'

  // A wait of kTries of up to a microsecond each; after an expired one a warp goes on
  // without waiting (the status word says so). Few instructions: there are many, and
  // the roles' code competes for the instruction caches.
  uint32_t tries = kTries;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    uint32_t left;
    asm volatile(
        "{\n .reg .pred p;\n .reg .u32 n;\n mov.u32 n, %3;\n"
        "W:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n @p bra D;\n"
        " sub.u32 n, n, 1;\n setp.ne.u32 p, n, 0;\n @p bra W;\n"
        "D:\n mov.u32 %0, n;\n}"
        : "=r"(left)
        : "r"(bar), "r"(parity), "r"(tries)
        : "memory");
    tries = left ? tries : 1u;
    __syncwarp();
  };
  auto arrive = [&](uint32_t bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  // Every product of this warp has ended before tensor memory is given back and the CTA
  // ends, also where the warp went on without waiting: with a wait's full time.
  auto drain = [&](uint32_t bar, uint32_t lead) {
    const bool gave_up = tries == 1;
    tries = kTries;
    tc_commit_el(bar, lead);
    wait(bar, 0);
    if (gave_up) tries = 1;
  };
  // Between the two passes: the parts' sums are there; the state at this part's start is
  // put together from those before it by all warps (a quarter of them took four times
  // as long: the cluster's shared memory answers late); `take` reads it; all have read.
  auto between = [&](auto take) {
    if (parts == 1) return;
    __syncwarp();
    cluster_sync();
    if (part > 0 && n2 > 0)
#pragma unroll 2
      for (int i = tid; i < DK * DV / 4; i += kThreads) {
        float4 x = peer_f128(peer(sums, 0) + i * 16);
#pragma unroll 1
        for (int r = 1; r < part; ++r) {
          const float4 y = peer_f128(peer(sums, r) + i * 16);
          const float e = peer_f32(peer(smem_u32(&s_part), r));
          x = make_float4(fmaf(x.x, e, y.x), fmaf(x.y, e, y.y), fmaf(x.z, e, y.z), fmaf(x.w, e, y.w));
        }
        st_s128(start + i * 16, __float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(x.z), __float_as_uint(x.w));
      }
    __syncthreads();
    take();
    __syncwarp();
    cluster_sync();
  };
  auto meet = [&] { between([] {}); };
  // the block of step i, and its token rows that are the sequence's
  const auto block_of = [&](int i) { return first + (i < n1 ? i : i - n1); };

  if (warp >= 20) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == 21) {
      // ================= TMA =================
      const uint32_t lead = elect_lane();
      auto load = [&](uint32_t dst, const CUtensorMap* m, int halves, int head, int row, uint32_t full) {
        if (lead) {
          mbar_expect_tx(full, (uint32_t)(halves * kHalf));
#pragma unroll 1
          for (int i = 0; i < halves; ++i) tma_load_3d(dst + i * kHalf, m, i * 64, head, row, full);
        }
        __syncwarp();
      };
      // the blocks after those come into L2 while the tiles are still in use
      auto ahead = [&](int c) {
        if (lead && c < n2) {
          const int row = s.row0 + (first + c) * kBlk;
#pragma unroll 1
          for (int x = 0; x < HK; ++x) {
            prefetch_3d(&p.tm_k, x * 64, hk, row);
            prefetch_3d(&p.tm_q, x * 64, hk, row);
          }
#pragma unroll 1
          for (int x = 0; x < HV; ++x) prefetch_3d(&p.tm_v, x * 64, h, row);
        }
        __syncwarp();
      };
#pragma unroll 1
      for (int c = 1; c < kAhead; ++c) ahead(c);
      auto step = [&](int i, bool full) {
        ahead(i + kAhead);
        const int row = s.row0 + block_of(i) * kBlk, x = i & 1, free = ((i >> 1) + 1) & 1;
        wait(k_empty + 8 * x, free);
        load(sk + x * kTile, &p.tm_k, HK, hk, row, k_full + 8 * x);
        if (full) {
          wait(q_empty, (i - n1 + 1) & 1);
          load(sq, &p.tm_q, HK, hk, row, q_full);
        }
        wait(v_empty + 8 * x, free);
        load(sv + x * kTile, &p.tm_v, HV, h, row, v_full + 8 * x);
      };
#pragma unroll 1
      for (int i = 0; i < n1; ++i) step(i, false);
      meet();
      fence_proxy_async_shared();
#pragma unroll 1
      for (int i = 0; i < n2; ++i) step(n1 + i, true);
      // no copy is under way when the CTA ends, also where a warp went on without
      // waiting: the last fill of every tile
      const bool gave_up = tries == 1;
      tries = kTries;
      const int n = n1 + n2;
      if (n2 > 0) wait(q_full, (n2 + 1) & 1);
#pragma unroll 1
      for (int x = 0; x < 2; ++x)
        if (n > x) {
          const int fills = (n - x + 1) >> 1;
          wait(k_full + 8 * x, (fills + 1) & 1);
          wait(v_full + 8 * x, (fills + 1) & 1);
        }
      if (gave_up) tries = 1;
    } else if (warp == 20) {
      // ================= products: A and O =================
      const uint32_t lead = elect_lane();
      const uint32_t id_a = idesc_16(F16, 128, kBlk, false), id_o = idesc_16(F16, 128, DV, true);
      const uint64_t qd = sdesc_sw128(sq), kd = sdesc_sw128(sk), vd = sdesc_sw128_n(sv, kHalf), sd = sdesc_sw128_n(ss, DK * 128);
#pragma unroll 1
      for (int i = 0; i < n1; ++i) {  // (K and V of the first pass are not this warp's)
        const int x = i & 1;
        wait(k_full + 8 * x, (i >> 1) & 1);
        arrive(k_empty + 8 * x);
        wait(v_full + 8 * x, (i >> 1) & 1);
        arrive(v_empty + 8 * x);
      }
      meet();
#pragma unroll 1
      for (int c = 0; c < n2; ++c) {
        const int i = n1 + c, x = i & 1;
        wait(k_full + 8 * x, (i >> 1) & 1);
        wait(q_full, c & 1);
        tc_fence_after();
        const uint64_t k = kd + (uint32_t)(x * kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) {
          const uint32_t o = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
          tc_mma_el(ta, qd + o, k + o, id_a, kk > 0, lead);
        }
        tc_commit_el(a_full, lead);
        tc_commit_el(q_empty, lead);
        tc_commit_el(k_empty + 8 * x, lead);
        wait(v_full + 8 * x, (i >> 1) & 1);
        if (s.n - block_of(i) * kBlk < kBlk) wait(v_ready, 0);  // (the sequence's last block)
        wait(s_ready, c & 1);
        wait(o_free, (c + 1) & 1);
        wait(p_ready, c & 1);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) tc_mma_ts_el(to, ta + 64 + kk * 8, sd + kk * 128, id_o, kk > 0, lead);
        const uint64_t v = vd + (uint32_t)(x * kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < kBlk / 16; ++kk) tc_mma_ts_el(to, ta + kk * 8, v + kk * 128, id_o, 1, lead);
        tc_commit_el(o_full, lead);
        tc_commit_el(v_empty + 8 * x, lead);
      }
      drain(drained, lead);
    } else if (warp == 23) {
      // ================= products: U =================
      const uint32_t lead = elect_lane(), id_o = idesc_16(F16, 128, DV, true);
      const uint64_t vd = sdesc_sw128_n(sv, kHalf);
#pragma unroll 1
      for (int i = 0; i < n1 + n2; ++i) {
        if (i == n1) {
          meet();
        }
        const int x = i & 1;
        wait(v_full + 8 * x, (i >> 1) & 1);
        if (s.n - block_of(i) * kBlk < kBlk) wait(v_ready, 0);
        wait(u_free, (i + 1) & 1);
        const uint64_t v = vd + (uint32_t)(x * kTile >> 4);
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {  // 32 tokens, by the groups of warps in turn
          const int y = j & 1;
          wait(kt_full + 8 * y, j >> 1);  // (two uses a step)
          tc_fence_after();
#pragma unroll
          for (int z = 0; z < kTerms; ++z)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
              tc_mma_ts_el(tu, tk + y * kKeyCols + z * 16 + kk * 8, v + (uint32_t)(j * 256) + kk * 128, id_o, j > 0 || z > 0 || kk > 0, lead);
          tc_commit_el(kt_empty + 8 * y, lead);
        }
        tc_commit_el(u_full, lead);
        tc_commit_el(v_empty + 8 * x, lead);
      }
      if (n2 == 0) {
        meet();
      }
      drain(u_drained, lead);
    } else {
      // ================= decays =================
      float next[4];
      const auto fetch = [&](int i) {
        const int t0 = block_of(i) * kBlk + lane * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) next[j] = t0 + j < s.n ? a.g[(s.row0 + t0 + j) * a.g_stride + h] : 0.f;
      };
      if (n1 + n2 > 0) fetch(0);
#pragma unroll 1
      for (int i = 0; i < n1 + n2; ++i) {
        if (i == n1) {
          meet();
        }
        const int slot = i & 1;
        // sums of logarithms to base 2 as pairs of fp32 values
        FF g[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = bounded_g(next[j]), hi = x * 0x1.715476p+0f;
          g[j] = ff_fast_two_sum(hi, fmaf(x, 0x1.4ae0cp-26f, fmaf(x, 0x1.715476p+0f, -hi)));
          if (j) g[j] = ff_add(g[j - 1], g[j]);
        }
        if (i + 1 < n1 + n2) fetch(i + 1);
        FF x = g[3];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const FF y = {__shfl_up_sync(0xffffffffu, x.h, o), __shfl_up_sync(0xffffffffu, x.l, o)};
          if (lane >= o) x = ff_add(y, x);
        }
        const FF total = {__shfl_sync(0xffffffffu, x.h, 31), __shfl_sync(0xffffffffu, x.l, 31)};
        FF before = {__shfl_up_sync(0xffffffffu, x.h, 1), __shfl_up_sync(0xffffffffu, x.l, 1)};
        if (lane == 0) before = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j] = ff_add(before, g[j]);
        const FF end = {__shfl_sync(0xffffffffu, g[3].h, lane | 7), __shfl_sync(0xffffffffu, g[3].l, lane | 7)};
        const float2 all = decay_of(total.h * 0x1.62e43p-1f + fmaf(total.l, 0x1.62e43p-1f, total.h * -0x1.05c61p-29f));
        const bool weak = total.h > -kWeak<F16>();
        wait(g_empty + 8 * slot, ((i >> 1) + 1) & 1);
        Decays& d = s_dec[slot];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          d.gh[lane * 4 + j] = -g[j].h;
          d.gl[lane * 4 + j] = -g[j].l;
          d.k[lane * 4 + j] = kv::ex2((total.h - g[j].h) + (total.l - g[j].l));
          d.q[lane * 4 + j] = kv::ex2(g[j].h + g[j].l);
          d.col[lane * 4 + j] = weak ? kv::ex2(-g[j].h - g[j].l) : kv::ex2((end.h - g[j].h) + (end.l - g[j].l));
        }
        if (lane == 0) {
          d.all = all;
          d.weak = weak;
        }
        arrive(g_full + 8 * slot);
      }
      if (n2 == 0) {
        meet();
      }
    }
  } else if (warp < 4) {
    // ================= A o D: a thread is a token's row =================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsScore));
#pragma unroll 1
    for (int i = 0; i < n1; ++i) {
      wait(g_full + 8 * (i & 1), (i >> 1) & 1);
      arrive(g_empty + 8 * (i & 1));
    }
    meet();
    const uint32_t tr = ta + ((uint32_t)(warp * 32) << 16);
#pragma unroll 1
    for (int c = 0; c < n2; ++c) {
      const int i = n1 + c;
      const Decays& d = s_dec[i & 1];
      const auto query = [&](int j) { return ld_s128(sq + (j >> 3) * kHalf + tid * 128 + (((j & 7) ^ (tid & 7)) << 4)); };
      wait(g_full + 8 * (i & 1), (i >> 1) & 1);
      wait(q_full, c & 1);
      const float gh = -d.gh[tid], gl = -d.gl[tid];
      const bool weak = d.weak;
      // of A o D; of Q' (weak: it is exact); of the output
      float up = 1.f, fq = weak ? 1.f : d.q[tid], out = weak ? d.q[tid] * a.scale : a.scale;
      uint32_t mq = 0;
      if constexpr (F16)
#pragma unroll 4
        for (int j = 0; j < DK / 8; ++j) {
          const uint4 v = query(j);
          mq = __vmaxu2(__vmaxu2(mq, __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu)), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
        }
      wait(a_full, c & 1);
      tc_fence_after();
      if constexpr (F16) {  // the largest of the row's weighted |q . k| and of its Q' (times S's scale) to about 2^13
        float m = 0.f;
#pragma unroll 1
        for (int j = 0; j <= warp; ++j) {
          uint32_t x[32];
          tc_ld32(tr + j * 32, x);
          tc_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (j < warp || e <= lane) m = fmaxf(m, fabsf(__uint_as_float(x[e])));
        }
        if (weak) m *= d.col[tid];
        wait(s_ready, c & 1);
        mq = min(max(mq & 0xffffu, mq >> 16), 0x7bffu);
        const int up_s = s_state_up[c & 1], e = max(-100, min(lift_of(m), lift_of(kv::unpack2<true>(mq).x * fq) + up_s));
        up = pow2(e);
        fq = e - up_s < -126 ? 0.f : fq * pow2(min(e - up_s, 127));
        out *= pow2(-e);
      }
      s_row[c & 1][tid] = out;
      // (rolled loops: with all roles' loops unrolled their code did not stay in the
      // instruction cache, and a block took twice as long)
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        uint32_t pk[16], x[32];
        if (j > warp) {
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = 0u;
        } else {
          tc_ld32(tr + j * 32, x);
          tc_ld_wait();
          if (weak || j < warp) {
            // weak: e^G_i is left to the output. Else 32 tokens before all of the warp's,
            // p the last of them: D_ij = e^(G_i - G_p) e^(G_p - G_j), neither above 1
            const float f = weak ? up : kv::ex2((gh + d.gh[j * 32 + 31]) + (gl + d.gl[j * 32 + 31])) * up;
            const float4* col = reinterpret_cast<const float4*>(d.col + j * 32);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 w = col[e];
              const float2 d0 = mul2(make_float2(w.x, w.y), make_float2(f, f)), d1 = mul2(make_float2(w.z, w.w), make_float2(f, f));
              const float2 p0 = mul2(d0, make_float2(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1])));
              const float2 p1 = mul2(d1, make_float2(__uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3])));
              pk[2 * e] = kv::pack2<F16>(p0.x, p0.y);
              pk[2 * e + 1] = kv::pack2<F16>(p1.x, p1.y);
            }
          } else {
            const float4* nh = reinterpret_cast<const float4*>(d.gh + j * 32);
            const float4* nl = reinterpret_cast<const float4*>(d.gl + j * 32);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 a4 = nh[e], b4 = nl[e];
              const float2 t0 = add2(add2(make_float2(gh, gh), make_float2(a4.x, a4.y)), add2(make_float2(gl, gl), make_float2(b4.x, b4.y)));
              const float2 t1 = add2(add2(make_float2(gh, gh), make_float2(a4.z, a4.w)), add2(make_float2(gl, gl), make_float2(b4.z, b4.w)));
              const float2 d0 = mul2(make_float2(kv::ex2(t0.x), kv::ex2(t0.y)), make_float2(up, up));
              const float2 d1 = mul2(make_float2(kv::ex2(t1.x), kv::ex2(t1.y)), make_float2(up, up));
              const float2 p0 = mul2(d0, make_float2(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1])));
              const float2 p1 = mul2(d1, make_float2(__uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3])));
              pk[2 * e] = kv::pack2<F16>(p0.x, p0.y);
              pk[2 * e + 1] = kv::pack2<F16>(p1.x, p1.y);
            }
          }
          if (j == warp)  // later tokens (what stands there may be NaN) are cleared as bits
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] &= (2 * e <= lane ? 0xffffu : 0u) | (2 * e + 1 <= lane ? 0xffff0000u : 0u);
        }
        tc_st16(tr + j * 16, pk);
      }
      arrive(g_empty + 8 * (i & 1));
      // Q' in the columns from 64 on, which the row has read
#pragma unroll 1
      for (int j = 0; j < DK / 32; ++j) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 v = query(j * 4 + e);
          w[4 * e] = v.x; w[4 * e + 1] = v.y; w[4 * e + 2] = v.z; w[4 * e + 3] = v.w;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 x = mul2(kv::unpack2<F16>(w[e]), make_float2(fq, fq));
          w[e] = kv::pack2<F16>(x.x, x.y);
        }
        tc_st16(tr + 64 + j * 16, w);
      }
      arrive(q_empty);
      tc_st_wait();
      tc_fence_before();
      arrive(p_ready);
    }
  } else if (warp < 8) {
    // ================= the state: a thread is a row =================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsState));
    const int row = tid - 128;
    const bool held = row < DK;  // (head size 64: two of the warps only take part)
    const uint32_t tr = tu + ((uint32_t)((warp & 3) * 32) << 16);
    float4* state = reinterpret_cast<float4*>(a.state + ((long long)s.slot * a.Hv + h) * DK * DV);
    float2 S[DV / 2];
    // The state from or to memory, 64 columns at a time through S's tile, so that
    // memory is touched along rows (16 pieces of 16 bytes each, in places that keep a
    // warp's rows in different banks). Coming in, all of a thread's pieces are under
    // way together.
    const int piece_row = row >> 4, piece = row & 15;
    const auto place = [&](int r, int j) { return ss + r * 256 + ((j ^ (r & 15)) << 4); };
    auto put = [&](int i, uint32_t at) {  // S[2 i], S[2 i + 1]
      st_s128(at, __float_as_uint(S[2 * i].x), __float_as_uint(S[2 * i].y), __float_as_uint(S[2 * i + 1].x), __float_as_uint(S[2 * i + 1].y));
    };
    auto get = [&](int i, uint32_t at) {
      const uint4 f = ld_s128(at);
      S[2 * i] = make_float2(__uint_as_float(f.x), __uint_as_float(f.y));
      S[2 * i + 1] = make_float2(__uint_as_float(f.z), __uint_as_float(f.w));
    };
    auto meet_state = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    auto bring = [&] {
#pragma unroll
      for (int i = 0; i < HV * DK / 8; ++i) {  // (DK / 8 <= 16: a thread's part of 64 columns)
        const int x = i / (DK / 8), r = i % (DK / 8) * 8 + piece_row, at = x * 16 + i % (DK / 8);
        const float4 f = state[r * (DV / 4) + x * 16 + piece];
        S[2 * at] = make_float2(f.x, f.y);
        S[2 * at + 1] = make_float2(f.z, f.w);
      }
#pragma unroll
      for (int x = 0; x < HV; ++x) {
        meet_state();
#pragma unroll
        for (int i = 0; i < DK / 8; ++i) put(x * 16 + i, place(i * 8 + piece_row, piece));
        meet_state();
        if (held)
#pragma unroll
          for (int j = 0; j < 16; ++j) get(x * 16 + j, place(row, j));
      }
      meet_state();  // S's tile is free for S
    };
    auto leave = [&] {
#pragma unroll
      for (int x = 0; x < HV; ++x) {
        meet_state();
        if (held)
#pragma unroll
          for (int j = 0; j < 16; ++j) put(x * 16 + j, place(row, j));
        meet_state();
#pragma unroll
        for (int i = 0; i < DK / 8; ++i) {
          const int r = i * 8 + piece_row;
          const uint4 f = ld_s128(place(r, piece));
          state[r * (DV / 4) + x * 16 + piece] = make_float4(__uint_as_float(f.x), __uint_as_float(f.y), __uint_as_float(f.z), __uint_as_float(f.w));
        }
      }
    };
    auto step = [&](int i, float* decay) {  // S <- e^G S + U
      wait(g_full + 8 * (i & 1), (i >> 1) & 1);
      const float2 e = s_dec[i & 1].all;
      if (decay) *decay = fmaf(*decay, e.x, *decay * e.y);
      wait(u_full, i & 1);
      tc_fence_after();
      const float up = F16 ? s_key_down[i & 1] : 1.f;
#pragma unroll
      for (int j = 0; j < DV / 32; ++j) {
        uint32_t x[32];
        tc_ld32(tr + j * 32, x);
        tc_ld_wait();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          float2 u = make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1]));
          if constexpr (F16) u = mul2(u, make_float2(up, up));
          S[j * 16 + c] = fma2(S[j * 16 + c], make_float2(e.x, e.x), fma2(S[j * 16 + c], make_float2(e.y, e.y), u));
        }
      }
      tc_fence_before();
      arrive(u_free);
      arrive(g_empty + 8 * (i & 1));
    };
    if (parts > 1) {
      float decay = 1.f;
      if (n1 > 0 && part == 0) {
        bring();
      } else {
#pragma unroll
        for (int j = 0; j < DV / 2; ++j) S[j] = make_float2(0.f, 0.f);
      }
#pragma unroll 1
      for (int i = 0; i < n1; ++i) step(i, &decay);
      if (n1 > 0) {  // columns 4 j of all rows side by side
        if (held)
#pragma unroll
          for (int j = 0; j < DV / 4; ++j) put(j, sums + (j * DK + row) * 16);
        if (row == 0) s_part = decay;
      }
      // The first part reads the initial state again here, before the cluster's second
      // barrier: behind it the part with the sequence's end may write the final one in
      // its place at any time. (A pointer that is either memory's or shared memory's: the
      // state by way of `start` as well was a loop more in every role's code, and the eight
      // prompts took 2 % longer.)
      between([&] {
        const float4* from = part == 0 ? state + row * (DV / 4) : reinterpret_cast<const float4*>(smem_linear + (start - smem_u32(smem_linear))) + row;
        const int pitch = part == 0 ? 1 : DK;
        if (n2 > 0 && held)
#pragma unroll
          for (int j = 0; j < DV / 4; ++j) {
            const float4 f = from[j * pitch];
            S[2 * j] = make_float2(f.x, f.y);
            S[2 * j + 1] = make_float2(f.z, f.w);
          }
      });
    }
    if (parts == 1) bring();
#pragma unroll 1
    for (int c = 0; c < n2; ++c) {
      float up = 1.f;
      if constexpr (F16) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < DV / 2; ++j) m = fmaxf(m, held ? fmaxf(fabsf(S[j].x), fabsf(S[j].y)) : 0.f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        asm volatile("bar.sync 1, 128;" ::: "memory");  // the last block's have been read
        if (lane == 0) s_max[warp & 3] = m;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const int e = lift_of(fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3])));
        up = pow2(e);
        if (row == 0) s_state_up[c & 1] = e;
      }
      if (c > 0) wait(o_full, (c + 1) & 1);  // the product with the S before
      if (held)
#pragma unroll
        for (int j = 0; j < DV / 8; ++j) {
          uint32_t x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 u = F16 ? mul2(S[4 * j + e], make_float2(up, up)) : S[4 * j + e];
            x[e] = kv::pack2<F16>(u.x, u.y);
          }
          st_s128(ss + (j >> 3) * (DK * 128) + row * 128 + (((j & 7) ^ (row & 7)) << 4), x[0], x[1], x[2], x[3]);
        }
      fence_proxy_async_shared();
      arrive(s_ready);
      step(n1 + c, nullptr);
    }
    if (last) {
      wait(o_full, (n2 + 1) & 1);  // the last product with S
      leave();
    }
  } else if (warp < 12) {
    // ================= the output: a thread is a token's row =================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOut));
    const int t = tid - 256;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    meet();
#pragma unroll 1
    for (int c = 0; c < n2; ++c) {
      wait(o_full, c & 1);
      tc_fence_after();
      const float scale = s_row[c & 1][t];
#pragma unroll 1
      for (int j = 0; j < DV / 32; ++j) {
        uint32_t x[32], w[16];
        tc_ld32(to + lanes + j * 32, x);
        tc_ld_wait();
        if (j == DV / 32 - 1) {
          tc_fence_before();
          arrive(o_free);
        }
#pragma unroll
        for (int y = 0; y < 16; ++y) {
          const float2 o = mul2(make_float2(__uint_as_float(x[2 * y]), __uint_as_float(x[2 * y + 1])), make_float2(scale, scale));
          w[y] = kv::pack2<F16>(o.x, o.y);
        }
        // rows of 64 values go out together, eight lanes a row: a store of one piece
        // per row and lane takes the load-store unit 32 cycles, and everything waits
        const uint32_t mine = so + (t >> 5) * (32 * kPitch);
#pragma unroll
        for (int y = 0; y < 4; ++y)
          st_s128(mine + lane * kPitch + (j & 1) * 64 + y * 16, w[4 * y], w[4 * y + 1], w[4 * y + 2], w[4 * y + 3]);
        if (j & 1) {
          __syncwarp();
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int r = y * 4 + (lane >> 3), tok = (first + c) * kBlk + (t & ~31) + r;
            const uint4 v = ld_s128(mine + r * kPitch + (lane & 7) * 16);
            if (tok < s.n)
              *reinterpret_cast<uint4*>(a.o + ((long long)(s.row0 + tok) * a.Hv + h) * DV + (j & ~1) * 32 + (lane & 7) * 8) = v;
          }
          __syncwarp();
        }
      }
    }
  } else {
    // ================= K'^T: a warp has 32 of its rows (values of a key) =================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsKey));
    const int w = warp & 3, part = (warp - 12) >> 2;  // (its place in shared memory: warp - 12)
    const bool held = w * 32 < DK;
#pragma unroll 1
    for (int i = 0; i < n1 + n2; ++i) {
      if (i == n1) {
        meet();
      }
      const int x = i & 1, rows = s.n - block_of(i) * kBlk;
      const Decays& d = s_dec[x];
      wait(g_full + 8 * x, (i >> 1) & 1);
      if (rows < kBlk && part == 0) {  // the sequence's last block: V behind its end becomes zeros
        wait(v_full + 8 * x, (i >> 1) & 1);
#pragma unroll 1
        for (int at = rows * 128 + (tid & 127) * 16; at < kHalf; at += 128 * 16)
#pragma unroll
          for (int y = 0; y < HV; ++y) st_s128(sv + x * kTile + y * kHalf + at, 0u, 0u, 0u, 0u);
        fence_proxy_async_shared();
        arrive(v_ready);
      }
      wait(k_full + 8 * x, (i >> 1) & 1);
      // this lane's row of the matrices: tokens (lane & 7) + 8 (lane >> 4), the warp's first or
      // second 8 values of 16 by (lane >> 3) & 1
      const uint32_t tile = sk + x * kTile + (w >> 1) * kHalf + ((lane & 7) + ((lane >> 4) << 3)) * 128;
      const auto fetch = [&](int t0, int half, uint32_t (&m)[4]) {  // 16 tokens from t0 on, 16 values
        const int at = (w & 1) * 4 + half * 2 + ((lane >> 3) & 1);
        ldmatrix4_t(tile + t0 * 128 + ((at ^ (lane & 7)) << 4), m);
        if (t0 + 16 > rows) {  // tokens behind the end (which may be NaN) become zeros
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int t = t0 + (y >> 1) * 8 + (lane & 3) * 2;
            m[y] &= (t < rows ? 0xffffu : 0u) | (t + 1 < rows ? 0xffff0000u : 0u);
          }
        }
      };
      float up = 1.f;
      if constexpr (F16) {  // the block's largest |k| (infinities and NaN apart) to about 2^13
        uint32_t m = 0;
        if (held)
#pragma unroll 2
          for (int y = 0; y < 8; ++y) {
            uint32_t v[4];
            fetch(part * 64 + (y >> 1) * 16, y & 1, v);
            m = __vmaxu2(__vmaxu2(m, __vmaxu2(v[0] & 0x7fff7fffu, v[1] & 0x7fff7fffu)),
                         __vmaxu2(v[2] & 0x7fff7fffu, v[3] & 0x7fff7fffu));
          }
        m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
        asm volatile("bar.sync 2, 256;" ::: "memory");  // the last block's have been read
        if (lane == 0) s_kmax[warp - 12] = m;
        asm volatile("bar.sync 2, 256;" ::: "memory");
#pragma unroll
        for (int y = 0; y < 8; ++y) m = max(m, s_kmax[y]);
        const int e = lift_of(kv::unpack2<true>(min(m, 0x7bffu)).x);
        up = pow2(e);
        if (tid == 32 * 12) s_key_down[x] = pow2(-e);
      }
      const uint32_t lanes = (uint32_t)(w * 32) << 16;
      // what is left of f without its upper 8 bits: three such values are all of an fp32
      const auto rest = [](float2 f) {
        return add2(f, make_float2(-__uint_as_float(__float_as_uint(f.x) & 0xffff0000u), -__uint_as_float(__float_as_uint(f.y) & 0xffff0000u)));
      };
      const auto upper = [](float2 f) { return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632); };
      // 32 tokens by 16 values of the head at a time, in 8 registers each of the values
      // that stand for K'
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        const int t0 = (j >> 1) * 64 + part * 32;
        uint32_t v[kTerms][8];
        if (held) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint32_t m[4];
            fetch(t0 + g * 16, j & 1, m);
#pragma unroll
            for (int z = 0; z < 4; ++z) v[0][4 * g + z] = m[z];
          }
          const float* e0 = d.k + t0 + (lane & 3) * 2;
#pragma unroll
          for (int z = 0; z < 8; ++z) {  // a pair of tokens
            float2 f = mul2(kv::unpack2<F16>(v[0][z]), *reinterpret_cast<const float2*>(e0 + (z >> 1) * 8));
            if constexpr (F16) {
              f = mul2(f, make_float2(up, up));
              v[0][z] = kv::pack2<true>(f.x, f.y);
              const float2 r = kv::unpack2<true>(v[0][z]);
              v[1][z] = kv::pack2<true>(f.x - r.x, f.y - r.y);
            } else {
              v[0][z] = upper(f);
              f = rest(f);
              v[1][z] = upper(f);
              v[kTerms - 1][z] = upper(rest(f));
            }
          }
        }
        if (!(j & 1)) {
          wait(kt_empty + 8 * part, (j >> 1) ^ 1);
          tc_fence_after();
        }
        if (held) {
#pragma unroll
          for (int y = 0; y < kTerms; ++y)
            tc_st_16x16(tk + lanes + ((uint32_t)((j & 1) * 16) << 16) + part * kKeyCols + y * 16, v[y]);
        }
        if (j & 1) {
          tc_st_wait();
          tc_fence_before();
          arrive(kt_full + 8 * part);
        }
      }
      arrive(k_empty + 8 * x);
      arrive(g_empty + 8 * x);
    }
    if (n2 == 0) {
      meet();
    }
  }

  if (tries == 1 && a.status && lane == 0) atomicOr(a.status, DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 20) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(ta));
  }
}

bool encode(CUtensorMap* m, const void* base, int D, int heads, int rows, long long stride) {
  const auto fn = kv::encode_fn();
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t str[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, kBlk}, es[3] = {1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims, str, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool F16, int DK, int DV>
cudaError_t launch_one(const ChunkArgs& g, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(linear_chunk_kernel<F16, DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)g.r.B * g.a.Hv * g.parts));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = g.parts;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = g.parts > 1 ? 2 : 1;
  launch_begin(K_LINEAR_CHUNK, st);
  e = cudaLaunchKernelEx(&cfg, linear_chunk_kernel<F16, DK, DV>, ChunkArgs(g));
  launch_end(st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool F16>
cudaError_t launch_type(const ChunkArgs& g, cudaStream_t st) {
  if (g.a.Dk == 128) return g.a.Dv == 128 ? launch_one<F16, 128, 128>(g, st) : launch_one<F16, 128, 64>(g, st);
  return g.a.Dv == 128 ? launch_one<F16, 64, 128>(g, st) : launch_one<F16, 64, 64>(g, st);
}

}  // namespace

bool linear_chunk_supported(const Linear& a) {
  return (a.Dk == 64 || a.Dk == 128) && (a.Dv == 64 || a.Dv == 128) && kv::encode_fn();
}

cudaError_t launch_linear_chunk(const Linear& a, const kv::Rows& r, bool f16, cudaStream_t st) {
  ChunkArgs g;
  g.a = a;
  g.r = r;
  if (!encode(&g.tm_q, a.q, a.Dk, a.Hk, r.n_rows, a.q_stride) || !encode(&g.tm_k, a.k, a.Dk, a.Hk, r.n_rows, a.k_stride) ||
      !encode(&g.tm_v, a.v, a.Dv, a.Hv, r.n_rows, a.v_stride))
    return cudaErrorInvalidValue;
  // CTAs per item: while the items leave half of the GPU's 152 SMs or more without one
  // and the mean sequence has two blocks or more for each.
  const long long items = (long long)r.B * a.Hv, mean = ((long long)r.n_rows / r.B + kBlk - 1) / kBlk;
  g.parts = 1;
  while (g.parts < kMostParts && items * g.parts * 2 <= 152 && mean >= 4 * g.parts) g.parts *= 2;
  return f16 ? launch_type<true>(g, st) : launch_type<false>(g, st);
}

}  // namespace block
}  // namespace moe
