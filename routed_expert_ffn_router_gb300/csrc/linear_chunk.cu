// Linear attention of prompt chunks on the 5th-generation tensor cores
// (include/moe_block.h), head sizes 64 and 128.
//
// Blocks of 128 tokens. With G_i the sum of the logarithms of the decays of a
// block's tokens up to i, G the sum of all of them, and S the state before it:
//   o_i = scale (e^G_i q_i S + sum_{j <= i} e^(G_i - G_j) (q_i . k_j) v_j)
//   S'  = e^G S + sum_j k_j (e^(G - G_j) v_j)^T
// Four products, accumulators in tensor memory:
//   A = Q K^T    X = Q S    U = K^T V'    Y = (A o D) V
// V' = e^(G - G_j) v_j, D_ij = e^(G_i - G_j) for j <= i, else 0; A o D goes back to
// tensor memory as the first operand of Y. U does not depend on S, so the blocks of
// a sequence wait for one another only in S' = e^G S + U, in registers.
//
// Rounding. The state is fp32 throughout: V' enters as two values of the type (its
// rounding and the rest, 2^-17 of it for bf16), and U is a fresh sum each block. S
// and A o D, which only o sees, are rounded once to the type (half a step each, as o
// itself is). In fp16, whose range is narrow and whose step is fixed below 2^-14, V'
// and S are scaled by a power of two per block and a row of A o D by one of its own,
// which bring the largest magnitude to 2^13 and are undone in fp32: the smallest
// values are then off by up to 2^-38 of the largest. Sums of logarithms are taken in fp64 and handed on as two fp32
// values, so that G_i - G_j is right next to large |G|.
//
// Work. An item is a sequence and a v head, by a cluster of 1 to 8 CTAs that have
// consecutive parts of its blocks. With more than one, each first sums up its own
// part's state (K and V only), the parts meet through the cluster's shared memory
// (S at a part's start: the initial state and the parts before it), and each then
// goes through its part. So a long prompt of few heads fills the GPU in one launch
// and without a workspace. Items are started longest first.
//
// Warps. 0-3: A o D; 4-7: the state (a thread is a row of it); 8-11: V' and the
// output; 12: issues the products; 13: TMA; 14: decays, two blocks ahead.
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
constexpr int kThreads = 512;
constexpr int kRegsScore = 112, kRegsState = 184, kRegsOut = 104, kRegsRest = 112;  // at most 4 x 128 together
constexpr uint32_t kTries = 1u << 22;   // of a wait, each up to a microsecond long
constexpr int kHalf = kBlk * 128;       // bytes of 128 rows of 64 values
constexpr int kTile = 2 * kHalf;
constexpr int kPitch = 144;             // bytes per row of a warp's output buffer (64 values and a pad)
constexpr int kSmem = 1024 + 6 * kTile + 4 * 32 * kPitch;  // Q, K, V, V' twice, S; outputs
constexpr int kSortB = 512;             // sequences that are put in order of their length
constexpr int kMostParts = 8;
constexpr int kAhead = 2;               // blocks that are fetched into L2 ahead

struct ChunkArgs {
  CUtensorMap tm_q, tm_k, tm_v;
  Linear a;
  kv::Rows r;
  int parts;  // CTAs of a cluster
};

// What the decays of a block come to.
struct Decays {
  float gh[kBlk], gl[kBlk];  // -G_j / ln 2 as two values
  float v[kBlk];      // e^(G - G_j); 0 behind the last token
  float q[kBlk];      // scale e^G_i
  float2 all;         // e^G (decay_of)
  float pad[2];
};

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
  extern __shared__ __align__(1024) uint8_t smem_linear[];
  __shared__ __align__(16) Decays s_dec[2];
  __shared__ __align__(8) uint64_t s_bar[20];
  __shared__ float s_row[2][kBlk];    // fp16, by block: what a row of A o D was scaled by, undone
  __shared__ float s_state_up[2], s_v_up[2];  // the same of S, of V'
  __shared__ float s_max[4];
  __shared__ uint32_t s_vmax[4];
  __shared__ float s_part;            // e^(sum of the part's logarithms)
  __shared__ uint32_t s_tmem;
  __shared__ int s_b;

  const Linear& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sq = (smem_u32(smem_linear) + 1023u) & ~1023u;
  const uint32_t sk = sq + kTile, sv = sk + kTile, svh = sv + kTile, svl = svh + kTile, ss = svl + kTile, so = ss + kTile;
  const uint32_t q_full = smem_u32(s_bar), k_full = q_full + 8, v_full = q_full + 16, q_empty = q_full + 24;
  const uint32_t k_empty = q_full + 32, v_empty = q_full + 40, a_full = q_full + 48, p_full = q_full + 56;
  const uint32_t s_ready = q_full + 64, w_ready = q_full + 72, u_full = q_full + 80, u_free = q_full + 88;
  const uint32_t o_full = q_full + 96, o_free = q_full + 104, g_full = q_full + 112, g_empty = q_full + 128;
  const uint32_t drained = q_full + 144;
  if (tid == 0) {
    mbar_init(q_full, 1); mbar_init(k_full, 1); mbar_init(v_full, 1);
    mbar_init(q_empty, 1); mbar_init(k_empty, 1); mbar_init(v_empty, 1);
    mbar_init(a_full, 1); mbar_init(p_full, 4);
    mbar_init(s_ready, 4); mbar_init(w_ready, 4);
    mbar_init(u_full, 1); mbar_init(u_free, 4);
    mbar_init(o_full, 1); mbar_init(o_free, 4);
    mbar_init(g_full, 1); mbar_init(g_full + 8, 1);
    mbar_init(g_empty, 12); mbar_init(g_empty + 8, 12);
    mbar_init(drained, 1);
    fence_barrier_init();
  }
  if (tid == 32 * 13) {
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

  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t ta = s_tmem, tx = ta + 128, ty = ta + 256, tu = ta + 384;

  bool dead = false;  // an expired wait: go on without waiting (the status word says so)
  auto wait = [&](uint32_t bar, uint32_t parity) {
    uint32_t n = dead ? 1u : kTries;
    while (!mbar_try_wait_ns(bar, parity, 1000) && --n) {
    }
    dead |= n == 0;
    __syncwarp();
  };
  auto arrive = [&](uint32_t bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  auto meet = [&] {  // between the two passes: the parts' sums are there; they have been read
    if (parts > 1) {
      __syncwarp();
      cluster_sync();
    }
  };

  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == 13) {
      // ================= TMA =================
      const uint32_t lead = elect_lane();
      auto load = [&](uint32_t dst, const CUtensorMap* m, int halves, int head, int row, uint32_t bar) {
        if (lead) {
          mbar_expect_tx(bar, (uint32_t)(halves * kHalf));
          for (int i = 0; i < halves; ++i) tma_load_3d(dst + i * kHalf, m, i * 64, head, row, bar);
        }
        __syncwarp();
      };
      // the next blocks come into L2 while the tiles are still in use
      auto ahead = [&](int c) {
        if (lead && c < n2) {
          const int row = s.row0 + (first + c) * kBlk;
          for (int x = 0; x < HK; ++x) {
            prefetch_3d(&p.tm_k, x * 64, hk, row);
            prefetch_3d(&p.tm_q, x * 64, hk, row);
          }
          for (int x = 0; x < HV; ++x) prefetch_3d(&p.tm_v, x * 64, h, row);
        }
        __syncwarp();
      };
      for (int c = 1; c < kAhead; ++c) ahead(c);
      auto step = [&](int i, bool full) {
        ahead(i + kAhead);
        const int row = s.row0 + (first + (i < n1 ? i : i - n1)) * kBlk;
        if (full) {
          wait(q_empty, (i - n1 + 1) & 1);
          load(sq, &p.tm_q, HK, hk, row, q_full);
        }
        wait(k_empty, (i + 1) & 1);
        load(sk, &p.tm_k, HK, hk, row, k_full);
        wait(v_empty, (i + 1) & 1);
        load(sv, &p.tm_v, HV, h, row, v_full);
      };
      for (int i = 0; i < n1; ++i) step(i, false);
      if (n2 > 0) step(n1, true);
      meet();
      meet();
      for (int i = 1; i < n2; ++i) step(n1 + i, true);
      // no copy is under way when the CTA ends, also where a warp went on without waiting
      const bool gave_up = dead;
      dead = false;
      const int n = n1 + n2;
      if (n2 > 0) wait(q_full, (n2 + 1) & 1);
      if (n > 0) {
        wait(k_full, (n + 1) & 1);
        wait(v_full, (n + 1) & 1);
      }
      dead |= gave_up;
    } else if (warp == 12) {
      // ================= products =================
      const uint32_t lead = elect_lane();
      const uint32_t id_a = idesc_16(F16, 128, kBlk, false), id_o = idesc_16(F16, 128, DV, true);
      const uint32_t id_u = id_o | 1u << 15;  // the first operand, too, lies along its rows' dimension
      const uint64_t qd = sdesc_sw128(sq), kd = sdesc_sw128(sk), kt = sdesc_sw128_n(sk, kHalf), vd = sdesc_sw128_n(sv, kHalf);
      const uint64_t vh = sdesc_sw128_n(svh, kHalf), vl = sdesc_sw128_n(svl, kHalf), sd = sdesc_sw128_n(ss, DK * 128);
      auto update = [&](int i) {  // U of step i
        wait(w_ready, i & 1);
        wait(u_free, (i + 1) & 1);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kBlk / 16; ++kk) tc_mma_el(tu, kt + kk * 128, vh + kk * 128, id_u, kk > 0, lead);
#pragma unroll
        for (int kk = 0; kk < kBlk / 16; ++kk) tc_mma_el(tu, kt + kk * 128, vl + kk * 128, id_u, 1, lead);
        tc_commit_el(u_full, lead);
        tc_commit_el(k_empty, lead);
      };
      for (int i = 0; i < n1; ++i) {
        wait(k_full, i & 1);
        update(i);
        tc_commit_el(v_empty, lead);
      }
      meet();
      meet();
      for (int c = 0; c < n2; ++c) {
        const int i = n1 + c;
        wait(k_full, i & 1);
        wait(q_full, c & 1);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) {
          const uint32_t o = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
          tc_mma_el(ta, qd + o, kd + o, id_a, kk > 0, lead);
        }
        tc_commit_el(a_full, lead);
        wait(s_ready, c & 1);
        wait(o_free, (c + 1) & 1);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) {
          const uint32_t o = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
          tc_mma_el(tx, qd + o, sd + kk * 128, id_o, kk > 0, lead);
        }
        tc_commit_el(q_empty, lead);
        update(i);
        wait(p_full, c & 1);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kBlk / 16; ++kk) tc_mma_ts_el(ty, ta + kk * 8, vd + kk * 128, id_o, kk > 0, lead);
        tc_commit_el(o_full, lead);
        tc_commit_el(v_empty, lead);
      }
      tc_commit_el(drained, lead);  // every product has ended before tensor memory is given back
      wait(drained, 0);
    } else if (warp == 14) {
      // ================= decays =================
      for (int i = 0; i < n1 + n2; ++i) {
        if (i == n1) {
          meet();
          meet();
        }
        const int t0 = (first + (i < n1 ? i : i - n1)) * kBlk + lane * 4, slot = i & 1;
        double g[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          g[j] = t0 + j < s.n ? (double)bounded_g(a.g[(s.row0 + t0 + j) * a.g_stride + h]) * 1.4426950408889634 : 0.0;
#pragma unroll
        for (int j = 1; j < 4; ++j) g[j] += g[j - 1];
        double x = g[3];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const double total = __shfl_sync(0xffffffffu, x, 31);
        const double before = __shfl_up_sync(0xffffffffu, x, 1);
        wait(g_empty + 8 * slot, ((i >> 1) + 1) & 1);
        Decays& d = s_dec[slot];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const double G = (lane ? before : 0.0) + g[j];
          const float hi = (float)G;
          d.gh[lane * 4 + j] = -hi;
          d.gl[lane * 4 + j] = (float)(hi - G);
          d.v[lane * 4 + j] = t0 + j < s.n ? exp2f((float)(total - G)) : 0.f;
          d.q[lane * 4 + j] = a.scale * exp2f(hi);
        }
        if (lane == 0) d.all = decay_of((float)(total * 0.6931471805599453));
        arrive(g_full + 8 * slot);
      }
      if (n2 == 0) {
        meet();
        meet();
      }
    } else {
      meet();
      meet();
    }
  } else if (warp < 4) {
    // ================= A o D: a thread is a token's row =================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsScore));
    for (int i = 0; i < n1; ++i) {
      wait(g_full + 8 * (i & 1), (i >> 1) & 1);
      arrive(g_empty + 8 * (i & 1));
    }
    meet();
    meet();
    const uint32_t tr = ta + ((uint32_t)(warp * 32) << 16);
    for (int c = 0; c < n2; ++c) {
      const int i = n1 + c;
      const Decays& d = s_dec[i & 1];
      wait(g_full + 8 * (i & 1), (i >> 1) & 1);
      wait(a_full, c & 1);
      tc_fence_after();
      const float2 gh = make_float2(-d.gh[tid], -d.gh[tid]), gl = make_float2(-d.gl[tid], -d.gl[tid]);
      float up = 1.f;
      if constexpr (F16) {  // the row's largest |q . k| to about 2^13
        float m = 0.f;
        for (int j = 0; j <= warp; ++j) {
          uint32_t x[32];
          tc_ld32(tr + j * 32, x);
          tc_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (j < warp || e <= lane) m = fmaxf(m, fabsf(__uint_as_float(x[e])));
        }
        const int e = lift_of(m);
        up = pow2(e);
        s_row[c & 1][tid] = pow2(-e);
      }
      // (rolled loops: with all roles' loops unrolled their code did not stay in the
      // instruction cache, and a block took twice as long)
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        uint32_t pk[16], x[32];
        if (j <= warp) {
          tc_ld32(tr + j * 32, x);
          tc_ld_wait();
          const float4* nh = reinterpret_cast<const float4*>(d.gh + j * 32);
          const float4* nl = reinterpret_cast<const float4*>(d.gl + j * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 a4 = nh[e], b4 = nl[e];
            const float2 t0 = add2(add2(gh, make_float2(a4.x, a4.y)), add2(gl, make_float2(b4.x, b4.y)));
            const float2 t1 = add2(add2(gh, make_float2(a4.z, a4.w)), add2(gl, make_float2(b4.z, b4.w)));
            float2 d0 = make_float2(kv::ex2(t0.x), kv::ex2(t0.y)), d1 = make_float2(kv::ex2(t1.x), kv::ex2(t1.y));
            if constexpr (F16) {
              d0 = mul2(d0, make_float2(up, up));
              d1 = mul2(d1, make_float2(up, up));
            }
            d0 = mul2(d0, make_float2(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1])));
            d1 = mul2(d1, make_float2(__uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3])));
            pk[2 * e] = kv::pack2<F16>(d0.x, d0.y);
            pk[2 * e + 1] = kv::pack2<F16>(d1.x, d1.y);
          }
          if (j == warp) {  // later tokens (what stands there may be NaN: cleared as bits)
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] &= (2 * e <= lane ? 0xffffu : 0u) | (2 * e + 1 <= lane ? 0xffff0000u : 0u);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = 0u;
        }
        tc_st16(tr + j * 16, pk);
      }
      tc_st_wait();
      tc_fence_before();
      arrive(p_full);
      arrive(g_empty + 8 * (i & 1));
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
    // memory is touched along rows (16 pieces of 16 bytes each, in places that
    // keep a warp's rows in different banks).
    auto exchange = [&](bool in) {
#pragma unroll
      for (int x = 0; x < HV; ++x) {
        const uint32_t mine = ss + row * 256;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (!in) {
          if (held)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 u = S[x * 32 + 2 * j], w = S[x * 32 + 2 * j + 1];
              st_s128(mine + ((j ^ (row & 15)) << 4), __float_as_uint(u.x), __float_as_uint(u.y), __float_as_uint(w.x), __float_as_uint(w.y));
            }
          asm volatile("bar.sync 1, 128;" ::: "memory");
        }
#pragma unroll 8
        for (int i = 0; i < DK / 8; ++i) {
          const int r = i * 8 + (row >> 4), j = row & 15;
          const uint32_t at = ss + r * 256 + ((j ^ (r & 15)) << 4);
          float4* m = state + r * (DV / 4) + x * 16 + j;
          if (in) {
            const float4 f = *m;
            st_s128(at, __float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(f.z), __float_as_uint(f.w));
          } else {
            const uint4 f = ld_s128(at);
            *m = make_float4(__uint_as_float(f.x), __uint_as_float(f.y), __uint_as_float(f.z), __uint_as_float(f.w));
          }
        }
        if (in) {
          asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint4 f = held ? ld_s128(mine + ((j ^ (row & 15)) << 4)) : make_uint4(0, 0, 0, 0);
            S[x * 32 + 2 * j] = make_float2(__uint_as_float(f.x), __uint_as_float(f.y));
            S[x * 32 + 2 * j + 1] = make_float2(__uint_as_float(f.z), __uint_as_float(f.w));
          }
        }
      }
      if (in) asm volatile("bar.sync 1, 128;" ::: "memory");  // S's tile is free for S
    };
    auto step = [&](int i, float* decay) {  // S <- e^G S + U
      wait(g_full + 8 * (i & 1), (i >> 1) & 1);
      const float2 e = s_dec[i & 1].all;
      if (decay) *decay = fmaf(*decay, e.x, *decay * e.y);
      wait(u_full, i & 1);
      tc_fence_after();
      const float up = F16 ? s_v_up[i & 1] : 1.f;
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
#pragma unroll
      for (int j = 0; j < DV / 2; ++j) S[j] = make_float2(0.f, 0.f);
      for (int i = 0; i < n1; ++i) step(i, &decay);
      if (n1 > 0) {  // columns 4 j of all rows side by side, where V' was
        if (held)
#pragma unroll
          for (int j = 0; j < DV / 4; ++j)
            st_s128(svh + (j * DK + row) * 16, __float_as_uint(S[2 * j].x), __float_as_uint(S[2 * j].y),
                    __float_as_uint(S[2 * j + 1].x), __float_as_uint(S[2 * j + 1].y));
        if (row == 0) s_part = decay;
      }
      meet();
    }
    if (n2 > 0) {
      exchange(true);
      for (int r = 0; r < part; ++r) {  // the parts before, in their order
        const float e = peer_f32(peer(smem_u32(&s_part), r));
        const uint32_t from = peer(svh, r);
        if (held)
#pragma unroll
          for (int j = 0; j < DV / 4; ++j) {
            const float4 x = peer_f128(from + (j * DK + row) * 16);
            S[2 * j] = fma2(S[2 * j], make_float2(e, e), make_float2(x.x, x.y));
            S[2 * j + 1] = fma2(S[2 * j + 1], make_float2(e, e), make_float2(x.z, x.w));
          }
      }
    }
    meet();
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
        if (row == 0) s_state_up[c & 1] = pow2(-e);
      }
      if (c > 0) wait(q_empty, (c + 1) & 1);  // the product with the S before
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
      wait(q_empty, (n2 + 1) & 1);  // the last product with S
      exchange(false);
    }
  } else {
    // ================= V' and the output =================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOut));
    const int t = tid - 256;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    auto scaled = [&](int i) {  // V' of step i; rows behind the last token become zeros, in K and V too
      const int nv = s.n - (first + (i < n1 ? i : i - n1)) * kBlk;
      const Decays& d = s_dec[i & 1];
      wait(g_full + 8 * (i & 1), (i >> 1) & 1);
      wait(v_full, i & 1);
      if (i > 0) wait(u_full, (i + 1) & 1);  // the product with the V' before
      float up = 1.f;
      if constexpr (F16) {  // the block's largest |v| (infinities and NaN apart) to about 2^13
        uint32_t m = 0;
#pragma unroll 4
        for (int j = 0; j < 8 * HV; ++j) {
          const int at = (j * 128 + t) * 16;
          const uint4 raw = ld_s128(sv + at);
          if ((at & (kHalf - 1)) >> 7 < nv)
            m = __vmaxu2(__vmaxu2(m, __vmaxu2(raw.x & 0x7fff7fffu, raw.y & 0x7fff7fffu)),
                         __vmaxu2(raw.z & 0x7fff7fffu, raw.w & 0x7fff7fffu));
        }
        m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
        asm volatile("bar.sync 2, 128;" ::: "memory");  // the last block's have been read
        if (lane == 0) s_vmax[warp & 3] = m;
        asm volatile("bar.sync 2, 128;" ::: "memory");
        m = min(max(max(s_vmax[0], s_vmax[1]), max(s_vmax[2], s_vmax[3])), 0x7bffu);
        const int e = lift_of(kv::unpack2<true>(m).x);
        up = pow2(e);
        if (t == 0) s_v_up[i & 1] = pow2(-e);
      }
#pragma unroll 2
      for (int j = 0; j < 8 * HV; ++j) {
        const int at = (j * 128 + t) * 16, row = (at & (kHalf - 1)) >> 7;
        const uint4 raw = ld_s128(sv + at);
        const float e = F16 ? d.v[row] * up : d.v[row];
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float2 f = mul2(kv::unpack2<F16>(w[x]), make_float2(e, e));
          hi[x] = kv::pack2<F16>(f.x, f.y);
          const float2 r = kv::unpack2<F16>(hi[x]), rest = add2(f, make_float2(-r.x, -r.y));
          lo[x] = kv::pack2<F16>(rest.x, rest.y);
        }
        const bool in = row < nv;
        if (!in) st_s128(sv + at, 0u, 0u, 0u, 0u);
        st_s128(svh + at, in ? hi[0] : 0u, in ? hi[1] : 0u, in ? hi[2] : 0u, in ? hi[3] : 0u);
        st_s128(svl + at, in ? lo[0] : 0u, in ? lo[1] : 0u, in ? lo[2] : 0u, in ? lo[3] : 0u);
      }
      if (nv < kBlk) {
        wait(k_full, i & 1);
        for (int at = nv * 128 + t * 16; at < kHalf; at += 128 * 16)
#pragma unroll
          for (int x = 0; x < HK; ++x) st_s128(sk + x * kHalf + at, 0u, 0u, 0u, 0u);
      }
      fence_proxy_async_shared();
      arrive(w_ready);
    };
    for (int i = 0; i < n1; ++i) {
      scaled(i);
      arrive(g_empty + 8 * (i & 1));
    }
    meet();
    meet();
    for (int c = 0; c < n2; ++c) {
      const int i = n1 + c;
      scaled(i);
      const float e = s_dec[i & 1].q[t];
      arrive(g_empty + 8 * (i & 1));
      wait(o_full, c & 1);
      tc_fence_after();
      const float ex = F16 ? e * s_state_up[c & 1] : e, ey = F16 ? a.scale * s_row[c & 1][t] : a.scale;
#pragma unroll 1
      for (int j = 0; j < DV / 32; ++j) {
        uint32_t x[32], y[32];
        tc_ld32(tx + lanes + j * 32, x);
        tc_ld32(ty + lanes + j * 32, y);
        tc_ld_wait();
        if (j == DV / 32 - 1) {
          tc_fence_before();
          arrive(o_free);
        }
        uint32_t w[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const float2 o = fma2(make_float2(ex, ex), make_float2(__uint_as_float(x[2 * q]), __uint_as_float(x[2 * q + 1])),
                                mul2(make_float2(ey, ey), make_float2(__uint_as_float(y[2 * q]), __uint_as_float(y[2 * q + 1]))));
          w[q] = kv::pack2<F16>(o.x, o.y);
        }
        // rows of 64 values go out together, eight lanes a row: a store of one piece
        // per row and lane takes the load-store unit 32 cycles, and everything waits
        const uint32_t mine = so + (t >> 5) * (32 * kPitch);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          st_s128(mine + lane * kPitch + (j & 1) * 64 + q * 16, w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
        if (j & 1) {
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int r = q * 4 + (lane >> 3), tok = (first + c) * kBlk + (t & ~31) + r;
            const uint4 v = ld_s128(mine + r * kPitch + (lane & 7) * 16);
            if (tok < s.n)
              *reinterpret_cast<uint4*>(a.o + ((long long)(s.row0 + tok) * a.Hv + h) * DV + (j & ~1) * 32 + (lane & 7) * 8) = v;
          }
          __syncwarp();
        }
      }
    }
  }

  if (dead && a.status && lane == 0) atomicOr(a.status, DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
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
  // CTAs per item: while the items leave half of the GPU's SMs or more without one
  // and the mean sequence has two blocks or more for each.
  const long long items = (long long)r.B * a.Hv, mean = ((long long)r.n_rows / r.B + kBlk - 1) / kBlk;
  g.parts = 1;
  while (g.parts < kMostParts && items * g.parts * 2 <= 152 && mean >= 4 * g.parts) g.parts *= 2;
  return f16 ? launch_type<true>(g, st) : launch_type<false>(g, st);
}

}  // namespace block
}  // namespace moe
