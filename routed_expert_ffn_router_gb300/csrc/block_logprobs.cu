// Log probabilities of given tokens, ranks, entropies and top alternatives over
// rows of logits (include/moe_block.h).
//
// One pass. With a running maximum m (scores in units of log2, c = log2 e /
// temperature, d_i = (z_i - m) c):
//   l = sum 2^d_i,  s = sum 2^d_i d_i      a larger maximum m': a = (m - m') c,
//   s' = 2^a (s + l a),  l' = 2^a l
// and at the end ln p_i = (z_i - m) / temperature - ln l, entropy = ln l - ln 2 s / l.
// z - m is taken before the product, so that rows of the type's lowest value are
// uniform and not NaN; d is bounded by -200, where 2^d is 0 in fp32 already, which
// makes the terms of -inf zeros.
//
// A row is read by a cluster of 1 to 8 CTAs, each by 16 warps that take chunks of
// 32 lanes x 64 bytes in turn; rows start anywhere, so the pieces of a row go by
// 16-byte boundaries of memory and the first and the last by single values. The
// parts meet through shared memory, then through the cluster's: few rows use many
// SMs without a workspace or a second launch.
//
// Top alternatives: each warp keeps its best 32 as sorted keys (order of the logit,
// then lower id: all distinct), one per lane. A chunk is looked through only if its
// maximum, which the sum needs anyway, reaches the k-th best of any warp of the CTA
// so far. The rank likewise counts only in chunks whose maximum reaches the token's
// logit.
#include "block_internal.h"
#include "kv_common.cuh"

namespace moe {
namespace block {

namespace {

typedef unsigned long long Key;

constexpr int kThreads = 512;
constexpr int kWarpsPerCta = kThreads / 32;
constexpr int kVecs = 4;  // 16-byte pieces of a lane's chunk

struct Part {
  float m, l, s;
  int rank;
};
struct Shared {
  Part part[kWarpsPerCta];
  Key key[kWarpsPerCta][32];
  float floor;  // some warp's k-th best logit: no smaller one is among the k best
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// NaN becomes -200
__device__ __forceinline__ float bounded(float d) { return fmaxf(d, -200.f); }

__device__ __forceinline__ void join(Part& a, const Part& b, float c) {
  const float m = max_nan(a.m, b.m);
  const float da = bounded((a.m - m) * c), db = bounded((b.m - m) * c);
  const float ea = kv::ex2(da), eb = kv::ex2(db);
  a.s = ea * (a.s + a.l * da) + eb * (b.s + b.l * db);
  a.l = ea * a.l + eb * b.l;
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

template <int TYPE>
__device__ __forceinline__ float value(uint32_t bits) {
  if constexpr (TYPE == MOE_T_F32) return __uint_as_float(bits);
  else return kv::unpack2<TYPE == MOE_T_F16>(bits).x;
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads, 2) logprobs_kernel(const __grid_constant__ moe_logprobs_args a, int parts) {
  constexpr int S = TYPE == MOE_T_F32 ? 4 : 2, E = 16 / S, N = kVecs * E;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x / parts, rank = parts > 1 ? (int)cluster_rank() : 0;
  const float c = 1.4426950408889634f / a.temperature;
  const char* row = static_cast<const char*>(a.logits) + (long long)t * a.stride * S;
  const int lead = (int)(reinterpret_cast<uintptr_t>(row) & 15) / S;  // values of the first piece before the row
  const char* base = row - lead * S;
  const int n_vec = (lead + a.V + E - 1) / E;
  const int token = a.tokens ? a.tokens[t] : -1;
  const bool has = token >= 0 && token < a.V;
  const auto one = [&](int id) {
    return TYPE == MOE_T_F32 ? value<TYPE>(*reinterpret_cast<const uint32_t*>(row + (long long)id * S))
                             : value<TYPE>(*reinterpret_cast<const uint16_t*>(row + (long long)id * S));
  };
  const float mine_raw = has ? one(token) : 0.f;
  // counts are of logits at or above it: with no token, of none
  const float mine = !has ? __int_as_float(0x7f800000) : mine_raw == mine_raw ? mine_raw : -__int_as_float(0x7f800000);
  const float kNone = -__int_as_float(0x7f800000);
  if (tid == 0) sh.floor = kNone;
  __syncthreads();

  Part p = {kNone, 0.f, 0.f, 0};
  Key best = 0;
  float floor = kNone;
  for (int v0 = (rank * kWarpsPerCta + warp) * 32 * kVecs; v0 < n_vec; v0 += parts * kWarpsPerCta * 32 * kVecs) {
    uint4 raw[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int j = v0 + u * 32 + lane;
      // whole pieces; -inf elsewhere, which the edges below overwrite
      const bool whole = j * E >= lead && (j + 1) * E <= lead + a.V;
      const uint32_t none = TYPE == MOE_T_F32 ? 0xff800000u : TYPE == MOE_T_BF16 ? 0xff80ff80u : 0xfc00fc00u;
      raw[u] = make_uint4(none, none, none, none);
      if (whole) raw[u] = __ldcs(reinterpret_cast<const uint4*>(base + (long long)j * 16));
    }
    float z[N];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (TYPE == MOE_T_F32) {
          z[u * E + i] = __uint_as_float(w[i]);
        } else {
          const float2 f = kv::unpack2<TYPE == MOE_T_F16>(w[i]);
          z[u * E + 2 * i] = f.x;
          z[u * E + 2 * i + 1] = f.y;
        }
      }
    }
    const auto id_of = [&](int i) { return (v0 + (i / E) * 32 + lane) * E + i % E - lead; };
    if (v0 == 0 || v0 + 32 * kVecs >= n_vec) {  // the row's first piece and its last
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        const int j = v0 + u * 32 + lane;
        if (j < n_vec && !(j * E >= lead && (j + 1) * E <= lead + a.V)) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int id = j * E + e - lead;
            if (id >= 0 && id < a.V) z[u * E + e] = one(id);
          }
        }
      }
    }
    float mx = z[0];
#pragma unroll
    for (int i = 1; i < N; ++i) mx = max_nan(mx, z[i]);
    if (mx > p.m || mx != mx) {
      const float m = max_nan(p.m, mx), d = bounded((p.m - m) * c), e = kv::ex2(d);
      p.s = e * (p.s + p.l * d);
      p.l *= e;
      p.m = m;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float d = bounded((z[i] - p.m) * c), e = kv::ex2(d);
      p.l += e;
      p.s = fmaf(e, d, p.s);
    }
    if (!(mx < mine)) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float x = z[i] == z[i] ? z[i] : kNone;
        p.rank += x > mine || (x == mine && (unsigned)id_of(i) < (unsigned)token) ? 1 : 0;
      }
    }
    if (a.top) {
      floor = fmaxf(floor, *const_cast<volatile float*>(&sh.floor));
      if (__any_sync(0xffffffffu, !(mx < floor))) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float x = z[i] == z[i] ? z[i] : kNone;
          const int id = id_of(i);
          const Key key = (unsigned)id < (unsigned)a.V ? (Key)order_key(x) << 32 | (uint32_t)~id : 0;
          unsigned todo = __ballot_sync(0xffffffffu, key != 0 && x >= floor);
          while (todo) {
            const Key k = shfl_key(key, __ffs(todo) - 1);
            todo &= todo - 1;
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
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Part q;
    q.m = __shfl_xor_sync(0xffffffffu, p.m, o);
    q.l = __shfl_xor_sync(0xffffffffu, p.l, o);
    q.s = __shfl_xor_sync(0xffffffffu, p.s, o);
    q.rank = __shfl_xor_sync(0xffffffffu, p.rank, o);
    if (lane & o) {  // both sides of a pair join in the same order
      join(q, p, c);
      p = q;
    } else {
      join(p, q, c);
    }
  }
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
  const float ln_l = logf(p.l);
  const auto log_p = [&](float z) { return broken ? nan : empty ? kNone : (z - p.m) / a.temperature - ln_l; };
  if (lane == 0) {
    if (a.logprob) a.logprob[t] = has ? log_p(mine_raw) : 0.f;
    if (a.rank) a.rank[t] = has ? p.rank : -1;
    if (a.entropy) a.entropy[t] = broken ? nan : empty ? 0.f : fmaxf(ln_l - 0.6931471805599453f * (p.s / p.l), 0.f);
  }
  if (lane < a.top && a.top_ids) {
    const Key k = sh.key[0][lane];
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
  // CTAs per row: while there are fewer than two per SM and each has a chunk or
  // more for every warp.
  int parts = 1;
  const long long chunk = (long long)kThreads * kVecs * (a.type == MOE_T_F32 ? 4 : 8);
  while (parts < 8 && (long long)a.T * parts * 2 <= 304 && a.V >= chunk * parts) parts *= 2;
  if (a.type == MOE_T_F32) return launch_type<MOE_T_F32>(a, parts, st);
  return a.type == MOE_T_F16 ? launch_type<MOE_T_F16>(a, parts, st) : launch_type<MOE_T_BF16>(a, parts, st);
}

}  // namespace block
}  // namespace moe
