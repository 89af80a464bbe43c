// The residual's addition and the root-mean-square norm of its rows, in 16 or 32
// bits or in e4m3 with scales (include/moe_block.h).
//
// One CTA per row: a thread holds its values of the row in registers from the one
// read of x and r to the write of y, so the row's sum of squares is the only
// exchange (a shuffle tree and one barrier). A pass over memory and nothing else:
// the raw loads of x, r and w are issued together before anything waits for them.
#include <cuda_fp8.h>

#include "block_internal.h"
#include "kv_common.cuh"

namespace moe {
namespace block {

namespace {

struct Raw {
  uint4 a, b;  // 8 values: 16 bytes, or 32 in fp32
};
__device__ __forceinline__ Raw load_raw(const void* p, int type, long long i) {
  Raw r;
  if (type == MOE_T_F32) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
    r.a = q[0];
    r.b = q[1];
  } else {
    r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    r.b = make_uint4(0, 0, 0, 0);
  }
  return r;
}
__device__ __forceinline__ void widen(const Raw& r, int type, float (&f)[8]) {
  const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  if (type == MOE_T_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = type == MOE_T_F16 ? kv::unpack2<true>(u[i]) : kv::unpack2<false>(u[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
}
// Rounds f to `type` and writes it; f then holds what was written.
__device__ __forceinline__ void store8(void* p, int type, long long i, float (&f)[8]) {
  if (type == MOE_T_F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else if (type == MOE_T_E4M3) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * j], f[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p) + i) = make_uint2(u[0] | u[1] << 16, u[2] | u[3] << 16);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = type == MOE_T_F16 ? kv::pack2<true>(f[2 * j], f[2 * j + 1]) : kv::pack2<false>(f[2 * j], f[2 * j + 1]);
      const float2 t = type == MOE_T_F16 ? kv::unpack2<true>(u[j]) : kv::unpack2<false>(u[j]);
      f[2 * j] = t.x;
      f[2 * j + 1] = t.y;
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}
__device__ __forceinline__ float load1(const void* p, int type, long long i) {
  if (type == MOE_T_F32) return static_cast<const float*>(p)[i];
  const uint32_t u = static_cast<const uint16_t*>(p)[i];
  return type == MOE_T_F16 ? kv::unpack2<true>(u).x : kv::unpack2<false>(u).x;
}
__device__ __forceinline__ float store1(void* p, int type, long long i, float f) {
  if (type == MOE_T_F32) {
    static_cast<float*>(p)[i] = f;
    return f;
  }
  if (type == MOE_T_E4M3) {
    static_cast<uint8_t*>(p)[i] = __nv_cvt_float_to_fp8(f, __NV_SATFINITE, __NV_E4M3);
    return f;
  }
  const uint32_t u = type == MOE_T_F16 ? kv::pack2<true>(f, 0.f) : kv::pack2<false>(f, 0.f);
  static_cast<uint16_t*>(p)[i] = (uint16_t)u;
  return type == MOE_T_F16 ? kv::unpack2<true>(u).x : kv::unpack2<false>(u).x;
}

// What a value of a group is multiplied by for its e4m3, in two factors: the
// reciprocal of a tiny scale would leave fp32.
struct Quant {
  float up, inv;
};
__device__ __forceinline__ Quant quant_of(float scale) {
  const float up = scale < 1e-30f ? 0x1p100f : 1.f;
  return {up, scale == 0.f ? 0.f : 1.f / (scale * up)};
}

// NV groups of 8 values per thread. VEC: 8 values that lie together (16-byte
// loads); else value j of a thread is column j * threads + thread (rows whose
// alignment allows single values only).
template <int NV, bool VEC>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) norm_kernel(const __grid_constant__ moe_norm_args a) {
  extern __shared__ int group_max[];  // e4m3: largest magnitude of each group, as bits (they are not negative)
  __shared__ float part[32];
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const long long t = blockIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const long long xo = t * a.x_stride, ro = t * a.res_stride, yo = t * a.y_stride;
  const bool fp8 = a.y_type == MOE_T_E4M3;
  const int G = a.group ? a.group : a.H, n_groups = a.H / G;
  if (fp8)
    for (int i = tid; i < n_groups; i += nt) group_max[i] = 0;

  float r[NV][8];
  Raw rw[NV];
  if constexpr (VEC) {
    Raw rx[NV], rr[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * nt + tid) * 8;
      if (c < a.H) {
        rx[j] = load_raw(a.x, a.x_type, xo + c);
        if (a.res) rr[j] = load_raw(a.res, a.res_type, ro + c);
        if (a.w) rw[j] = load_raw(a.w, a.w_type, c);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * nt + tid) * 8;
      if (c < a.H) {
        widen(rx[j], a.x_type, r[j]);
        if (a.res) {
          float f[8];
          widen(rr[j], a.res_type, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) r[j][i] += f[i];
          store8(a.res, a.res_type, ro + c, r[j]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[j][i] = 0.f;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (j * 8 + i) * nt + tid;
        r[j][i] = 0.f;
        if (c < a.H) {
          r[j][i] = load1(a.x, a.x_type, xo + c);
          if (a.res) r[j][i] = store1(a.res, a.res_type, ro + c, r[j][i] + load1(a.res, a.res_type, ro + c));
        }
      }
  }

  float s = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(r[j][i], r[j][i], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) part[warp] = s;
  __syncthreads();
  s = lane < (nt >> 5) ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float root = 1.f / sqrtf(s / (float)a.H + a.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float w[8];
    if constexpr (VEC) {
      if (a.w) widen(rw[j], a.w_type, w);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (j * 8 + i) * nt + tid;
        w[i] = a.w && c < a.H ? load1(a.w, a.w_type, c) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) r[j][i] = a.w ? r[j][i] * root * (w[i] + a.w_offset) : r[j][i] * root;
  }

  if (!fp8) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (VEC) {
        const int c = (j * nt + tid) * 8;
        if (c < a.H) store8(a.y, a.y_type, yo + c, r[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = (j * 8 + i) * nt + tid;
          if (c < a.H) store1(a.y, a.y_type, yo + c, r[j][i]);
        }
      }
    }
    return;
  }

  // e4m3. A group of up to 256 columns lies within a warp (G / 8 lanes, H a
  // multiple of G): its maximum by shuffles alone. A wider one, or the whole row,
  // through shared memory.
  const bool in_warp = VEC && G <= 256 && a.group;
  float scale[NV];
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * nt + tid) * 8;
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(c < a.H ? r[j][i] : 0.f));
      const int lanes = in_warp ? G >> 3 : 32;
      for (int o = 1; o < lanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      scale[j] = m / 448.f;
      // a warp's 256 columns are of one wide group
      if (!in_warp && lane == 0 && c < a.H) atomicMax(&group_max[c / G], __float_as_int(m));
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (j * 8 + i) * nt + tid;
        if (c < a.H) atomicMax(&group_max[c / G], __float_as_int(fmaxf(0.f, fabsf(r[j][i]))));
      }
  }
  if (!in_warp) {
    __syncthreads();
    for (int i = tid; i < n_groups; i += nt) a.scales[t * n_groups + i] = __int_as_float(group_max[i]) / 448.f;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if constexpr (VEC) {
      const int c = (j * nt + tid) * 8;
      if (c >= a.H) continue;
      const float sc = in_warp ? scale[j] : __int_as_float(group_max[c / G]) / 448.f;
      if (in_warp && c % G == 0) a.scales[t * n_groups + c / G] = sc;
      const Quant q = quant_of(sc);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[j][i] = r[j][i] * q.up * q.inv;
      store8(a.y, a.y_type, yo + c, r[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (j * 8 + i) * nt + tid;
        if (c >= a.H) continue;
        const Quant q = quant_of(__int_as_float(group_max[c / G]) / 448.f);
        store1(a.y, a.y_type, yo + c, r[j][i] * q.up * q.inv);
      }
    }
  }
}

template <int NV>
cudaError_t launch_nv(const moe_norm_args& a, bool vec, int threads, size_t smem, cudaStream_t st) {
  return vec ? launch_pdl(K_NORM, norm_kernel<NV, true>, dim3(a.T), threads, smem, st, a)
             : launch_pdl(K_NORM, norm_kernel<NV, false>, dim3(a.T), threads, smem, st, a);
}

}  // namespace

cudaError_t launch_rms_norm(const moe_norm_args& a, bool vec, cudaStream_t st) {
  const int per = (a.H + 7) / 8;  // groups of 8 values of a row
  const int nv = per <= 1024 ? 1 : 4;
  const int threads = ((per + nv - 1) / nv + 31) / 32 * 32;
  const size_t smem = a.y_type == MOE_T_E4M3 ? (size_t)(a.H / (a.group ? a.group : a.H)) * 4 : 0;
  return nv == 1 ? launch_nv<1>(a, vec, threads, smem, st) : launch_nv<4>(a, vec, threads, smem, st);
}

}  // namespace block
}  // namespace moe
