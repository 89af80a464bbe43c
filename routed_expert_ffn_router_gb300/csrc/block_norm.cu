// The residual's addition and the root-mean-square norm of its rows, in 16 or 32
// bits or in e4m3 with scales (include/moe_block.h).
//
// A CTA has a row at a time: a thread holds its values in registers from the one read
// of x and r to the write of y, so the row's sum of squares is the only exchange (a
// shuffle tree and one barrier). With more rows than the grid has CTAs (at most six, three
// or one per SM: see launch_rows) a CTA goes on
// to the row a grid further, whose loads are under way meanwhile; its weights stay in
// registers, widened, and its addresses go forward by a step. A pass over memory and
// nothing else; what kept it from memory's rate were instructions per value (the
// 8-bit form: 82 us with conversions chosen per value, divisions and a CTA per row, 47
// without, 44 with rows fetched ahead, 39.5 with the weights widened once).
//
// Measured, back to back in a graph: 8 rows of 2,048 (fp32 to a bf16 residual and
// result) 1.8 us, a launch's latency; 2,048 such rows 5.9 us for 42 MB (7.1 TB/s, part
// of it from the L2); 8,192 x 4,096 with residual to e4m3 39.5 us for 235 MB (6.0 TB/s,
// 0.88 of a copy's rate: what remains are the issue slots and the ends of rows). The grid
// suits 2,048 and 4,096 columns. Others, with 16-bit x, residual and result, the same
// buffers each call: 4,096 x 8,192 44 us (floor 40), 4,096 x 5,120 33 (25), 16,384 x 512 11
// (10, with help of the L2), but 65,536 x 128 36 us (floor 10), where an SM has six warps.
// Value by value, 4,096 x 5,121 takes 261 us (floor 25). The kernel for more than 8,192
// columns with fp32 among its types spills 112 bytes by stores and 56 by loads.
#include <atomic>

#include <type_traits>

#include "block_internal.h"
#include "kv_common.cuh"
#include "packed.cuh"

namespace moe {
namespace block {

namespace {

// 8 values as they lie in memory; WIDE: fp32 among the types of a call.
template <bool WIDE>
struct Raw;
template <>
struct Raw<false> {
  uint4 a;
};
template <>
struct Raw<true> {
  uint4 a, b;
};
template <bool WIDE>
__device__ __forceinline__ Raw<WIDE> load_raw(const void* p, int type, int i) {
  Raw<WIDE> r;
  if constexpr (WIDE) {
    if (type == MOE_T_F32) {
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
      r.a = q[0];
      r.b = q[1];
      return r;
    }
    r.b = make_uint4(0, 0, 0, 0);
  }
  r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  return r;
}
// (One branch around all eight values, not a choice per value: with both types'
// conversions and a select each, the instructions were what bound the kernel.)
template <bool WIDE>
__device__ __forceinline__ void widen(const Raw<WIDE>& r, int type, float2 (&f)[4]) {
  const auto two = [&](auto f16) {
    const uint32_t u[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = kv::unpack2<decltype(f16)::value>(u[i]);
  };
  if (type == MOE_T_BF16) {
    two(std::false_type());
  } else if (!WIDE || type == MOE_T_F16) {
    two(std::true_type());
  } else if constexpr (WIDE) {
    f[0] = make_float2(__uint_as_float(r.a.x), __uint_as_float(r.a.y));
    f[1] = make_float2(__uint_as_float(r.a.z), __uint_as_float(r.a.w));
    f[2] = make_float2(__uint_as_float(r.b.x), __uint_as_float(r.b.y));
    f[3] = make_float2(__uint_as_float(r.b.z), __uint_as_float(r.b.w));
  }
}
// Two e4m3 values, x in the low byte; to the nearest, saturating, NaN kept.
__device__ __forceinline__ uint32_t e4m3x2(float x, float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}
// Rounds f to `type` and writes it; f then holds what was written (but for e4m3).
__device__ __forceinline__ void store8(void* p, int type, int i, float2 (&f)[4]) {
  const auto two = [&](auto f16) {
    constexpr bool F16 = decltype(f16)::value;
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = kv::pack2<F16>(f[j].x, f[j].y);
      f[j] = kv::unpack2<F16>(u[j]);
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(u[0], u[1], u[2], u[3]);
  };
  if (type == MOE_T_BF16) {
    two(std::false_type());
  } else if (type == MOE_T_F16) {
    two(std::true_type());
  } else if (type == MOE_T_F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    q[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = e4m3x2(f[j].x, f[j].y);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p) + i) = make_uint2(u[0] | u[1] << 16, u[2] | u[3] << 16);
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
    static_cast<uint8_t*>(p)[i] = (uint8_t)e4m3x2(f, 0.f);
    return f;
  }
  const uint32_t u = type == MOE_T_F16 ? kv::pack2<true>(f, 0.f) : kv::pack2<false>(f, 0.f);
  static_cast<uint16_t*>(p)[i] = (uint16_t)u;
  return type == MOE_T_F16 ? kv::unpack2<true>(u).x : kv::unpack2<false>(u).x;
}

// What a value is multiplied by for its e4m3, in two factors: the reciprocal of a tiny
// scale would leave fp32.
struct Quant {
  float up, inv;
};
__device__ __forceinline__ Quant quant_of(float scale) {
  const float up = scale < 1e-30f ? 0x1p100f : 1.f;
  return {up, scale == 0.f ? 0.f : __fdividef(1.f, scale * up)};
}

struct Args {
  moe_norm_args a;
  float inv_H;
  int shift, n_groups;  // log2 of a group's columns (of a power of two: not the whole row), groups of a row
};

// The sum of s over the CTA (all threads); part: a buffer that the row before did not use.
__device__ __forceinline__ float cta_sum(float s, float* part) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  s = lane < (blockDim.x >> 5) ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Rows on 16-byte boundaries: NV pieces of 8 values per thread.
template <int NV, bool FP8, bool WIDE, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 1024 ? 1 : (WIDE ? 1280 : 1536) / MAXT) norm_kernel(const __grid_constant__ Args g) {
  __shared__ float part[2][32];
  __shared__ int row_max[2];  // e4m3 with one scale a row, or groups wider than a warp: see below
  extern __shared__ int group_max[];
  const moe_norm_args& a = g.a;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
  griddep_wait();
  griddep_launch_dependents();
  Raw<WIDE> rx[NV], rr[NV];
  // the row that is fetched next, and the one that is written
  const int xs = a.x_type == MOE_T_F32 ? 4 : 2, rs = a.res_type == MOE_T_F32 ? 4 : 2, ys = FP8 ? 1 : a.y_type == MOE_T_F32 ? 4 : 2;
  int t = blockIdx.x;
  const char* x = static_cast<const char*>(a.x) + t * a.x_stride * xs;
  char* res = static_cast<char*>(a.res) + t * a.res_stride * rs;
  char* y = static_cast<char*>(a.y) + t * a.y_stride * ys;
  float* scales = FP8 ? a.scales + (long long)t * g.n_groups : nullptr;
  const long long x_step = gridDim.x * a.x_stride * xs, r_step = gridDim.x * a.res_stride * rs, y_step = gridDim.x * a.y_stride * ys;
  const auto fetch = [&](const char* r) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * nt + tid) * 8;
      if (c < a.H) {
        rx[j] = load_raw<WIDE>(x, a.x_type, c);
        if (a.res) rr[j] = load_raw<WIDE>(r, a.res_type, c);
      }
    }
  };
  fetch(res);
  float2 w[NV][4];  // the weights, their offset added
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * nt + tid) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[j][i] = make_float2(1.f, 1.f);
    if (a.w && c < a.H) {
      const Raw<WIDE> rw = load_raw<WIDE>(a.w, a.w_type, c);
      widen(rw, a.w_type, w[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[j][i] = add2(w[j][i], make_float2(a.w_offset, a.w_offset));
    }
  }
  for (int turn = 0;; turn ^= 1) {
    float2 r[NV][4];
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * nt + tid) * 8;
      if (c < a.H) {
        widen(rx[j], a.x_type, r[j]);
        if (a.res) {
          float2 f[4];
          widen(rr[j], a.res_type, f);
#pragma unroll
          for (int i = 0; i < 4; ++i) r[j][i] = add2(r[j][i], f[i]);
          store8(res, a.res_type, c, r[j]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[j][i] = make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sum = fma2(r[j][i], r[j][i], sum);
    }
    t += gridDim.x;
    x += x_step;
    res += r_step;
    if (t < a.T) fetch(res);
    if (FP8 && g.shift < 0 && tid == 0) row_max[turn] = 0;
    const float root = rsqrtf(cta_sum(sum.x + sum.y, part[turn]) * g.inv_H + a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[j][i] = mul2(mul2(r[j][i], make_float2(root, root)), w[j][i]);
    }
    if constexpr (!FP8) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * nt + tid) * 8;
        if (c < a.H) store8(y, a.y_type, c, r[j]);
      }
    } else {
      // The largest magnitude: a group of up to 256 columns lies within a warp; a wider
      // one takes its warps' together through shared memory, as does a whole row.
      float m[NV];
      const int lanes = g.shift >= 0 && g.shift < 8 ? 1 << (g.shift - 3) : 32;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        m[j] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) m[j] = fmaxf(m[j], fmaxf(fabsf(r[j][i].x), fabsf(r[j][i].y)));
        if ((j * nt + tid) * 8 >= a.H) m[j] = 0.f;
        for (int o = 1; o < lanes; o <<= 1) m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], o));
      }
      if (g.shift < 0) {
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) top = fmaxf(top, m[j]);
        if (lane == 0) atomicMax(&row_max[turn], __float_as_int(top));
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NV; ++j) m[j] = __int_as_float(row_max[turn]);
        if (tid == 0) scales[0] = m[0] * (1.f / 448.f);
      } else if (g.shift > 8) {
        __syncthreads();  // the row before has been read
        for (int i = tid; i < g.n_groups; i += nt) group_max[i] = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = (j * nt + tid) * 8;
          if (lane == 0 && c < a.H) atomicMax(&group_max[c >> g.shift], __float_as_int(m[j]));
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = (j * nt + tid) * 8;
          if (c < a.H) m[j] = __int_as_float(group_max[c >> g.shift]);
        }
        for (int i = tid; i < g.n_groups; i += nt) scales[i] = __int_as_float(group_max[i]) * (1.f / 448.f);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * nt + tid) * 8;
        if (c >= a.H) continue;
        const float scale = m[j] * (1.f / 448.f);
        if (g.shift >= 0 && g.shift <= 8 && (c & ((1 << g.shift) - 1)) == 0) scales[c >> g.shift] = scale;
        const Quant q = quant_of(scale);
        if (q.up != 1.f)
#pragma unroll
          for (int i = 0; i < 4; ++i) r[j][i] = mul2(r[j][i], make_float2(q.up, q.up));
#pragma unroll
        for (int i = 0; i < 4; ++i) r[j][i] = mul2(r[j][i], make_float2(q.inv, q.inv));
        store8(y, MOE_T_E4M3, c, r[j]);
      }
    }
    if (t >= a.T) break;
    y += y_step;
    if (FP8) scales += (long long)gridDim.x * g.n_groups;
  }
}

// Any alignment and row length, value by value: value j of a thread is column
// j * threads + thread.
template <int NV>
__global__ void __launch_bounds__(NV == 8 ? 1024 : 512) norm_values_kernel(const __grid_constant__ Args g) {
  __shared__ float part[32];
  extern __shared__ int group_max[];
  const moe_norm_args& a = g.a;
  const int tid = threadIdx.x, nt = blockDim.x;
  griddep_wait();
  griddep_launch_dependents();
  const long long t = blockIdx.x, xo = t * a.x_stride, ro = t * a.res_stride, yo = t * a.y_stride;
  const bool fp8 = a.y_type == MOE_T_E4M3;
  const auto group_of = [&](int c) { return g.shift < 0 ? 0 : c >> g.shift; };
  if (fp8)
    for (int i = tid; i < g.n_groups; i += nt) group_max[i] = 0;
  float r[NV], s = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = j * nt + tid;
    r[j] = 0.f;
    if (c < a.H) {
      r[j] = load1(a.x, a.x_type, xo + c);
      if (a.res) r[j] = store1(a.res, a.res_type, ro + c, r[j] + load1(a.res, a.res_type, ro + c));
    }
    s = fmaf(r[j], r[j], s);
  }
  const float root = rsqrtf(cta_sum(s, part) * g.inv_H + a.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = j * nt + tid;
    if (c >= a.H) continue;
    r[j] *= root;
    if (a.w) r[j] *= load1(a.w, a.w_type, c) + a.w_offset;
    if (fp8) atomicMax(&group_max[group_of(c)], __float_as_int(fmaxf(0.f, fabsf(r[j]))));
    else store1(a.y, a.y_type, yo + c, r[j]);
  }
  if (!fp8) return;
  __syncthreads();
  for (int i = tid; i < g.n_groups; i += nt) a.scales[t * g.n_groups + i] = __int_as_float(group_max[i]) * (1.f / 448.f);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = j * nt + tid;
    if (c >= a.H) continue;
    const Quant q = quant_of(__int_as_float(group_max[group_of(c)]) * (1.f / 448.f));
    store1(a.y, a.y_type, yo + c, r[j] * q.up * q.inv);
  }
}

// A grid of what fits on the GPU at once with the most threads that this kernel is launched
// with, or a CTA per row where there are fewer: for less wide rows more CTAs would fit (the
// figures at the top), and no more than this are launched.
template <int NV, bool FP8, bool WIDE, int MAXT>
cudaError_t launch_rows(const Args& g, int threads, size_t smem, cudaStream_t st) {
  static std::atomic<int> fits{0};
  int n = fits.load(std::memory_order_relaxed);
  if (n == 0) {
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, norm_kernel<NV, FP8, WIDE, MAXT>, MAXT, 0);
    if (e != cudaSuccess) return e;
    n = sms * (per_sm > 0 ? per_sm : 1);
    fits.store(n, std::memory_order_relaxed);
  }
  const int grid = g.a.T < n ? g.a.T : n;
  return launch_pdl(K_NORM, norm_kernel<NV, FP8, WIDE, MAXT>, dim3(grid), threads, smem, st, g);
}
template <bool FP8, bool WIDE>
cudaError_t launch_types(const Args& g, size_t smem, cudaStream_t st) {
  const int per = g.a.H / 8;  // pieces of a row
  const int nv = per <= 1024 ? 1 : 2, threads = ((per + nv - 1) / nv + 31) / 32 * 32;
  if (nv == 2) return launch_rows<2, FP8, WIDE, 1024>(g, threads, smem, st);
  if (threads <= 256) return launch_rows<1, FP8, WIDE, 256>(g, threads, smem, st);
  if (threads <= 512) return launch_rows<1, FP8, WIDE, 512>(g, threads, smem, st);
  return launch_rows<1, FP8, WIDE, 1024>(g, threads, smem, st);
}

}  // namespace

cudaError_t launch_rms_norm(const moe_norm_args& a, bool vec, cudaStream_t st) {
  Args g;
  g.a = a;
  g.inv_H = 1.f / (float)a.H;
  g.n_groups = a.group ? a.H / a.group : 1;
  g.shift = -1;
  if (a.group)
    for (g.shift = 0; (1 << g.shift) < a.group;) ++g.shift;
  const bool fp8 = a.y_type == MOE_T_E4M3;
  const size_t smem = fp8 ? (size_t)g.n_groups * 4 : 0;
  if (!vec) {
    const int nv = a.H <= 8192 ? 8 : 32, threads = ((a.H + nv - 1) / nv + 31) / 32 * 32;
    return nv == 8 ? launch_pdl(K_NORM, norm_values_kernel<8>, dim3(a.T), threads, smem, st, g)
                   : launch_pdl(K_NORM, norm_values_kernel<32>, dim3(a.T), threads, smem, st, g);
  }
  const bool wide = a.x_type == MOE_T_F32 || (a.res && a.res_type == MOE_T_F32) || (a.w && a.w_type == MOE_T_F32);
  if (fp8) return wide ? launch_types<true, true>(g, smem, st) : launch_types<true, false>(g, smem, st);
  return wide ? launch_types<false, true>(g, smem, st) : launch_types<false, false>(g, smem, st);
}

}  // namespace block
}  // namespace moe
