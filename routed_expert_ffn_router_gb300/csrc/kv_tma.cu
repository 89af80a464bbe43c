// TMA descriptors of the cache's pools.
#include "kv_tma.h"

#include <mutex>

namespace moe {
namespace kv {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    else
      cudaGetLastError();
  });
  return fn;
}

namespace {
bool encode(CUtensorMap* m, void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  const auto fn = encode_fn();
  const cuuint32_t es[3] = {1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, rank, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace

bool pool_maps(const Cache& c, CUtensorMap* k, CUtensorMap* v, int box_rows) {
  const cuuint64_t dims[3] = {64, (cuuint64_t)c.n_pages * c.Hkv * c.page, (cuuint64_t)c.D / 64};
  const cuuint64_t str[2] = {(cuuint64_t)c.D * 2, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)c.D / 64};
  return encode(k, c.k, 3, dims, str, box) && encode(v, c.v, 3, dims, str, box);
}

bool pool_maps_2d(const Cache& c, CUtensorMap* k, CUtensorMap* v, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)c.D, (cuuint64_t)c.n_pages * c.Hkv * c.page};
  const cuuint64_t str[1] = {(cuuint64_t)c.D * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  return encode(k, c.k, 2, dims, str, box) && encode(v, c.v, 2, dims, str, box);
}

bool query_map(const Attn& a, int D, int n_rows, int tq, CUtensorMap* q) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.Hq, (cuuint64_t)n_rows};
  const cuuint64_t str[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.q_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)a.G, (cuuint32_t)tq};
  return encode(q, const_cast<uint16_t*>(a.q), 3, dims, str, box);
}

}  // namespace kv
}  // namespace moe
