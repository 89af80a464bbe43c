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

bool pool_maps(const Cache& c, CUtensorMap* k, CUtensorMap* v, int box_rows) {
  const auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {64, (cuuint64_t)c.n_pages * c.Hkv * c.page, (cuuint64_t)c.D / 64};
  const cuuint64_t str[2] = {(cuuint64_t)c.D * 2, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)c.D / 64};
  const cuuint32_t es[3] = {1, 1, 1};
  for (int i = 0; i < 2; ++i)
    if (fn(i ? v : k, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, i ? c.v : c.k, dims, str, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  return true;
}

}  // namespace kv
}  // namespace moe
