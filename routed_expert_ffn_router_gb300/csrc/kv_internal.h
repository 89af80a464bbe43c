// Internal declarations of the paged key-value cache's translation units.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "moe_internal.h"
#include "moe_kv.h"

namespace moe {
namespace kv {

enum : int32_t {
  DEV_NO_PAGES = 32,   // a page operation needs more free pages than there are
  DEV_REFUSED = 64,    // a page operation refuses an argument
};

// Device view of a cache (one layer's pools for the calls that take a layer).
struct Cache {
  uint16_t *k, *v;
  int n_layers, n_pages, page, Hkv, D, n_slots, max_pages;
  int32_t *table, *lens, *refs, *free_pages, *n_free;
};

// The rows of a call: sequence b has rows row_start[b] .., or n_q each.
struct Rows {
  int B, n_rows, n_q;
  const int32_t *slots, *row_start;
};

struct Attn {
  int Hq, G, window, n_sink;
  float scale;
  const uint16_t *q;
  long long q_stride;
  uint16_t *o;
  float *lse;
};

// Workspace: the head (status word, cross-CTA counters), then one region that
// each call lays out for itself.
size_t pages_ws_bytes(int n_pages, int n);

// One sequence of a call, as the device sees it.
struct Seq {
  int slot;    // -1: out of range
  int len;     // tokens, at most max_pages * page
  int row0, n; // its rows
};

__device__ __forceinline__ Seq load_seq(const Cache& c, const Rows& r, int b, int32_t* status) {
  Seq s;
  s.row0 = r.row_start ? r.row_start[b] : b * r.n_q;
  const int row1 = r.row_start ? r.row_start[b + 1] : s.row0 + r.n_q;
  s.row0 = max(0, min(s.row0, r.n_rows));
  s.n = max(0, min(row1, r.n_rows) - s.row0);
  s.slot = r.slots ? r.slots[b] : b;
  s.len = 0;
  if (s.slot < 0 || s.slot >= c.n_slots) {
    if (status) atomicOr(status, DEV_BAD_SLOT);
    s.slot = -1;
    return s;
  }
  const long long cap = (long long)c.max_pages * c.page;
  int len = c.lens[s.slot];
  if (len > cap) {
    if (status) atomicOr(status, DEV_BAD_SLOT);
    len = (int)cap;
  }
  s.len = max(0, len);
  return s;
}

// Launch that may be scheduled before the stream's previous kernel has ended:
// a kernel launched this way waits (griddep_wait) before it touches memory and
// then lets its own successor be scheduled, so that in a chain of short calls
// a kernel's launch latency and prologue are paid during the one before.
template <class... P, class... A>
cudaError_t launch_pdl(int kind, void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  launch_begin(kind, st);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(a)...);
  launch_end(st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_append(const Cache& c, const Rows& r, const uint16_t* k, const uint16_t* v, long long stride,
                          int32_t* status, cudaStream_t st);
cudaError_t launch_append_rope(const Cache& c, const Rows& r, const moe_rope_desc& d, const int32_t* positions, int Hq,
                               const uint16_t* q, long long q_stride, uint16_t* q_out, long long q_out_stride, const uint16_t* k,
                               const uint16_t* v, long long stride, bool f16, int32_t* status, cudaStream_t st);
cudaError_t launch_attn_rows(const Cache& c, const Rows& r, const Attn& a, bool f16, bool decode, int32_t* status,
                             cudaStream_t st);
// The one-launch decode kernel (kv_decode.cu): D 64 or 128, pages of a power of
// two of at least 8 tokens.
bool decode_supported(int D, int page, int Hkv, int G, int n_q, int max_pages);
size_t decode_ws_bytes(int page, int max_pages, int Hkv, int G, int D, int max_rows);
cudaError_t launch_attn_decode(const Cache& c, const Rows& r, const Attn& a, bool f16, int32_t* status, int32_t* sync,
                               void* scratch, cudaStream_t st);
// The tensor-core prompt-chunk kernels (kv_chunk.cu): D 64 or 128, pages of a
// power of two of at least 8 tokens, up to 128 query heads per KV head, a scale
// above zero.
bool chunk_supported(int D, int page, int Hkv, int G, int B, int n_rows, int max_pages, float scale);
size_t chunk_ws_bytes(int D);
cudaError_t launch_attn_chunk(const Cache& c, const Rows& r, const Attn& a, bool f16, int32_t* status, int32_t* sync,
                              void* scratch, cudaStream_t st);
cudaError_t launch_grow(const Cache& c, const int32_t* slots, const int32_t* add, int n, int32_t* status, void* scratch,
                        cudaStream_t st);
cudaError_t launch_fork(const Cache& c, const int32_t* src, const int32_t* dst, int n, int32_t* status, void* scratch,
                        cudaStream_t st);
cudaError_t launch_free(const Cache& c, const int32_t* slots, int n, int32_t* status, cudaStream_t st);
cudaError_t launch_compact(const Cache& c, int32_t* n_moved, int32_t* status, void* scratch, cudaStream_t st);
cudaError_t launch_copy_pages(const Cache& c, const int32_t* src, const int32_t* dst, int n, int32_t* status,
                              cudaStream_t st);

}  // namespace kv
}  // namespace moe
