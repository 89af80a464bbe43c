// C ABI of the paged key-value cache and its attention (include/moe_kv.h):
// argument validation, workspace layout, choice of kernel.
#include <algorithm>
#include <climits>

#include "kv_internal.h"

using namespace moe;
using namespace moe::kv;

namespace {

constexpr int kMostHeads = 65535;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

moe_status check_kv(const moe_kv_desc* d) {
  if (!d) return MOE_ERR_INVALID;
  if (d->dtype != MOE_KV_BF16 && d->dtype != MOE_KV_F16) return MOE_ERR_INVALID;
  if (d->n_layers < 1 || d->n_pages < 1 || d->page_size < 1 || d->Hkv < 1 || d->D < 1 || d->n_slots < 1 ||
      d->max_pages < 1)
    return MOE_ERR_INVALID;
  if (!d->k || !d->v || !d->table || !d->lens || !d->refs || !d->free_pages || !d->n_free) return MOE_ERR_INVALID;
  if (!aligned(d->k, 16) || !aligned(d->v, 16) || !aligned(d->table, 4) || !aligned(d->lens, 4) ||
      !aligned(d->refs, 4) || !aligned(d->free_pages, 4) || !aligned(d->n_free, 4))
    return MOE_ERR_INVALID;
  if (d->D % 8 || d->D > 256 || d->max_pages > (1 << 20) || d->n_slots > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  // rows of one layer's pool, tokens of one slot
  if ((int64_t)d->Hkv * d->page_size > INT32_MAX || (int64_t)d->Hkv * d->page_size * d->n_pages > INT32_MAX ||
      (int64_t)d->max_pages * d->page_size > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

Cache cache_of(const moe_kv_desc* d, int layer) {
  const size_t off = (size_t)layer * d->n_pages * d->Hkv * d->page_size * d->D;
  Cache c;
  c.k = static_cast<uint16_t*>(d->k) + off;
  c.v = static_cast<uint16_t*>(d->v) + off;
  c.n_layers = d->n_layers; c.n_pages = d->n_pages; c.page = d->page_size; c.Hkv = d->Hkv; c.D = d->D;
  c.n_slots = d->n_slots; c.max_pages = d->max_pages;
  c.table = d->table; c.lens = d->lens; c.refs = d->refs; c.free_pages = d->free_pages; c.n_free = d->n_free;
  return c;
}

moe_status check_rows(const moe_kv_desc* d, int32_t layer, const moe_kv_rows* r) {
  if (!r || layer < 0 || layer >= d->n_layers || r->B < 0 || r->n_rows < 0) return MOE_ERR_INVALID;
  if (!aligned(r->slots, 4) || !aligned(r->row_start, 4)) return MOE_ERR_INVALID;
  if (r->n_rows > 0 && r->B < 1) return MOE_ERR_INVALID;
  if (r->B > 0 && !r->row_start && r->n_rows % r->B) return MOE_ERR_INVALID;
  return MOE_OK;
}

Rows rows_of(const moe_kv_rows* r) {
  Rows o;
  o.B = r->B;
  o.n_rows = r->n_rows;
  o.n_q = r->row_start ? 0 : r->n_rows / r->B;
  o.slots = r->slots;
  o.row_start = r->row_start;
  return o;
}

// The workspace: the head that moe_workspace_init zeroes, then one region that
// every call lays out for itself. The kernel for any head and page size has none.
bool tiled(const moe_kv_desc* d) {
  return (d->D == 64 || d->D == 128) && d->page_size >= 8 && !(d->page_size & (d->page_size - 1));
}
size_t decode_region(const moe_kv_desc* d, int32_t Hq, int32_t max_rows) {
  return tiled(d) ? decode_ws_bytes(d->page_size, d->max_pages, d->Hkv, Hq / d->Hkv, d->D, max_rows) : 0;
}
size_t chunk_region(const moe_kv_desc* d) { return tiled(d) ? chunk_ws_bytes(d->D) : 0; }

moe_status check_ws(const void* ws, size_t ws_bytes, size_t region) {
  if (!ws || !aligned(ws, 256) || ws_bytes < kWsHeadBytes + region) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

int32_t* status_of(void* ws) { return static_cast<int32_t*>(ws); }
int32_t* sync_of(void* ws) { return reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + 512); }  // kSyncInts counters
void* region_of(void* ws) { return static_cast<uint8_t*>(ws) + kWsHeadBytes; }

moe_status attention(const moe_kv_desc* d, int32_t layer, const moe_kv_rows* r, const moe_attn_args* a, void* ws,
                     size_t ws_bytes, void* stream, bool decode) {
  launch_count_reset();
  moe_status s = check_kv(d);
  if (s != MOE_OK) return s;
  if ((s = check_rows(d, layer, r)) != MOE_OK) return s;
  if (!a || a->Hq < 1 || a->Hq % d->Hkv || a->window < 0 || a->n_sink < 0) return MOE_ERR_INVALID;
  if (!(a->scale > -3.0e38f && a->scale < 3.0e38f)) return MOE_ERR_INVALID;
  if (decode && r->row_start) return MOE_ERR_INVALID;
  if (decode && r->B > 0 && r->n_rows / r->B > 16) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)a->Hq * r->n_rows > INT32_MAX || a->Hq > kMostHeads) return MOE_ERR_UNSUPPORTED;
  if (r->n_rows == 0) return MOE_OK;
  if (!a->q || !a->o || !aligned(a->q, 16) || !aligned(a->o, 16) || !aligned(a->lse, 4)) return MOE_ERR_INVALID;
  if (a->q_stride % 8 || a->q_stride < (int64_t)a->Hq * d->D) return MOE_ERR_INVALID;
  if ((s = check_ws(ws, ws_bytes, decode ? decode_region(d, a->Hq, r->n_rows) : chunk_region(d))) != MOE_OK) return s;
  const Cache c = cache_of(d, layer);
  const Rows rw = rows_of(r);
  Attn at;
  // Neither a window nor first tokens beyond what a table holds mean more than all
  // of it: bounded so, their sums with tokens' positions stay in int32.
  const int32_t most = d->max_pages * d->page_size;
  at.window = a->window < most ? a->window : most;
  at.n_sink = a->n_sink < most ? a->n_sink : most;
  at.Hq = a->Hq; at.G = a->Hq / d->Hkv; at.scale = a->scale;
  at.q = static_cast<const uint16_t*>(a->q);
  at.q_stride = a->q_stride;
  at.o = static_cast<uint16_t*>(a->o);
  at.lse = a->lse;
  const bool f16 = d->dtype == MOE_KV_F16;
  if (decode && decode_supported(d->D, d->page_size, d->Hkv, at.G, rw.n_q, d->max_pages))
    return cuda_status(launch_attn_decode(c, rw, at, f16, status_of(ws), sync_of(ws), region_of(ws),
                                          static_cast<cudaStream_t>(stream)));
  if (!decode && chunk_supported(d->D, d->page_size, d->Hkv, at.G, rw.B, rw.n_rows, d->max_pages, at.scale))
    return cuda_status(launch_attn_chunk(c, rw, at, f16, status_of(ws), sync_of(ws), region_of(ws),
                                         static_cast<cudaStream_t>(stream)));
  return cuda_status(launch_attn_rows(c, rw, at, f16, decode, status_of(ws), static_cast<cudaStream_t>(stream)));
}

// Checks shared by the page operations over n slots.
moe_status check_pages(const moe_kv_desc* d, int32_t n, void* ws, size_t ws_bytes) {
  launch_count_reset();
  moe_status s = check_kv(d);
  if (s != MOE_OK) return s;
  if (n < 0 || n > d->n_slots) return MOE_ERR_INVALID;
  return check_ws(ws, ws_bytes, pages_ws_bytes(d->n_pages, d->n_slots));
}

}  // namespace

extern "C" {

size_t moe_kv_workspace_bytes(const moe_kv_desc* d, int32_t Hq, int32_t max_rows) {
  if (check_kv(d) != MOE_OK || Hq < 1 || Hq > kMostHeads || Hq % d->Hkv || max_rows < 0) return 0;
  return kWsHeadBytes + std::max({pages_ws_bytes(d->n_pages, d->n_slots), decode_region(d, Hq, max_rows), chunk_region(d)});
}

moe_status moe_kv_append(const moe_kv_desc* d, int32_t layer, const moe_kv_rows* r, const void* k, const void* v,
                         int64_t row_stride, void* ws, size_t ws_bytes, void* stream) {
  launch_count_reset();
  moe_status s = check_kv(d);
  if (s != MOE_OK) return s;
  if ((s = check_rows(d, layer, r)) != MOE_OK) return s;
  if (r->n_rows == 0) return MOE_OK;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return MOE_ERR_INVALID;
  if (row_stride % 8 || row_stride < (int64_t)d->Hkv * d->D) return MOE_ERR_INVALID;
  if ((s = check_ws(ws, ws_bytes, 0)) != MOE_OK) return s;
  return cuda_status(launch_append(cache_of(d, layer), rows_of(r), static_cast<const uint16_t*>(k),
                                   static_cast<const uint16_t*>(v), row_stride, status_of(ws),
                                   static_cast<cudaStream_t>(stream)));
}

moe_status moe_kv_append_rope(const moe_kv_desc* d, int32_t layer, const moe_kv_rows* r, const moe_rope_desc* rope,
                              const int32_t* positions, int32_t Hq, const void* q, int64_t q_stride, void* q_out,
                              int64_t q_out_stride, const void* k, const void* v, int64_t row_stride, void* ws,
                              size_t ws_bytes, void* stream) {
  launch_count_reset();
  moe_status s = check_kv(d);
  if (s != MOE_OK) return s;
  if ((s = check_rows(d, layer, r)) != MOE_OK) return s;
  if (!rope || rope->rot < 2 || rope->rot % 2 || rope->rot > d->D) return MOE_ERR_INVALID;
  if (rope->layout != MOE_ROPE_HALF && rope->layout != MOE_ROPE_INTERLEAVED) return MOE_ERR_INVALID;
  if (!(rope->gain > -3.0e38f && rope->gain < 3.0e38f) || !rope->freq || !aligned(rope->freq, 8)) return MOE_ERR_INVALID;
  if (Hq < 1 || !aligned(positions, 4)) return MOE_ERR_INVALID;
  if (Hq > kMostHeads) return MOE_ERR_UNSUPPORTED;
  if (r->n_rows == 0) return MOE_OK;
  if (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16)) return MOE_ERR_INVALID;
  if (q_stride % 8 || q_stride < (int64_t)Hq * d->D || q_out_stride % 8 || q_out_stride < (int64_t)Hq * d->D)
    return MOE_ERR_INVALID;
  if (q == q_out && q_stride != q_out_stride) return MOE_ERR_INVALID;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return MOE_ERR_INVALID;
  if (row_stride % 8 || row_stride < (int64_t)d->Hkv * d->D) return MOE_ERR_INVALID;
  if ((s = check_ws(ws, ws_bytes, 0)) != MOE_OK) return s;
  return cuda_status(launch_append_rope(cache_of(d, layer), rows_of(r), *rope, positions, Hq, static_cast<const uint16_t*>(q),
                                        q_stride, static_cast<uint16_t*>(q_out), q_out_stride,
                                        static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), row_stride,
                                        d->dtype == MOE_KV_F16, status_of(ws), static_cast<cudaStream_t>(stream)));
}

moe_status moe_attn_decode(const moe_kv_desc* d, int32_t layer, const moe_kv_rows* r, const moe_attn_args* a, void* ws,
                           size_t ws_bytes, void* stream) {
  return attention(d, layer, r, a, ws, ws_bytes, stream, true);
}

moe_status moe_attn_chunk(const moe_kv_desc* d, int32_t layer, const moe_kv_rows* r, const moe_attn_args* a, void* ws,
                          size_t ws_bytes, void* stream) {
  return attention(d, layer, r, a, ws, ws_bytes, stream, false);
}

moe_status moe_kv_grow(const moe_kv_desc* d, const int32_t* slots, const int32_t* add, int32_t n, void* ws,
                       size_t ws_bytes, void* stream) {
  moe_status s = check_pages(d, n, ws, ws_bytes);
  if (s != MOE_OK || n == 0) return s;
  if (!slots || !add || !aligned(slots, 4) || !aligned(add, 4)) return MOE_ERR_INVALID;
  return cuda_status(launch_grow(cache_of(d, 0), slots, add, n, status_of(ws), region_of(ws),
                                 static_cast<cudaStream_t>(stream)));
}

moe_status moe_kv_fork(const moe_kv_desc* d, const int32_t* src, const int32_t* dst, int32_t n, void* ws,
                       size_t ws_bytes, void* stream) {
  moe_status s = check_pages(d, n, ws, ws_bytes);
  if (s != MOE_OK || n == 0) return s;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return MOE_ERR_INVALID;
  return cuda_status(launch_fork(cache_of(d, 0), src, dst, n, status_of(ws), region_of(ws),
                                 static_cast<cudaStream_t>(stream)));
}

moe_status moe_kv_free(const moe_kv_desc* d, const int32_t* slots, int32_t n, void* ws, size_t ws_bytes, void* stream) {
  moe_status s = check_pages(d, n, ws, ws_bytes);
  if (s != MOE_OK || n == 0) return s;
  if (!slots || !aligned(slots, 4)) return MOE_ERR_INVALID;
  return cuda_status(launch_free(cache_of(d, 0), slots, n, status_of(ws), static_cast<cudaStream_t>(stream)));
}

moe_status moe_kv_compact(const moe_kv_desc* d, int32_t* n_moved, void* ws, size_t ws_bytes, void* stream) {
  moe_status s = check_pages(d, 0, ws, ws_bytes);
  if (s != MOE_OK) return s;
  if (!aligned(n_moved, 4)) return MOE_ERR_INVALID;
  return cuda_status(launch_compact(cache_of(d, 0), n_moved, status_of(ws), region_of(ws), static_cast<cudaStream_t>(stream)));
}

moe_status moe_kv_copy_pages(const moe_kv_desc* d, const int32_t* src, const int32_t* dst, int32_t n, void* ws,
                             size_t ws_bytes, void* stream) {
  moe_status s = check_pages(d, 0, ws, ws_bytes);
  if (s != MOE_OK) return s;
  if (n < 0 || n > d->n_pages) return MOE_ERR_INVALID;
  if (n == 0) return MOE_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return MOE_ERR_INVALID;
  return cuda_status(launch_copy_pages(cache_of(d, 0), src, dst, n, status_of(ws),
                                       static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
