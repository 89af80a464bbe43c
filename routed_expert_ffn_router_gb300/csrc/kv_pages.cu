// Pages of the key-value cache: growing, forking, freeing and compacting
// slots, copying pages, and writing new tokens' keys and values.
//
// The bookkeeping (tables, lengths, reference counts, the free stack) lives in
// device memory and every decision is taken there, so a serving loop queues
// these calls without knowing how many pages they touch. Each operation that
// moves data is two launches: one CTA decides (block prefix sums give every
// new page its place in the free stack's order, so the outcome does not depend
// on timing), then the whole GPU copies and rewrites. The copies are bound by
// HBM, the small calls by the launches; the second launch of a pair is scheduled
// while the first runs.
//
// Measured: forking 4 slots over 48 layers (a page of 16 tokens each) and freeing
// them 8.6 us; 64 forks (82 MB of pages of 32 tokens) and their freeing 28 us,
// 5.8 TB/s read and written (0.86 of a measured copy); compacting 2.6 GB of moves
// 408 us, 6.4 TB/s (0.94).
#include "kv_common.cuh"

namespace moe {
namespace kv {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;

// Scratch of the page operations, int32: a header, then the move list (source
// page, destination page), the remapping of pages and one entry per slot.
constexpr int kHdr = 64;
struct Scratch {
  int32_t *hdr, *msrc, *mdst, *remap, *len, *rank;
};
__host__ __device__ Scratch scratch_of(void* p, int n_pages, int n_slots) {
  int32_t* b = static_cast<int32_t*>(p);
  Scratch s;
  s.hdr = b;
  s.msrc = b + kHdr;
  s.mdst = s.msrc + n_pages;
  s.remap = s.mdst + n_pages;
  s.len = s.remap + n_pages;
  s.rank = s.len + n_slots;
  return s;
}

// Exclusive prefix sum of v over the CTA's threads; total in *sum (all threads).
__device__ int block_scan(int v, int* sum, int* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // sh is free again
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int t = lane < nw ? sh[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    sh[lane] = t;
  }
  __syncthreads();
  *sum = sh[nw - 1];
  return (warp ? sh[warp - 1] : 0) + x - v;
}

// The first thing of every kernel here (launch_pdl).
__device__ __forceinline__ void start() {
  griddep_wait();
  griddep_launch_dependents();
}

__device__ __forceinline__ int pages_of(int len, int page) { return (int)(((long long)len + page - 1) / page); }

// ------------------------------------------------------------------ append
// One CTA per row; a thread moves 16-byte pieces of the row's keys and values.
__global__ void __launch_bounds__(128) append_kernel(Cache c, Rows r, const uint16_t* k, const uint16_t* v,
                                                     long long stride, int32_t* status) {
  const int t = blockIdx.x;
  start();
  const int vd = c.D >> 3, per = c.Hkv * vd;
  auto src = [&](int i) {
    const int j = i < per ? i : i - per;
    return reinterpret_cast<const uint4*>((i < per ? k : v) + (long long)t * stride) + j;
  };
  // the thread's first piece is on its way while the row's page is looked up
  uint4 x = make_uint4(0, 0, 0, 0);
  if (threadIdx.x < 2 * per) x = *src(threadIdx.x);
  const Seq s = load_seq(c, r, seq_of_row(r, t), threadIdx.x == 0 ? status : nullptr);
  if (s.slot < 0 || t < s.row0 || t >= s.row0 + s.n) return;
  const int tok = s.len - s.n + (t - s.row0);
  if (tok < 0) return;
  const int pg = c.table[(long long)s.slot * c.max_pages + tok / c.page];
  if (pg < 0 || pg >= c.n_pages) {
    if (threadIdx.x == 0) atomicOr(status, DEV_BAD_SLOT);
    return;
  }
  const long long base = (long long)pg * c.Hkv * c.page + tok % c.page;
  for (int i = threadIdx.x; i < 2 * per; i += blockDim.x) {
    if (i != threadIdx.x) x = *src(i);
    const int j = i < per ? i : i - per;
    const int h = j / vd, d = (j - h * vd) * 8;
    uint16_t* dst = (i < per ? c.k : c.v) + (base + (long long)h * c.page) * c.D + d;
    *reinterpret_cast<uint4*>(dst) = x;
  }
}

// ------------------------------------------------------------------ grow
__global__ void __launch_bounds__(kPlanThreads) grow_kernel(Cache c, const int32_t* slots, const int32_t* add, int n,
                                                            int32_t* status, Scratch s) {
  __shared__ int sh[32];
  __shared__ int bad;
  const int tid = threadIdx.x;
  start();
  if (tid == 0) bad = 0;
  __syncthreads();
  const long long cap = (long long)c.max_pages * c.page;
  const int nf = *c.n_free;
  long long total = 0;
  for (int b0 = 0; b0 < n; b0 += kPlanThreads) {
    const int i = b0 + tid;
    int need = 0;
    if (i < n) {
      const int slot = slots[i], a = add[i];
      const int len = slot >= 0 && slot < c.n_slots ? c.lens[slot] : -1;
      if (len < 0 || a < 0 || (long long)len + a > cap) bad = 1;
      else need = pages_of(len + a, c.page) - pages_of(len, c.page);
      s.len[i] = len;
    }
    int sum;
    const int x = block_scan(need, &sum, sh);
    if (i < n) s.rank[i] = (int)(total < nf ? total : nf) + x;  // only used when the total fits
    total += sum;
  }
  __syncthreads();
  if (bad || total > nf || nf > c.n_pages) {
    if (tid == 0) atomicOr(status, bad || nf > c.n_pages ? DEV_REFUSED : DEV_NO_PAGES);
    return;
  }
  const int lane = tid & 31;
  for (int i = tid >> 5; i < n; i += kPlanThreads / 32) {  // a warp per slot
    const int slot = slots[i], len = s.len[i], a = add[i];
    const int p0 = pages_of(len, c.page), p1 = pages_of(len + a, c.page);
    for (int q = p0 + lane; q < p1; q += 32) {
      const int pg = c.free_pages[nf - 1 - (s.rank[i] + q - p0)];
      if (pg < 0 || pg >= c.n_pages) {
        atomicOr(status, DEV_BAD_SLOT);
        continue;
      }
      c.table[(long long)slot * c.max_pages + q] = pg;
      c.refs[pg] = 1;
    }
    if (lane == 0) c.lens[slot] = len + a;
  }
  if (tid == 0) *c.n_free = nf - (int)total;
}

// ------------------------------------------------------------------ fork
// The plan: which fork takes which free page, and the copies (source page of
// the partly filled last page, destination page).
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(Cache c, const int32_t* src, const int32_t* dst, int n,
                                                                 int32_t* status, Scratch s) {
  __shared__ int sh[32];
  __shared__ int bad;
  const int tid = threadIdx.x;
  start();
  if (tid == 0) bad = 0;
  __syncthreads();
  const long long cap = (long long)c.max_pages * c.page;
  const int nf = *c.n_free;
  int total = 0;
  for (int b0 = 0; b0 < n; b0 += kPlanThreads) {
    const int i = b0 + tid;
    int need = 0, len = 0, last = -1;
    if (i < n) {
      const int a = src[i], d = dst[i];
      len = a >= 0 && a < c.n_slots ? c.lens[a] : -1;
      if (len < 0 || len > cap || d < 0 || d >= c.n_slots || a == d || c.lens[d] != 0) {
        bad = 1;
        len = 0;
      } else if (len % c.page) {
        last = c.table[(long long)a * c.max_pages + len / c.page];
        if (last < 0 || last >= c.n_pages) bad = 1;
        need = 1;
      }
      s.len[i] = len;
    }
    int sum;
    const int x = block_scan(need, &sum, sh) + total;
    if (i < n) s.rank[i] = x;
    if (need && x < nf && nf <= c.n_pages) {
      const int to = c.free_pages[nf - 1 - x];
      if (to < 0 || to >= c.n_pages) bad = 1;
      s.msrc[x] = last;
      s.mdst[x] = to;
      s.remap[x] = len % c.page;  // rows to copy
    }
    total += sum;
  }
  __syncthreads();
  const bool ok = !bad && total <= nf && nf <= c.n_pages;
  if (tid == 0) {
    if (!ok) atomicOr(status, bad || nf > c.n_pages ? DEV_REFUSED : DEV_NO_PAGES);
    else *c.n_free = nf - total;
    s.hdr[0] = ok ? total : -1;
  }
}

// Copy `vecs` 16-byte pieces by one warp, eight loads in flight per lane.
constexpr int kPiece = 256;
__device__ __forceinline__ void warp_copy(uint4* dst, const uint4* src, int vecs) {
  const int lane = threadIdx.x & 31;
  for (int j = lane; j < vecs; j += kPiece) {
    uint4 t[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (j + 32 * u < vecs) t[u] = __ldcs(src + j + 32 * u);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (j + 32 * u < vecs) __stcs(dst + j + 32 * u, t[u]);
  }
}

// The walk of a warp over (move, plane, part): plane 2 l + (0 keys, 1 values) of
// layer l, `parts` pieces of a page each. One division per warp, then additions.
struct Walk {
  long long m, dm;
  int pl, part, dpl, dpart, planes, parts;
  __device__ Walk(int planes_, int parts_) : planes(planes_), parts(parts_) {
    const unsigned w = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5), nw = gridDim.x * (kMoveThreads / 32);
    split(w, m, pl, part);
    split(nw, dm, dpl, dpart);
  }
  __device__ void split(unsigned w, long long& a, int& b, int& c) const {
    const unsigned t = w / parts;
    c = (int)(w - t * parts);
    a = t / planes;
    b = (int)(t - (unsigned)a * planes);
  }
  __device__ void next() {
    part += dpart;
    pl += dpl;
    m += dm;
    if (part >= parts) part -= parts, ++pl;
    if (pl >= planes) pl -= planes, ++m;
  }
};

// Pages moved whole: a page's rows of all heads are contiguous in a layer's
// pool; a warp copies pieces of 4 KB of it.
__device__ void move_pages(const Cache& c, const int32_t* msrc, const int32_t* mdst, long long n, int32_t* status) {
  const long long vecs = (long long)c.Hkv * c.page * c.D / 8;  // of a page in one pool
  for (Walk w(2 * c.n_layers, (int)((vecs + kPiece - 1) / kPiece)); w.m < n; w.next()) {
    const int a = msrc[w.m], b = mdst[w.m];
    if (a < 0 || a >= c.n_pages || b < 0 || b >= c.n_pages) {
      if ((threadIdx.x & 31) == 0) atomicOr(status, DEV_BAD_SLOT);
      continue;
    }
    const long long at = (long long)w.part * kPiece, left = vecs - at;
    uint4* pool = reinterpret_cast<uint4*>((w.pl & 1) ? c.v : c.k) + (long long)(w.pl >> 1) * c.n_pages * vecs + at;
    warp_copy(pool + b * vecs, pool + a * vecs, (int)(left < kPiece ? left : kPiece));
  }
}

__global__ void __launch_bounds__(kMoveThreads) fork_apply_kernel(Cache c, const int32_t* src, const int32_t* dst, int n,
                                                                  int32_t* status, Scratch s) {
  start();
  const int moves = s.hdr[0];
  if (moves < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long gw = (long long)blockIdx.x * (kMoveThreads / 32) + warp, nw = (long long)gridDim.x * (kMoveThreads / 32);
  // a warp copies the rows in use of one head of one layer's keys or values
  const int vd = c.D >> 3;
  const long long head = (long long)c.page * vd;
  for (Walk w(2 * c.n_layers, c.Hkv); w.m < moves; w.next()) {
    uint4* pool = reinterpret_cast<uint4*>((w.pl & 1) ? c.v : c.k) +
                  ((long long)(w.pl >> 1) * c.n_pages * c.Hkv + w.part) * head;
    warp_copy(pool + s.mdst[w.m] * c.Hkv * head, pool + s.msrc[w.m] * c.Hkv * head, s.remap[w.m] * vd);
  }
  // a warp rewrites 32 entries of one fork's table row
  const int segs = (c.max_pages + 31) / 32;
  for (long long it = gw; it < (long long)n * segs; it += nw) {
    const int i = (int)(it / segs), q = (int)(it - (long long)i * segs) * 32 + lane;
    const int len = s.len[i], full = len / c.page;
    if (q < full) {
      const int pg = c.table[(long long)src[i] * c.max_pages + q];
      c.table[(long long)dst[i] * c.max_pages + q] = pg;
      if (pg >= 0 && pg < c.n_pages) atomicAdd(c.refs + pg, 1);
      else atomicOr(status, DEV_BAD_SLOT);
    } else if (q == full && len % c.page) {
      const int pg = s.mdst[s.rank[i]];
      c.table[(long long)dst[i] * c.max_pages + q] = pg;
      c.refs[pg] = 1;
    }
    if (q == 0) c.lens[dst[i]] = len;
  }
}

// ------------------------------------------------------------------ free
// refs - 1 for page q of slot slots[i]; a page that reaches 0 is marked -1, to
// be pushed afterwards (in page order, so the stack does not depend on timing).
__device__ __forceinline__ void release(const Cache& c, int slot, int q, int32_t* status) {
  int32_t* e = c.table + (long long)slot * c.max_pages + q;
  if (q < pages_of(max(0, c.lens[slot]), c.page)) {
    const int pg = *e;
    if (pg >= 0 && pg < c.n_pages) {
      const int old = atomicSub(c.refs + pg, 1);
      if (old == 1) {
        atomicExch(c.refs + pg, -1);
      } else if (old <= 0) {  // not a held page: the books were wrong
        atomicAdd(c.refs + pg, 1);
        atomicOr(status, DEV_BAD_SLOT);
      }
    } else {
      atomicOr(status, DEV_BAD_SLOT);
    }
  }
  *e = -1;
}

__global__ void __launch_bounds__(kMoveThreads) free_refs_kernel(Cache c, const int32_t* slots, int n, int32_t* status) {
  const int i = blockIdx.x, q = blockIdx.y * kMoveThreads + threadIdx.x;
  start();
  const int slot = slots[i];
  if (slot < 0 || slot >= c.n_slots) {
    if (q == 0) atomicOr(status, DEV_BAD_SLOT);
  } else if (q < c.max_pages) {
    release(c, slot, q, status);
  }
}

// Few table entries are released here too, by the one CTA that pushes: a launch
// less (4 slots of 65 entries, with their forks, 8.6 us against 9.1 and 2 us less
// for the host; 1,040 entries 12.2 against 11.4). Counted are the entries of the
// tables, whatever the slots hold: what n * max_pages is, the host knows.
constexpr int kFewEntries = 512;
__global__ void __launch_bounds__(kPlanThreads) free_push_kernel(Cache c, const int32_t* slots, int n, int few,
                                                                 int32_t* status) {
  __shared__ int sh[32];
  const int tid = threadIdx.x;
  start();
  if (few) {
    for (int k = tid; k < n * c.max_pages; k += kPlanThreads) {
      const int i = k / c.max_pages, slot = slots[i], q = k - i * c.max_pages;
      if (slot >= 0 && slot < c.n_slots) release(c, slot, q, status);
      else if (q == 0) atomicOr(status, DEV_BAD_SLOT);
    }
    __syncthreads();
  }
  const int nf = *c.n_free;
  int at = nf;
  constexpr int kPer = 8;
  for (int b0 = 0; b0 < c.n_pages; b0 += kPlanThreads * kPer) {
    // thread tid looks at pages top - kPer * tid - u, u = 0 .. kPer - 1
    const int top = c.n_pages - 1 - b0 - kPer * tid;
    unsigned gone = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (top - u >= 0 && __ldcg(c.refs + top - u) == -1) gone |= 1u << u;
    int sum;
    int x = block_scan(__popc(gone), &sum, sh) + at;
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (gone >> u & 1) {
        c.refs[top - u] = 0;
        if (x >= 0 && x < c.n_pages) c.free_pages[x] = top - u;
        else atomicOr(status, DEV_BAD_SLOT);
        ++x;
      }
    at += sum;
  }
  for (int i = tid; i < n; i += kPlanThreads)
    if (slots[i] >= 0 && slots[i] < c.n_slots) c.lens[slots[i]] = 0;
  if (tid == 0) *c.n_free = min(at, c.n_pages);
}

// ------------------------------------------------------------------ compact
// hdr[0] = moves, hdr[1] = live pages; move list in ascending order; remap[p]
// = the new place of a moved page p.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(Cache c, Scratch s, int32_t* n_moved) {
  __shared__ int sh[32];
  const int tid = threadIdx.x;
  start();
  int n_live = 0;
  for (int p = tid; p < c.n_pages; p += kPlanThreads) n_live += c.refs[p] > 0 ? 1 : 0;
  int dummy = n_live;
  block_scan(dummy, &n_live, sh);
  constexpr int kPer = 8;
  int holes = 0, movers = 0;
  for (int b0 = 0; b0 < c.n_pages; b0 += kPlanThreads * kPer) {
    const int lo = b0 + kPer * tid;
    unsigned live = 0;
    int nh = 0, nm = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int p = lo + u;
      if (p >= c.n_pages) continue;
      const bool l = c.refs[p] > 0;
      if (l) live |= 1u << u;
      nh += !l && p < n_live;
      nm += l && p >= n_live;
    }
    int sumh, summ;
    int xh = block_scan(nh, &sumh, sh) + holes;
    int xm = block_scan(nm, &summ, sh) + movers;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int p = lo + u;
      if (p >= c.n_pages) continue;
      const bool l = live >> u & 1;
      if (!l && p < n_live) s.mdst[xh++] = p;
      if (l && p >= n_live) s.msrc[xm++] = p;
      if (!l && p >= n_live) s.remap[p] = p;
    }
    holes += sumh;
    movers += summ;
  }
  __syncthreads();  // the lists are complete (holes == movers)
  for (int i = tid; i < movers; i += kPlanThreads) s.remap[s.msrc[i]] = s.mdst[i];
  if (tid == 0) {
    s.hdr[0] = movers;
    s.hdr[1] = n_live;
    if (n_moved) *n_moved = movers;
    *c.n_free = c.n_pages - n_live;
  }
}

__global__ void __launch_bounds__(kMoveThreads) compact_apply_kernel(Cache c, Scratch s, int32_t* status) {
  start();
  const int moves = s.hdr[0], n_live = s.hdr[1];
  const long long gt = (long long)blockIdx.x * kMoveThreads + threadIdx.x, nt = (long long)gridDim.x * kMoveThreads;
  move_pages(c, s.msrc, s.mdst, moves, status);
  for (long long i = gt; i < moves; i += nt) {
    c.refs[s.mdst[i]] = c.refs[s.msrc[i]];
    c.refs[s.msrc[i]] = 0;
  }
  for (long long i = gt; i < c.n_pages - n_live; i += nt) c.free_pages[i] = c.n_pages - 1 - (int)i;
  if (moves == 0) return;
  for (long long i = gt; i < (long long)c.n_slots * c.max_pages; i += nt) {
    const int slot = (int)(i / c.max_pages), q = (int)(i - (long long)slot * c.max_pages);
    if (q >= pages_of(max(0, c.lens[slot]), c.page)) continue;
    const int pg = c.table[i];
    if (pg < 0 || pg >= c.n_pages) atomicOr(status, DEV_BAD_SLOT);
    else if (pg >= n_live) c.table[i] = s.remap[pg];
  }
}

__global__ void __launch_bounds__(kMoveThreads) copy_pages_kernel(Cache c, const int32_t* src, const int32_t* dst, int n,
                                                                  int32_t* status) {
  start();
  move_pages(c, src, dst, n, status);
}

int move_grid() {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return (sms > 0 ? sms : 1) * 6;
}

}  // namespace

size_t pages_ws_bytes(int n_pages, int n_slots) {
  return align256(((size_t)kHdr + 3 * (size_t)n_pages + 2 * (size_t)n_slots) * 4);
}

cudaError_t launch_append(const Cache& c, const Rows& r, const uint16_t* k, const uint16_t* v, long long stride,
                          int32_t* status, cudaStream_t st) {
  return launch_pdl(K_KV_APPEND, append_kernel, dim3(r.n_rows), 128, 0, st, c, r, k, v, stride, status);
}

cudaError_t launch_grow(const Cache& c, const int32_t* slots, const int32_t* add, int n, int32_t* status, void* scratch,
                        cudaStream_t st) {
  return launch_pdl(K_KV_PAGES, grow_kernel, dim3(1), kPlanThreads, 0, st, c, slots, add, n, status,
                    scratch_of(scratch, c.n_pages, c.n_slots));
}

cudaError_t launch_fork(const Cache& c, const int32_t* src, const int32_t* dst, int n, int32_t* status, void* scratch,
                        cudaStream_t st) {
  const Scratch s = scratch_of(scratch, c.n_pages, c.n_slots);
  const cudaError_t e = launch_pdl(K_KV_PAGES, fork_plan_kernel, dim3(1), kPlanThreads, 0, st, c, src, dst, n, status, s);
  return e != cudaSuccess
             ? e
             : launch_pdl(K_KV_MOVE, fork_apply_kernel, dim3(move_grid()), kMoveThreads, 0, st, c, src, dst, n, status, s);
}

cudaError_t launch_free(const Cache& c, const int32_t* slots, int n, int32_t* status, cudaStream_t st) {
  const int few = (long long)n * c.max_pages <= kFewEntries;
  if (!few) {
    const cudaError_t e = launch_pdl(K_KV_PAGES, free_refs_kernel, dim3(n, (c.max_pages + kMoveThreads - 1) / kMoveThreads),
                                     kMoveThreads, 0, st, c, slots, n, status);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(K_KV_PAGES, free_push_kernel, dim3(1), kPlanThreads, 0, st, c, slots, n, few, status);
}

cudaError_t launch_compact(const Cache& c, int32_t* n_moved, int32_t* status, void* scratch, cudaStream_t st) {
  const Scratch s = scratch_of(scratch, c.n_pages, c.n_slots);
  const cudaError_t e = launch_pdl(K_KV_PAGES, compact_plan_kernel, dim3(1), kPlanThreads, 0, st, c, s, n_moved);
  return e != cudaSuccess ? e : launch_pdl(K_KV_MOVE, compact_apply_kernel, dim3(move_grid()), kMoveThreads, 0, st, c, s, status);
}

cudaError_t launch_copy_pages(const Cache& c, const int32_t* src, const int32_t* dst, int n, int32_t* status,
                              cudaStream_t st) {
  return launch_pdl(K_KV_MOVE, copy_pages_kernel, dim3(move_grid()), kMoveThreads, 0, st, c, src, dst, n, status);
}

}  // namespace kv
}  // namespace moe
