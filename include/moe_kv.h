/*
 * moe_kv.h - C ABI of a paged key-value cache and the attention that reads it,
 * for sm_103a: the attention side of the layers whose routed-expert FFN moe.h
 * runs. The cache serves the same calls: decode windows of one row per
 * conversation or token + proposal, and prompt chunks.
 *
 * Cache. Keys and values of every layer live in two pools of pages
 *   k, v  [n_layers][n_pages][Hkv][page_size][D]   bf16 or fp16
 * shared by all layers' page numbers: token j of slot s is row j % page_size
 * of page table[s][j / page_size] in every layer. lens[s] counts slot s's
 * tokens, those of the call included: moe_kv_grow first, then moe_kv_append
 * and the attention of every layer. The page operations keep lens, table and
 * refs together: a program that lowers a length itself (a refused proposal) must
 * stay within the slot's last page, since no later call gives back a page that
 * lies past the new length. refs[p] is the number of slots that hold
 * page p (0: free); free_pages[0 .. n_free) is a stack, popped from its end.
 * A program that starts empty sets table to -1, lens and refs to 0,
 * free_pages[i] = n_pages - 1 - i and n_free to n_pages.
 *
 * Conventions are those of moe.h: every pointer is a DEVICE pointer unless its
 * comment says host, the caller owns every buffer, calls are asynchronous on
 * `stream` and never synchronise, may be captured into a CUDA graph after one
 * warm-up call per kind, and report host-detected errors before anything is
 * launched. The workspace is initialised by moe_workspace_init, its status
 * word is read by moe_read_status, and it serves one call at a time. Results
 * are deterministic: the same call gives the same bits.
 *
 * Device-detected problems are OR-ed into the status word: 2 a slot outside
 * [0, n_slots) (its rows are treated as a sequence of length 0), a page number
 * outside [0, n_pages) (its tokens are treated as not visible, or not
 * written), or a length beyond max_pages pages (taken as max_pages pages);
 * 4 a bounded wait expired (the call's results are incomplete, and the
 * workspace has to be initialised before its next call); 32 not enough
 * free pages, 64 an argument that a page operation refuses (named at each):
 * after 32 or 64 the operation has changed nothing.
 */
#ifndef MOE_KV_GB300_H
#define MOE_KV_GB300_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_KV_BF16 = 1, MOE_KV_F16 = 2 } moe_kv_dtype;

/* The cache (a HOST struct of DEVICE pointers). k and v 16-byte aligned, the
 * other buffers 4-byte aligned. D a multiple of 8 up to 256; n_pages * Hkv *
 * page_size at most 2^31 - 1 (rows of one layer's pool). */
typedef struct {
  void *k, *v;
  moe_kv_dtype dtype;
  int32_t n_layers, n_pages, page_size, Hkv, D;
  int32_t n_slots, max_pages;
  int32_t *table;      /* [n_slots][max_pages] */
  int32_t *lens;       /* [n_slots] */
  int32_t *refs;       /* [n_pages] */
  int32_t *free_pages; /* [n_pages] */
  int32_t *n_free;     /* [1] */
} moe_kv_desc;

/* The rows of a call (a HOST struct): B sequences, sequence b being slot
 * slots[b] (NULL: slot b). Its new tokens are rows row_start[b] ..
 * row_start[b + 1) (row_start [B + 1], ascending from 0 to n_rows), or n_rows
 * / B rows each when row_start is NULL. Row i of the n rows of a sequence of
 * length L is token L - n + i (a row with a negative token is no token: it is
 * not written and sees nothing). */
typedef struct {
  int32_t B, n_rows;
  const int32_t *slots;
  const int32_t *row_start;
} moe_kv_rows;

/* Attention of a call's rows over their sequences. Query head h reads KV head
 * h / (Hq / Hkv). Row at token p sees token j when j <= p, j < lens and
 * (window == 0 or j > p - window or j < n_sink): a sliding window of `window`
 * tokens with the first n_sink tokens always visible.
 *   lse[t][h] = ln sum_j exp(scale q_t,h . k_j)   over the visible tokens j
 *   o[t][h]   = sum_j exp(scale q_t,h . k_j - lse[t][h]) v_j
 * Hq is a multiple of Hkv up to 65,535. A row that sees nothing gets o = 0 and
 * lse = -inf. q [n_rows][Hq][D] with q_stride elements from row to row (heads
 * contiguous, so q may be a part of a larger projection); o [n_rows][Hq][D]
 * contiguous; both in the cache's type and 16-byte aligned, q_stride a multiple
 * of 8. lse [n_rows][Hq] fp32 or NULL. Products are of the cache's type, sums and
 * softmax in fp32. A token that no row of the call sees (past the length, outside
 * every row's window) is not used and may hold anything, NaN included; pages
 * wholly of such tokens are not read and their table entries may be anything (in
 * these calls: the page operations below go by every entry of a slot's length). */
typedef struct {
  int32_t Hq;
  float scale;
  int32_t window, n_sink;
  const void *q;
  int64_t q_stride;
  void *o;
  float *lse;
} moe_attn_args;

/* Workspace bytes of every call on this cache with up to max_rows rows (and
 * sequences) and Hq query heads (256-byte aligned base, moe_workspace_init
 * once). Only moe_attn_decode's part grows with max_rows: the bytes for 0 rows
 * serve chunks and page operations of any size. kv: HOST. 0 for an invalid
 * description. */
size_t moe_kv_workspace_bytes(const moe_kv_desc *kv, int32_t Hq, int32_t max_rows);

/* Write the rows' keys and values of one layer into their pages. k, v
 * [n_rows][Hkv][D] of the cache's type, row_stride elements from row to row (a
 * multiple of 8, at least Hkv * D), 16-byte aligned. */
moe_status moe_kv_append(const moe_kv_desc *kv, int32_t layer, const moe_kv_rows *rows,
                         const void *k, const void *v, int64_t row_stride, void *ws,
                         size_t ws_bytes, void *stream);

/* Rotary positions (a HOST struct). The first rot of a head's D values are
 * turned in pairs, the rest is left: pair i is (i, i + rot / 2) in the HALF
 * layout, (2 i, 2 i + 1) INTERLEAVED, and a token at position p turns it by
 * the angle of p freq[i] turns / 2^64:
 *   (x, y) -> gain (x cos - y sin, y cos + x sin)
 * freq [rot / 2] holds turns per token as fractions of 2^64 (radians / 2 pi
 * times 2^64, modulo 2^64), so that p freq[i] modulo 2^64 is the angle without
 * an error that grows with p. Contexts are lengthened by other frequencies
 * (and a gain). rot even, 2 .. D; freq 8-byte aligned. */
typedef enum { MOE_ROPE_HALF = 0, MOE_ROPE_INTERLEAVED = 1 } moe_rope_layout;
typedef struct {
  int32_t rot;
  moe_rope_layout layout;
  float gain;
  const uint64_t *freq;
} moe_rope_desc;

/* moe_kv_append with rotary positions: the rows' keys are turned on their way
 * into the pages, their values written as they are, and their queries q
 * [n_rows][Hq][D] turned into q_out [n_rows][Hq][D] (q_out_stride elements from
 * row to row; q_out may be q with the same stride; both 16-byte aligned,
 * strides a multiple of 8). positions [n_rows] int32 (4-byte aligned) or NULL:
 * each row's token number in its sequence. Angles, products in fp32, one
 * rounding. A row that is no token has its q copied; rows behind the last
 * sequence are left as they were. Hq up to 65,535. */
moe_status moe_kv_append_rope(const moe_kv_desc *kv, int32_t layer, const moe_kv_rows *rows,
                              const moe_rope_desc *rope, const int32_t *positions, int32_t Hq,
                              const void *q, int64_t q_stride, void *q_out, int64_t q_out_stride,
                              const void *k, const void *v, int64_t row_stride, void *ws,
                              size_t ws_bytes, void *stream);

/* Attention of a decode window: the same number of rows (1 .. 16) for every
 * sequence, row_start NULL. With D 64 or 128 and pages of a power of two of at
 * least 8 tokens the key-value pairs are read once per 16 query rows of a KV
 * head, the work split over the sequences' lengths and joined; other shapes read
 * them once per row and query head, one CTA each. A row's result depends on its
 * own sequence only, bit for bit: not on the other sequences of the call, nor on
 * where the pages lie. A NaN or an infinity in a token reaches only the rows that
 * see the token (an infinite value as an infinity or as NaN). */
moe_status moe_attn_decode(const moe_kv_desc *kv, int32_t layer, const moe_kv_rows *rows,
                           const moe_attn_args *a, void *ws, size_t ws_bytes, void *stream);

/* Attention of prompt chunks: any number of rows per sequence. On the tensor
 * cores with the shapes named above, up to 128 query heads per KV head and a
 * scale above zero; else the keys are read once per row and query head, by a CTA
 * or a warp each. A probability is rounded to the cache's type for its product
 * with a value (decode keeps twice as many bits). How a long sequence is split
 * depends on the call, so a row's last bits may differ in another call. Values
 * that some rows of a sequence see must be finite: as in a plain product of
 * probabilities and values, a NaN or an infinity may reach rows that do not see
 * it. */
moe_status moe_attn_chunk(const moe_kv_desc *kv, int32_t layer, const moe_kv_rows *rows,
                          const moe_attn_args *a, void *ws, size_t ws_bytes, void *stream);

/* Pages for add[i] >= 0 more tokens of slot slots[i] (i < n, distinct slots):
 * lens[slots[i]] += add[i], new pages popped in slot order, then token order,
 * each with refs 1. Refused (64): a slot out of range, a negative add, a
 * length beyond max_pages pages. */
moe_status moe_kv_grow(const moe_kv_desc *kv, const int32_t *slots, const int32_t *add, int32_t n,
                       void *ws, size_t ws_bytes, void *stream);

/* Fork slot src[i] into the empty slot dst[i] (i < n; the dst distinct, a src
 * may repeat): the full pages are shared (refs + 1); the rows in use of a
 * partly filled last page are copied, in every layer, into a page popped in
 * order of i. Refused (64): a slot out of range, a dst of non-zero length, a
 * source beyond max_pages pages, a page number out of range among the last pages
 * or the free ones. */
moe_status moe_kv_fork(const moe_kv_desc *kv, const int32_t *src, const int32_t *dst, int32_t n,
                       void *ws, size_t ws_bytes, void *stream);

/* Empty the slots (i < n, distinct): refs - 1 for each of their pages; pages
 * that reach 0 are pushed in descending page order (the lowest is popped
 * first); lens = 0, the table rows = -1. A slot out of range is skipped (2). */
moe_status moe_kv_free(const moe_kv_desc *kv, const int32_t *slots, int32_t n, void *ws,
                       size_t ws_bytes, void *stream);

/* Move the live pages to the page numbers below their count L: the i-th live
 * page at or above L (ascending) moves, in every layer, to the i-th free page
 * below L; tables and refs follow and the free stack becomes n_pages - 1 ..
 * L. n_moved [1] (nullable) receives the number of moves. Only free pages are
 * written, so work already queued that reads the old places is not disturbed. */
moe_status moe_kv_compact(const moe_kv_desc *kv, int32_t *n_moved, void *ws, size_t ws_bytes,
                          void *stream);

/* Copy page src[i] to page dst[i] in every layer (i < n; no dst is a src or
 * another dst). The bookkeeping is the caller's. A pair with a page out of
 * range is skipped (2). */
moe_status moe_kv_copy_pages(const moe_kv_desc *kv, const int32_t *src, const int32_t *dst,
                             int32_t n, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_KV_GB300_H */
