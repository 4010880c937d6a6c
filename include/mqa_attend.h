/*
 * mqa_attend.h -- C ABI of the paged 8-bit key/value cache in libmqa_topk.so:
 * storing tokens (mqa_kv_append), reading them back (mqa_kv_read), attention
 * over each row's range of positions (mqa_attend_paged), through a sliding window
 * with sinks (mqa_attend_window), over trees of drafted tokens (mqa_attend_tree)
 * and over each row's listed positions (mqa_attend_topk, which takes the output of
 * the mqa_topk_* calls as it is).
 *
 * The cache. A page holds page_size tokens of kv_heads key heads and as many
 * value heads of head_dim 8-bit codes:
 *     codes  [2][kv_heads][page_size][head_dim] bytes   (keys, then values)
 *     scales [2][kv_heads][page_size / block]   fp32
 * padded to mqa_kv_page_bytes(). A code stands for its own value (e4m3 or
 * int8) times the scale of its block of `block` consecutive slots and head.
 * Position j of request i is slot j % page_size of page table[i][j /
 * page_size]. Several layers may interleave their pages (page_stride).
 *
 * Rows. Row r belongs to request r / R, R rows a request, and sees positions
 * [s, e) of it: s = clamp(starts[r], 0, K), e = clamp(ends[r], s, K), K =
 * min(table_stride * page_size, MQA_MAX_KEYS). A chunk of one request, or of
 * several requests laid out in one key numbering (as mqa_topk_prefill_paged
 * takes them), is requests = 1 with R rows; decode is R = 1; speculative rows
 * are R > 1; a sliding window or an encoder's states are ranges like any other.
 *
 * The conventions of mqa_topk.h hold (device pointers, no allocation, no
 * state, asynchronous on `stream`, nothing launched on an error, checks in the
 * order NULL, ALIGN, SHAPE, DEVICE, WORKSPACE, the return codes).
 */
#ifndef MQA_ATTEND_H
#define MQA_ATTEND_H

#include <stddef.h>
#include <stdint.h>

#include "mqa_topk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MQA_CODES_E4M3 0 /* OCP e4m3fn: 448 the largest, 0x7F / 0xFF NaN */
#define MQA_CODES_INT8 1 /* two's complement, -127 .. 127 written */

#define MQA_BF16 0
#define MQA_FP16 1
#define MQA_FP32 2 /* mqa_kv_append and mqa_kv_read only */

#define MQA_MAX_ATTEND_HEADS 1024
#define MQA_MAX_LIST (1 << 16) /* listed positions per row of mqa_attend_topk */
#define MQA_MAX_DRAFT_WORDS 32  /* mask words per row of mqa_attend_tree */

typedef struct mqa_kv_cache {
  void* pages;          /* first page, 16-B aligned */
  const int32_t* table; /* [requests][table_stride] int32, 4-B aligned */
  int64_t page_stride;  /* bytes from a page to the next: a multiple of 16,
                           >= mqa_kv_page_bytes() */
  int32_t num_pages;    /* >= 1; num_pages * page_size < 2^32 - 1 */
  int32_t table_stride; /* >= 1 */
  int32_t kv_heads;     /* 1 .. MQA_MAX_ATTEND_HEADS */
  int32_t head_dim;     /* 64 or 128 */
  int32_t page_size;    /* a power of two, 16 .. 65536 */
  int32_t block;        /* a power of two, 16 .. page_size */
  int32_t codes;        /* MQA_CODES_* */
} mqa_kv_cache;

/* Bytes of one page, padded to a multiple of 128; 0 for sizes out of range. */
size_t mqa_kv_page_bytes(int kv_heads, int head_dim, int page_size, int block);

/*
 * Stores count_i new tokens of each request i at its positions starts[i] ..
 * starts[i] + count_i - 1: row i * R + t of k and v is its token t.
 *   k, v      [requests * R, kv_heads, head_dim] of `dtype`, 16-B aligned, the
 *             last axis dense; row and head strides in elements, each a
 *             multiple of 16 bytes
 *   starts    [requests] int32; counts [requests] int32, or NULL for R each
 *             (clamped to [0, R]). Tokens at negative positions or at K and
 *             past it, and tokens whose table entry names no page, are not
 *             stored.
 * A block's scale is the smallest 2^e >= 2^-126 with amax <= M 2^e, amax the
 * largest finite magnitude among its new tokens and M = 448 (e4m3) or 127
 * (int8); a block that keeps tokens from before the call (starts[i] inside
 * it) never lowers its scale, and where it grows the kept codes are rounded
 * again under the new one. Rounding is to nearest, ties to even. Powers of two
 * make x / scale exact, so that codes do not depend on how a GPU divides.
 * Infinities become the largest code, NaN code 0x7F (e4m3) or 0 (int8).
 * Tokens come in the order of their positions: the new ones are the request's
 * last, and what their last block held behind them (a longer draft that was taken
 * back, a page's earlier use) stands for nothing afterwards -- its codes stay as
 * they are, under a scale that may be another. To change tokens in the middle,
 * store all from there on again. Requests must not share a page that they write
 * to.
 */
int mqa_kv_append(const mqa_kv_cache* cache, const void* k, int64_t k_row_stride,
                  int64_t k_head_stride, const void* v, int64_t v_row_stride,
                  int64_t v_head_stride, int dtype, const int32_t* starts, const int32_t* counts,
                  int requests, int R, void* stream);

/*
 * Reads positions starts[i] .. starts[i] + count_i - 1 of each request back:
 * row i * R + t of k and v (dense [requests * R, kv_heads, head_dim] of
 * `dtype`, 16-B aligned) is position starts[i] + t: its code times its scale in
 * fp32 (exact for append's scales), rounded to `dtype`; rows at and past count_i
 * (counts NULL: R), outside [0, K) or without a page are zero.
 */
int mqa_kv_read(const mqa_kv_cache* cache, void* k, void* v, int dtype, const int32_t* starts,
                const int32_t* counts, int requests, int R, void* stream);

/*
 * Bytes of workspace on `device` that suffice for every attention call of up to
 * `requests` requests, up to R rows of each and up to `positions` positions a row
 * may see (mqa_attend_topk: the list's width; else table_stride * page_size; more than
 * MQA_MAX_KEYS count as that), with `heads` query heads: what a caller allocates once, for
 * its largest batch. 256 where no such call needs any; 0 for sizes out of range or a device
 * that is not gfx950.
 */
size_t workspace_size_attend(int requests, int R, int heads, int kv_heads, int head_dim,
                             int positions, int device);

/*
 * Bytes that one call of exactly these sizes needs (kind: 0 mqa_attend_paged, 1
 * mqa_attend_topk, 3 mqa_attend_tree), or that suffice for mqa_attend_window (2) with
 * any window and sinks whose min(window + sinks + R - 1, table_stride * page_size) is
 * `positions`. Few rows need more than many, as their keys are split over more
 * workgroups. 256 where it needs none (its workspace may then be NULL); 0 for another kind.
 */
size_t workspace_size_attend_call(int requests, int R, int heads, int kv_heads, int head_dim,
                                  int positions, int kind, int device);

/* Bytes that one mqa_attend_window of exactly these sizes needs (positions: table_stride *
 * page_size); 256 where it needs none. */
size_t workspace_size_attend_window(int requests, int R, int heads, int kv_heads, int head_dim,
                                    int positions, int window, int sinks, int device);

/*
 * How a call of these sizes is cut on a device of so many compute units: cut[0] columns (a
 * row of a query head each) a tile, cut[1] tiles of a request (of a row, for lists) and
 * key head, cut[2] parts of a tile's keys. kind as above; positions: table_stride *
 * page_size, or the list's width; window and sinks are looked at for kind 2 only. Needs
 * no device. MQA_ERR_SHAPE for sizes out of range.
 */
int mqa_attend_cut(int kind, int requests, int R, int heads, int kv_heads, int head_dim,
                   int positions, int window, int sinks, int compute_units, int32_t* cut);

/*
 * Attention of every row over its range: with h = query head / (heads /
 * kv_heads), k_j and v_j the values of position j's codes,
 *     S_j = scale * (q . k_j);  lse = ln sum_{s <= j < e} exp S_j
 *     out = sum_{s <= j < e} exp(S_j - lse) v_j
 * A row that sees nothing gives out = 0 and lse = -inf.
 *   q         [requests * R, heads, head_dim] of `dtype` (MQA_BF16 or
 *             MQA_FP16), 16-B aligned, the last axis dense, row and head
 *             strides in elements (multiples of 8)
 *   starts, ends [requests * R] int32, 4-B aligned
 *   out       dense [requests * R, heads, head_dim] of `dtype`, 16-B aligned
 *   lse       dense [requests * R, heads] fp32 or NULL, 4-B aligned
 *   heads     a multiple of kv_heads, at most MQA_MAX_ATTEND_HEADS
 *   scale     finite, >= 0
 *   requests * R <= MQA_MAX_ROWS
 *   workspace >= workspace_size_attend_call(requests, R, heads, kv_heads,
 *             head_dim, table_stride * page_size, 0, device) bytes, 256-B aligned,
 *             owned by the call until the stream reaches its end; nothing needs
 *             clearing
 * Scores, softmax sums and the output's sums are held in fp32. Positions that
 * no row sees may hold anything (also NaN codes and NaN or infinite scales); a
 * table entry outside [0, num_pages) is clamped into it. Scales of seen
 * positions must be >= 0, the values' at most 2^100. Probabilities times value
 * scales are rounded to 11 bits for the output's sums, down to 2^-24 of the row's
 * and head's largest such product (whatever other rows see); smaller ones, and
 * those of value scales below 2^-97, lose bits. A row that sees a NaN code becomes NaN (of a value's,
 * at least in its column), and no other row does.
 */
int mqa_attend_paged(const mqa_kv_cache* cache, const void* q, int64_t q_row_stride,
                     int64_t q_head_stride, int dtype, const int32_t* starts, const int32_t* ends,
                     void* out, float* lse, int requests, int R, int heads, float scale,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same sums over listed positions only: entry x of indices[r] names
 * position s + x of the row's request where x >= 0 and s + x < e, and nothing
 * otherwise -- the output of mqa_topk_prefill_paged and mqa_topk_decode_paged
 * with the same starts and ends. Entries may come in any order; one that is
 * there twice counts twice.
 *   indices   [requests * R, width] int32, dense, 16-B aligned, width in [1,
 *             MQA_MAX_LIST]
 *   workspace >= workspace_size_attend_call(requests, R, heads, kv_heads,
 *             head_dim, width, 1, device) bytes
 */
int mqa_attend_topk(const mqa_kv_cache* cache, const void* q, int64_t q_row_stride,
                    int64_t q_head_stride, int dtype, const int32_t* indices, int width,
                    const int32_t* starts, const int32_t* ends, void* out, float* lse,
                    int requests, int R, int heads, float scale, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * mqa_attend_paged through a sliding window: a row sees the last `window`
 * positions of its range [s, e) and the first `sinks` of it, j with e - window <=
 * j < e or s <= j < min(s + sinks, e), each once. Only these are read: pages that hold
 * none of them may be in other use, their table entries anything.
 *   window    >= 1; sinks >= 0
 *   workspace >= workspace_size_attend_window(requests, R, heads, kv_heads, head_dim,
 *             table_stride * page_size, window, sinks, device) bytes
 */
int mqa_attend_window(const mqa_kv_cache* cache, const void* q, int64_t q_row_stride,
                      int64_t q_head_stride, int dtype, const int32_t* starts, const int32_t* ends,
                      int window, int sinks, void* out, float* lse, int requests, int R, int heads,
                      float scale, void* workspace, size_t workspace_bytes, void* stream);

/*
 * mqa_attend_paged over a tree of drafted tokens, which stand in the cache behind
 * the tokens that are settled: a row sees its range [s, e) and those positions e + x
 * below K whose bit x % 32 of mask[r][x / 32] is set -- itself and its ancestors,
 * where drafts are stored in any order.
 *   mask      [requests * R, words] int32, dense, 4-B aligned, words in [1,
 *             MQA_MAX_DRAFT_WORDS]
 *   workspace >= workspace_size_attend_call(requests, R, heads, kv_heads, head_dim,
 *             table_stride * page_size, 3, device) bytes
 */
int mqa_attend_tree(const mqa_kv_cache* cache, const void* q, int64_t q_row_stride,
                    int64_t q_head_stride, int dtype, const int32_t* starts, const int32_t* ends,
                    const int32_t* mask, int words, void* out, float* lse, int requests, int R,
                    int heads, float scale, void* workspace, size_t workspace_bytes,
                    void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MQA_ATTEND_H */
