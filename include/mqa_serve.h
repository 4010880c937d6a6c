/*
 * mqa_serve.h -- C ABI of what a serving step does around attention over the paged
 * 8-bit key/value cache of mqa_attend.h, in libmqa_topk.so: norm and rotation of queries
 * and keys before they go there (mqa_norm_rotate), and eviction: the attention weight
 * that positions receive (mqa_kv_weigh), which of them stay (mqa_kv_select), and moving
 * these together (mqa_kv_keep, also for the accepted tokens of a draft's tree).
 *
 * The conventions of mqa_topk.h and mqa_attend.h hold (device pointers, no allocation,
 * no state, asynchronous on `stream`, nothing launched on an error, checks in the order
 * NULL, ALIGN, SHAPE, DEVICE, WORKSPACE, the return codes).
 */
#ifndef MQA_SERVE_H
#define MQA_SERVE_H

#include <stddef.h>
#include <stdint.h>

#include "mqa_attend.h"

#ifdef __cplusplus
extern "C" {
#endif

/* [rows, heads, head_dim] of a 16-bit type, the last axis dense. */
typedef struct mqa_head_rows {
  void* data;          /* 16-B aligned */
  int64_t row_stride;  /* in elements, multiples of 8, >= 0 */
  int64_t head_stride;
} mqa_head_rows;

/*
 * RMS norm of every query and key head, then the rotation of its position, in one pass:
 *     y_d = w_d x_d / sqrt(mean_d x_d^2 + eps)          (norm != 0; else y = x)
 *     a_i = positions[r] * inv_freq[i]
 *     (y_p, y_s) -> (y_p cos a_i - y_s sin a_i, y_s cos a_i + y_p sin a_i)
 * for i < rot / 2 with (p, s) = (i, i + rot / 2), or (2 i, 2 i + 1) where pairs != 0;
 * elements from rot on are y. Sums and products are held in fp32 (x^2 of 1.8e19 and more
 * overflows there), the angle in 64 bits, its sine and cosine are within 2^-20; the result
 * is rounded once.
 *   q, q_out   [rows, heads, head_dim] of `dtype` (MQA_BF16 or MQA_FP16)
 *   k, k_out   [rows, kv_heads, head_dim]; kv_heads = 0: no keys (k, k_out are not read)
 *   *_out may be what they are computed from (the same address and strides); no other
 *   overlap, and no stride of 0 over more than one row or head
 *   q_weight, k_weight   [head_dim] of weight_dtype (dtype or MQA_FP32), 16-B aligned, or
 *   NULL for ones
 *   positions  [rows] int32, 4-B aligned; inv_freq [rot / 2] fp32, 16-B aligned
 *   rot        a multiple of 16 in [0, head_dim]; 0: no rotation (positions and inv_freq
 *              are not read)
 *   rows in [1, MQA_MAX_ROWS], heads and kv_heads at most MQA_MAX_ATTEND_HEADS, head_dim
 *   64, 128 or 256, eps finite, >= 0
 */
int mqa_norm_rotate(const mqa_head_rows* q, const mqa_head_rows* q_out, int heads,
                    const mqa_head_rows* k, const mqa_head_rows* k_out, int kv_heads,
                    const void* q_weight, const void* k_weight, int weight_dtype,
                    const int32_t* positions, const float* inv_freq, int rot, int pairs, int rows,
                    int head_dim, int dtype, int norm, float eps, void* stream);

#define MQA_MAX_KEPT (1 << 26) /* listed positions of all requests of a call */

/*
 * Adds to every position's weight what the rows' attention gave it:
 *     weights[i][j] += sum over request i's rows r and heads h with s_r <= j < e_r of
 *                      exp(S_j - lse[r][h]),   S_j, s_r and e_r as in mqa_attend_paged
 * With the lse that mqa_attend_paged returned for the same q, ranges and scale, a row's
 * heads share out `heads` in all. Rows are weighed over whole ranges: what a row saw through
 * mqa_attend_window or mqa_attend_tree cannot be (the lse of either leaves positions of the
 * range out, or has others, and the sums above would not be the weights of that attention).
 *   lse       dense [requests * R, heads] fp32, 4-B aligned; a row and head of -inf adds
 *             nothing
 *   weights   dense [requests, width] fp32, 4-B aligned, width >= 1; positions from width
 *             on are left out
 *   workspace >= workspace_size_weigh(requests, R, heads, kv_heads, head_dim,
 *             table_stride * page_size, device) bytes, 256-B aligned, owned by the call
 *             until the stream reaches its end; nothing needs clearing. NULL where that is
 *             256.
 *   q, starts, ends, R, heads and scale as in mqa_attend_paged
 * Scores and sums are held in fp32, added in a fixed order. Positions that no row sees
 * may hold anything; one whose key holds a NaN becomes NaN if some row sees it.
 */
int mqa_kv_weigh(const mqa_kv_cache* cache, const void* q, int64_t q_row_stride,
                 int64_t q_head_stride, int dtype, const int32_t* starts, const int32_t* ends,
                 const float* lse, float* weights, int width, int requests, int R, int heads,
                 float scale, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Bytes of workspace on `device` that suffice for every mqa_kv_weigh of up to so many
 * requests, rows of each and positions (more than MQA_MAX_KEYS count as that); 256 where
 * none is needed, 0 for sizes out of range or a device that is not gfx950.
 */
size_t workspace_size_weigh(int requests, int R, int heads, int kv_heads, int head_dim,
                            int positions, int device);

/*
 * Which positions of each request stay: of its n = clamp(lengths[i], 0, width) positions
 * the first `sinks`, the last `recent`, and of those between the largest weights, until
 * counts[i] = min(n, keep) are chosen. Equal weights: the smallest positions; NaN counts
 * as larger than any number.
 *   weights   dense [requests, width] fp32; lengths [requests] int32
 *   positions [requests, keep] int32: the chosen ones in ascending order, then -1
 *   counts    [requests] int32
 *   kept      dense [requests, width] fp32 or NULL, not overlapping weights: the chosen
 *             positions' weights in the same order, then 0 -- what mqa_kv_weigh goes on
 *             with after mqa_kv_keep
 *   workspace >= workspace_size_select(requests, width) bytes, 256-B aligned, owned by the
 *             call until the stream reaches its end; nothing needs clearing. NULL where that
 *             is 256.
 *   keep, width in [1, MQA_MAX_KEYS], requests in [1, MQA_MAX_ROWS], requests * keep <=
 *   MQA_MAX_KEPT, sinks and recent >= 0, sinks + recent <= keep; other pointers 4-B aligned
 */
int mqa_kv_select(const float* weights, int width, const int32_t* lengths, int keep, int sinks,
                  int recent, int32_t* positions, int32_t* counts, float* kept, int requests,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace that suffice for every mqa_kv_select of up to so many requests and
 * weights of each; 256 where none is needed, 0 for sizes out of range. */
size_t workspace_size_select(int requests, int width);

/*
 * Moves the first counts[i] (clamped to [0, width]) listed positions of request i to its
 * positions starts[i] .. (starts NULL: 0 ..): what mqa_kv_append makes of what
 * mqa_kv_read returns for them in fp32, but for blocks whose tokens all stay where they
 * are, which stay as they are. Tokens move towards the front, or stay: entry t of a list
 * names no position before starts[i] + t, as ascending positions from starts[i] on do
 * (where one does, what the request holds from starts[i] on is unspecified). An entry
 * without a position in [0, K) or without a page stands for zeros, wherever it is; a position
 * may be named twice. What stood behind the moved tokens stands for nothing afterwards: the
 * request is starts[i] + counts[i] long. Requests must not share a page that they write to.
 *   positions [requests, width] int32, counts and starts [requests] int32, 4-B aligned
 *   workspace >= workspace_size_keep(requests, width, kv_heads, head_dim, block) bytes,
 *             256-B aligned, owned by the call until the stream reaches its end; nothing
 *             needs clearing. NULL where that is 256.
 *   width in [1, MQA_MAX_KEYS], requests in [1, MQA_MAX_ROWS], requests * width <=
 *   MQA_MAX_KEPT
 */
int mqa_kv_keep(const mqa_kv_cache* cache, const int32_t* positions, const int32_t* counts,
                const int32_t* starts, int width, int requests, void* workspace,
                size_t workspace_bytes, void* stream);

/* Bytes of workspace that suffice for every mqa_kv_keep of up to so many requests and
 * listed positions; 256 where none is needed, 0 for sizes out of range. */
size_t workspace_size_keep(int requests, int width, int kv_heads, int head_dim, int block);

#ifdef __cplusplus
}
#endif

#endif /* MQA_SERVE_H */
