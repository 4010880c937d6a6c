/*
 * mqa_serve.h -- C ABI of what a serving step does around attention over the paged
 * 8-bit key/value cache of mqa_attend.h, in libmqa_topk.so: norm and rotation of queries
 * and keys before they go there (mqa_norm_rotate).
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

#ifdef __cplusplus
}
#endif

#endif /* MQA_SERVE_H */
