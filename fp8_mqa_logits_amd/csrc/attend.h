// The paged 8-bit key/value cache as its kernels see it, parameter blocks and
// launch entry points of kvcache.hip and attend.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <stdint.h>

namespace mqa {

enum { kE4m3 = 0, kInt8 = 1 };
enum { kBf16 = 0, kFp16 = 1, kFp32 = 2 };
constexpr int kMaxSplits = 256;  // parts of a tile's keys, a multiple of 64
// What a row sees: its range; the first and the last positions of it; its range and
// some of the positions behind it.
enum { kRange = 0, kWindow = 1, kTree = 2 };

struct KvCache {
  uint8_t* pages;
  const int32_t* table;
  int64_t page_stride;
  int32_t num_pages, table_stride;
  int32_t kv_heads, head_dim;
  int32_t page_shift, block_shift;
  int32_t codes;
  int32_t cap;         // positions a request can have
  int32_t scales_at;   // byte of a page's first scale
};

struct KvMoveParams {  // append and read
  KvCache c;
  const void* k;
  const void* v;
  void* ko;
  void* vo;
  int64_t k_row, k_head, v_row, v_head;  // elements
  const int32_t* starts;
  const int32_t* counts;
  int requests, R, dtype;
};

struct AttendParams {
  KvCache c;
  const void* q;
  int64_t q_row, q_head;  // elements
  const int32_t* starts;
  const int32_t* ends;
  const int32_t* indices;  // [rows][width]; nullptr: every position of the range
  int width;
  int sight;               // kRange, kWindow, kTree
  int window, sinks;       // kWindow
  const int32_t* mask;     // kTree: [rows][words]
  int words;
  void* out;
  float* lse;
  int requests, R, rows, heads, group, dtype;
  float scale;
  // How the work is cut: tiles of `cols` columns (rows x the query heads of a
  // key head) per request or listed row, each tile's keys in `splits` parts.
  int cols, tiles, splits;
  int64_t block0;  // first workgroup of this launch
  float* part_ml;  // [item][split][cols][2] reference point and sum
  float* part_o;   // [item][split][cols][head_dim]
};

// Byte offsets of a page's parts: all below 2^31 (checked on the host).
__device__ __forceinline__ int code_at(const KvCache& c, int w, int h, int slot) {
  return (((w * c.kv_heads + h) << c.page_shift) + slot) * c.head_dim;
}
__device__ __forceinline__ int scale_at(const KvCache& c, int w, int h, int slot) {
  return c.scales_at +
         (((w * c.kv_heads + h) << (c.page_shift - c.block_shift)) + (slot >> c.block_shift)) * 4;
}

}  // namespace mqa

extern "C" {
int mqa_kv_append_launch(const mqa::KvMoveParams* p, hipStream_t stream);
int mqa_kv_read_launch(const mqa::KvMoveParams* p, hipStream_t stream);
int mqa_attend_launch(const mqa::AttendParams* p, hipStream_t stream);
}
