// Argument checks that the C ABI's calls on the paged cache share.
#pragma once

#include "attend.h"
#include "mqa_attend.h"

namespace mqa {

constexpr size_t kNoWorkspace = 256;  // what is asked for where nothing is needed

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool power_of_two(int x) { return x > 0 && (x & (x - 1)) == 0; }

// Bytes of a page (0: sizes out of range). A page stays below 2^31 bytes, so
// that offsets inside it fit 32 bits.
inline int64_t page_bytes(int kv_heads, int head_dim, int page_size, int block) {
  if (kv_heads < 1 || kv_heads > MQA_MAX_ATTEND_HEADS || (head_dim != 64 && head_dim != 128) ||
      !power_of_two(page_size) || page_size < 16 || page_size > 65536 || !power_of_two(block) ||
      block < 16 || block > page_size)
    return 0;
  const int64_t n = 2 * (int64_t)kv_heads * ((int64_t)page_size * head_dim + page_size / block * 4);
  const int64_t padded = (n + 127) / 128 * 128;
  return padded < ((int64_t)1 << 31) ? padded : 0;
}

// NULL and ALIGN part of a cache's checks.
inline int cache_pointers(const mqa_kv_cache* c) {
  if (!c || !c->pages || !c->table) return MQA_ERR_NULL;
  return aligned(c->pages, 16) && aligned(c->table, 4) && c->page_stride % 16 == 0 ? MQA_OK
                                                                                  : MQA_ERR_ALIGN;
}

inline bool cache_shape(const mqa_kv_cache* c) {
  const int64_t n = page_bytes(c->kv_heads, c->head_dim, c->page_size, c->block);
  return n > 0 && c->page_stride >= n && c->page_stride < ((int64_t)1 << 40) && c->num_pages >= 1 &&
         (int64_t)c->num_pages * c->page_size < ((int64_t)1 << 32) - 1 && c->table_stride >= 1 &&
         (c->codes == MQA_CODES_E4M3 || c->codes == MQA_CODES_INT8);
}

inline KvCache kernel_cache(const mqa_kv_cache* c) {
  KvCache k{};
  k.pages = static_cast<uint8_t*>(c->pages);
  k.table = c->table;
  k.page_stride = c->page_stride;
  k.num_pages = c->num_pages;
  k.table_stride = c->table_stride;
  k.kv_heads = c->kv_heads;
  k.head_dim = c->head_dim;
  k.page_shift = __builtin_ctz((unsigned)c->page_size);
  k.block_shift = __builtin_ctz((unsigned)c->block);
  k.codes = c->codes;
  const int64_t cap = (int64_t)c->table_stride * c->page_size;
  k.cap = (int)(cap < MQA_MAX_KEYS ? cap : MQA_MAX_KEYS);
  k.scales_at = 2 * c->kv_heads * c->page_size * c->head_dim;
  return k;
}

inline bool rows_ok(int requests, int R) {
  return requests >= 1 && R >= 1 && (int64_t)requests * R <= MQA_MAX_ROWS;
}

// Positions that a request's table has room for.
inline int64_t positions_of(const mqa_kv_cache* cache) {
  return cache ? (int64_t)cache->table_stride * cache->page_size : 0;
}

inline int at_most_keys(int64_t positions) {
  return (int)(positions < MQA_MAX_KEYS ? positions : MQA_MAX_KEYS);
}

}  // namespace mqa
