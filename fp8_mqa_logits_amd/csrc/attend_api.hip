// C ABI of the paged 8-bit key/value cache: argument checks, workspace layout
// and launches. The declarations and their contracts are in
// include/mqa_attend.h.
#include <hip/hip_runtime.h>

#include "attend.h"
#include "launch.h"
#include "mqa_attend.h"

namespace {

using mqa::AttendParams;
using mqa::KvCache;
using mqa::KvMoveParams;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool power_of_two(int x) { return x > 0 && (x & (x - 1)) == 0; }

// Bytes of a page (0: sizes out of range). A page stays below 2^31 bytes, so
// that offsets inside it fit 32 bits.
int64_t page_bytes(int kv_heads, int head_dim, int page_size, int block) {
  if (kv_heads < 1 || kv_heads > MQA_MAX_ATTEND_HEADS || (head_dim != 64 && head_dim != 128) ||
      !power_of_two(page_size) || page_size < 16 || page_size > 65536 || !power_of_two(block) ||
      block < 16 || block > page_size)
    return 0;
  const int64_t n = 2 * (int64_t)kv_heads * ((int64_t)page_size * head_dim + page_size / block * 4);
  const int64_t padded = (n + 127) / 128 * 128;
  return padded < ((int64_t)1 << 31) ? padded : 0;
}

// NULL and ALIGN part of a cache's checks.
int cache_pointers(const mqa_kv_cache* c) {
  if (!c || !c->pages || !c->table) return MQA_ERR_NULL;
  return aligned(c->pages, 16) && aligned(c->table, 4) && c->page_stride % 16 == 0 ? MQA_OK
                                                                                  : MQA_ERR_ALIGN;
}

bool cache_shape(const mqa_kv_cache* c) {
  const int64_t n = page_bytes(c->kv_heads, c->head_dim, c->page_size, c->block);
  return n > 0 && c->page_stride >= n && c->page_stride < ((int64_t)1 << 40) && c->num_pages >= 1 &&
         (int64_t)c->num_pages * c->page_size < ((int64_t)1 << 32) - 1 && c->table_stride >= 1 &&
         (c->codes == MQA_CODES_E4M3 || c->codes == MQA_CODES_INT8);
}

KvCache kernel_cache(const mqa_kv_cache* c) {
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

bool rows_ok(int requests, int R) {
  return requests >= 1 && R >= 1 && (int64_t)requests * R <= MQA_MAX_ROWS;
}

constexpr size_t kNoWorkspace = 256;  // what is asked for where nothing is needed

// How an attention call is cut (AttendParams), from what the host knows.
struct Plan {
  int cols, tiles, splits;
  size_t ml, o, total;  // workspace offsets
};

constexpr int kMostRounds = 4;  // of resident workgroups, where keys are split

// Workgroups that the device holds at once, by their registers.
int64_t resident(int cols, int head_dim, bool list, int cus) {
  const int held = list ? 2 : cols == 16 ? 4 : cols == 32 ? (head_dim == 64 ? 4 : 2)
                                                       : cols == 128 ? 2 : 1;
  return (int64_t)held * cus;
}

// The widest tile for so many columns.
int widest(int columns, bool list) {
  int cols = 16;
  while (cols < columns && cols < (list ? 64 : 256)) cols *= 2;
  return cols;
}

// Workspace offsets for so many columns of parts.
void lay_out(Plan& a, int64_t slots, int head_dim) {
  a.ml = 0;
  a.o = (size_t)((slots * 8 + 255) / 256 * 256);
  a.total = a.o + (size_t)slots * head_dim * 4;
  if (a.total == 0) a.total = kNoWorkspace;
}

// Tiles: the widest whose workgroups, with 512 keys each at least, give every
// compute unit one, else the narrowest (333 rows of 12 heads, each its own key
// head, over a window of 83: 6 us on 16 columns, 20 on 256 with the keys split).
// Parts of a tile's keys: every round of resident workgroups takes the time of
// its keys and of a start and an end that 512 keys' time stands for (1024 for
// the wide tiles, whose sums are larger); the join takes twice that. One round
// comes out where the keys allow it: 32 x 131072 positions of 2 heads 373 us in
// 16 parts, 384 in 24, 425 in 64; 48 uneven requests of 4 heads 123.5 us in 5,
// 124.5 in 8; one request of 777 positions 10 us in one, 13 in two.
Plan plan(int requests, int R, int heads, int kv_heads, int head_dim, int positions, bool list,
          int cus) {
  Plan a{};
  const int group = heads / kv_heads, columns = list ? group : R * group;
  const int64_t units = (int64_t)(list ? requests * R : requests) * kv_heads;
  a.cols = widest(columns, list);
  auto items = [&]() { return units * ((columns + a.cols - 1) / a.cols); };
  const int64_t most = positions < 1024 ? 1 : positions / 512;
  while (!list && a.cols > 16 && items() * most < cus) a.cols /= 2;
  a.tiles = (columns + a.cols - 1) / a.cols;
  const int64_t room = resident(a.cols, head_dim, list, cus), n = items();
  const int64_t ends = a.cols > 64 ? 1024 : 512;
  int64_t best = 0;
  for (int s = 1; s <= mqa::kMaxSplits && (s == 1 || s * 256 <= positions); ++s) {
    const int64_t rounds = (n * s + room - 1) / room;
    const int64_t cost = rounds * ((positions + s - 1) / s + ends) + (s > 1 ? 2 * ends : 0);
    if (s > 1 && rounds > kMostRounds) break;
    if (s > 1 && cost >= best) continue;
    best = cost;
    a.splits = s;
  }
  lay_out(a, a.splits > 1 ? n * a.splits * a.cols : 0, head_dim);
  return a;
}

// Bytes that suffice for every plan of up to so many requests, rows of each and
// positions: no plan has more parts than the positions allow, nor more than
// kMostRounds rounds of workgroups.
size_t most_workspace(int requests, int R, int heads, int kv_heads, int head_dim, int positions,
                      bool list, int cus) {
  const int group = heads / kv_heads, columns = list ? group : R * group;
  const int64_t units = (int64_t)(list ? requests * R : requests) * kv_heads;
  const int64_t splits = positions / 256 < mqa::kMaxSplits ? positions / 256 : mqa::kMaxSplits;
  int64_t most = 0;
  for (int cols = widest(columns, list); cols >= 16 && splits > 1; cols /= 2) {
    const int64_t by_keys = units * ((columns + cols - 1) / cols) * splits;
    const int64_t by_rounds = kMostRounds * resident(cols, head_dim, list, cus);
    const int64_t slots = (by_keys < by_rounds ? by_keys : by_rounds) * cols;
    most = slots > most ? slots : most;
  }
  Plan a{};
  lay_out(a, most, head_dim);
  return a.total;
}

// What either size function refuses.
bool sizes_ok(int requests, int R, int heads, int kv_heads, int head_dim, int positions) {
  return rows_ok(requests, R) && kv_heads >= 1 && heads >= kv_heads &&
         heads <= MQA_MAX_ATTEND_HEADS && heads % kv_heads == 0 &&
         (head_dim == 64 || head_dim == 128) && positions >= 1;
}

int at_most_keys(int64_t positions) {
  return (int)(positions < MQA_MAX_KEYS ? positions : MQA_MAX_KEYS);
}

int move(const mqa_kv_cache* cache, KvMoveParams& p, int (*launch)(const KvMoveParams*, hipStream_t),
         void* stream) {
  if (!mqa::current_device_cus()) return MQA_ERR_DEVICE;
  p.c = kernel_cache(cache);
  const int rc = launch(&p, static_cast<hipStream_t>(stream));
  return rc != 0 ? mqa::launch_failed(rc) : MQA_OK;
}

int attend(const mqa_kv_cache* cache, const void* q, int64_t q_row, int64_t q_head, int dtype,
           const int32_t* indices, int width, const int32_t* starts, const int32_t* ends,
           void* out, float* lse, int requests, int R, int heads, float scale, void* workspace,
           size_t workspace_bytes, int positions, void* stream) {
  if (!cache || !q || !starts || !ends || !out) return MQA_ERR_NULL;
  const int rc = cache_pointers(cache);
  if (rc != MQA_OK) return rc;
  if (!aligned(q, 16) || q_row % 8 != 0 || q_head % 8 != 0 || !aligned(starts, 4) ||
      !aligned(ends, 4) || !aligned(indices, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 256))
    return MQA_ERR_ALIGN;
  if (!cache_shape(cache) || !rows_ok(requests, R) || heads < 1 || heads > MQA_MAX_ATTEND_HEADS ||
      heads % cache->kv_heads != 0 || (dtype != MQA_BF16 && dtype != MQA_FP16) || q_row < 0 ||
      q_head < 0 || !(scale >= 0.f) || scale > 3.4e38f ||
      (indices && (width < 1 || width > MQA_MAX_LIST)))
    return MQA_ERR_SHAPE;
  const int cus = mqa::current_device_cus();
  if (!cus) return MQA_ERR_DEVICE;
  const Plan a = plan(requests, R, heads, cache->kv_heads, cache->head_dim, positions,
                      indices != nullptr, cus);
  if (!workspace && a.total > kNoWorkspace) return MQA_ERR_NULL;
  if (workspace && workspace_bytes < a.total)
    return mqa::workspace_failed("the workspace is smaller than workspace_size_attend_call()");
  AttendParams p{};
  p.c = kernel_cache(cache);
  p.q = q;
  p.q_row = q_row;
  p.q_head = q_head;
  p.starts = starts;
  p.ends = ends;
  p.indices = indices;
  p.width = width;
  p.out = out;
  p.lse = lse;
  p.requests = requests;
  p.R = R;
  p.rows = requests * R;
  p.heads = heads;
  p.group = heads / cache->kv_heads;
  p.dtype = dtype;
  p.scale = scale;
  p.cols = a.cols;
  p.tiles = a.tiles;
  p.splits = a.splits;
  p.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + a.ml);
  p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + a.o);
  const int err = mqa_attend_launch(&p, static_cast<hipStream_t>(stream));
  return err != 0 ? mqa::launch_failed(err) : MQA_OK;
}

}  // namespace

extern "C" {

size_t mqa_kv_page_bytes(int kv_heads, int head_dim, int page_size, int block) {
  return (size_t)page_bytes(kv_heads, head_dim, page_size, block);
}

int mqa_kv_append(const mqa_kv_cache* cache, const void* k, int64_t k_row_stride,
                  int64_t k_head_stride, const void* v, int64_t v_row_stride,
                  int64_t v_head_stride, int dtype, const int32_t* starts, const int32_t* counts,
                  int requests, int R, void* stream) {
  if (!cache || !k || !v || !starts) return MQA_ERR_NULL;
  const int rc = cache_pointers(cache);
  if (rc != MQA_OK) return rc;
  const int unit = dtype == MQA_FP32 ? 4 : 8;  // elements in 16 bytes
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(starts, 4) || !aligned(counts, 4) ||
      k_row_stride % unit != 0 || k_head_stride % unit != 0 || v_row_stride % unit != 0 ||
      v_head_stride % unit != 0)
    return MQA_ERR_ALIGN;
  if (!cache_shape(cache) || !rows_ok(requests, R) || dtype < MQA_BF16 || dtype > MQA_FP32 ||
      k_row_stride < 0 || k_head_stride < 0 || v_row_stride < 0 || v_head_stride < 0)
    return MQA_ERR_SHAPE;
  KvMoveParams p{};
  p.k = k;
  p.v = v;
  p.k_row = k_row_stride;
  p.k_head = k_head_stride;
  p.v_row = v_row_stride;
  p.v_head = v_head_stride;
  p.starts = starts;
  p.counts = counts;
  p.requests = requests;
  p.R = R;
  p.dtype = dtype;
  return move(cache, p, mqa_kv_append_launch, stream);
}

int mqa_kv_read(const mqa_kv_cache* cache, void* k, void* v, int dtype, const int32_t* starts,
                const int32_t* counts, int requests, int R, void* stream) {
  if (!cache || !k || !v || !starts) return MQA_ERR_NULL;
  const int rc = cache_pointers(cache);
  if (rc != MQA_OK) return rc;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(starts, 4) || !aligned(counts, 4))
    return MQA_ERR_ALIGN;
  if (!cache_shape(cache) || !rows_ok(requests, R) || dtype < MQA_BF16 || dtype > MQA_FP32)
    return MQA_ERR_SHAPE;
  KvMoveParams p{};
  p.ko = k;
  p.vo = v;
  p.starts = starts;
  p.counts = counts;
  p.requests = requests;
  p.R = R;
  p.dtype = dtype;
  return move(cache, p, mqa_kv_read_launch, stream);
}

size_t workspace_size_attend(int requests, int R, int heads, int kv_heads, int head_dim,
                             int positions, int device) {
  if (!sizes_ok(requests, R, heads, kv_heads, head_dim, positions)) return 0;
  const int cus = mqa::device_cus(device);
  if (!cus) return 0;
  auto most = [&](bool list) {
    return most_workspace(requests, R, heads, kv_heads, head_dim, at_most_keys(positions), list,
                          cus);
  };
  const size_t range = most(false), list = most(true);
  return range > list ? range : list;
}

size_t workspace_size_attend_call(int requests, int R, int heads, int kv_heads, int head_dim,
                                  int positions, int listed, int device) {
  if (!sizes_ok(requests, R, heads, kv_heads, head_dim, positions)) return 0;
  const int cus = mqa::device_cus(device);
  if (!cus) return 0;
  return plan(requests, R, heads, kv_heads, head_dim, at_most_keys(positions), listed != 0, cus)
      .total;
}

int mqa_attend_paged(const mqa_kv_cache* cache, const void* q, int64_t q_row_stride,
                     int64_t q_head_stride, int dtype, const int32_t* starts, const int32_t* ends,
                     void* out, float* lse, int requests, int R, int heads, float scale,
                     void* workspace, size_t workspace_bytes, void* stream) {
  const int64_t cap = cache ? (int64_t)cache->table_stride * cache->page_size : 0;
  return attend(cache, q, q_row_stride, q_head_stride, dtype, nullptr, 0, starts, ends, out, lse,
                requests, R, heads, scale, workspace, workspace_bytes,
                at_most_keys(cap), stream);
}

int mqa_attend_topk(const mqa_kv_cache* cache, const void* q, int64_t q_row_stride,
                    int64_t q_head_stride, int dtype, const int32_t* indices, int width,
                    const int32_t* starts, const int32_t* ends, void* out, float* lse,
                    int requests, int R, int heads, float scale, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!indices) return MQA_ERR_NULL;
  return attend(cache, q, q_row_stride, q_head_stride, dtype, indices, width, starts, ends, out,
                lse, requests, R, heads, scale, workspace, workspace_bytes, width, stream);
}

}  // extern "C"
