// C ABI of eviction from the paged 8-bit cache: argument checks, workspace layout and
// launches. The declarations and their contracts are in include/mqa_serve.h.
#include <hip/hip_runtime.h>

#include "cache_api.h"
#include "launch.h"
#include "mqa_serve.h"
#include "serve.h"

namespace {

using namespace mqa;

// Blocks that `width` tokens from any position on can fall into.
int64_t blocks_of(int width, int block) {
  return ((int64_t)block - 1 + width - 1) / block + 1;
}

// Calls of more columns (rows x query heads of a key head) run on the wide kernel: 9000
// positions of 8 key heads of 4 query heads, 64 rows (256 columns) 33 us on the narrow one,
// 44 on the wide one, 128 rows (512) 61 and 40.
constexpr int kNarrowColumns = 384;
constexpr int kWeighGroups = 256;  // workgroups that the wide kernel's work is cut for

struct WeighLayout {
  bool wide;
  int tiles, slots, row_tiles;  // of a request: workgroups; sums of 512 keys; 32 rows
  size_t columns, sight, part, cut, total;
};
WeighLayout weigh_layout(int requests, int R, int heads, int kv_heads, int head_dim,
                         int positions) {
  WeighLayout a{};
  a.wide = (int64_t)R * (heads / kv_heads) > kNarrowColumns;
  if (!a.wide) {
    a.total = kNoWorkspace;
    return a;
  }
  const int keys = (positions + kWeighKeys - 1) / kWeighKeys;
  a.tiles = kWeighGroups / requests < 1 ? 1 : kWeighGroups / requests;
  a.slots = keys > kWeighRounds * a.tiles ? keys : kWeighRounds * a.tiles;
  a.row_tiles = (R + 31) / 32;
  const size_t tiles =
      (size_t)requests * kv_heads * ((heads / kv_heads * (size_t)a.row_tiles + 1) / 2 * 2);
  // (fewer requests have more workgroups each: never more than kWeighGroups in all)
  const size_t slots = (size_t)requests * a.slots, few = kWeighRounds * kWeighGroups;
  a.columns = tiles * 32 * head_dim * 2;
  a.sight = a.columns + tiles * 32 * sizeof(float2);
  a.part = a.sight + tiles * sizeof(int4);
  a.cut = a.part + (slots > few ? slots : few) * kWeighKeys * 4;
  a.total = a.cut + (size_t)requests * 2 * sizeof(int4);
  return a;
}

// Parts of a request's positions in mqa_kv_select. Up to 16384 weights stay in one
// workgroup's registers (32 requests of 9001: 18 us, in three parts 27); more are cut into
// as many parts as fill the card, of 4096 or more (65536 weights of one request: 16 parts,
// 33 us in four launches, in one part 99); 512 requests and more have one workgroup each.
constexpr int kSelectWhole = 16384;
int64_t select_parts(int width) { return width <= kSelectWhole ? 1 : (width + 4095) / 4096; }

struct SelectLayout {
  int parts, part;
  size_t total;
};
SelectLayout select_layout(int requests, int width) {
  SelectLayout a{};
  const int most = 512 / requests < 64 ? 512 / requests : 64, want = (int)select_parts(width);
  const int parts = most < 1 ? 1 : want < most ? want : most;
  a.part = ((width + parts - 1) / parts + 1023) / 1024 * 1024;
  a.parts = (width + a.part - 1) / a.part;
  a.total = a.parts > 1 ? (size_t)requests * a.parts * 3 * 2048 * 4 : kNoWorkspace;
  return a;
}

// Whether mqa_kv_keep works in place: a workgroup for the keys or the values of a
// request's head, where these are enough to fill half the card or lists are so short that
// none has more than two rounds to go. Selecting, moving and reading 2048 of 9001 positions
// of 8 heads: 1 request 57 us in place, 45 through the workspace, 4 64 and 64, 8 72 and 86,
// 16 96 and 142; accepted drafts of one request 10 and 12.
constexpr int kDirectGroups = 128;
bool keep_direct(int requests, int width, int kv_heads, int block) {
  return block <= 64 &&
         ((int64_t)requests * kv_heads * 2 >= kDirectGroups || width + block <= 1024);
}

struct KeepLayout {
  size_t scales, total;
};
KeepLayout keep_layout(int requests, int width, int kv_heads, int head_dim, int block) {
  KeepLayout none{};
  none.total = kNoWorkspace;
  if (keep_direct(requests, width, kv_heads, block)) return none;
  const size_t items = (size_t)requests * blocks_of(width, block) * 2 * kv_heads;
  KeepLayout a{};
  a.scales = (items * block * head_dim + 255) / 256 * 256;
  a.total = a.scales + (items * 4 + 255) / 256 * 256;
  return a;
}

bool keep_sizes_ok(int requests, int width) {
  return requests >= 1 && requests <= MQA_MAX_ROWS && width >= 1 && width <= MQA_MAX_KEYS &&
         (int64_t)requests * width <= (int64_t)MQA_MAX_KEPT;
}

}  // namespace

extern "C" {

size_t workspace_size_weigh(int requests, int R, int heads, int kv_heads, int head_dim,
                            int positions, int device) {
  if (!rows_ok(requests, R) || kv_heads < 1 || heads < kv_heads || heads > MQA_MAX_ATTEND_HEADS ||
      heads % kv_heads != 0 || (head_dim != 64 && head_dim != 128) || positions < 1)
    return 0;
  if (!device_cus(device)) return 0;
  return weigh_layout(requests, R, heads, kv_heads, head_dim, at_most_keys(positions)).total;
}

int mqa_kv_weigh(const mqa_kv_cache* cache, const void* q, int64_t q_row_stride,
                 int64_t q_head_stride, int dtype, const int32_t* starts, const int32_t* ends,
                 const float* lse, float* weights, int width, int requests, int R, int heads,
                 float scale, void* workspace, size_t workspace_bytes, void* stream) {
  if (!cache || !q || !starts || !ends || !lse || !weights) return MQA_ERR_NULL;
  const int rc = cache_pointers(cache);
  if (rc != MQA_OK) return rc;
  if (!aligned(q, 16) || q_row_stride % 8 != 0 || q_head_stride % 8 != 0 || !aligned(starts, 4) ||
      !aligned(ends, 4) || !aligned(lse, 4) || !aligned(weights, 4) || !aligned(workspace, 256))
    return MQA_ERR_ALIGN;
  if (!cache_shape(cache) || !rows_ok(requests, R) || heads < 1 || heads > MQA_MAX_ATTEND_HEADS ||
      heads % cache->kv_heads != 0 || (dtype != MQA_BF16 && dtype != MQA_FP16) ||
      q_row_stride < 0 || q_head_stride < 0 || !(scale >= 0.f) || scale > 3.4e38f || width < 1)
    return MQA_ERR_SHAPE;
  const int cus = current_device_cus();
  if (!cus) return MQA_ERR_DEVICE;
  const WeighLayout l =
      weigh_layout(requests, R, heads, cache->kv_heads, cache->head_dim,
                   at_most_keys(positions_of(cache)));
  if (!workspace && l.total > kNoWorkspace) return MQA_ERR_NULL;
  if (workspace && workspace_bytes < l.total)
    return workspace_failed("the workspace is smaller than workspace_size_weigh()");
  WeighParams p{};
  p.a.c = kernel_cache(cache);
  p.a.q = q;
  p.a.q_row = q_row_stride;
  p.a.q_head = q_head_stride;
  p.a.starts = starts;
  p.a.ends = ends;
  p.a.requests = requests;
  p.a.R = R;
  p.a.rows = requests * R;
  p.a.heads = heads;
  p.a.group = heads / cache->kv_heads;
  p.a.dtype = dtype;
  p.a.scale = scale;
  p.lse = lse;
  p.weights = weights;
  p.width = width;
  p.wide = l.wide;
  p.tiles = l.tiles;
  p.slots = l.slots;
  p.row_tiles = l.row_tiles;
  uint8_t* const base = static_cast<uint8_t*>(workspace);
  p.queries = reinterpret_cast<uint16_t*>(base);
  p.columns = reinterpret_cast<float2*>(base + l.columns);
  p.part = reinterpret_cast<float*>(base + l.part);
  p.sight = reinterpret_cast<int4*>(base + l.sight);
  p.cut = reinterpret_cast<int4*>(base + l.cut);
  if (!l.wide) {
    // Few columns: 256 keys a workgroup where that gives every compute unit four, else 64,
    // whose heads its waves share. One row each of 32 heads on 8 key heads of 128: 1 x 32768
    // positions 12.6 us shared, 16.5 not, 8 x 30000 54 and 58, 16 x 16384 59 and 51, 32 x
    // 32768 245 and 199. (Where all keys fit into one round of three workgroups a compute
    // unit, not sharing is faster already: 8 x 16384 32.5 and 27.4; but not for many rows or
    // a little more of them: 40 rows 114 and 133, 8 x 30000 205 and 255.)
    p.split = (int64_t)requests * p.a.c.cap < (int64_t)4 * 256 * cus;
    const int keys = p.split ? 64 : 256;
    const int most = (p.a.c.cap + keys - 1) / keys, share = 16 * cus / requests;
    p.tiles = most < share ? most : share < 1 ? 1 : share;
  }
  const int err = mqa_kv_weigh_launch(&p, static_cast<hipStream_t>(stream));
  return err != 0 ? launch_failed(err) : MQA_OK;
}

int mqa_kv_select(const float* weights, int width, const int32_t* lengths, int keep, int sinks,
                  int recent, int32_t* positions, int32_t* counts, float* kept, int requests,
                  void* workspace, size_t workspace_bytes, void* stream) {
  if (!weights || !lengths || !positions || !counts) return MQA_ERR_NULL;
  if (!aligned(weights, 4) || !aligned(lengths, 4) || !aligned(positions, 4) ||
      !aligned(counts, 4) || !aligned(kept, 4) || !aligned(workspace, 256))
    return MQA_ERR_ALIGN;
  if (!keep_sizes_ok(requests, keep) || width < 1 || width > MQA_MAX_KEYS || sinks < 0 ||
      recent < 0 || (int64_t)sinks + recent > keep)
    return MQA_ERR_SHAPE;
  if (!current_device_cus()) return MQA_ERR_DEVICE;
  const SelectLayout l = select_layout(requests, width);
  if (!workspace && l.total > kNoWorkspace) return MQA_ERR_NULL;
  if (workspace && workspace_bytes < l.total)
    return workspace_failed("the workspace is smaller than workspace_size_select()");
  SelectParams p{};
  p.parts = l.parts;
  p.part = l.part;
  p.hist = static_cast<uint32_t*>(workspace);
  p.weights = weights;
  p.lengths = lengths;
  p.positions = positions;
  p.counts = counts;
  p.kept = kept;
  p.width = width;
  p.keep = keep;
  p.sinks = sinks;
  p.recent = recent;
  p.requests = requests;
  const int err = mqa_kv_select_launch(&p, static_cast<hipStream_t>(stream));
  return err != 0 ? launch_failed(err) : MQA_OK;
}

size_t workspace_size_select(int requests, int width) {
  if (requests < 1 || requests > MQA_MAX_ROWS || width < 1 || width > MQA_MAX_KEYS) return 0;
  // fewer requests may have more parts each, but never more than 512 in all
  const int64_t most = select_parts(width), parts = requests * most < 512 ? requests * most : 512;
  return most > 1 ? (size_t)parts * 3 * 2048 * 4 : kNoWorkspace;
}

size_t workspace_size_keep(int requests, int width, int kv_heads, int head_dim, int block) {
  if (!keep_sizes_ok(requests, width) || page_bytes(kv_heads, head_dim, block, block) == 0) return 0;
  // (more requests may need none)
  int most = requests;
  if (keep_direct(requests, width, kv_heads, block)) {
    const int few = (kDirectGroups - 1) / (2 * kv_heads);
    most = few < requests ? few : requests;
    if (most < 1) return kNoWorkspace;
  }
  return keep_layout(most, width, kv_heads, head_dim, block).total;
}

int mqa_kv_keep(const mqa_kv_cache* cache, const int32_t* positions, const int32_t* counts,
                const int32_t* starts, int width, int requests, void* workspace,
                size_t workspace_bytes, void* stream) {
  if (!cache || !positions || !counts) return MQA_ERR_NULL;
  const int rc = cache_pointers(cache);
  if (rc != MQA_OK) return rc;
  if (!aligned(positions, 4) || !aligned(counts, 4) || !aligned(starts, 4) ||
      !aligned(workspace, 256))
    return MQA_ERR_ALIGN;
  if (!cache_shape(cache) || !keep_sizes_ok(requests, width)) return MQA_ERR_SHAPE;
  if (!current_device_cus()) return MQA_ERR_DEVICE;
  const KeepLayout a =
      keep_layout(requests, width, cache->kv_heads, cache->head_dim, cache->block);
  if (!workspace && a.total > kNoWorkspace) return MQA_ERR_NULL;
  if (workspace && workspace_bytes < a.total)
    return workspace_failed("the workspace is smaller than workspace_size_keep()");
  KeepParams p{};
  p.c = kernel_cache(cache);
  p.positions = positions;
  p.counts = counts;
  p.starts = starts;
  p.width = width;
  p.requests = requests;
  p.blocks = (int)blocks_of(width, cache->block);
  p.direct = a.total == kNoWorkspace;
  p.codes = static_cast<uint8_t*>(workspace);
  p.scales = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + a.scales);
  const int err = mqa_kv_keep_launch(&p, static_cast<hipStream_t>(stream));
  return err != 0 ? launch_failed(err) : MQA_OK;
}

}  // extern "C"
