// C ABI of the paged 8-bit key/value cache: argument checks, workspace layout
// and launches. The declarations and their contracts are in
// include/mqa_attend.h.
#include <hip/hip_runtime.h>

#include "attend.h"
#include "cache_api.h"
#include "launch.h"

namespace {

using namespace mqa;

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

// The plan of windows and trees (window: how many positions a row sees at most, 0: any
// number; positions: what the rows of a request may span). Narrower tiles span fewer
// positions of their rows' windows and waste fewer columns, wider ones take less time a
// column and key: a workgroup's time for a key, with its compute unit full, was measured as
// `ns`, for heads of 64 and of 128 (0: not taken. Tiles of 64 columns are the slowest a
// column; for heads of 64 those of 256 take between 0.91 and 1.6 times those of 128). A start and an end take the time of 640
// keys, of 1024 for the wide tiles; a join 7 us, or 2 and its parts' way to memory and back
// where they are many (8192 rows of 12 heads through 8196 positions: 335 us in two parts,
// 259 in one).
// Where the table's room, not the window, bounds what rows span (a prompt that fills its
// table), the first of them see less than a window: the rounds take the mean row's time, and
// all of it no less than the longest workgroup's.
// All rows of a prompt of 12 heads of 128, each its own key head, in a table of its size:
// 16384 through 8196 positions 700 us on 256 columns, 946 on 32; 8192 through 2052 225 and
// 174; 4096 through 4100 136 and 108. 2000 through 504 73 and 29; 4096 of 32 heads on 4 key
// heads through 1027 of many positions 129 and 158; 8 uneven trees of 13 drafts, 40 heads of
// 64 on 8 key heads, up to 9001 positions: 37 on 128, 45 on 32.
Plan fitted_plan(int requests, int R, int heads, int kv_heads, int head_dim, int positions,
                 int window, int cus) {
  static const struct {
    int cols;
    double ns[2];
  } kTiles[] = {{16, {12, 22}}, {32, {17, 12.5}}, {128, {18, 39}}, {256, {0, 31}}};
  Plan a{};
  const int group = heads / kv_heads, columns = R * group, most = widest(columns, false);
  const int64_t units = (int64_t)requests * kv_heads;
  // positions that a row sees in the mean: the first see lo, lo + 1, ..
  const int64_t lo = positions >= R ? positions - R + 1 : 1;
  const int64_t fewer = window <= lo ? 0 : window - lo < R ? window - lo : R;
  const double mean = window > 0 ? ((2 * lo + fewer - 1) * 0.5 * fewer +
                                    (double)(R - fewer) * window) / R : positions;
  double best = 0;
  int64_t slots = 0;
  for (const auto& t : kTiles) {
    const double ns = t.ns[head_dim == 128];
    if (t.cols > most || ns == 0) continue;
    const int64_t tiles = (columns + t.cols - 1) / t.cols, n = units * tiles;
    const int64_t room = resident(t.cols, head_dim, false, cus), ends = t.cols > 64 ? 1024 : 640;
    const int64_t rows = (t.cols + group - 1) / group;
    const int64_t span = window > 0 && window + rows < positions ? window + rows : positions;
    const double usual = mean + rows < span ? mean + rows : span;
    for (int s = 1; s <= mqa::kMaxSplits && (s == 1 || s * 256 <= span); ++s) {
      const int64_t rounds = (n * s + room - 1) / room;
      if (s > 1 && rounds > kMostRounds) break;
      // (a round that leaves compute units part of their workgroups takes less)
      const int64_t full = n * s / room, rest = n * s % room, held = room / cus;
      const double part = rest ? 0.4 + 0.6 * (double)((rest + cus - 1) / cus) / held : 0;
      const double all = ns * (usual / s + ends) * (full + part);
      const double longest = ns * ((double)span / s + ends) * (full ? 1 : part);
      const double parts = (double)units * columns * s * (4 * head_dim + 8);  // bytes
      const double join = 2000 + 2 * parts / 5000 > 7000 ? 2000 + 2 * parts / 5000 : 7000;
      const double cost = (all > longest ? all : longest) + (s > 1 ? join : 0);
      if (a.cols > 0 && cost >= best) continue;
      best = cost;
      a.cols = t.cols;
      a.tiles = (int)tiles;
      a.splits = s;
      slots = s > 1 ? n * s * t.cols : 0;
    }
  }
  lay_out(a, slots, head_dim);
  return a;
}

// kind: 0 ranges, 1 lists, 2 windows (window: of a row, its sinks among them), 3 trees.
Plan plan_of(int kind, int requests, int R, int heads, int kv_heads, int head_dim, int positions,
             int window, int cus) {
  if (kind < 2) return plan(requests, R, heads, kv_heads, head_dim, positions, kind == 1, cus);
  return fitted_plan(requests, R, heads, kv_heads, head_dim, positions, kind == 2 ? window : 0, cus);
}

// What the windows of a request's R rows span of `room` positions, in a row.
int64_t spanned(int64_t window, int R, int64_t room) {
  return window + R - 1 < room ? window + R - 1 : room;
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

int move(const mqa_kv_cache* cache, KvMoveParams& p, int (*launch)(const KvMoveParams*, hipStream_t),
         void* stream) {
  if (!mqa::current_device_cus()) return MQA_ERR_DEVICE;
  p.c = kernel_cache(cache);
  const int rc = launch(&p, static_cast<hipStream_t>(stream));
  return rc != 0 ? mqa::launch_failed(rc) : MQA_OK;
}

// What the entry points differ in: p holds what rows see (sight and its fields, or a
// list), `good` says whether that is in range, and `positions` bounds what a row's tile
// of keys may span.
int attend(const mqa_kv_cache* cache, const void* q, int64_t q_row, int64_t q_head, int dtype,
           AttendParams p, bool good, const int32_t* starts, const int32_t* ends,
           void* out, float* lse, int requests, int R, int heads, float scale, void* workspace,
           size_t workspace_bytes, int64_t positions, void* stream) {
  if (!cache || !q || !starts || !ends || !out) return MQA_ERR_NULL;
  const int rc = cache_pointers(cache);
  if (rc != MQA_OK) return rc;
  if (!aligned(q, 16) || q_row % 8 != 0 || q_head % 8 != 0 || !aligned(starts, 4) ||
      !aligned(ends, 4) || !aligned(p.indices, 16) || !aligned(p.mask, 4) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(workspace, 256))
    return MQA_ERR_ALIGN;
  if (!cache_shape(cache) || !rows_ok(requests, R) || heads < 1 || heads > MQA_MAX_ATTEND_HEADS ||
      heads % cache->kv_heads != 0 || (dtype != MQA_BF16 && dtype != MQA_FP16) || q_row < 0 ||
      q_head < 0 || !(scale >= 0.f) || scale > 3.4e38f || !good)
    return MQA_ERR_SHAPE;
  const int cus = mqa::current_device_cus();
  if (!cus) return MQA_ERR_DEVICE;
  const int kind = p.indices ? 1 : p.sight == mqa::kWindow ? 2 : p.sight == mqa::kTree ? 3 : 0;
  const Plan a = plan_of(kind, requests, R, heads, cache->kv_heads, cache->head_dim,
                         at_most_keys(positions), at_most_keys((int64_t)p.window + p.sinks), cus);
  if (!workspace && a.total > kNoWorkspace) return MQA_ERR_NULL;
  if (workspace && workspace_bytes < a.total)
    return mqa::workspace_failed(kind == 2
                                     ? "the workspace is smaller than workspace_size_attend_window()"
                                     : "the workspace is smaller than workspace_size_attend_call()");
  p.c = kernel_cache(cache);
  p.q = q;
  p.q_row = q_row;
  p.q_head = q_head;
  p.starts = starts;
  p.ends = ends;
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
                                  int positions, int kind, int device) {
  if (!sizes_ok(requests, R, heads, kv_heads, head_dim, positions) || kind < 0 || kind > 3) return 0;
  const int cus = mqa::device_cus(device), most = at_most_keys(positions);
  if (!cus) return 0;
  // Windows: `positions` may be the table's room and says nothing of a row's window then.
  // Where the narrowest tile holds all rows they span it all, else any plan is possible.
  if (kind == 2 && (int64_t)R * (heads / kv_heads) > 16)
    return most_workspace(requests, R, heads, kv_heads, head_dim, most, false, cus);
  return plan_of(kind, requests, R, heads, kv_heads, head_dim, most, 0, cus).total;
}

size_t workspace_size_attend_window(int requests, int R, int heads, int kv_heads, int head_dim,
                                    int positions, int window, int sinks, int device) {
  if (!sizes_ok(requests, R, heads, kv_heads, head_dim, positions) || window < 1 || sinks < 0)
    return 0;
  const int cus = mqa::device_cus(device);
  if (!cus) return 0;
  const int64_t seen = (int64_t)window + sinks;
  return plan_of(2, requests, R, heads, kv_heads, head_dim,
                 at_most_keys(spanned(seen, R, positions)), at_most_keys(seen), cus)
      .total;
}

int mqa_attend_cut(int kind, int requests, int R, int heads, int kv_heads, int head_dim,
                   int positions, int window, int sinks, int compute_units, int32_t* cut) {
  if (!cut) return MQA_ERR_NULL;
  if (!sizes_ok(requests, R, heads, kv_heads, head_dim, positions) || kind < 0 || kind > 3 ||
      compute_units < 1 || compute_units > 4096 || (kind == 2 && (window < 1 || sinks < 0)))
    return MQA_ERR_SHAPE;
  const int64_t seen = (int64_t)window + sinks;
  const Plan a = plan_of(kind, requests, R, heads, kv_heads, head_dim,
                         at_most_keys(kind == 2 ? spanned(seen, R, positions) : positions),
                         at_most_keys(seen), compute_units);
  cut[0] = a.cols;
  cut[1] = a.tiles;
  cut[2] = a.splits;
  return MQA_OK;
}

int mqa_attend_paged(const mqa_kv_cache* cache, const void* q, int64_t q_row_stride,
                     int64_t q_head_stride, int dtype, const int32_t* starts, const int32_t* ends,
                     void* out, float* lse, int requests, int R, int heads, float scale,
                     void* workspace, size_t workspace_bytes, void* stream) {
  return attend(cache, q, q_row_stride, q_head_stride, dtype, AttendParams{}, true, starts, ends,
                out, lse, requests, R, heads, scale, workspace, workspace_bytes, positions_of(cache),
                stream);
}

int mqa_attend_topk(const mqa_kv_cache* cache, const void* q, int64_t q_row_stride,
                    int64_t q_head_stride, int dtype, const int32_t* indices, int width,
                    const int32_t* starts, const int32_t* ends, void* out, float* lse,
                    int requests, int R, int heads, float scale, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!indices) return MQA_ERR_NULL;
  AttendParams p{};
  p.indices = indices;
  p.width = width;
  return attend(cache, q, q_row_stride, q_head_stride, dtype, p,
                width >= 1 && width <= MQA_MAX_LIST, starts, ends, out, lse, requests, R, heads,
                scale, workspace, workspace_bytes, width, stream);
}

int mqa_attend_window(const mqa_kv_cache* cache, const void* q, int64_t q_row_stride,
                      int64_t q_head_stride, int dtype, const int32_t* starts, const int32_t* ends,
                      int window, int sinks, void* out, float* lse, int requests, int R, int heads,
                      float scale, void* workspace, size_t workspace_bytes, void* stream) {
  AttendParams p{};
  p.sight = mqa::kWindow;
  p.window = window;
  p.sinks = sinks;
  return attend(cache, q, q_row_stride, q_head_stride, dtype, p, window >= 1 && sinks >= 0, starts,
                ends, out, lse, requests, R, heads, scale, workspace, workspace_bytes,
                spanned((int64_t)window + sinks, R, positions_of(cache)), stream);
}

int mqa_attend_tree(const mqa_kv_cache* cache, const void* q, int64_t q_row_stride,
                    int64_t q_head_stride, int dtype, const int32_t* starts, const int32_t* ends,
                    const int32_t* mask, int words, void* out, float* lse, int requests, int R,
                    int heads, float scale, void* workspace, size_t workspace_bytes,
                    void* stream) {
  if (!mask) return MQA_ERR_NULL;
  AttendParams p{};
  p.sight = mqa::kTree;
  p.mask = mask;
  p.words = words;
  return attend(cache, q, q_row_stride, q_head_stride, dtype, p,
                words >= 1 && words <= MQA_MAX_DRAFT_WORDS, starts, ends, out, lse, requests, R,
                heads, scale, workspace, workspace_bytes, positions_of(cache), stream);
}

}  // extern "C"
