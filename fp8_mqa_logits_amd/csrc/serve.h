// Parameter blocks and launch entry points of weigh.hip and evict.hip.
#pragma once

#include "attend.h"

namespace mqa {

struct WeighParams {
  AttendParams a;    // q, ranges, heads, scale; out and lists unused
  const float* lse;  // [rows][heads]
  float* weights;    // [requests][width]
  int width;
  int tiles;  // workgroups of a request
  // Many columns: what is known of a column, {lse', its factor}, [request][head][32 *
  // row_tiles]; of 32 columns, {largest start, smallest end, smallest start, largest end};
  // of a request, {first position, tiles of keys, shares of a tile, -} and its span; and
  // the sums of a workgroup's share [request][slots][kWeighKeys].
  bool wide;
  int slots, row_tiles;
  float2* columns;
  int4* sight;
  int4* cut;  // [requests][2]
  float* part;
};

// Tiles of keys that a workgroup of the wide kernel takes.
constexpr int kWeighKeys = 512;

struct SelectParams {
  const float* weights;  // [requests][width]
  const int32_t* lengths;
  int32_t* positions;  // [requests][keep]
  int32_t* counts;
  float* kept;  // [requests][width] or nullptr
  int width, keep, sinks, recent, requests;
};

struct KeepParams {
  KvCache c;
  const int32_t* positions;  // [requests][width]
  const int32_t* counts;
  const int32_t* starts;  // nullptr: 0
  int width, requests, blocks;  // blocks of a request that moved tokens can fall into
  // moved blocks on their way: codes [item][B][head_dim], scales [item], item =
  // ((request * blocks + block) * 2 + w) * kv_heads + head
  uint8_t* codes;
  float* scales;
};

}  // namespace mqa

extern "C" {
int mqa_kv_weigh_launch(const mqa::WeighParams* p, hipStream_t stream);
int mqa_kv_select_launch(const mqa::SelectParams* p, hipStream_t stream);
int mqa_kv_keep_launch(const mqa::KeepParams* p, hipStream_t stream);
}
