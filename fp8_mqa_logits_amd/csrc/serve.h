// Parameter blocks and launch entry points of weigh.hip and evict.hip.
#pragma once

#include "attend.h"

namespace mqa {

struct WeighParams {
  AttendParams a;    // q, ranges, heads, scale; out and lists unused
  const float* lse;  // [rows][heads]
  float* weights;    // [requests][width]
  int width;
  int tiles;   // workgroups of a request
  bool split;  // few columns: waves share keys
  // Many columns, tile by tile of 32 (row_tiles for a query head's rows, an even number
  // for a key head's): the queries [tile][32][head_dim]; {lse', its factor} [tile][32];
  // {largest start, smallest end, smallest start, largest end} [tile]. The sums of a
  // workgroup's share [request][slots][kWeighKeys]. Of a request, {first position, tiles of
  // keys, shares of a tile, -} and its span [request][2].
  bool wide;
  int slots, row_tiles;
  uint16_t* queries;
  float2* columns;
  int4* sight;
  float* part;
  int4* cut;
};

// Tiles of keys that a workgroup of the wide kernel takes.
constexpr int kWeighKeys = 512;
constexpr int kWeighRounds = 4;  // of workgroups, at most, unless there are more tiles

struct SelectParams {
  const float* weights;  // [requests][width]
  const int32_t* lengths;
  int32_t* positions;  // [requests][keep]
  int32_t* counts;
  float* kept;  // [requests][width] or nullptr
  int width, keep, sinks, recent, requests;
  int parts, part;  // of a request's positions, their length (a multiple of 1024)
  uint32_t* hist;   // parts > 1: [requests][parts][3][2048]
};

struct KeepParams {
  KvCache c;
  const int32_t* positions;  // [requests][width]
  const int32_t* counts;
  const int32_t* starts;  // nullptr: 0
  int width, requests, blocks;  // blocks of a request that moved tokens can fall into
  bool direct;                  // in place, without the workspace
  int chunks;
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
