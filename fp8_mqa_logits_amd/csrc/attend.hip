// Attention calls: which tiles they run on, and the join of split keys.
#include "attend_tiles.h"

namespace mqa {
namespace {

// Joins the splits of a (row, query head), in order, a wave each: a lane a
// split for the weights, then D / 64 columns of the output. A split that saw
// nothing has l = 0.
template <int T, int D>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendParams p) {
  constexpr int EACH = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t pair = (p.block0 + blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (pair >= (int64_t)p.rows * p.heads) return;
  const int row = (int)(pair / p.heads), head = (int)(pair % p.heads), h = head / p.group;
  const int per_unit = p.indices ? 1 : p.R;
  const int column = row % per_unit * p.group + head % p.group;
  const int64_t item = ((int64_t)(row / per_unit) * p.tiles + column / p.cols) * p.c.kv_heads + h;
  const int64_t first = item * p.splits * p.cols + column % p.cols;
  static_assert(kMaxSplits == 64, "a lane a split");
  const bool mine = lane < p.splits;
  const float* ml = p.part_ml + 2 * (first + (int64_t)(mine ? lane : 0) * p.cols);
  const float ls = mine ? ml[1] : 0.f;
  const float ms = ls != 0.f ? ml[0] : kLowest;
  const float top = wave_max(ms);
  const float w = ls != 0.f ? __builtin_amdgcn_exp2f(ms - top) : 0.f;
  float sum = ls * w;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o, 64);
  const float* o = p.part_o + first * D + EACH * lane;
  float v[EACH] = {};
#pragma unroll 8
  for (int s = 0; s < p.splits; ++s) {
    const float ws = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), s));
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      const float x = o[(int64_t)s * p.cols * D + e];
      v[e] = ws == 0.f ? v[e] : __builtin_fmaf(x, ws, v[e]);
    }
  }
  uint16_t* const out = static_cast<uint16_t*>(p.out) + pair * D + EACH * lane;
#pragma unroll
  for (int e = 0; e < EACH; ++e) out[e] = to_type(sum == 0.f ? 0.f : v[e] / sum, T);
  if (lane == 0 && p.lse)
    p.lse[pair] = sum == 0.f ? -__builtin_inff() : (top - kBias) * kLn2 + __builtin_logf(sum);
}

// A launch's grid stays below 2^32 threads: more workgroups go in several.
template <class Launch>
void in_pieces(AttendParams p, int64_t blocks, Launch launch) {
  constexpr int64_t kMost = 1 << 22;
  for (p.block0 = 0; p.block0 < blocks; p.block0 += kMost)
    launch(p, dim3((unsigned)(blocks - p.block0 < kMost ? blocks - p.block0 : kMost)));
}

}  // namespace
}  // namespace mqa

extern "C" int mqa_attend_launch(const mqa::AttendParams* all, hipStream_t s) {
  using namespace mqa;
  const int64_t units = all->indices ? all->rows : all->requests;
  in_pieces(*all, units * all->tiles * all->c.kv_heads * all->splits,
            [&](const AttendParams& p, dim3 grid) {
              if (p.indices)
                attend_list(p, grid, s);
              else if (p.cols <= 64)
                attend_narrow(p, grid, s);
              else
                attend_wide(p, grid, s);
            });
  if (all->splits > 1)
    in_pieces(*all, ((int64_t)all->rows * all->heads + 3) / 4, [&](const AttendParams& p, dim3 grid) {
      dispatch(p, [&](auto t, auto, auto d) {
        attend_join_kernel<t.value, d.value><<<grid, 256, 0, s>>>(p);
      });
    });
  return (int)hipGetLastError();
}
