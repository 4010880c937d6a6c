// Attention calls: which tiles they run on, and the join of split keys.
#include "attend_tiles.h"

namespace mqa {
namespace {

// Joins the splits of a (row, query head), in order, one workgroup each: the
// splits' weights first, then 256 / head_dim groups of threads take every
// such-and-such split, a thread a column of the output. A split that saw
// nothing has l = 0.
template <int T, int D>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendParams p) {
  constexpr int GROUPS = 256 / D;
  __shared__ float s_w[kMaxSplits];
  __shared__ float s_v[GROUPS][D];
  const int64_t pair = p.block0 + blockIdx.x;
  const int t = threadIdx.x, lane = t & 63;
  const int row = (int)(pair / p.heads), head = (int)(pair % p.heads), h = head / p.group;
  const int per_unit = p.indices ? 1 : p.R;
  const int column = row % per_unit * p.group + head % p.group;
  const int64_t item = ((int64_t)(row / per_unit) * p.tiles + column / p.cols) * p.c.kv_heads + h;
  const int64_t first = item * p.splits * p.cols + column % p.cols;
  static_assert(kMaxSplits == 64, "a lane a split");
  const float* ml = p.part_ml + 2 * (first + (int64_t)lane * p.cols);
  const float ls = lane < p.splits ? ml[1] : 0.f;
  const float ms = ls != 0.f ? ml[0] : kLowest;
  const float top = wave_max(ms);
  const float w = ls != 0.f ? __builtin_amdgcn_exp2f(ms - top) : 0.f;
  float sum = ls * w;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o, 64);
  if (t < 64) s_w[lane] = w;
  __syncthreads();
  const int d = t % D, group = t / D;
  const float* o = p.part_o + first * D + d;
  float v = 0.f;
#pragma unroll 8
  for (int s = group; s < p.splits; s += GROUPS) {
    const float x = o[(int64_t)s * p.cols * D], ws = s_w[s];
    v = ws == 0.f ? v : __builtin_fmaf(x, ws, v);
  }
  s_v[group][d] = v;
  __syncthreads();
  if (group != 0) return;
  v = s_v[0][d];
#pragma unroll
  for (int g = 1; g < GROUPS; ++g) v += s_v[g][d];
  static_cast<uint16_t*>(p.out)[pair * D + d] = to_type(sum == 0.f ? 0.f : v / sum, T);
  if (d == 0 && p.lse)
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
    in_pieces(*all, (int64_t)all->rows * all->heads, [&](const AttendParams& p, dim3 grid) {
      dispatch(p, [&](auto t, auto, auto d) {
        attend_join_kernel<t.value, d.value><<<grid, 256, 0, s>>>(p);
      });
    });
  return (int)hipGetLastError();
}
