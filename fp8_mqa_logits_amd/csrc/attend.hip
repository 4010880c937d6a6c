// Attention calls: which tiles they run on, and the join of split keys.
#include "attend_tiles.h"

namespace mqa {
namespace {

// Joins the splits of a (row, query head), in order, with WAYS waves each: a
// lane every 64th split for the weights, then D / 64 columns of the output of
// every WAYS-th split. A split that saw nothing has l = 0 and sums of 0 (but for a
// row that sees nothing at all, whose output is 0 whatever they are). Few
// splits: one wave, many rows a workgroup; many: their reads in parallel.
template <int T, int D, int WAYS>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendParams p) {
  constexpr int EACH = D / 64, MANY = kMaxSplits / 64;
  __shared__ float s_v[4][D];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, way = wave % WAYS;
  const int64_t pair = (p.block0 + blockIdx.x) * (4 / WAYS) + wave / WAYS;
  const bool real = pair < (int64_t)p.rows * p.heads;
  if (WAYS == 1 && !real) return;
  const int row = (int)(real ? pair / p.heads : 0), head = (int)(real ? pair % p.heads : 0);
  const int h = head / p.group;
  const int per_unit = p.indices ? 1 : p.R;
  const int column = row % per_unit * p.group + head % p.group;
  const int64_t item = ((int64_t)(row / per_unit) * p.tiles + column / p.cols) * p.c.kv_heads + h;
  const int64_t first = item * p.splits * p.cols + column % p.cols;
  float ms[MANY], ls[MANY], w[MANY], top = kLowest, sum = 0.f;
#pragma unroll
  for (int k = 0; k < MANY; ++k) {
    const int s = lane + 64 * k;
    const float* ml = p.part_ml + 2 * (first + (int64_t)(s < p.splits ? s : 0) * p.cols);
    ls[k] = s < p.splits ? ml[1] : 0.f;
    ms[k] = ls[k] != 0.f ? ml[0] : kLowest;
    top = __builtin_fmaxf(top, ms[k]);
  }
  top = wave_max(top);
#pragma unroll
  for (int k = 0; k < MANY; ++k) {
    w[k] = ls[k] != 0.f ? __builtin_amdgcn_exp2f(ms[k] - top) : 0.f;
    sum = __builtin_fmaf(ls[k], w[k], sum);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o, 64);
  typedef float Cols __attribute__((ext_vector_type(EACH)));
  const float* const o = p.part_o + first * D + EACH * lane;
  const int64_t stride = (int64_t)p.cols * D;
  Cols v = 0.f;
#pragma unroll
  for (int k = 0; k < MANY; ++k) {
    constexpr int AHEAD = 8;  // reads on their way
    const int end = min(p.splits - 64 * k, 64);
    for (int s0 = way; s0 < end; s0 += WAYS * AHEAD) {
      Cols x[AHEAD];
#pragma unroll
      for (int a = 0; a < AHEAD; ++a)
        x[a] = *reinterpret_cast<const Cols*>(o + (64 * k + min(s0 + WAYS * a, end - 1)) * stride);
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        const int s = s0 + WAYS * a;
        const float ws = s < end ? __int_as_float(__builtin_amdgcn_readlane(
                                       __float_as_int(w[k]), s & 63)) : 0.f;
        // (also where a part's weight is 0: what it holds may be NaN)
#pragma unroll
        for (int e = 0; e < EACH; ++e) v[e] = __builtin_fmaf(x[a][e], ws, v[e]);
      }
    }
  }
  if constexpr (WAYS > 1) {
#pragma unroll
    for (int e = 0; e < EACH; ++e) s_v[wave][EACH * lane + e] = v[e];
    __syncthreads();
    if (way != 0 || !real) return;
#pragma unroll
    for (int k = 1; k < WAYS; ++k)
#pragma unroll
      for (int e = 0; e < EACH; ++e) v[e] += s_v[wave + k][EACH * lane + e];
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
  if (all->splits > 1) {
    const int64_t pairs = (int64_t)all->rows * all->heads;
    const bool many = all->splits > 16;
    in_pieces(*all, many ? pairs : (pairs + 3) / 4, [&](const AttendParams& p, dim3 grid) {
      dispatch(p, [&](auto t, auto, auto d) {
        if (many)
          attend_join_kernel<t.value, d.value, 4><<<grid, 256, 0, s>>>(p);
        else
          attend_join_kernel<t.value, d.value, 1><<<grid, 256, 0, s>>>(p);
      });
    });
  }
  return (int)hipGetLastError();
}
