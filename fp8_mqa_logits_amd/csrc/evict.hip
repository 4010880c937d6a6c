// Eviction from the paged 8-bit cache: which positions stay (by accumulated weight),
// and moving what stays together.
#include <type_traits>

#include "kvcodes.h"
#include "serve.h"

namespace mqa {
namespace {

// ------------------------------------------------------------------ selection

constexpr int kSelectThreads = 1024, kSelectWaves = kSelectThreads / 64;

// Weights in an order of unsigned integers: NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t rank_of(float w) {
  if (w != w) return ~0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A workgroup selects for one request. Of the positions between the sinks and the
// recent ones the `need` largest weights stay, those of the smallest positions where
// they are equal. The need-th largest is found digit by digit (11, 11 and 10 bits) by
// histograms in LDS; then every wave goes through a part of the positions in their
// order, once to count and once to write.
__global__ __launch_bounds__(kSelectThreads) void kv_select_kernel(SelectParams p) {
  const int i = blockIdx.x, t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  int n = p.lengths[i];
  n = n < 0 ? 0 : (n > p.width ? p.width : n);
  const float* const w = p.weights + (int64_t)i * p.width;
  const int count = n < p.keep ? n : p.keep;
  const int lo = n < p.sinks ? n : p.sinks, hi = n - p.recent > lo ? n - p.recent : lo;
  const int need = count - lo - (n - hi);  // of [lo, hi); sinks + recent <= keep

  __shared__ uint32_t s_hist[2048];
  __shared__ uint32_t s_wave[kSelectWaves], s_ties[kSelectWaves];
  __shared__ uint32_t s_digit, s_rest;

  uint32_t found = 0, left = (uint32_t)need;  // the digits so far; how many of them stay
  const bool all = need >= hi - lo;
  if (!all && need > 0) {
    for (int shift = 21, bits = 11; shift >= 0; bits = shift >= 11 ? 11 : 10, shift -= bits) {
      for (int b = t; b < 2048; b += kSelectThreads) s_hist[b] = 0;
      __syncthreads();
      const uint32_t above = shift == 21 ? 0u : ~0u << (shift + bits);
      for (int j = lo + t; j < hi; j += kSelectThreads) {
        const uint32_t u = rank_of(w[j]);
        if (((u ^ found) & above) == 0) atomicAdd(&s_hist[u >> shift & ((1u << bits) - 1)], 1u);
      }
      __syncthreads();
      // the largest digit d with at least `left` elements at or above it: two bins a
      // thread, sums from above
      const uint32_t b1 = s_hist[2047 - 2 * t], b0 = s_hist[2046 - 2 * t];
      uint32_t sum = b1 + b0;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const uint32_t x = __shfl_up(sum, o, 64);
        if (lane >= o) sum += x;
      }
      if (lane == 63) s_wave[wave] = sum;
      __syncthreads();
      for (int v = 0; v < wave; ++v) sum += s_wave[v];
      const uint32_t before = sum - b1 - b0;  // above this thread's bins
      if (before < left && before + b1 >= left) {
        s_digit = 2047 - 2 * t;
        s_rest = left - before;
      } else if (before + b1 < left && sum >= left) {
        s_digit = 2046 - 2 * t;
        s_rest = left - before - b1;
      }
      __syncthreads();
      found |= s_digit << shift;
      left = s_rest;
      if (shift == 0) break;
    }
  }

  // of a position: whether it stays for sure, whether it is one of the equal ones
  auto look = [&](int j, bool& stays, bool& tie) {
    stays = tie = false;
    if (j >= n) return;
    if (j < lo || j >= hi || all) {
      stays = true;
    } else if (need > 0) {
      const uint32_t u = rank_of(w[j]);
      stays = u > found;
      tie = u == found;
    }
  };
  const int part = (n + kSelectThreads - 1) / kSelectThreads * 64;  // a wave's positions
  const int from = wave * part, to = min(from + part, n);
  uint32_t sure = 0, ties = 0;
  for (int j = from; j < to; j += 64) {
    bool stays, tie;
    look(j + lane < to ? j + lane : n, stays, tie);
    sure += __popcll(__ballot(stays));
    ties += __popcll(__ballot(tie));
  }
  __syncthreads();
  if (lane == 0) {
    s_wave[wave] = sure;
    s_ties[wave] = ties;
  }
  __syncthreads();
  uint32_t at = 0, tied = 0;
  for (int v = 0; v < wave; ++v) {
    at += s_wave[v];
    tied += s_ties[v];
  }
  at += tied < left ? tied : left;
  int32_t* const list = p.positions + (int64_t)i * p.keep;
  float* const kept = p.kept ? p.kept + (int64_t)i * p.width : nullptr;
  const uint64_t below = (1ull << lane) - 1;
  for (int j = from; j < to; j += 64) {
    bool stays, tie;
    look(j + lane < to ? j + lane : n, stays, tie);
    const uint64_t mt = __ballot(tie);
    stays = stays || (tie && tied + __popcll(mt & below) < left);
    const uint64_t m = __ballot(stays);
    if (stays) {
      const uint32_t x = at + __popcll(m & below);
      list[x] = j + lane;
      if (kept) kept[x] = w[j + lane];
    }
    at += __popcll(m);
    tied += __popcll(mt);
  }
  for (int x = count + t; x < p.keep; x += kSelectThreads) list[x] = -1;
  if (kept)
    for (int x = count + t; x < p.width; x += kSelectThreads) kept[x] = 0.f;
  if (t == 0) p.counts[i] = count;
}

// -------------------------------------------------------------------- moving

constexpr int kKeepThreads = 256;

// What a workgroup moves: tokens lo <= t < hi of a request fall into one block of its
// positions, `kept` tokens of which stand there before them.
struct Target {
  int request, item_block, lo, hi, kept;
  int64_t first;  // position of token 0
  int begin;      // position of the block
};

// Whether there is anything to do: false where nothing is moved here, or every token
// stays where it is.
__device__ __forceinline__ bool target(const KeepParams& p, int block_index, Target& x) {
  const KvCache& c = p.c;
  x.request = block_index / p.blocks;
  const int B = 1 << c.block_shift;
  int count = p.counts[x.request];
  count = count < 0 ? 0 : (count > p.width ? p.width : count);
  x.first = p.starts ? p.starts[x.request] : 0;
  const int64_t begin = (x.first & ~(int64_t)(B - 1)) + (int64_t)(block_index % p.blocks) * B;
  const int64_t lo = begin > x.first ? begin : x.first;
  const int64_t hi = begin + B < x.first + count ? begin + B : x.first + count;
  if (begin < 0 || begin >= c.cap || lo >= hi) return false;
  x.begin = (int)begin;
  x.lo = (int)(lo - x.first);
  x.hi = (int)(hi - x.first);
  x.kept = (int)(lo - begin);
  if (page_of(c, x.request, x.begin) < 0) return false;
  const int32_t* const list = p.positions + (int64_t)x.request * p.width;
  bool moves = false;
  for (int t = x.lo + threadIdx.x; t < x.hi; t += kKeepThreads) moves |= list[t] != x.first + t;
  return __syncthreads_or(moves);
}

// Gathers a block's tokens: their values, the block's scale (the smallest power of two
// that holds the largest of them), and their codes under it, into the workspace.
template <int C, int D>
__global__ __launch_bounds__(kKeepThreads) void kv_gather_kernel(KeepParams p) {
  constexpr int PER = D / 8;
  const KvCache& c = p.c;
  const int h = blockIdx.y, w = blockIdx.z;
  Target x;
  if (!target(p, blockIdx.x, x)) return;
  const int64_t item = ((int64_t)blockIdx.x * 2 + w) * c.kv_heads + h;
  const int32_t* const list = p.positions + (int64_t)x.request * p.width;
  const int n = (x.hi - x.lo) * PER;
  // values of piece i: eight elements of a token (0 where the list names none)
  auto piece = [&](int i, float* v) {
    const int pos = list[x.lo + i / PER];
    uint2 code{0, 0};
    float s = 0.f;
    if (pos >= 0 && pos < c.cap) {
      const int page = page_of(c, x.request, pos);
      if (page >= 0) {
        const uint8_t* const base = c.pages + (int64_t)page * c.page_stride;
        const int slot = pos & ((1 << c.page_shift) - 1);
        s = *reinterpret_cast<const float*>(base + scale_at(c, w, h, slot));
        code = *reinterpret_cast<const uint2*>(base + code_at(c, w, h, slot) + i % PER * 8);
      }
    }
    decode8<C>(code, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= s;
  };
  float amax = 0.f, v[8];
  for (int i = threadIdx.x; i < n; i += kKeepThreads) {
    piece(i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = __builtin_fabsf(v[j]);
      amax = a < __builtin_inff() ? __builtin_fmaxf(amax, a) : amax;
    }
  }
  __shared__ float part[kKeepThreads / 64];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) amax = __builtin_fmaxf(amax, __shfl_xor(amax, o, 64));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kKeepThreads / 64; ++i) amax = __builtin_fmaxf(amax, part[i]);
  float scale = __builtin_ldexpf(1.f, scale_exponent<C>(amax));
  if (x.kept) {
    const int page = page_of(c, x.request, x.begin), slot = x.begin & ((1 << c.page_shift) - 1);
    const float was = *reinterpret_cast<const float*>(
        c.pages + (int64_t)page * c.page_stride + scale_at(c, w, h, slot));
    scale = scale > was ? scale : was;
  }
  const float inv = 1.f / scale;
  uint8_t* const codes = p.codes + item * ((int64_t)D << c.block_shift);
  for (int i = threadIdx.x; i < n; i += kKeepThreads) {
    piece(i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= inv;
    *reinterpret_cast<uint2*>(codes + x.kept * D + i * 8) = encode8<C>(v);
  }
  if (threadIdx.x == 0) p.scales[item] = scale;
}

// Puts the gathered blocks where they belong; what a first block keeps is rounded again
// where its scale grew.
template <int C, int D>
__global__ __launch_bounds__(kKeepThreads) void kv_place_kernel(KeepParams p) {
  constexpr int PER = D / 8;
  const KvCache& c = p.c;
  const int h = blockIdx.y, w = blockIdx.z;
  Target x;
  if (!target(p, blockIdx.x, x)) return;
  const int64_t item = ((int64_t)blockIdx.x * 2 + w) * c.kv_heads + h;
  uint8_t* const base =
      c.pages + (int64_t)page_of(c, x.request, x.begin) * c.page_stride;
  const int slot = x.begin & ((1 << c.page_shift) - 1);
  float* const scale_p = reinterpret_cast<float*>(base + scale_at(c, w, h, slot));
  const float was = x.kept ? *scale_p : 0.f, scale = p.scales[item];
  uint8_t* const to = base + code_at(c, w, h, slot);
  const uint8_t* const from = p.codes + item * ((int64_t)D << c.block_shift);
  __syncthreads();
  for (int i = threadIdx.x; i < (x.hi - x.lo) * PER; i += kKeepThreads)
    *reinterpret_cast<uint2*>(to + x.kept * D + i * 8) =
        *reinterpret_cast<const uint2*>(from + x.kept * D + i * 8);
  if (x.kept && scale > was) {
    const float shrink = was * (1.f / scale);
    for (int i = threadIdx.x; i < x.kept * PER; i += kKeepThreads) {
      uint2* const at = reinterpret_cast<uint2*>(to + i * 8);
      float v[8];
      decode8<C>(*at, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= shrink;
      *at = encode8<C>(v);
    }
  }
  if (threadIdx.x == 0 && !(x.kept && scale == was)) *scale_p = scale;
}

// f(codes, head_dim) as compile-time values.
template <class F>
void dispatch(const KvCache& c, F f) {
  auto with = [&](auto codes) {
    if (c.head_dim == 64)
      f(codes, std::integral_constant<int, 64>{});
    else
      f(codes, std::integral_constant<int, 128>{});
  };
  if (c.codes == kE4m3)
    with(std::integral_constant<int, kE4m3>{});
  else
    with(std::integral_constant<int, kInt8>{});
}

}  // namespace
}  // namespace mqa

extern "C" int mqa_kv_select_launch(const mqa::SelectParams* p, hipStream_t s) {
  mqa::kv_select_kernel<<<dim3(p->requests), mqa::kSelectThreads, 0, s>>>(*p);
  return (int)hipGetLastError();
}

extern "C" int mqa_kv_keep_launch(const mqa::KeepParams* p, hipStream_t s) {
  using namespace mqa;
  dispatch(p->c, [&](auto c, auto d) {
    const dim3 grid((unsigned)p->requests * p->blocks, p->c.kv_heads, 2);
    kv_gather_kernel<c.value, d.value><<<grid, kKeepThreads, 0, s>>>(*p);
    kv_place_kernel<c.value, d.value><<<grid, kKeepThreads, 0, s>>>(*p);
  });
  return (int)hipGetLastError();
}
