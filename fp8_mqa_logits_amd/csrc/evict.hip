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

// Of the positions between the sinks and the recent ones the `need` largest weights stay,
// those of the smallest positions where they are equal. The need-th largest is found
// digit by digit (11, 11 and 10 bits) by histograms in LDS; then every wave goes through
// its part of the positions in their order, once to count and once to write. Its weights
// stay in registers meanwhile (HOLD a lane; 0: they are read again).
//
// LEVEL kWhole: a workgroup for a request. Long rows of few requests are cut into
// p.parts of p.part positions: launches of LEVEL 0, 1 and 2 leave each part's histogram
// of a digit in the workspace, among the positions that agree with the digits before,
// which every workgroup finds from the sums of the histograms so far; the last launch
// finds from them also what stays of the parts before its own, and writes. (A request of
// 65536 weights: 99 us in one workgroup, whose vector unit is what bounds it.)
//
// The other workgroups of a request clear what lies behind the chosen weights.
enum { kWhole = 4, kWrite = 3 };

__device__ __forceinline__ int digit_shift(int level) { return level == 0 ? 21 : level == 1 ? 10 : 0; }
__device__ __forceinline__ uint32_t digit_mask(int level) { return level == 2 ? 0x3FFu : 0x7FFu; }

template <int LEVEL, int HOLD>
__global__ __launch_bounds__(kSelectThreads) void kv_select_kernel(SelectParams p, int fillers) {
  const int blocks = p.parts + fillers;
  const int i = blockIdx.x / blocks, g = blockIdx.x % blocks;
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  int n = p.lengths[i];
  n = n < 0 ? 0 : (n > p.width ? p.width : n);
  const int count = n < p.keep ? n : p.keep;
  float* const kept = p.kept ? p.kept + (int64_t)i * p.width : nullptr;
  int32_t* const list = p.positions + (int64_t)i * p.keep;
  if (g >= p.parts) {
    const int step = fillers * kSelectThreads, at = count + (g - p.parts) * kSelectThreads + t;
    for (int x = at; x < p.keep; x += step) list[x] = -1;
    if (kept)
      for (int x = at; x < p.width; x += step) kept[x] = 0.f;
    return;
  }
  const float* const w = p.weights + (int64_t)i * p.width;
  const int lo = n < p.sinks ? n : p.sinks, hi = n - p.recent > lo ? n - p.recent : lo;
  const int need = count - lo - (n - hi);  // of [lo, hi); sinks + recent <= keep
  const bool search = need > 0 && need < hi - lo;
  // the workgroup's positions, and the wave's
  const int begin = min(g * p.part, n), end = min(begin + p.part, n);
  const int rounds = (end - begin + kSelectThreads - 1) / kSelectThreads;  // of 64 a wave
  const int from = min(begin + wave * rounds * 64, end), to = min(from + rounds * 64, end);

  __shared__ uint32_t s_hist[2048];
  __shared__ uint32_t s_wave[kSelectWaves], s_ties[kSelectWaves];
  __shared__ uint32_t s_digit, s_rest;

  // f(position, weight) for the lane's positions, in their order
  float held[HOLD ? HOLD : 1];
  if constexpr (HOLD > 0) {
#pragma unroll
    for (int r = 0; r < HOLD; ++r) {
      const int j = from + 64 * r + lane;
      held[r] = j < to ? w[j] : 0.f;
    }
  }
  auto each = [&](auto f) {
    if constexpr (HOLD > 0) {
#pragma unroll
      for (int r = 0; r < HOLD; ++r) {
        if (64 * r < to - from) f(from + 64 * r + lane, held[r]);
        __builtin_amdgcn_sched_barrier(0);  // (rounds side by side would need too many registers)
      }
    } else {
      constexpr int AHEAD = 8;  // reads on their way
      for (int j0 = from; j0 < to; j0 += 64 * AHEAD) {
        float x[AHEAD];
#pragma unroll
        for (int r = 0; r < AHEAD; ++r) {
          const int j = j0 + 64 * r + lane;
          x[r] = j < to ? w[j] : 0.f;
        }
#pragma unroll
        for (int r = 0; r < AHEAD; ++r)
          if (j0 + 64 * r < to) f(j0 + 64 * r + lane, x[r]);
      }
    }
  };

  uint32_t found = 0, left = (uint32_t)need;  // the digits so far; how many of them stay
  // the histogram of a level's digit, over what agrees with `found` above it
  auto histogram = [&](int level) {
    const int shift = digit_shift(level);
    const uint32_t mask = digit_mask(level), above = ~(mask << shift | ((1u << shift) - 1));
    for (int b = t; b < 2048; b += kSelectThreads) s_hist[b] = 0;
    __syncthreads();
    each([&](int j, float x) {
      const uint32_t u = rank_of(x);
      const bool counts = j >= lo && j < hi && j < to && ((u ^ found) & above) == 0;
      const uint32_t digit = u >> shift & mask;
      // (what is equal in the whole wave is one addition: weights may all be)
      const uint64_t m = __ballot(counts);
      if (m == 0) return;
      const uint32_t one = __builtin_amdgcn_readlane(digit, __builtin_ctzll(m));
      const uint64_t same = __ballot(counts && digit == one);
      if (counts && digit != one) atomicAdd(&s_hist[digit], 1u);
      if (lane == __builtin_ctzll(m)) atomicAdd(&s_hist[one], (uint32_t)__popcll(same));
    });
    __syncthreads();
  };
  // the largest digit with at least `left` elements at or above it: two bins a thread,
  // 2047 - 2 t with b1 elements and the one below it with b0, sums from above
  auto pick = [&](uint32_t b1, uint32_t b0) {
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
    left = s_rest;
    return s_digit;
  };
  uint32_t sure_before = 0, ties_before = 0;  // of the parts before this one
  if (search) {
    if constexpr (LEVEL == kWhole) {
      for (int level = 0; level < 3; ++level) {
        histogram(level);
        found |= pick(s_hist[2047 - 2 * t], s_hist[2046 - 2 * t]) << digit_shift(level);
        __syncthreads();
      }
    } else {
      uint32_t* const mine = p.hist + ((int64_t)i * p.parts + g) * 3 * 2048;
      uint32_t sure = 0, ties = 0;  // in this thread's bins
      for (int level = 0; level < LEVEL; ++level) {
        const uint32_t* h = p.hist + (int64_t)i * p.parts * 3 * 2048 + level * 2048 + 2046 - 2 * t;
        uint32_t b1 = 0, b0 = 0, p1 = 0, p0 = 0;
#pragma unroll 8
        for (int v = 0; v < p.parts; ++v) {
          const uint2 x = *reinterpret_cast<const uint2*>(h + v * (3 * 2048));
          b0 += x.x;
          b1 += x.y;
          p0 += v < g ? x.x : 0;
          p1 += v < g ? x.y : 0;
        }
        const uint32_t digit = pick(b1, b0), top = 2047 - 2 * t;
        sure += (top > digit ? p1 : 0) + (top - 1 > digit ? p0 : 0);
        if (level == 2) ties = top == digit ? p1 : top - 1 == digit ? p0 : 0;
        found |= digit << digit_shift(level);
        __syncthreads();
      }
      if constexpr (LEVEL < kWrite) {
        histogram(LEVEL);
        for (int b = t; b < 2048; b += kSelectThreads) mine[LEVEL * 2048 + b] = s_hist[b];
      } else {
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          sure += __shfl_xor(sure, o, 64);
          ties += __shfl_xor(ties, o, 64);
        }
        if (lane == 0) {
          s_wave[wave] = sure;
          s_ties[wave] = ties;
        }
        __syncthreads();
        for (int v = 0; v < kSelectWaves; ++v) {
          sure_before += s_wave[v];
          ties_before += s_ties[v];
        }
        __syncthreads();
      }
    }
  }
  if constexpr (LEVEL < kWrite) return;

  // of a position: whether it stays for sure, whether it is one of the equal ones
  auto look = [&](int j, float x, bool& stays, bool& tie) {
    const bool middle = j >= lo && j < hi;
    const uint32_t u = rank_of(x);
    stays = j < to && (!middle || (search ? u > found : need > 0));
    tie = j < to && middle && search && u == found;
  };
  uint32_t sure = 0, ties = 0;
  each([&](int j, float x) {
    bool stays, tie;
    look(j, x, stays, tie);
    sure += __popcll(__ballot(stays));
    ties += __popcll(__ballot(tie));
  });
  if (lane == 0) {
    s_wave[wave] = sure;
    s_ties[wave] = ties;
  }
  __syncthreads();
  // what stays before the workgroup's positions: of the ends, and in between
  const int middle = min(max(begin - lo, 0), hi - lo);
  uint32_t at = begin - middle + (search ? sure_before : need > 0 ? middle : 0);
  uint32_t tied = ties_before;
  for (int v = 0; v < wave; ++v) {
    at += s_wave[v];
    tied += s_ties[v];
  }
  at += tied < left ? tied : (search ? left : 0);
  const uint64_t below = (1ull << lane) - 1;
  each([&](int j, float x) {
    bool stays, tie;
    look(j, x, stays, tie);
    const uint64_t mt = __ballot(tie);
    stays = stays || (tie && tied + __popcll(mt & below) < left);
    const uint64_t m = __ballot(stays);
    if (stays) {
      const uint32_t to_at = at + __popcll(m & below);
      list[to_at] = j;
      if (kept) kept[to_at] = x;
    }
    at += __popcll(m);
    tied += __popcll(mt);
  });
  if (g == 0 && t == 0) p.counts[i] = count;
}

template <int LEVEL, int HOLD>
void select(const SelectParams& p, int fillers, hipStream_t s) {
  kv_select_kernel<LEVEL, HOLD>
      <<<dim3((unsigned)p.requests * (p.parts + fillers)), kSelectThreads, 0, s>>>(p, fillers);
}
template <int HOLD>
void select(const SelectParams& p, int fillers, hipStream_t s) {
  if (p.parts == 1) {
    select<kWhole, HOLD>(p, fillers, s);
  } else {
    select<0, HOLD>(p, 0, s);
    select<1, HOLD>(p, 0, s);
    select<2, HOLD>(p, 0, s);
    select<kWrite, HOLD>(p, fillers, s);
  }
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
  using namespace mqa;
  const int fillers = p->width > 4 * kSelectThreads || p->keep > 4 * kSelectThreads ? 4 : 1;
  if (p->part <= 4 * kSelectThreads)
    select<4>(*p, fillers, s);
  else if (p->part <= 16 * kSelectThreads)
    select<16>(*p, fillers, s);
  else
    select<0>(*p, fillers, s);
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
