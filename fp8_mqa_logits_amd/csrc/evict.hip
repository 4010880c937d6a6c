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
// 65536 weights: 99 us in one workgroup, whose vector unit is what bounds it; 4 + 7 + 8 + 14
// in these four launches, chains of loads and barriers.)
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
#pragma unroll
    for (int v = 0; v < kSelectWaves; ++v) sum += v < wave ? s_wave[v] : 0;
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
      // sums over all parts and those before this one, of all levels at once: what other
      // workgroups wrote comes from far
      uint32_t b1[3] = {}, b0[3] = {}, p1[3] = {}, p0[3] = {};
      const uint32_t* const h = p.hist + (int64_t)i * p.parts * 3 * 2048 + 2046 - 2 * t;
#pragma unroll 8
      for (int v = 0; v < p.parts; ++v)
#pragma unroll
        for (int level = 0; level < (LEVEL < 3 ? LEVEL : 3); ++level) {
          const uint2 x = *reinterpret_cast<const uint2*>(h + (v * 3 + level) * 2048);
          b0[level] += x.x;
          b1[level] += x.y;
          p0[level] += v < g ? x.x : 0;
          p1[level] += v < g ? x.y : 0;
        }
#pragma unroll
      for (int level = 0; level < (LEVEL < 3 ? LEVEL : 3); ++level) {
        const uint32_t digit = pick(b1[level], b0[level]), top = 2047 - 2 * t;
        sure += (top > digit ? p1[level] : 0) + (top - 1 > digit ? p0[level] : 0);
        if (level == 2) ties = top == digit ? p1[2] : top - 1 == digit ? p0[2] : 0;
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
#pragma unroll
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
#pragma unroll
  for (int v = 0; v < kSelectWaves; ++v) {
    at += v < wave ? s_wave[v] : 0;
    tied += v < wave ? s_ties[v] : 0;
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
//
// A moved block is made in three steps: its tokens' codes and scales are gathered, its
// scale is found (the smallest power of two that holds the largest of them), and the
// codes are written under it. Entry t of a list names no position before its place, starts
// + t (the caller sees to it). Hence what a workgroup gathers for later blocks is still
// there when it has written the earlier ones, and one that goes through a request's blocks
// in their order, of one head's keys or values, can work in place: kv_move_kernel<DIRECT>.
// With too few requests and heads for that, blocks are gathered by all workgroups at once
// into the workspace (kv_move_kernel) and put in place by a second launch
// (kv_place_kernel).
//
// 32 requests cut to 2048 positions of 4 heads of 128 in place: 37 us, 3.4 TB/s read
// and written (selecting, moving and reading back 112 us, 197 with gather and place);
// 8192 positions of one request's 8 heads through the workspace 14 + 8 us; accepted paths
// of 64 trees 7 us, the chain of loads.

// What a block keeps, `bytes` codes, under its larger scale; thread t of `threads`.
template <int C>
__device__ __forceinline__ void round_again(uint8_t* codes, int bytes, float was, float scale, int t,
                                            int threads) {
  const float shrink = was * (1.f / scale);
  constexpr int AHEAD = 8;  // reads on their way
  for (int i0 = t; i0 < bytes / 8; i0 += AHEAD * threads) {
    uint2 x[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (i0 + k * threads < bytes / 8) x[k] = *reinterpret_cast<uint2*>(codes + (i0 + k * threads) * 8);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (i0 + k * threads >= bytes / 8) continue;
      float v[8];
      decode8<C>(x[k], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= shrink;
      *reinterpret_cast<uint2*>(codes + (i0 + k * threads) * 8) = encode8<C>(v);
    }
  }
}

// A wave moves TOK tokens at a time (blocks of B <= 64): 16 codes a lane and read, every
// read within one block. Its largest is sought among the codes themselves, four in a word,
// and codes are rounded without regard to what is not finite, where neither a NaN nor an
// overflow nor a scale that is no power of two is there.
// The largest magnitude of 16 codes; odd: whether one is NaN.
template <int C>
__device__ __forceinline__ float largest_code(const uint4& code, bool& odd) {
  typedef uint16_t U2 __attribute__((ext_vector_type(2)));
  typedef int16_t I2 __attribute__((ext_vector_type(2)));
  const uint32_t word[4] = {code.x, code.y, code.z, code.w};
  if constexpr (C == kE4m3) {
    // magnitudes are ordered as their bits
    U2 lo{0, 0}, hi{0, 0};
    uint32_t nan = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      lo = __builtin_elementwise_max(lo, __builtin_bit_cast(U2, word[k] & 0x007F007Fu));
      hi = __builtin_elementwise_max(hi, __builtin_bit_cast(U2, word[k] & 0x7F007F00u));
      nan |= (word[k] & 0x7F7F7F7Fu) + 0x01010101u;
    }
    odd |= (nan & 0x80808080u) != 0;
    const U2 top = __builtin_elementwise_max(lo, (U2)(hi >> 8));
    return __builtin_amdgcn_cvt_f32_fp8(max((int)top.x, (int)top.y), 0);
  } else {
    I2 most{0, 0}, least{0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const I2 hi = __builtin_bit_cast(I2, word[k] & 0xFF00FF00u);
      const I2 lo = __builtin_bit_cast(I2, word[k]) << 8;
      most = __builtin_elementwise_max(most, __builtin_elementwise_max(hi, lo));
      least = __builtin_elementwise_min(least, __builtin_elementwise_min(hi, lo));
    }
    const int up = max((int)most.x, (int)most.y), down = min((int)least.x, (int)least.y);
    return (float)(max(up, -down) >> 8);
  }
}

// Four codes of scale s under the power of two 1 / inv, where all is finite and no result
// is too large.
template <int C>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float s, float inv) {
  if constexpr (C == kE4m3) {
    float v[4] = {__builtin_amdgcn_cvt_f32_fp8((int)w, 0), __builtin_amdgcn_cvt_f32_fp8((int)w, 1),
                  __builtin_amdgcn_cvt_f32_fp8((int)w, 2), __builtin_amdgcn_cvt_f32_fp8((int)w, 3)};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = v[j] * s * inv;
    const int d = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], d, true);
  } else {
    // added to 1.5 * 2^23, a number is rounded to the integer in the sum's last byte
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      u[j] = __float_as_uint(
          __builtin_fmaf((float)(int8_t)(w >> (8 * j)) * s, inv, 12582912.f));
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(u[3], u[2], 0x0C0C0400u),
                                 __builtin_amdgcn_perm(u[1], u[0], 0x0C0C0400u), 0x05040100u);
  }
}

template <int C, int D, int B, bool DIRECT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 4) void kv_move_kernel(KeepParams p) {
  constexpr int TOK = 64, PER = D / 16, AT = 64 / PER;  // tokens a read
  constexpr int NL = TOK / AT, LB = B / AT, NB = TOK / B;            // reads; of a block; blocks
  const KvCache& c = p.c;
  const int h = blockIdx.y, w = blockIdx.z, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int request = DIRECT ? blockIdx.x : blockIdx.x / p.chunks;
  int count = p.counts[request];
  count = count < 0 ? 0 : (count > p.width ? p.width : count);
  const int64_t first = p.starts ? p.starts[request] : 0;
  if (count == 0) return;
  const int64_t begin = first & ~(int64_t)(B - 1);
  const int kept = (int)(first - begin);  // tokens of the first block that stand before
  const int32_t* const list = p.positions + (int64_t)request * p.width;
  const int chunks = (kept + count + WAVES * TOK - 1) / (WAVES * TOK);

  struct Held {
    uint4 code[NL];
    float s[NL];
    uint32_t moves;  // bit i: read i's token does not stay where it is
  };
  // tokens of a chunk, from - kept ..: token 0's place is `first`
  auto from_of = [&](int chunk) { return (chunk * WAVES + wave) * TOK - kept; };
  auto fetch = [&](Held& f, int chunk) {
    // (what has no place or no source is read from some page, and cleared)
    int pos[NL], page[NL];
    uint32_t none = 0;  // bit i: read i stands for zeros
    f.moves = 0;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int t = from_of(chunk) + i * AT + lane / PER;
      pos[i] = list[min(max(t, 0), count - 1)];
      const bool real = t >= 0 && t < count;
      f.moves |= (real && pos[i] != first + t ? 1u : 0u) << i;
      none |= (!real || pos[i] < 0 || pos[i] >= c.cap ? 1u : 0u) << i;
    }
    const int32_t* const table = c.table + (int64_t)request * c.table_stride;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      pos[i] = min(max(pos[i], 0), c.cap - 1);
      page[i] = table[pos[i] >> c.page_shift];
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      none |= (page[i] < 0 || page[i] >= c.num_pages ? 1u : 0u) << i;
      const uint8_t* const base =
          c.pages + (int64_t)min(max(page[i], 0), c.num_pages - 1) * c.page_stride;
      const int slot = pos[i] & ((1 << c.page_shift) - 1);
      f.s[i] = *reinterpret_cast<const float*>(base + scale_at(c, w, h, slot));
      f.code[i] = *reinterpret_cast<const uint4*>(base + code_at(c, w, h, slot) + lane % PER * 16);
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      if (none >> i & 1) {
        f.s[i] = 0.f;
        f.code[i] = uint4{0, 0, 0, 0};
      }
    }
  };
  // half k of read i, in loops that are not unrolled (what is seldom needed stays small)
  auto half = [&](const Held& f, int i, int k, float& s) {
    uint2 x{0, 0};
    s = 0.f;
#pragma unroll
    for (int r = 0; r < NL; ++r) {
      x.x = i == r ? (k ? f.code[r].z : f.code[r].x) : x.x;
      x.y = i == r ? (k ? f.code[r].w : f.code[r].y) : x.y;
      s = i == r ? f.s[r] : s;
    }
    return x;
  };
  // the block's new codes, in place of its old ones; its scale
  auto round = [&](Held& f, int b, float was) {
    // the largest magnitude among a lane's codes of a read, times its scale
    float amax = 0.f;
    bool odd = false;  // NaN or overflow
#pragma unroll
    for (int i = b * LB; i < (b + 1) * LB; ++i) {
      const float a = largest_code<C>(f.code[i], odd) * f.s[i];
      odd |= !(a >= 0.f && a < __builtin_inff());
      amax = __builtin_fmaxf(amax, a);
    }
    const bool plain = !__any(odd);
    if (!plain) {
      amax = 0.f;
#pragma unroll 1
      for (int i = b * LB; i < (b + 1) * LB; ++i)
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          float v[8], s;
          decode8<C>(half(f, i, k, s), v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float a = __builtin_fabsf(v[j] * s);
            amax = a < __builtin_inff() ? __builtin_fmaxf(amax, a) : amax;
          }
        }
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) amax = __builtin_fmaxf(amax, __shfl_xor(amax, o, 64));
    const float fresh = __builtin_ldexpf(1.f, scale_exponent<C>(amax));
    const float scale = fresh > was ? fresh : was, inv = 1.f / scale;
    // (a kept scale may be any; a subnormal inverse would lose bits)
    if (plain && (__float_as_uint(scale) & 0x807FFFFFu) == 0 && scale < 0x1p120f) {
#pragma unroll
      for (int i = b * LB; i < (b + 1) * LB; ++i) {
        uint32_t* const word = &f.code[i].x;
#pragma unroll
        for (int k = 0; k < 4; ++k) word[k] = rescale4<C>(word[k], f.s[i], inv);
      }
    } else {
#pragma unroll 1
      for (int i = b * LB; i < (b + 1) * LB; ++i)
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          float v[8], s;
          decode8<C>(half(f, i, k, s), v);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = v[j] * s * inv;
          const uint2 x = encode8<C>(v);
#pragma unroll
          for (int r = 0; r < NL; ++r) {
            f.code[r].x = i == r && k == 0 ? x.x : f.code[r].x;
            f.code[r].y = i == r && k == 0 ? x.y : f.code[r].y;
            f.code[r].z = i == r && k == 1 ? x.x : f.code[r].z;
            f.code[r].w = i == r && k == 1 ? x.y : f.code[r].w;
          }
        }
    }
    return scale;
  };
  // whether block b of a chunk has a place and something moves in it; its page and slot
  struct Place {
    uint8_t* base;
    int slot, kept;
    bool any;
  };
  auto place = [&](const Held& f, int chunk, int b) {
    Place x{nullptr, 0, 0, false};
    const int t = from_of(chunk) + b * B;  // of the block's first token
    const int64_t at = first + t;
    if (t >= count || at < 0 || at >= c.cap) return x;
    if (!__any(f.moves >> (b * LB) & ((1ull << LB) - 1))) return x;
    const int page = page_of(c, request, (int)at);
    if (page < 0) return x;
    return Place{c.pages + (int64_t)page * c.page_stride, (int)at & ((1 << c.page_shift) - 1),
                 t < 0 ? -t : 0, true};
  };

  Held f;
  for (int chunk = DIRECT ? 0 : blockIdx.x % p.chunks; chunk < chunks; ++chunk) {
    fetch(f, chunk);
    float scale[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const Place x = place(f, chunk, b);
      const float was =
          x.any && x.kept ? *reinterpret_cast<const float*>(x.base + scale_at(c, w, h, x.slot)) : 0.f;
      scale[b] = x.any ? round(f, b, was) : 0.f;
    }
    if (DIRECT) __syncthreads();  // (every wave has what it gathers from these places)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const Place x = place(f, chunk, b);
      if (!x.any) continue;
      uint8_t* to;
      if constexpr (DIRECT) {
        to = x.base + code_at(c, w, h, x.slot);
      } else {
        const int64_t item =
            (((int64_t)request * p.blocks + (chunk * WAVES + wave) * NB + b) * 2 + w) *
                c.kv_heads + h;
        to = p.codes + item * (B * D);
        if (lane == 0) p.scales[item] = scale[b];
      }
#pragma unroll
      for (int i = b * LB; i < (b + 1) * LB; ++i) {
        const int t = from_of(chunk) + i * AT + lane / PER;
        if (t >= 0 && t < count)
          *reinterpret_cast<uint4*>(to + ((i - b * LB) * 64 + lane) * 16) = f.code[i];
      }
      if constexpr (DIRECT) {
        float* const scale_p = reinterpret_cast<float*>(x.base + scale_at(c, w, h, x.slot));
        const float was = x.kept ? *scale_p : 0.f;
        if (x.kept && scale[b] > was) round_again<C>(to, x.kept * D, was, scale[b], lane, 64);
        if (lane == 0 && !(x.kept && scale[b] == was)) *scale_p = scale[b];
      }
    }
    if (!DIRECT) break;
  }
}

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

// kv_move_kernel's part for blocks of more than 64 tokens, a workgroup each, which reads
// them twice. Gathers a block's tokens: their values, the block's scale (the smallest power of two
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
  constexpr int PER = D / 16;
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
    *reinterpret_cast<uint4*>(to + x.kept * D + i * 16) =
        *reinterpret_cast<const uint4*>(from + x.kept * D + i * 16);
  if (x.kept && scale > was) round_again<C>(to, x.kept * D, was, scale, threadIdx.x, kKeepThreads);
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
  // (requests that fill the card many times over take one each, so that a grid stays below
  // 2^32 threads; rows cut into parts are of fewer than 512 requests)
  const bool much = p->width > 4 * kSelectThreads || p->keep > 4 * kSelectThreads;
  const int fillers = much && p->requests < 1 << 16 ? 4 : 1;
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
    auto move = [&](auto block) {
      constexpr int B = block.value;
      if (p->direct) {
        // short lists: as many workgroups a compute unit as there are
        const dim3 grid(p->requests, p->c.kv_heads, 2);
        if (p->width + B <= 128)
          kv_move_kernel<c.value, d.value, B, true, 2><<<grid, 128, 0, s>>>(*p);
        else
          kv_move_kernel<c.value, d.value, B, true, 16><<<grid, 1024, 0, s>>>(*p);
      } else {
        KeepParams all = *p;
        all.chunks = (int)(((int64_t)p->blocks * B + 255) / 256);
        kv_move_kernel<c.value, d.value, B, false, 4>
            <<<dim3((unsigned)p->requests * all.chunks, p->c.kv_heads, 2), 256, 0, s>>>(all);
      }
    };
    const dim3 grid((unsigned)p->requests * p->blocks, p->c.kv_heads, 2);
    const int B = 1 << p->c.block_shift;
    if (B == 16) move(std::integral_constant<int, 16>{});
    if (B == 32) move(std::integral_constant<int, 32>{});
    if (B == 64) move(std::integral_constant<int, 64>{});
    if (B > 64) kv_gather_kernel<c.value, d.value><<<grid, kKeepThreads, 0, s>>>(*p);
    if (!p->direct) kv_place_kernel<c.value, d.value><<<grid, kKeepThreads, 0, s>>>(*p);
  });
  return (int)hipGetLastError();
}
