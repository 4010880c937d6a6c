// Attention of query rows over a paged 8-bit key/value cache.
//
//     S_j = scale * ks_j * (q . kc_j)        (kc, vc: codes; ks, vs: block scales)
//     m = max_j S_j,  l = sum_j exp(S_j - m)
//     out = sum_j exp(S_j - m) * vs_j * vc_j / l,   lse = m + ln l
// over the positions j of the row's range, or over its listed positions.
//
// Numbers. Codes of either kind are exact in bf16 and in fp16, so q . kc runs
// on the matrix unit in q's own type with fp32 sums, and the scales come in
// afterwards, in fp32. The probabilities go to the second product in fp16
// whatever q's type (11 bits; bf16's 8 would add an error as large as the
// rounding of a bf16 output; outputs in fp16 are up to 1.4 times as far from the
// exact ones as a computation in fp32 rounded once, 2.9e-4 relative to 2.1e-4), as
// P = 2^10 e vs, where the exponentials e = 2^7 exp2(S' - m), S' in units of ln 2,
// are what l sums in fp32, before P's rounding.
// Every (row, head) column has its own reference point m, the largest of its S' +
// log2(vs / kVref) when m last moved: its loudest weight exp2(S') vs has P = 2^10 or
// more, at most 65504, and weights down to 2^-24 of it keep full precision, whatever
// other rows see and however loud the blocks are to which it gives no weight. m
// moves only when the P that a lane forms could pass 65504 (no search for a largest
// weight in the common step: 374 -> 367 us for 32 rows of 16 heads over 131072
// positions), and the sums are rescaled then. kVref is a value scale such as
// activations have; it keeps e near 2^7, where l costs lse no bits. In m, vs / kVref
// counts as 2^kLeast at least: e of a block of zeros stays finite, and value scales
// below 2^-97 lose precision.
// (2^10 is a choice between the two ends of fp16: at 2^7 outputs near 2^-20, made
// up of values of such weights, were off by up to twice an fp16 output's own
// rounding; the higher P starts the more often m moves: 4096 rows of 32 heads over
// 49152 positions 2.92 ms at 2^7, 2.95 at 2^10, 2.96 at 2^11, on one card.)

#pragma once

#include <type_traits>

#include "attend.h"
#include "launch.h"

namespace mqa {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.4028234e38f;  // m of a column that has seen nothing
constexpr float kVref = 0x1p-7f;
constexpr float kBias = 7.f;               // e is 2^kBias at m, for a value scale of kVref
constexpr float kTop = 10.f;               // and P 2^kTop
constexpr float kUp = 0x1p10f;             // P = kUp vs e: 2^(kTop - kBias) / kVref
constexpr float kMost = 65504.f;           // most that eight P may add up to
constexpr float kFar = 0x1p-88f;           // eight e times kFar, too
constexpr float kLeast = -90.f;            // least log2(vs / kVref) in m

// 4 codes of one dword -> 4 values of the matrix unit's type.
template <int T, int C>
__device__ __forceinline__ uint2 widen4(uint32_t w) {
  if constexpr (C == kE4m3) {
    if constexpr (T == kBf16) {
      return uint2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.f, true))};
    } else {
      return uint2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.f, true))};
    }
  } else if constexpr (T == kBf16) {
    const v2bf a{(__bf16)(float)(int8_t)w, (__bf16)(float)(int8_t)(w >> 8)};
    const v2bf b{(__bf16)(float)(int8_t)(w >> 16), (__bf16)(float)(int8_t)(w >> 24)};
    return uint2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
  } else {
    // the byte as the low mantissa bits of 1024 + (code + 128), exact in fp16
    w ^= 0x80808080u;
    const v2h off{(_Float16)-1152.f, (_Float16)-1152.f};
    const v2h a = __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) + off;
    const v2h b = __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) + off;
    return uint2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
  }
}

template <int T, int C>
__device__ __forceinline__ v4u widen8(uint32_t lo, uint32_t hi) {
  const uint2 a = widen4<T, C>(lo), b = widen4<T, C>(hi);
  return v4u{a.x, a.y, b.x, b.y};
}

template <int T>
__device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
  if constexpr (T == kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

template <int T>
__device__ __forceinline__ v16f mfma32(v4u a, v4u b, v16f c) {
  if constexpr (T == kBf16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Bytes w[i] of four dwords (rows) -> t[b] = bytes b of the four rows.
__device__ __forceinline__ void transpose4(const uint32_t* w, uint32_t* t) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u);  // w0.0 w1.0 w0.1 w1.1
  const uint32_t b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
  const uint32_t d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  t[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  t[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  t[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  t[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// 0xFF in each byte of w that is an e4m3 NaN (0x7F or 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  const uint32_t t = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return (t >> 7) * 0xFFu;
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) x = __builtin_fmaxf(x, __shfl_xor(x, o, 64));
  return x;
}

__device__ __forceinline__ uint16_t to_type(float x, int type) {
  return type == kBf16 ? __builtin_bit_cast(uint16_t, (__bf16)x)
                       : __builtin_bit_cast(uint16_t, (_Float16)x);
}

// A row's range, clamped as the contract says.
__device__ __forceinline__ void row_range(const AttendParams& p, int row, int& s, int& e) {
  s = p.starts[row];
  e = p.ends[row];
  s = s < 0 ? 0 : (s > p.c.cap ? p.c.cap : s);
  e = e < s ? s : (e > p.c.cap ? p.c.cap : e);
}

__device__ __forceinline__ int clamp_page(const KvCache& c, int entry) {
  return min(max(entry, 0), c.num_pages - 1);
}

// A pointer to what no one writes during the call: uniform loads through it
// are scalar.
template <class X>
__device__ __forceinline__ auto constant(const X* x) {
  return (const __attribute__((address_space(4))) X*)(uintptr_t)x;
}

// log2(vs / kVref) as m takes it, of kUp vs.
__device__ __forceinline__ float loudness(float vr) {
  return __builtin_fmaxf(__builtin_amdgcn_logf(vr) - (kTop - kBias), kLeast);
}

// Bits of the positions pos .. pos + 31 that lie in [s, e).
__device__ __forceinline__ uint32_t seen_bits(int pos, int s, int e) {
  const int from = max(s - pos, 0), to = min(e - pos, 32);
  return from >= to ? 0u : ~0u << from & ~0u >> (32 - to);
}

// All ones where bit `at` of mask is set: masks are applied to the scores' and
// probabilities' bits, as what is unseen may be NaN.
__device__ __forceinline__ uint32_t bit(uint32_t mask, int at) {
  return (uint32_t)__builtin_amdgcn_sbfe((int)mask, at, 1);
}
__device__ __forceinline__ float or_zero(float x, uint32_t see) {
  return __uint_as_float(__float_as_uint(x) & see);
}
__device__ __forceinline__ float or_lowest(float x, uint32_t see) {
  return __uint_as_float((__float_as_uint(x) & see) | (~see & 0xFF800000u));
}

// What a row sees (M: kRange, kWindow, kTree), by the range [s, e) that row_range
// gives: all of it; its first p.sinks and its last p.window positions; all of it and
// positions e + x for the set bits x of the row's mask, up to the table's end.
__device__ __forceinline__ int sinks_end(const AttendParams& p, int s, int e) {
  return e - s < p.sinks ? e : s + p.sinks;
}
__device__ __forceinline__ int window_start(const AttendParams& p, int s, int e) {
  return e - s < p.window ? s : e - p.window;
}

// 32 bits of the row's mask from bit x on; none before its first and behind its last.
__device__ __forceinline__ uint32_t mask_bits(const AttendParams& p, int row, int x) {
  const int32_t* const at = p.mask + (int64_t)row * p.words;
  const int word = x >> 5;
  const uint32_t lo = (uint32_t)word < (uint32_t)p.words ? at[word] : 0;
  const uint32_t hi = (uint32_t)(word + 1) < (uint32_t)p.words ? at[word + 1] : 0;
  return (uint32_t)(((uint64_t)hi << 32 | lo) >> (x & 31));
}

// Bits of the positions pos .. pos + 31 that the row sees.
template <int M>
__device__ __forceinline__ uint32_t row_bits(const AttendParams& p, int row, int pos, int s, int e) {
  uint32_t bits = seen_bits(pos, M == kWindow ? window_start(p, s, e) : s, e);
  if constexpr (M == kWindow) bits |= seen_bits(pos, s, sinks_end(p, s, e));
  if constexpr (M == kTree)
    if (pos + 32 > e) bits |= mask_bits(p, row, pos - e) & seen_bits(pos, e, p.c.cap);
  return bits;
}

// The lowest (-1: none) and the highest position behind e that the row's mask names.
struct Drafts {
  int lo, hi;
};
__device__ __forceinline__ Drafts drafts(const AttendParams& p, int row, int e) {
  Drafts d{-1, -1};
  for (int w = 0; w < p.words && e + 32 * w < p.c.cap; ++w) {
    const uint32_t bits = mask_bits(p, row, 32 * w) & seen_bits(e + 32 * w, e, p.c.cap);
    if (!bits) continue;
    if (d.lo < 0) d.lo = e + 32 * w + __builtin_ctz(bits);
    d.hi = e + 32 * w + 31 - __builtin_clz(bits);
  }
  return d;
}

template <int M>
__device__ __forceinline__ bool sees_nothing(const AttendParams& p, int row, int s, int e) {
  if constexpr (M == kTree)
    if (s >= e) return drafts(p, row, e).lo < 0;
  return s >= e;
}

// Of `rows` rows from row_lo, those that see nothing left out: the positions that some
// of them see lie in [lo, hi), where kWindow: in [lo, hi) or among the sinks' [s_lo,
// s_hi); those that all of them see hold [in_lo, in_hi). A lane takes every step-th row
// from `first`; the result is the wave's.
struct Span {
  int lo, hi, in_lo, in_hi, s_lo, s_hi;
};
template <int M>
__device__ __forceinline__ Span join(const Span& a, const Span& b) {
  Span c{min(a.lo, b.lo), max(a.hi, b.hi), max(a.in_lo, b.in_lo), min(a.in_hi, b.in_hi), 0, 0};
  if constexpr (M == kWindow) {
    c.s_lo = min(a.s_lo, b.s_lo);
    c.s_hi = max(a.s_hi, b.s_hi);
  }
  return c;
}
template <int M>
__device__ __forceinline__ Span row_span(const AttendParams& p, int row_lo, int rows, int first,
                                         int step) {
  Span a{p.c.cap, 0, 0, p.c.cap, p.c.cap, 0};
  for (int r = first; r < rows; r += step) {
    int s, e;
    row_range(p, row_lo + r, s, e);
    Span b{s, e, s, e, p.c.cap, 0};
    if constexpr (M == kTree) {
      const Drafts d = drafts(p, row_lo + r, e);
      if (s >= e) b.lo = d.lo < 0 ? p.c.cap : d.lo;
      if (s >= e && d.lo < 0) continue;
      if (d.hi >= 0) b.hi = d.hi + 1;
    } else {
      if (s >= e) continue;
    }
    if constexpr (M == kWindow) {
      b.lo = b.in_lo = window_start(p, s, e);
      if (p.sinks > 0 && s < b.lo) {
        b.s_lo = s;
        b.s_hi = sinks_end(p, s, e);
      }
    }
    a = join<M>(a, b);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    Span b{__shfl_xor(a.lo, o, 64), __shfl_xor(a.hi, o, 64), __shfl_xor(a.in_lo, o, 64),
           __shfl_xor(a.in_hi, o, 64), 0, 0};
    if constexpr (M == kWindow) {
      b.s_lo = __shfl_xor(a.s_lo, o, 64);
      b.s_hi = __shfl_xor(a.s_hi, o, 64);
    }
    a = join<M>(a, b);
  }
  return a;
}
__device__ __forceinline__ Span uniform(Span a) {
  return {__builtin_amdgcn_readfirstlane(a.lo),    __builtin_amdgcn_readfirstlane(a.hi),
          __builtin_amdgcn_readfirstlane(a.in_lo), __builtin_amdgcn_readfirstlane(a.in_hi),
          __builtin_amdgcn_readfirstlane(a.s_lo),  __builtin_amdgcn_readfirstlane(a.s_hi)};
}

// The keys that a tile of columns walks over, STEP at a time from a multiple of 16:
// its span, and before it the sinks' (kWindow), where they do not meet. A window costs its
// tile the keys that some of its rows see, masked steps at both ends among them, and a
// step for the sinks: 4096 rows of 32 heads on 4 key heads, 4095 + 5 positions each, 311
// to 319 us, up to 0.88 PFLOP/s. (When it took 322, 253 of them went by the keys, at 1.09
// PFLOP/s as in chunks, 57 were starts, ends and masked steps of two rounds, 12 the
// sinks'.) Trees: 16 x 64 drafts of 32 heads on 8 key heads behind 32768 positions 655 to
// 680 us, up to 0.84 PFLOP/s, of which the join of split keys takes 21.
template <int M, int STEP>
struct Walk {
  Span span;
  int first, steps;     // of all steps, where there are no sinks
  int s_first, s_steps; // the sinks' steps come first
  __device__ __forceinline__ explicit Walk(const Span& of) : span(of) {
    s_first = s_steps = 0;
    if constexpr (M == kWindow) {
      if (span.s_hi > span.s_lo) {
        span.s_lo = min(span.s_lo, span.lo);  // (a short row's window, before others' sinks)
        s_first = span.s_lo & ~15;
        s_steps = (span.s_hi - s_first + STEP - 1) / STEP;
        // what windows see of the sinks' steps is walked over there
        const int end = s_first + s_steps * STEP;
        if (span.lo < end) {
          span.s_hi = max(span.s_hi, min(span.hi, end));
          span.lo = end;
        }
      } else {
        span.s_lo = span.s_hi = 0;
      }
    }
    first = span.lo & ~15;
    steps = s_steps + (span.hi > span.lo ? (span.hi - first + STEP - 1) / STEP : 0);
  }
  // Position of step st's first key.
  __device__ __forceinline__ int pos(int st) const {
    if constexpr (M == kWindow)
      return st < s_steps ? s_first + st * STEP : first + (st - s_steps) * STEP;
    else
      return first + st * STEP;
  }
  // Where the 16 keys from `at` keys into step st are read: those behind what some row
  // sees, or before it, from the nearest that some row sees; what lies between the sinks
  // and the windows (kWindow), as it is.
  __device__ __forceinline__ int read_pos(int st, int at) const {
    if constexpr (M == kWindow)
      return min(pos(st) + at, max(span.hi, span.s_hi) - 1) & ~15;
    else
      return min(max(pos(st) + at, span.lo), span.hi - 1) & ~15;
  }
  __device__ __forceinline__ bool inside(int at) const {  // every row sees keys at .. at + STEP - 1
    return at >= span.in_lo && at + STEP <= span.in_hi;
  }
  // Position `at` is in what some rows see (kWindow: is not asked, as its values have no
  // weight and are not NaN).
  __device__ __forceinline__ bool some(int at) const {
    return M == kWindow || (at >= span.lo && at < span.hi);
  }
  __device__ __forceinline__ uint32_t some_bits(int at) const {
    return M == kWindow ? ~0u : seen_bits(at, span.lo, span.hi);
  }
};

// The end of a workgroup whose waves hold O^T sums in v_mfma_f32_16x16x32's
// layout: wave kb * HW + hw has 16 NT columns from 16 NT hw, over part kb of the
// keys; lane (g, n) holds element d of column n's output in acc[t][u][i], d =
// 16 u + 4 g + i (INLINE) or D / 16 * (4 g + i) + u. The KW waves of a column are brought to one reference
// point and added, US products a round, through LDS; then the rows are written,
// or the parts when the keys are split over workgroups.
template <int D, int NT, int HW, int KW>
struct Finish {
  static constexpr int U = D / 16, COLS = 16 * NT * HW;
  static constexpr int US = U < 8 / NT ? U : 8 / NT;
  float part[KW][US * 16][COLS];
  float m[KW][COLS], l[KW][COLS];
};

template <int T, bool INLINE, int D, int NT, int HW, int KW>
__device__ __forceinline__ void finish(const AttendParams& p, Finish<D, NT, HW, KW>& sh,
                                       int64_t block, int first_row, int columns, int tile, int h,
                                       int wave, const float (&m)[NT], const float (&l_in)[NT],
                                       const v4f (&acc)[NT][D / 16]) {
  using F = Finish<D, NT, HW, KW>;
  constexpr int U = F::U, US = F::US, COLS = F::COLS;
  const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
  const int hw = wave % HW, kb = wave / HW;
  float part[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float l = l_in[t];
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (g == 0) {
      sh.m[kb][16 * (NT * hw + t) + n] = m[t];
      sh.l[kb][16 * (NT * hw + t) + n] = l;
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float top = kLowest;
#pragma unroll
    for (int w = 0; w < KW; ++w) top = __builtin_fmaxf(top, sh.m[w][16 * (NT * hw + t) + n]);
    part[t] = __builtin_amdgcn_exp2f(m[t] - top) * (1.f / kUp);
  }
  const int col = threadIdx.x % COLS, at_col = tile * COLS + col;  // what this thread writes
  const bool real = at_col < columns;
  const int row = first_row + (real ? at_col / p.group : 0);
  const int head = h * p.group + (real ? at_col % p.group : 0);
  float top = kLowest, sum = 0.f;
#pragma unroll
  for (int w = 0; w < KW; ++w) top = __builtin_fmaxf(top, sh.m[w][col]);
#pragma unroll
  for (int w = 0; w < KW; ++w)
    sum += sh.l[w][col] * __builtin_amdgcn_exp2f(sh.m[w][col] - top);
  const bool direct = p.splits == 1;
  const float inv = 1.f / sum;
  const int64_t slot = block * COLS + col;
  if (threadIdx.x < COLS) {
    if (!direct) {
      p.part_ml[2 * slot] = top;
      p.part_ml[2 * slot + 1] = sum;
    } else if (real && p.lse) {
      p.lse[(int64_t)row * p.heads + head] =
          sum == 0.f ? -__builtin_inff() : (top - kBias) * kLn2 + __builtin_logf(sum);
    }
  }
  uint16_t* const out = static_cast<uint16_t*>(p.out) + ((int64_t)row * p.heads + head) * D;
#pragma unroll
  for (int u0 = 0; u0 < U; u0 += US) {
    if (u0) __syncthreads();
#pragma unroll
    for (int u = 0; u < US; ++u)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sh.part[kb][u * 16 + 4 * g + i][16 * (NT * hw + t) + n] = acc[t][u0 + u][i] * part[t];
    __syncthreads();
    for (int r = threadIdx.x / COLS; r < 16; r += (int)blockDim.x / COLS) {
      float v[US];
#pragma unroll
      for (int u = 0; u < US; ++u) {
        v[u] = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) v[u] += sh.part[w][INLINE ? US * r + u : u * 16 + r][col];
      }
      const int d = INLINE ? 16 * u0 + US * r : U * r + u0;
      if (!real) continue;
      if (!direct) {
        float* const o = p.part_o + slot * D + d;
#pragma unroll
        for (int u = 0; u < US; u += 2)
          *reinterpret_cast<float2*>(o + u) = float2{v[u], v[u + 1]};
      } else {
#pragma unroll
        for (int u = 0; u < US; u += 2) {
          const float x = sum == 0.f ? 0.f : v[u] * inv, y = sum == 0.f ? 0.f : v[u + 1] * inv;
          *reinterpret_cast<uint32_t*>(out + d + u) = to_type(x, T) | (uint32_t)to_type(y, T) << 16;
        }
      }
    }
  }
}

// f(type of q, codes, head_dim) as compile-time values.
template <class F>
void dispatch(const AttendParams& p, F f) {
  auto with = [&](auto t, auto c) {
    if (p.c.head_dim == 64)
      f(t, c, std::integral_constant<int, 64>{});
    else
      f(t, c, std::integral_constant<int, 128>{});
  };
  auto of = [&](auto t) {
    if (p.c.codes == kE4m3)
      with(t, std::integral_constant<int, kE4m3>{});
    else
      with(t, std::integral_constant<int, kInt8>{});
  };
  if (p.dtype == kBf16)
    of(std::integral_constant<int, kBf16>{});
  else
    of(std::integral_constant<int, kFp16>{});
}

// One launch of p.block0 .. each: tiles of up to 64 columns, lists, and tiles of 128
// or 256 columns.
template <int M>
void attend_narrow(const AttendParams& p, dim3 grid, hipStream_t s);
void attend_list(const AttendParams& p, dim3 grid, hipStream_t s);
template <int M>
void attend_wide(const AttendParams& p, dim3 grid, hipStream_t s);

}  // namespace mqa
