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

// The positions that some of `rows` rows from row_lo see, [lo, hi), and those
// that all of them see, [in_lo, in_hi); rows that see nothing are left out. A
// lane takes every step-th row from `first`; the result is the wave's.
struct Span {
  int lo, hi, in_lo, in_hi;
};
__device__ __forceinline__ Span row_span(const AttendParams& p, int row_lo, int rows, int first,
                                         int step) {
  Span a{p.c.cap, 0, 0, p.c.cap};
  for (int r = first; r < rows; r += step) {
    int s, e;
    row_range(p, row_lo + r, s, e);
    if (s < e) a = {min(a.lo, s), max(a.hi, e), max(a.in_lo, s), min(a.in_hi, e)};
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    a.lo = min(a.lo, __shfl_xor(a.lo, o, 64));
    a.hi = max(a.hi, __shfl_xor(a.hi, o, 64));
    a.in_lo = max(a.in_lo, __shfl_xor(a.in_lo, o, 64));
    a.in_hi = min(a.in_hi, __shfl_xor(a.in_hi, o, 64));
  }
  return a;
}
__device__ __forceinline__ Span uniform(Span a) {
  return {__builtin_amdgcn_readfirstlane(a.lo), __builtin_amdgcn_readfirstlane(a.hi),
          __builtin_amdgcn_readfirstlane(a.in_lo), __builtin_amdgcn_readfirstlane(a.in_hi)};
}

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

// One launch of p.block0 .. each (attend_narrow.hip, attend_list.hip,
// attend_wide.hip).
void attend_narrow(const AttendParams& p, dim3 grid, hipStream_t s);
void attend_list(const AttendParams& p, dim3 grid, hipStream_t s);
void attend_wide(const AttendParams& p, dim3 grid, hipStream_t s);

}  // namespace mqa
