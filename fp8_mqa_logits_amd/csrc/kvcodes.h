// Codes under power-of-two scales. For a block of B tokens and one head,
//     scale = smallest 2^e >= 2^-126 with amax <= M 2^e   (M: 448 or 127)
//     code  = round_to_nearest_even(x / scale)
// x / scale only moves x's exponent, so the one rounding is the code's own and
// the codes are the same on every path that follows the definition. The
// exponent comes from amax's bits: with amax = f 2^x, f in [1, 2), and M =
// m 2^t, m in [1, 2), e = x - t + (f > m).
#pragma once

#include "attend.h"

namespace mqa {

// 8 codes (two dwords) -> their values.
template <int C>
__device__ __forceinline__ void decode8(uint2 c, float* x) {
  if constexpr (C == kE4m3) {
    const int w[2] = {(int)c.x, (int)c.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i + 0] = __builtin_amdgcn_cvt_f32_fp8(w[i], 0);
      x[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8(w[i], 1);
      x[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8(w[i], 2);
      x[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8(w[i], 3);
    }
  } else {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)(int8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

// Values already divided by their scale -> 8 codes. The clamp only acts on
// infinities (and on kept codes whose scale a caller wrote himself). A NaN
// becomes 0x7F, whatever its sign (the conversion itself would write 0xFF).
template <int C>
__device__ __forceinline__ uint2 encode8(const float* x) {
  uint32_t w[2];
  if constexpr (C == kE4m3) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float y[4];
      uint32_t nan = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = x[4 * i + j];
        y[j] = __builtin_fminf(__builtin_fmaxf(v, -448.f), 448.f);
        nan |= v != v ? 0xFFu << (8 * j) : 0u;
      }
      int d = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
      w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], d, true);
      w[i] = (w[i] & ~nan) | (nan & 0x7F7F7F7Fu);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = x[4 * i + j];
        const float y =
            v != v ? 0.f : __builtin_rintf(__builtin_fminf(__builtin_fmaxf(v, -127.f), 127.f));
        w[i] |= ((uint32_t)(int)y & 0xFFu) << (8 * j);
      }
    }
  }
  return uint2{w[0], w[1]};
}

template <int C>
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  constexpr uint32_t m = C == kE4m3 ? 0x600000u : 0x7E0000u;  // mantissas of 1.75, 1.984375
  constexpr int t = C == kE4m3 ? 8 : 6;
  const int e = (int)(u >> 23) - 127 - t + ((u & 0x7FFFFFu) > m ? 1 : 0);
  return e < -126 ? -126 : e;
}

// Page of the position, or -1 where the table names none.
__device__ __forceinline__ int page_of(const KvCache& c, int request, int pos) {
  const int page = c.table[(int64_t)request * c.table_stride + (pos >> c.page_shift)];
  return page >= 0 && page < c.num_pages ? page : -1;
}

}  // namespace mqa
