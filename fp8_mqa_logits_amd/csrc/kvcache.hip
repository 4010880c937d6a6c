// Storing tokens into the paged 8-bit key/value cache and reading them back.
//
// Codes under power-of-two scales. For a block of B tokens and one head,
//     scale = smallest 2^e >= 2^-126 with amax <= M 2^e   (M: 448 or 127)
//     code  = round_to_nearest_even(x / scale)
// x / scale only moves x's exponent, so the one rounding is the code's own and
// the codes are the same on every path that follows the definition. The
// exponent comes from amax's bits: with amax = f 2^x, f in [1, 2), and M =
// m 2^t, m in [1, 2), e = x - t + (f > m).
#include "attend.h"
#include "launch.h"

namespace mqa {
namespace {

constexpr int kThreads = 256;

// 8 consecutive elements as fp32.
template <int T>
__device__ __forceinline__ void load8(const void* base, int64_t at, float* x) {
  if constexpr (T == kFp32) {
    const float4 a = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at)[0];
    const float4 b = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (T == kBf16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        x[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)w[i]);
        x[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] >> 16));
      }
    }
  }
}

template <int T>
__device__ __forceinline__ void store8(void* base, int64_t at, const float* x) {
  if constexpr (T == kFp32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    o[0] = float4{x[0], x[1], x[2], x[3]};
    o[1] = float4{x[4], x[5], x[6], x[7]};
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (T == kBf16) {
        w[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i]) |
               (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i + 1]) << 16;
      } else {
        w[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x[2 * i]) |
               (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x[2 * i + 1]) << 16;
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = uint4{w[0], w[1], w[2], w[3]};
  }
}

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

// One workgroup per (block that new tokens fall into, head, keys or values):
// its new tokens are read twice, the second time from the cache that the first
// read filled (a block of 64 x 128 bf16 is 16 KiB); kept tokens only where the
// scale grows.
template <int T, int C>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvMoveParams p, int blocks) {
  const KvCache& c = p.c;
  const int request = blockIdx.x / blocks, h = blockIdx.y, w = blockIdx.z;
  const int B = 1 << c.block_shift;
  int count = p.counts ? p.counts[request] : p.R;
  count = count < 0 ? 0 : (count > p.R ? p.R : count);
  // tokens lo <= t < hi of the request fall into this block and the table
  const int64_t first = p.starts[request];
  const int64_t begin = (first & ~(int64_t)(B - 1)) + (int64_t)(blockIdx.x % blocks) * B;
  int64_t lo = begin > first ? begin : first;
  int64_t hi = begin + B < first + count ? begin + B : first + count;
  if (begin < 0 || begin >= c.cap || lo >= hi) return;
  const int page = page_of(c, request, (int)begin);
  if (page < 0) return;
  uint8_t* const base = c.pages + (int64_t)page * c.page_stride;
  const int slot0 = (int)begin & ((1 << c.page_shift) - 1);
  const void* src = w ? p.v : p.k;
  const int64_t row_stride = w ? p.v_row : p.k_row, head_stride = w ? p.v_head : p.k_head;
  const int per = c.head_dim / 8;  // 8-element pieces of a token
  const int n = (int)(hi - lo) * per;
  const int64_t row0 = (int64_t)request * p.R + (lo - first);

  float amax = 0.f;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    float x[8];
    load8<T>(src, (row0 + i / per) * row_stride + h * head_stride + i % per * 8, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = __builtin_fabsf(x[j]);
      if (a < __builtin_inff()) amax = __builtin_fmaxf(amax, a);
    }
  }
  __shared__ float part[kThreads / 64];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) amax = __builtin_fmaxf(amax, __shfl_xor(amax, o, 64));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = amax;
  float* const scale_p = reinterpret_cast<float*>(base + scale_at(c, w, h, slot0));
  const bool keeps = lo > begin;
  const float was = keeps ? *scale_p : 0.f;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) amax = __builtin_fmaxf(amax, part[i]);
  const float fresh = __builtin_ldexpf(1.f, scale_exponent<C>(amax));
  const float scale = fresh > was ? fresh : was;
  const float inv = 1.f / scale;  // a power of two unless the kept scale is none

  for (int i = threadIdx.x; i < n; i += kThreads) {
    float x[8];
    load8<T>(src, (row0 + i / per) * row_stride + h * head_stride + i % per * 8, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= inv;
    const int slot = slot0 + (int)(lo - begin) + i / per;
    *reinterpret_cast<uint2*>(base + code_at(c, w, h, slot) + i % per * 8) = encode8<C>(x);
  }
  if (keeps && scale > was) {
    const float shrink = was * inv;
    for (int i = threadIdx.x; i < (int)(lo - begin) * per; i += kThreads) {
      uint2* const at = reinterpret_cast<uint2*>(base + code_at(c, w, h, slot0) + i * 8);
      float x[8];
      decode8<C>(*at, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= shrink;
      *at = encode8<C>(x);
    }
  }
  if (threadIdx.x == 0 && !(keeps && scale == was)) *scale_p = scale;
}

// A thread reads 8 codes and writes 8 values; consecutive threads go along a
// token, then to the next one of the same head (contiguous in its page).
template <int T, int C>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvMoveParams p) {
  const KvCache& c = p.c;
  const int per = c.head_dim / 8;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t row = i / per;
  if (row >= (int64_t)p.requests * p.R) return;
  const int request = (int)(row / p.R), t = (int)(row % p.R), h = blockIdx.y, w = blockIdx.z;
  const int count = p.counts ? p.counts[request] : p.R;
  const int64_t pos = (int64_t)p.starts[request] + t;
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (t < count && pos >= 0 && pos < c.cap) {
    const int page = page_of(c, request, (int)pos);
    if (page >= 0) {
      const uint8_t* base = c.pages + (int64_t)page * c.page_stride;
      const int slot = (int)pos & ((1 << c.page_shift) - 1);
      const float s = *reinterpret_cast<const float*>(base + scale_at(c, w, h, slot));
      decode8<C>(*reinterpret_cast<const uint2*>(base + code_at(c, w, h, slot) + i % per * 8), x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= s;
    }
  }
  store8<T>(w ? p.vo : p.ko, (row * c.kv_heads + h) * c.head_dim + i % per * 8, x);
}

template <int T, int C>
void append(const KvMoveParams& p, hipStream_t s) {
  const int B = 1 << p.c.block_shift;
  const int blocks = (B - 1 + p.R - 1) / B + 1;  // blocks R tokens can fall into
  kv_append_kernel<T, C><<<dim3(p.requests * blocks, p.c.kv_heads, 2), kThreads, 0, s>>>(p, blocks);
}

template <int T, int C>
void read(const KvMoveParams& p, hipStream_t s) {
  const int64_t n = (int64_t)p.requests * p.R * (p.c.head_dim / 8);
  kv_read_kernel<T, C><<<dim3((unsigned)((n + kThreads - 1) / kThreads), p.c.kv_heads, 2), kThreads,
                         0, s>>>(p);
}

}  // namespace
}  // namespace mqa

extern "C" int mqa_kv_append_launch(const mqa::KvMoveParams* p, hipStream_t s) {
  using namespace mqa;
  const bool e = p->c.codes == kE4m3;
  if (p->dtype == kBf16) e ? append<kBf16, kE4m3>(*p, s) : append<kBf16, kInt8>(*p, s);
  if (p->dtype == kFp16) e ? append<kFp16, kE4m3>(*p, s) : append<kFp16, kInt8>(*p, s);
  if (p->dtype == kFp32) e ? append<kFp32, kE4m3>(*p, s) : append<kFp32, kInt8>(*p, s);
  return (int)hipGetLastError();
}

extern "C" int mqa_kv_read_launch(const mqa::KvMoveParams* p, hipStream_t s) {
  using namespace mqa;
  const bool e = p->c.codes == kE4m3;
  if (p->dtype == kBf16) e ? read<kBf16, kE4m3>(*p, s) : read<kBf16, kInt8>(*p, s);
  if (p->dtype == kFp16) e ? read<kFp16, kE4m3>(*p, s) : read<kFp16, kInt8>(*p, s);
  if (p->dtype == kFp32) e ? read<kFp32, kE4m3>(*p, s) : read<kFp32, kInt8>(*p, s);
  return (int)hipGetLastError();
}
