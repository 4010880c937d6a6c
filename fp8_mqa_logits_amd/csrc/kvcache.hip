// Storing tokens into the paged 8-bit key/value cache and reading them back (codes and
// scales: kvcodes.h).
#include <type_traits>

#include "attend.h"
#include "kvcodes.h"
#include "launch.h"

namespace mqa {
namespace {

constexpr int kThreads = 256;

// 8 values -> consecutive elements, rounded to the type.
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

// 8 consecutive elements as they are stored.
template <int T>
struct Raw {
  uint4 x[T == kFp32 ? 2 : 1];
};
template <int T>
__device__ __forceinline__ Raw<T> load_raw(const void* base, int64_t at) {
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) +
                                                  at * (T == kFp32 ? 4 : 2));
  Raw<T> r;
  r.x[0] = p[0];
  if constexpr (T == kFp32) r.x[1] = p[1];
  return r;
}
template <int T>
__device__ __forceinline__ void widen(const Raw<T>& r, float* x) {
#pragma unroll
  for (int h = 0; h < (T == kFp32 ? 2 : 1); ++h) {
    const uint32_t w[4] = {r.x[h].x, r.x[h].y, r.x[h].z, r.x[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (T == kFp32) {
        x[4 * h + i] = __uint_as_float(w[i]);
      } else if constexpr (T == kBf16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        x[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)w[i]);
        x[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] >> 16));
      }
    }
  }
}

// One workgroup per (block that new tokens fall into, head, keys or values).
// HELD: its tokens stay in registers between the search for the largest and
// the rounding (blocks of up to kHold pieces of 8 elements a thread: 128 tokens
// of 128); larger blocks are read twice. Kept tokens are read only where the
// scale grows. Bound by the bytes of long inputs: 16384 tokens of 8 heads of 128
// in bf16 take 21.6 us, 4.7 TB/s in and out.
constexpr int kHold = 8;

template <int T, int C, int D, bool HELD>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvMoveParams p, int blocks) {
  constexpr int PER = D / 8;  // pieces of a token
  const KvCache& c = p.c;
  const int request = blockIdx.x / blocks, h = blockIdx.y, w = blockIdx.z;
  const int B = 1 << c.block_shift;
  int count = p.counts ? p.counts[request] : p.R;
  count = count < 0 ? 0 : (count > p.R ? p.R : count);
  // tokens lo <= t < hi of the request fall into this block and the table
  const int64_t first = p.starts[request];
  const int64_t begin = (first & ~(int64_t)(B - 1)) + (int64_t)(blockIdx.x % blocks) * B;
  const int64_t lo = begin > first ? begin : first;
  const int64_t hi = begin + B < first + count ? begin + B : first + count;
  if (begin < 0 || begin >= c.cap || lo >= hi) return;
  const int page = page_of(c, request, (int)begin);
  if (page < 0) return;
  uint8_t* const base = c.pages + (int64_t)page * c.page_stride;
  const int slot0 = (int)begin & ((1 << c.page_shift) - 1), kept = (int)(lo - begin);
  const void* src = w ? p.v : p.k;
  const int64_t row_stride = w ? p.v_row : p.k_row;
  const int64_t src0 = ((int64_t)request * p.R + (lo - first)) * row_stride +
                       h * (w ? p.v_head : p.k_head);
  const int n = (int)(hi - lo) * PER;
  auto piece = [&](int i) { return load_raw<T>(src, src0 + i / PER * row_stride + i % PER * 8); };
  float* const scale_p = reinterpret_cast<float*>(base + scale_at(c, w, h, slot0));
  const float was = kept ? *scale_p : 0.f;

  float amax = 0.f;
  auto look = [&](const Raw<T>& r) {
    float x[8];
    widen<T>(r, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = __builtin_fabsf(x[j]);
      amax = a < __builtin_inff() ? __builtin_fmaxf(amax, a) : amax;
    }
  };
  Raw<T> held[HELD ? kHold : 1];
  if constexpr (HELD) {
#pragma unroll
    for (int k = 0; k < kHold; ++k)
      if ((int)threadIdx.x + k * kThreads < n) held[k] = piece(threadIdx.x + k * kThreads);
#pragma unroll
    for (int k = 0; k < kHold; ++k)
      if ((int)threadIdx.x + k * kThreads < n) look(held[k]);
  } else {
    for (int i = threadIdx.x; i < n; i += kThreads) look(piece(i));
  }
  __shared__ float part[kThreads / 64];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) amax = __builtin_fmaxf(amax, __shfl_xor(amax, o, 64));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) amax = __builtin_fmaxf(amax, part[i]);
  const float fresh = __builtin_ldexpf(1.f, scale_exponent<C>(amax));
  const float scale = fresh > was ? fresh : was;
  const float inv = 1.f / scale;  // a power of two unless the kept scale is none

  uint8_t* const codes = base + code_at(c, w, h, slot0);
  auto put = [&](int i, const Raw<T>& r) {
    float x[8];
    widen<T>(r, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= inv;
    *reinterpret_cast<uint2*>(codes + kept * D + i * 8) = encode8<C>(x);
  };
  if constexpr (HELD) {
#pragma unroll
    for (int k = 0; k < kHold; ++k)
      if ((int)threadIdx.x + k * kThreads < n) put(threadIdx.x + k * kThreads, held[k]);
  } else {
    for (int i = threadIdx.x; i < n; i += kThreads) put(i, piece(i));
  }
  if (kept && scale > was) {
    const float shrink = was * inv;
    for (int i = threadIdx.x; i < kept * PER; i += kThreads) {
      uint2* const at = reinterpret_cast<uint2*>(codes + i * 8);
      float x[8];
      decode8<C>(*at, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= shrink;
      *at = encode8<C>(x);
    }
  }
  if (threadIdx.x == 0 && !(kept && scale == was)) *scale_p = scale;
}

// A thread reads kRows times 8 codes and writes as many values: consecutive
// threads go along a token, then to the next ones of the same head (contiguous
// in its page); its rows are kThreads / PER apart, each with its own chain of
// lookups under way (16384 tokens of 8 heads of 128 to bf16: 20.8 us, 4.8 TB/s;
// append and read together 54.6 us with one row a thread here and two looks at
// the tokens there, 47.6 us now).
constexpr int kRows = 4;

template <int T, int C, int D>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvMoveParams p) {
  constexpr int PER = D / 8;
  const KvCache& c = p.c;
  const int h = blockIdx.y, w = blockIdx.z, part = threadIdx.x % PER * 8;
  const int64_t rows = (int64_t)p.requests * p.R;
  const int64_t row0 = (int64_t)blockIdx.x * (kRows * kThreads / PER) + threadIdx.x / PER;
  uint2 code[kRows];
  float s[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t row = row0 + k * (kThreads / PER);
    code[k] = uint2{0, 0};
    s[k] = 0.f;
    if (row >= rows) continue;
    const int request = (int)(row / p.R), t = (int)(row % p.R);
    const int64_t pos = (int64_t)p.starts[request] + t;
    if (t >= (p.counts ? p.counts[request] : p.R) || pos < 0 || pos >= c.cap) continue;
    const int page = page_of(c, request, (int)pos);
    if (page < 0) continue;
    const uint8_t* base = c.pages + (int64_t)page * c.page_stride;
    const int slot = (int)pos & ((1 << c.page_shift) - 1);
    s[k] = *reinterpret_cast<const float*>(base + scale_at(c, w, h, slot));
    code[k] = *reinterpret_cast<const uint2*>(base + code_at(c, w, h, slot) + part);
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t row = row0 + k * (kThreads / PER);
    if (row >= rows) continue;
    float x[8];
    decode8<C>(code[k], x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= s[k];
    store8<T>(w ? p.vo : p.ko, (row * c.kv_heads + h) * D + part, x);
  }
}

template <int T, int C, int D>
void append(const KvMoveParams& p, hipStream_t s) {
  const int B = 1 << p.c.block_shift;
  const int blocks = (B - 1 + p.R - 1) / B + 1;  // blocks R tokens can fall into
  const dim3 grid(p.requests * blocks, p.c.kv_heads, 2);
  if ((B < p.R ? B : p.R) * (D / 8) <= kHold * kThreads)
    kv_append_kernel<T, C, D, true><<<grid, kThreads, 0, s>>>(p, blocks);
  else
    kv_append_kernel<T, C, D, false><<<grid, kThreads, 0, s>>>(p, blocks);
}

template <int T, int C, int D>
void read(const KvMoveParams& p, hipStream_t s) {
  const int64_t rows = (int64_t)p.requests * p.R, each = kRows * kThreads / (D / 8);
  kv_read_kernel<T, C, D><<<dim3((unsigned)((rows + each - 1) / each), p.c.kv_heads, 2), kThreads,
                            0, s>>>(p);
}

// f(type, codes, head_dim) as compile-time values.
template <class F>
void dispatch(const KvMoveParams& p, F f) {
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
  if (p.dtype == kBf16) of(std::integral_constant<int, kBf16>{});
  if (p.dtype == kFp16) of(std::integral_constant<int, kFp16>{});
  if (p.dtype == kFp32) of(std::integral_constant<int, kFp32>{});
}

}  // namespace
}  // namespace mqa

extern "C" int mqa_kv_append_launch(const mqa::KvMoveParams* p, hipStream_t s) {
  mqa::dispatch(*p, [&](auto t, auto c, auto d) { mqa::append<t.value, c.value, d.value>(*p, s); });
  return (int)hipGetLastError();
}

extern "C" int mqa_kv_read_launch(const mqa::KvMoveParams* p, hipStream_t s) {
  mqa::dispatch(*p, [&](auto t, auto c, auto d) { mqa::read<t.value, c.value, d.value>(*p, s); });
  return (int)hipGetLastError();
}
