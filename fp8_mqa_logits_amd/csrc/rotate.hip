// RMS norm of query and key heads and the rotation of their positions in one pass.
//
//     y = w x / sqrt(mean x^2 + eps),  a_i = position * inv_freq_i
//     (y_p, y_s) -> (y_p cos a_i - y_s sin a_i, y_s cos a_i + y_p sin a_i)
//
// Angles. position * inv_freq is formed in 64 bits and, in turns, reduced to [-1/2, 1/2]
// there, so that far positions lose nothing; the sine and cosine of what is left are
// taken in fp32 by the unit that takes turns: within 2^-20 (1.3e-7 at most where it
// was measured), below a hundredth of a last place of a 16-bit result.
//
// A wave takes EACH times 64 / (D / 8) heads, of the queries or of the keys, of one
// row, eight elements a lane, so that a row's angles are formed once for all of them.
// The other element of a pair i, i + rot / 2 comes from another lane as it was read
// (four words, and normed again there, instead of eight sums).
//
// Bound by the bytes of long inputs: 16384 rows of 32 + 8 heads of 128 take 69 to 74 us,
// 4.5 to 4.9 TB/s read and written, where a large copy reaches 4.7 to 5.2.
#include <type_traits>

#include "attend.h"
#include "launch.h"
#include "mqa_serve.h"

namespace mqa {
namespace {

struct Heads {
  const uint16_t* x;
  uint16_t* y;
  const void* weight;
  int64_t x_row, x_head, y_row, y_head;
  int heads, waves;  // waves a row
};
struct RotateParams {
  Heads of[2];  // queries, keys
  const int32_t* positions;
  const float* inv_freq;
  int rot, rows, dtype, weight_fp32, norm, pairs;
  float eps;
  uint32_t wave0;
};

template <int T>
__device__ __forceinline__ void widen2(uint32_t w, float* x) {
  if constexpr (T == kBf16) {
    x[0] = __uint_as_float(w << 16);
    x[1] = __uint_as_float(w & 0xFFFF0000u);
  } else {
    x[0] = (float)__builtin_bit_cast(_Float16, (uint16_t)w);
    x[1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16));
  }
}
template <int T>
__device__ __forceinline__ void widen8(uint4 w, float* x) {
  widen2<T>(w.x, x);
  widen2<T>(w.y, x + 2);
  widen2<T>(w.z, x + 4);
  widen2<T>(w.w, x + 6);
}
template <int T>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  if constexpr (T == kBf16)
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)a) |
           (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)b) << 16;
  else
    return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)a) |
           (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)b) << 16;
}

// Eight weights from element `at`.
template <int T>
__device__ __forceinline__ void weights8(const RotateParams& p, const void* weight, int at, float* w) {
  if (!weight) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f;
  } else if (p.weight_fp32) {
    const float4* const f = reinterpret_cast<const float4*>(static_cast<const float*>(weight) + at);
    const float4 a = f[0], b = f[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  } else {
    widen8<T>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(weight) + at), w);
  }
}

// Sine and cosine of position * f.
__device__ __forceinline__ void turn(int position, float f, float& s, float& c) {
  double turns = (double)position * (double)f * 0.15915494309189533577;  // 1 / (2 pi)
  turns -= __builtin_rint(turns);
  s = __builtin_amdgcn_sinf((float)turns);
  c = __builtin_amdgcn_cosf((float)turns);
}

template <int T, int D, bool PAIRS, int EACH>
__global__ __launch_bounds__(256) void norm_rotate_kernel(RotateParams p) {
  constexpr int LANES = D / 8, AT_ONCE = 64 / LANES;  // lanes of a head, heads of a wave
  const int lane = threadIdx.x & 63, li = lane % LANES;
  const uint32_t wave = p.wave0 + blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t per_row = p.of[0].waves + p.of[1].waves;
  const int row = (int)(wave / per_row);
  int part = (int)(wave % per_row);
  if (row >= p.rows) return;
  const bool keys = part >= p.of[0].waves;
  const Heads& of = p.of[keys];
  if (keys) part -= p.of[0].waves;

  const int head0 = part * EACH * AT_ONCE + lane / LANES;
  uint4 in[EACH];
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int head = head0 + e * AT_ONCE;
    in[e] = uint4{0, 0, 0, 0};
    if (head < of.heads)
      in[e] = *reinterpret_cast<const uint4*>(of.x + row * of.x_row + head * of.x_head + 8 * li);
  }

  // this lane's part of the rotation: elements 8 li .. + 7 and, unless pairs are
  // neighbours, those of lane `other`
  const int half = p.rot / 16;  // lanes of half of what is rotated
  const bool turns = li < 2 * half;
  const int other = lane - li + (li < half ? li + half : turns ? li - half : li);
  float c[PAIRS ? 4 : 8], s[PAIRS ? 4 : 8];
  if (p.rot > 0) {
    const int position = p.positions[row];
    const int first = !turns ? 0 : PAIRS ? 4 * li : 8 * (li < half ? li : li - half);
#pragma unroll
    for (int j = 0; j < (PAIRS ? 4 : 8); ++j) {
      turn(position, p.inv_freq[first + j], s[j], c[j]);
      if (!PAIRS && li < half) s[j] = -s[j];
    }
  }
  float w[8], w_other[8];
  weights8<T>(p, of.weight, 8 * li, w);
  if (!PAIRS) weights8<T>(p, of.weight, 8 * (other % LANES), w_other);

#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    float x[8], inv = 1.f;
    widen8<T>(in[e], x);
    if (p.norm) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(x[j], x[j], sum);
#pragma unroll
      for (int o = 1; o < LANES; o <<= 1) sum += __shfl_xor(sum, o, 64);
      inv = __builtin_amdgcn_rsqf(__builtin_fmaf(sum, 1.f / D, p.eps));
    }
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = x[j] * inv * w[j];
    if (p.rot > 0) {
      if constexpr (PAIRS) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a = y[2 * j], b = y[2 * j + 1];
          if (turns) {
            y[2 * j] = a * c[j] - b * s[j];
            y[2 * j + 1] = b * c[j] + a * s[j];
          }
        }
      } else {
        uint4 q;
        q.x = __shfl((int)in[e].x, other, 64);
        q.y = __shfl((int)in[e].y, other, 64);
        q.z = __shfl((int)in[e].z, other, 64);
        q.w = __shfl((int)in[e].w, other, 64);
        float z[8];
        widen8<T>(q, z);
        if (turns) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = y[j] * c[j] + z[j] * inv * w_other[j] * s[j];
        }
      }
    }
    const int head = head0 + e * AT_ONCE;
    if (head < of.heads) {
      uint4 out;
      out.x = narrow2<T>(y[0], y[1]);
      out.y = narrow2<T>(y[2], y[3]);
      out.z = narrow2<T>(y[4], y[5]);
      out.w = narrow2<T>(y[6], y[7]);
      *reinterpret_cast<uint4*>(of.y + row * of.y_row + head * of.y_head + 8 * li) = out;
    }
  }
}

// A launch's grid stays below 2^32 threads: more waves (at most 2^20 rows of 256) go in
// several.
template <int T, int D, bool PAIRS, int EACH>
void launch(RotateParams p, hipStream_t s) {
  constexpr int kAtOnce = 64 / (D / 8) * EACH;
  for (Heads& of : p.of) of.waves = (of.heads + kAtOnce - 1) / kAtOnce;
  const uint32_t waves = (uint32_t)p.rows * (p.of[0].waves + p.of[1].waves);
  constexpr uint32_t kMost = 1u << 24;
  for (p.wave0 = 0; p.wave0 < waves; p.wave0 += kMost) {
    const uint32_t n = waves - p.wave0 < kMost ? waves - p.wave0 : kMost;
    norm_rotate_kernel<T, D, PAIRS, EACH><<<dim3((n + 3) / 4), 256, 0, s>>>(p);
  }
}

// f(type, head_dim, pairs) as compile-time values.
template <class F>
void dispatch(const RotateParams& p, int head_dim, F f) {
  auto with = [&](auto t, auto d) {
    if (p.pairs)
      f(t, d, std::true_type{});
    else
      f(t, d, std::false_type{});
  };
  auto of = [&](auto t) {
    if (head_dim == 64) with(t, std::integral_constant<int, 64>{});
    if (head_dim == 128) with(t, std::integral_constant<int, 128>{});
    if (head_dim == 256) with(t, std::integral_constant<int, 256>{});
  };
  if (p.dtype == kBf16)
    of(std::integral_constant<int, kBf16>{});
  else
    of(std::integral_constant<int, kFp16>{});
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool aligned(const mqa_head_rows* x) {
  return aligned(x->data, 16) && x->row_stride % 8 == 0 && x->head_stride % 8 == 0;
}
bool strides_ok(const mqa_head_rows* x, const mqa_head_rows* y, int rows, int heads) {
  return x->row_stride >= 0 && x->head_stride >= 0 && y->row_stride >= (rows > 1) &&
         y->head_stride >= (heads > 1);
}

}  // namespace
}  // namespace mqa

extern "C" int mqa_norm_rotate(const mqa_head_rows* q, const mqa_head_rows* q_out, int heads,
                               const mqa_head_rows* k, const mqa_head_rows* k_out, int kv_heads,
                               const void* q_weight, const void* k_weight, int weight_dtype,
                               const int32_t* positions, const float* inv_freq, int rot, int pairs,
                               int rows, int head_dim, int dtype, int norm, float eps,
                               void* stream) {
  using namespace mqa;
  const bool keys = kv_heads != 0;
  if (!q || !q_out || !q->data || !q_out->data ||
      (keys && (!k || !k_out || !k->data || !k_out->data)) ||
      (rot != 0 && (!positions || !inv_freq)))
    return MQA_ERR_NULL;
  if (!aligned(q) || !aligned(q_out) || (keys && (!aligned(k) || !aligned(k_out))) ||
      !aligned(q_weight, 16) || (keys && !aligned(k_weight, 16)) ||
      (rot != 0 && (!aligned(positions, 4) || !aligned(inv_freq, 16))))
    return MQA_ERR_ALIGN;
  if (rows < 1 || rows > MQA_MAX_ROWS || heads < 1 || heads > MQA_MAX_ATTEND_HEADS ||
      kv_heads < 0 || kv_heads > MQA_MAX_ATTEND_HEADS ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      (dtype != MQA_BF16 && dtype != MQA_FP16) ||
      (weight_dtype != dtype && weight_dtype != MQA_FP32) || rot < 0 || rot > head_dim ||
      rot % 16 != 0 || !(eps >= 0.f) || eps > 3.4e38f || !strides_ok(q, q_out, rows, heads) ||
      (keys && !strides_ok(k, k_out, rows, kv_heads)))
    return MQA_ERR_SHAPE;
  if (!current_device_cus()) return MQA_ERR_DEVICE;
  RotateParams p{};
  auto set = [](Heads& of, const mqa_head_rows* x, const mqa_head_rows* y, const void* weight,
                int n) {
    of.x = static_cast<const uint16_t*>(x->data);
    of.y = static_cast<uint16_t*>(y->data);
    of.weight = weight;
    of.x_row = x->row_stride;
    of.x_head = x->head_stride;
    of.y_row = y->row_stride;
    of.y_head = y->head_stride;
    of.heads = n;
  };
  set(p.of[0], q, q_out, norm ? q_weight : nullptr, heads);
  if (keys) set(p.of[1], k, k_out, norm ? k_weight : nullptr, kv_heads);
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.rot = rot;
  p.rows = rows;
  p.dtype = dtype;
  p.weight_fp32 = weight_dtype == MQA_FP32;
  p.norm = norm != 0;
  p.pairs = pairs != 0;
  p.eps = eps;
  hipStream_t s = static_cast<hipStream_t>(stream);
  dispatch(p, head_dim, [&](auto t, auto d, auto pr) {
    // Few rows: a wave for every four (D = 128) heads, for a short chain; many: four times
    // as many heads, for angles formed once. 32 + 8 heads of 128: 256 rows 4.8 us on the
    // first, 5.4 on the second, 512 6.0 and 6.1, 1024 8.5 and 7.7, 16384 94 and 74.
    if ((int64_t)rows * (heads + kv_heads) * head_dim < (int64_t)1 << 21)
      launch<t.value, d.value, pr.value, 1>(p, s);
    else
      launch<t.value, d.value, pr.value, 4>(p, s);
  });
  const int rc = (int)hipGetLastError();
  return rc != 0 ? launch_failed(rc) : MQA_OK;
}
