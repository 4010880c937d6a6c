// Attention of query rows over a paged 8-bit key/value cache.
//
//     S_j = scale * ks_j * (q . kc_j)        (kc, vc: codes; ks, vs: block scales)
//     m = max_j S_j,  l = sum_j exp(S_j - m)
//     out = sum_j exp(S_j - m) * vs_j * vc_j / l,   lse = m + ln l
// over the positions j of the row's range, or over its listed positions.
#include "attend.h"
#include "launch.h"

namespace mqa {
namespace {

constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float element(const void* base, int64_t at, int type) {
  const uint16_t u = static_cast<const uint16_t*>(base)[at];
  return type == kBf16 ? __uint_as_float((uint32_t)u << 16) : (float)__builtin_bit_cast(_Float16, u);
}

__device__ __forceinline__ float code_value(uint32_t byte, int codes) {
  return codes == kE4m3 ? __builtin_amdgcn_cvt_f32_fp8((int)byte, 0) : (float)(int8_t)byte;
}

// One wave per (row, query head): a lane scores one of 64 positions at a time,
// then the wave adds the 64 value rows, a lane owning head_dim / 64 columns.
__global__ __launch_bounds__(64) void attend_wave_kernel(AttendParams p) {
  const KvCache& c = p.c;
  const int row = blockIdx.x, head = blockIdx.y, h = head / p.group;
  const int l = threadIdx.x, D = c.head_dim, request = row / p.R;
  __shared__ float q[128];
  __shared__ float prob[64];
  __shared__ int64_t vrow[64];
  for (int d = l; d < D; d += 64)
    q[d] = element(p.q, row * p.q_row + head * p.q_head + d, p.dtype);
  __syncthreads();
  int s = p.starts[row], e = p.ends[row];
  s = s < 0 ? 0 : (s > c.cap ? c.cap : s);
  e = e < s ? s : (e > c.cap ? c.cap : e);
  const int n = p.indices ? p.width : e - s;
  float m = -__builtin_inff(), sum = 0.f, acc[2] = {0.f, 0.f};
  for (int at = 0; at < n; at += 64) {
    bool seen = at + l < n;
    int x = at + l;
    if (p.indices && seen) {
      x = p.indices[(int64_t)row * p.width + at + l];
      seen = x >= 0 && x < e - s;
    }
    const int pos = seen ? s + x : s;
    float score = -__builtin_inff(), vs = 0.f;
    if (seen) {
      int page = c.table[(int64_t)request * c.table_stride + (pos >> c.page_shift)];
      page = page < 0 ? 0 : (page >= c.num_pages ? c.num_pages - 1 : page);
      const uint8_t* base = c.pages + (int64_t)page * c.page_stride;
      const int slot = pos & ((1 << c.page_shift) - 1);
      const uint8_t* k = base + code_at(c, 0, h, slot);
      float dot = 0.f;
      for (int d = 0; d < D; ++d) dot = __builtin_fmaf(q[d], code_value(k[d], c.codes), dot);
      score = dot * *reinterpret_cast<const float*>(base + scale_at(c, 0, h, slot)) *
              (p.scale * kLog2e);
      vs = *reinterpret_cast<const float*>(base + scale_at(c, 1, h, slot));
      vrow[l] = (int64_t)page * c.page_stride + code_at(c, 1, h, slot);
    }
    float top = score;
    for (int o = 32; o >= 1; o >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o, 64));
    top = __builtin_fmaxf(top, m);
    const float ref = top == -__builtin_inff() ? 0.f : top;
    const float keep = __builtin_amdgcn_exp2f(m - ref);
    const float pr = seen ? __builtin_amdgcn_exp2f(score - ref) : 0.f;
    float add = pr;
    for (int o = 32; o >= 1; o >>= 1) add += __shfl_xor(add, o, 64);
    sum = sum * keep + add;
    m = top;
    acc[0] *= keep;
    acc[1] *= keep;
    prob[l] = pr * vs;
    const uint64_t live = __ballot(seen);
    __syncthreads();
    for (int j = 0; j < 64; ++j) {
      if (!(live >> j & 1)) continue;
      for (int i = 0; i < D / 64; ++i)
        acc[i] = __builtin_fmaf(prob[j], code_value(c.pages[vrow[j] + l + 64 * i], c.codes), acc[i]);
    }
    __syncthreads();
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int i = 0; i < D / 64; ++i) {
    const int64_t o = ((int64_t)row * p.heads + head) * D + l + 64 * i;
    const float v = acc[i] * inv;
    static_cast<uint16_t*>(p.out)[o] = p.dtype == kBf16 ? __builtin_bit_cast(uint16_t, (__bf16)v)
                                                        : __builtin_bit_cast(uint16_t, (_Float16)v);
  }
  if (l == 0 && p.lse) p.lse[(int64_t)row * p.heads + head] = m * kLn2 + __builtin_logf(sum);
}

}  // namespace
}  // namespace mqa

extern "C" int mqa_attend_launch(const mqa::AttendParams* p, hipStream_t s) {
  mqa::attend_wave_kernel<<<dim3(p->rows, p->heads), 64, 0, s>>>(*p);
  return (int)hipGetLastError();
}
