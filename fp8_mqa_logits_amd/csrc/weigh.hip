// Attention weight that positions of the cache receive, summed over the query heads of
// a request's rows:
//     W_j += sum_{r, h} exp(S_rhj - lse_rh),  S as in attend_tiles.h
// The first of attention's two products and its exponentials, with the sums along the
// other axis: a lane's scores of one column (row and head) are added to those of its
// other columns, keys staying where they are, and lanes are joined once at the end. A
// position's sums are formed by one workgroup in a fixed order: the same bits every time.
//
// Numbers. S' = S log2 e and lse' = lse log2 e go into one fp32 exponent; lse' is off
// by up to half a last place, 2^-20 for lse' in [8, 16), and what it lacks is put
// back as a factor, 2^-(what it lacks), by which the exponential enters its sum.
#include "attend_tiles.h"
#include "serve.h"

namespace mqa {
namespace {

constexpr float kLog2eLow = 1.9259629911266175e-8f;  // log2 e - kLog2e

// Few columns: a wave takes 32 keys of every HW-th key head, widened once for all
// column tiles of 16; HW waves that share keys are joined through LDS.
template <int T, int C, int D>
__global__ __launch_bounds__(256, 4) void weigh_narrow_kernel(WeighParams p) {
  constexpr int KC = D / 64;  // 16-byte pieces of a key per lane
  const AttendParams& a = p.a;
  const KvCache& c = a.c;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, n = lane & 15;
  const int unit = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles;
  const int columns = a.R * a.group;
  const int HW = c.kv_heads >= 4 ? 4 : c.kv_heads >= 2 ? 2 : 1, KW = 4 / HW;
  const int hw = wave % HW, kb = wave / HW;
  __shared__ float s_part[4][32];

  const Span span = uniform(row_span<kRange>(a, unit * a.R, a.R, lane, 64));
  const int first = span.lo & ~15;
  const float cs = a.scale * kLog2e;
  const int32_t* const table = c.table + (int64_t)unit * c.table_stride;

  for (int at = first + tile * KW * 32; at < span.hi; at += p.tiles * KW * 32) {
    const int pos0 = at + kb * 32;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    if (pos0 < span.hi) {
      const uint8_t* page[2];
      int slot[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int pos = min(pos0 + 16 * b, (span.hi - 1) & ~15);
        page[b] = c.pages + (int64_t)clamp_page(c, table[pos >> c.page_shift]) * c.page_stride;
        slot[b] = pos & ((1 << c.page_shift) - 1);
      }
      const bool clean = pos0 >= span.in_lo && pos0 + 32 <= span.in_hi;
      for (int h = hw; h < c.kv_heads; h += HW) {
        v4u kf[2][2 * KC];
        float f[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint8_t* const k = page[b] + code_at(c, 0, h, slot[b]) + n * D + 16 * g;
#pragma unroll
          for (int x = 0; x < KC; ++x) {
            const v4u raw = *reinterpret_cast<const v4u*>(k + 64 * x);
            kf[b][2 * x] = widen8<T, C>(raw[0], raw[1]);
            kf[b][2 * x + 1] = widen8<T, C>(raw[2], raw[3]);
          }
          f[b] = *reinterpret_cast<const float*>(page[b] + scale_at(c, 0, h, slot[b])) * cs;
        }
        for (int col0 = 0; col0 < columns; col0 += 16) {
          const int col = col0 + n;
          const bool real = col < columns;
          const int row = unit * a.R + (real ? col / a.group : 0);
          const int head = h * a.group + (real ? col % a.group : 0);
          const uint16_t* src =
              static_cast<const uint16_t*>(a.q) + row * a.q_row + head * a.q_head;
          v4u q[2 * KC];
#pragma unroll
          for (int k = 0; k < 2 * KC; ++k)
            q[k] = *reinterpret_cast<const v4u*>(src + 64 * (k >> 1) + 16 * g + 8 * (k & 1));
          const float lse = p.lse[(int64_t)row * a.heads + head];
          const float to = lse * kLog2e;
          // exp(-lse) = 2^-to * by
          float by = __builtin_amdgcn_exp2f(
              -(__builtin_fmaf(lse, kLog2e, -to) + lse * kLog2eLow));
          if (!(__builtin_fabsf(to) < 3e38f)) by = 1.f;
          int s, e;
          row_range(a, row, s, e);
          uint32_t sees = real && lse != -__builtin_inff() ? ~0u : 0u;
          if (!clean) sees &= seen_bits(pos0, s, e);
          sees >>= 4 * g;
          if (s >= e) sees = 0;
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            v4f x = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 2 * KC; ++k) x = mfma<T>(kf[b][k], q[k], x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], f[b], -to)) * by;
              acc[4 * b + i] += or_zero(w, bit(sees, 16 * b + i));
            }
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) acc[j] += __shfl_xor(acc[j], o, 64);
      if (n == 0) s_part[wave][16 * (j >> 2) + 4 * g + (j & 3)] = acc[j];
    }
    __syncthreads();
    if ((int)threadIdx.x < 32 * KW) {
      const int k = threadIdx.x / 32, pos = at + threadIdx.x;
      float sum = 0.f;
      for (int w = 0; w < HW; ++w) sum += s_part[k * HW + w][threadIdx.x % 32];
      if (pos >= span.lo && pos < span.hi && pos < p.width)
        p.weights[(int64_t)unit * p.width + pos] += sum;
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace mqa

extern "C" int mqa_kv_weigh_launch(const mqa::WeighParams* p, hipStream_t s) {
  using namespace mqa;
  const dim3 grid((unsigned)p->a.requests * p->tiles);
  dispatch(p->a, [&](auto t, auto c, auto d) {
    weigh_narrow_kernel<t.value, c.value, d.value><<<grid, 256, 0, s>>>(*p);
  });
  return (int)hipGetLastError();
}
