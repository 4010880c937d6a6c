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

// exp(-lse) 2^to, to = lse log2 e as it was rounded (1 where that is none).
__device__ __forceinline__ float lacking(float lse, float to) {
  const float by =
      __builtin_amdgcn_exp2f(-(__builtin_fmaf(lse, kLog2e, -to) + lse * kLog2eLow));
  return __builtin_fabsf(to) < 3e38f ? by : 1.f;
}

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
          const float by = lacking(lse, to);
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

// Many columns: a wave holds 64 keys of one head, widened, in registers as the first
// operand of v_mfma_f32_32x32x16; 512 keys a workgroup. Queries pass through LDS, 64
// columns at a time, with what belongs to a column: lse', its factor, its range. So a
// staged query meets 512 keys, and a wave's only traffic per 64 keys x 32 columns is one
// read of the columns from LDS.
//
// A request's columns of all heads are cut into shares so that about p.tiles workgroups
// have work, whatever its span turns out to be; a workgroup goes from head to head in its
// share with the same sums, and weigh_join_kernel adds up a position's shares.
struct Column {
  float to, by;  // lse' and the factor of what it lacks
  int s, e;      // its range, empty where it adds nothing
};

template <int T, int C, int D>
__global__ __launch_bounds__(512, 2) void weigh_wide_kernel(WeighParams p) {
  constexpr int KS = D / 16, COLS = 64, QROW = 2 * D + 16;
  constexpr int EACH = COLS * D / 8 / 512;  // pieces of 8 elements a thread stages
  const AttendParams& a = p.a;
  const KvCache& c = a.c;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int hh = lane >> 5, n = lane & 31;
  const int unit = blockIdx.x / p.tiles, g0 = blockIdx.x % p.tiles;
  const int columns = a.R * a.group, per_head = (columns + COLS - 1) / COLS;
  const int all = per_head * c.kv_heads;

  __shared__ __align__(16) uint8_t s_q[2][COLS * QROW];
  __shared__ __align__(16) Column s_col[2][COLS];
  __shared__ int4 s_sight[2][2];  // of 32 columns: {largest s, smallest e, smallest s, largest e}
  __shared__ Span s_span[8];

  Span span = row_span<kRange>(a, unit * a.R, a.R, t, 512);
  if (lane == 0) s_span[wave] = span;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) span = join<kRange>(span, s_span[w]);
  const int lo = __builtin_amdgcn_readfirstlane(span.lo), hi = __builtin_amdgcn_readfirstlane(span.hi);
  const int first = lo & ~15;
  const int tiles = hi > first ? (hi - first + kWeighKeys - 1) / kWeighKeys : 0;
  const int shares = tiles > 0 ? min(max(p.tiles / tiles, 1), all) : 1;
  if (g0 == 0 && t == 0) {
    p.cut[2 * unit] = int4{first, tiles, shares, 0};
    p.cut[2 * unit + 1] = int4{lo, hi, 0, 0};
  }
  const int share = (all + shares - 1) / shares;
  const float cs = a.scale * kLog2e;
  const int32_t* const table = c.table + (int64_t)unit * c.table_stride;

  // stage x: 64 columns of head x / per_head
  v4u q_reg[EACH];
  float lse_reg = 0.f;
  int s_reg = 0, e_reg = 0;
  auto load = [&](int x) {
    const int h = x / per_head, col0 = x % per_head * COLS;
#pragma unroll
    for (int r = 0; r < EACH; ++r) {
      const int piece = t + 512 * r, col = col0 + piece / (D / 8);
      const bool real = col < columns;
      const int row = unit * a.R + (real ? col / a.group : 0);
      const int head = h * a.group + (real ? col % a.group : 0);
      q_reg[r] = *reinterpret_cast<const v4u*>(static_cast<const uint16_t*>(a.q) + row * a.q_row +
                                               head * a.q_head + piece % (D / 8) * 8);
      if (!real) q_reg[r] = v4u{0, 0, 0, 0};
    }
    if (wave == 0) {
      const int col = col0 + lane;
      const bool real = col < columns;
      const int row = unit * a.R + (real ? col / a.group : 0);
      const int head = h * a.group + (real ? col % a.group : 0);
      lse_reg = p.lse[(int64_t)row * a.heads + head];
      row_range(a, row, s_reg, e_reg);
      if (!real) e_reg = s_reg;
    }
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int r = 0; r < EACH; ++r) {
      const int piece = t + 512 * r;
      *reinterpret_cast<v4u*>(s_q[buf] + piece / (D / 8) * QROW + piece % (D / 8) * 16) = q_reg[r];
    }
    if (wave == 0) {
      const bool adds = s_reg < e_reg && lse_reg != -__builtin_inff();
      Column k;
      k.to = lse_reg * kLog2e;
      k.by = lacking(lse_reg, k.to);
      k.s = adds ? s_reg : 0;
      k.e = adds ? e_reg : 0;
      s_col[buf][lane] = k;
      int4 m{k.s, k.e, adds ? k.s : c.cap, k.e};
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        m.x = max(m.x, __shfl_xor(m.x, o, 64));
        m.y = min(m.y, __shfl_xor(m.y, o, 64));
        m.z = min(m.z, __shfl_xor(m.z, o, 64));
        m.w = max(m.w, __shfl_xor(m.w, o, 64));
      }
      if (n == 0) s_sight[buf][hh] = m;
    }
  };

  int count = 0;  // of stages: which buffer
  for (int item = g0; item < tiles * shares; item += p.tiles) {
    const int x_lo = item / tiles * share, x_hi = min(x_lo + share, all);
    const int pos0 = first + item % tiles * kWeighKeys + wave * 64;
    float acc[2][16];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[b][e] = 0.f;
    v4u kf[2][KS];
    float f[2][2];
    int at_head = -1;
    if (x_lo < x_hi) load(x_lo);
    for (int x = x_lo; x < x_hi; ++x, ++count) {
      const int buf = count & 1;
      stage(buf);
      if (x + 1 < x_hi) load(x + 1);
      const int h = x / per_head;
      if (h != at_head) {
        at_head = h;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int pos = min(pos0 + 32 * b + n, ((hi - 1) & ~15) + (n & 15));
          const uint8_t* const page =
              c.pages + (int64_t)clamp_page(c, table[pos >> c.page_shift]) * c.page_stride;
          const int slot = pos & ((1 << c.page_shift) - 1);
#pragma unroll
          for (int j = 0; j < KS / 2; ++j) {
            const v4u raw = *reinterpret_cast<const v4u*>(page + code_at(c, 0, h, slot) +
                                                          16 * (2 * j + hh));
            kf[b][2 * j] = widen8<T, C>(raw[0], raw[1]);
            kf[b][2 * j + 1] = widen8<T, C>(raw[2], raw[3]);
          }
          const float scale = *reinterpret_cast<const float*>(page + scale_at(c, 0, h, slot)) * cs;
          f[b][0] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scale), 0));
          f[b][1] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scale), 16));
        }
      }
      __syncthreads();
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const int4 sight = s_sight[buf][sub];
        const int smax = __builtin_amdgcn_readfirstlane(sight.x);
        const int emin = __builtin_amdgcn_readfirstlane(sight.y);
        const int smin = __builtin_amdgcn_readfirstlane(sight.z);
        const int emax = __builtin_amdgcn_readfirstlane(sight.w);
        if (emax <= pos0 || smin >= pos0 + 64) continue;
        const Column col = s_col[buf][32 * sub + n];
        const uint8_t* const from = s_q[buf] + (32 * sub + n) * QROW + 32 * hh;
        v16f s[2] = {v16f{}, v16f{}};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const v4u q = *reinterpret_cast<const v4u*>(from + 64 * (k >> 1) + 16 * (k & 1));
#pragma unroll
          for (int b = 0; b < 2; ++b) s[b] = mfma32<T>(kf[b][k], q, s[b]);
        }
        const bool clean = smax <= pos0 && emin >= pos0 + 64;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint32_t sees =
              clean ? ~0u : seen_bits(pos0 + 32 * b, col.s, col.e) >> (4 * hh);
          if (clean) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              acc[b][e] = __builtin_fmaf(
                  __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][e], f[b][e >> 3], -col.to)), col.by,
                  acc[b][e]);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][e], f[b][e >> 3], -col.to));
              acc[b][e] += or_zero(w * col.by, bit(sees, 8 * (e >> 2) + (e & 3)));
            }
          }
        }
      }
    }
    float* const part = p.part + ((int64_t)unit * p.slots + item) * kWeighKeys + wave * 64;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float v = acc[b][e];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) v += __shfl_xor(v, o, 64);
        if (n == 0) part[32 * b + 8 * (e >> 2) + 4 * hh + (e & 3)] = v;
      }
  }
}

// Adds a request's shares to its weights, in their order.
__global__ __launch_bounds__(256) void weigh_join_kernel(WeighParams p, int blocks) {
  const int unit = blockIdx.x / blocks;
  const int4 cut = p.cut[2 * unit], span = p.cut[2 * unit + 1];
  const int end = min(span.y, p.width);
  for (int pos = cut.x + (blockIdx.x % blocks) * 256 + (int)threadIdx.x; pos < end;
       pos += blocks * 256) {
    if (pos < span.x) continue;
    const float* part = p.part + (int64_t)unit * p.slots * kWeighKeys + (pos - cut.x);
    float sum = 0.f;
    for (int s = 0; s < cut.z; ++s) sum += part[(int64_t)s * cut.y * kWeighKeys];
    p.weights[(int64_t)unit * p.width + pos] += sum;
  }
}

}  // namespace
}  // namespace mqa

extern "C" int mqa_kv_weigh_launch(const mqa::WeighParams* p, hipStream_t s) {
  using namespace mqa;
  const dim3 grid((unsigned)p->a.requests * p->tiles);
  if (!p->wide) {
    dispatch(p->a, [&](auto t, auto c, auto d) {
      weigh_narrow_kernel<t.value, c.value, d.value><<<grid, 256, 0, s>>>(*p);
    });
    return (int)hipGetLastError();
  }
  dispatch(p->a, [&](auto t, auto c, auto d) {
    weigh_wide_kernel<t.value, c.value, d.value><<<grid, 512, 0, s>>>(*p);
  });
  const int cap = p->a.c.cap < p->width ? p->a.c.cap : p->width;
  const int most = (cap + 15 + 255) / 256, want = 2048 / p->a.requests;
  const int blocks = want < 1 ? 1 : want < most ? want : most;
  weigh_join_kernel<<<dim3((unsigned)p->a.requests * blocks), 256, 0, s>>>(*p, blocks);
  return (int)hipGetLastError();
}
