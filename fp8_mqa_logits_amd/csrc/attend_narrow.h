// Attention over what rows see of the cache for few columns (see attend_tiles.h for
// the sums).
#pragma once

#include "attend_tiles.h"

namespace mqa {
namespace {

// A column is a (row, query head) pair; the columns of one request and key
// head see the same keys and share a workgroup, 16 NT of them. The keys are
// split over the workgroup's four waves and over p.splits workgroups, 32 at a
// time.
//
// Per wave and step, with g = lane / 16 and n = lane % 16:
//   S^T = K Q^T, 16 keys x 16 columns per v_mfma_f32_16x16x32: lane (g, n)
//     loads 16-byte pieces of key n and gets the scores of keys 4g + i,
//     column n;
//   O^T += V^T P^T: the lane's eight scores (keys 4g + i of both halves of
//     the step) are its own operand as they stand, without a move between
//     lanes, when V's operand takes its keys in the same order: lane (g, n)
//     loads D / 16 consecutive codes of each of those eight keys (a wave's
//     load covers whole rows), and a byte transpose in registers makes them
//     the operands of D / 16 products, product u holding columns
//     d = D/16 * (4g + i) + u of the output.
// Nothing passes through LDS. A half step of 16 keys lies in one page and one
// block, so that its page, its addresses (but for an offset that each lane
// keeps) and its scales are scalars. The next step's keys are loaded when this
// step's are widened, its values when this step's are, table entries a step
// earlier; a single set of registers leaves room for several waves per SIMD, which
// hide what that does not.
//
// Bound by the cache's bytes in long contexts: 32 requests x 131072 positions of
// 2 key heads of 128 take 367 us, 5.86 TB/s; 48 uneven ones of up to 20011
// positions 121 to 124 us, 4.4 TB/s, as the longest parts end last. Heads of 64 cost
// as many instructions a key for half the bytes: 24 x 4 rows over up
// to 9001 positions 36 to 38 us with the join, 3.6 TB/s.
//
// Waves per SIMD: as many as hold the sums. Four of (D, NT) = (64, 2) spill five
// registers outside the loop; three, without them, took 40.4 us when four took 37.6.
template <int M, int T, int C, int D, int NT>
__global__ __launch_bounds__(256, NT == 4 ? 1 : NT == 2 && D == 128 ? 2 : 4)
void attend_narrow_kernel(AttendParams p) {
  constexpr int KC = D / 64;       // 16-byte pieces of a key per lane
  constexpr int U = D / 16;        // products per step and column tile
  constexpr int VW = D / 64;       // dwords of a value per lane
  constexpr int COLS = 16 * NT, WAVES = 4;
  const KvCache& c = p.c;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, n = lane & 15;
  const int64_t block = p.block0 + blockIdx.x;
  const int split = (int)(block % p.splits);
  const int64_t item = block / p.splits;
  const int h = (int)(item % c.kv_heads), tile = (int)(item / c.kv_heads % p.tiles);
  const int unit = (int)(item / c.kv_heads / p.tiles);
  const int columns = p.R * p.group;

  __shared__ Finish<D, NT, 1, WAVES> s_finish;

  const int row_lo = unit * p.R + tile * COLS / p.group;
  const int last = min(tile * COLS + COLS, columns);
  const int row_hi = unit * p.R + (last - 1) / p.group;
  const Walk<M, 32> walk(uniform(row_span<M>(p, row_lo, row_hi - row_lo + 1, lane, 64)));

  int col_row[NT], col_s[NT], col_e[NT];
  v4u q[NT][2 * KC];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int col = tile * COLS + 16 * t + n;
    const bool real = col < columns;
    const int row = unit * p.R + (real ? col / p.group : 0);
    const int head = h * p.group + (real ? col % p.group : 0);
    col_row[t] = row;
    row_range(p, row, col_s[t], col_e[t]);
    const uint16_t* src = static_cast<const uint16_t*>(p.q) + row * p.q_row + head * p.q_head;
#pragma unroll
    for (int k = 0; k < 2 * KC; ++k) {
      q[t][k] = *reinterpret_cast<const v4u*>(src + 64 * (k >> 1) + 16 * g + 8 * (k & 1));
      if (!real) q[t][k] = v4u{0, 0, 0, 0};
    }
  }
  // the part of the keys that this workgroup takes
  const int steps = walk.steps;
  const int per_split = ((steps + p.splits - 1) / p.splits + WAVES - 1) / WAVES * WAVES;
  const int step_lo = split * per_split + wave;
  const int step_hi = min(steps, (split + 1) * per_split);

  const float cs = p.scale * kLog2e;
  float m[NT], l[NT];
  v4f acc[NT][U];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = kLowest;
    l[t] = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) acc[t][u] = v4f{0.f, 0.f, 0.f, 0.f};
  }

  // A half step that no row sees is read from the nearest one that some row
  // sees, and masked later.
  const auto* const table = constant(c.table + (int64_t)unit * c.table_stride);
  auto half_pos = [&](int st, int b) { return walk.read_pos(st, 16 * b); };
  const uint32_t k_lane = n * D + 16 * g, v_lane = 4 * g * D + 4 * VW * n;
  v4u k_reg[2][KC];
  uint32_t v_reg[8][VW];
  float k_scale[2], v_scale[2];
  int entry[2];
  auto find = [&](int st) {
#pragma unroll
    for (int b = 0; b < 2; ++b) entry[b] = table[half_pos(st, b) >> c.page_shift];
  };
  const uint8_t* page[2];
  auto load_k = [&](int st) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      page[b] = c.pages + (int64_t)clamp_page(c, entry[b]) * c.page_stride;
      const int slot = half_pos(st, b) & ((1 << c.page_shift) - 1);
      const uint8_t* const k = page[b] + code_at(c, 0, h, slot);
#pragma unroll
      for (int x = 0; x < KC; ++x)
        k_reg[b][x] = *reinterpret_cast<const v4u*>(k + k_lane + 64 * x);
      k_scale[b] = *constant(reinterpret_cast<const float*>(page[b] + scale_at(c, 0, h, slot)));
    }
  };
  auto load_v = [&](int st) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int slot = half_pos(st, b) & ((1 << c.page_shift) - 1);
      const uint8_t* const v = page[b] + code_at(c, 1, h, slot);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (VW == 2) {
          const uint2 x = *reinterpret_cast<const uint2*>(v + v_lane + i * D);
          v_reg[4 * b + i][0] = x.x;
          v_reg[4 * b + i][1] = x.y;
        } else {
          v_reg[4 * b + i][0] = *reinterpret_cast<const uint32_t*>(v + v_lane + i * D);
        }
      }
      v_scale[b] = *constant(reinterpret_cast<const float*>(page[b] + scale_at(c, 1, h, slot)));
    }
  };

  if (step_lo < step_hi) {
    find(step_lo);
    load_k(step_lo);
    load_v(step_lo);
    find(step_lo + WAVES);
  }
  for (int st = step_lo; st < step_hi; st += WAVES) {
    // scores; the next step's keys are loaded as soon as these are widened
    const float f[2] = {k_scale[0] * cs, k_scale[1] * cs};
    v4f x[NT][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      v4u kf[2 * KC];
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        kf[2 * k] = widen8<T, C>(k_reg[b][k][0], k_reg[b][k][1]);
        kf[2 * k + 1] = widen8<T, C>(k_reg[b][k][2], k_reg[b][k][3]);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        x[t][b] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2 * KC; ++k) x[t][b] = mfma<T>(kf[k], q[t][k], x[t][b]);
      }
    }
    load_k(st + WAVES);
    find(st + 2 * WAVES);

    const int pos0 = walk.pos(st);
    const bool clean = walk.inside(pos0);
    uint32_t sees[NT], ill = 0;  // bit 16 b + i: key 16 b + 4 g + i
#pragma unroll
    for (int t = 0; t < NT; ++t) sees[t] = ~0u;
    if (!clean) {
      uint32_t any = 0;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        sees[t] = row_bits<M>(p, col_row[t], pos0, col_s[t], col_e[t]) >> (4 * g);
        any |= sees[t];
      }
      // (what lies between the rows' ranges may hold anything)
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (!__any(any & (0xFu << (16 * b)))) v_scale[b] = 0.f;
      // values that no row sees become 0; a NaN code, which some rows may
      // see and others not, becomes 0 too and is put back through the P of
      // the rows that see it (0 * NaN would reach the others)
      const uint32_t some = walk.some_bits(pos0) >> (4 * g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t bad = 0;
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          v_reg[j][w] &= bit(some, 16 * (j >> 2) + (j & 3));
          if constexpr (C == kE4m3) {
            const uint32_t nan = nan_bytes(v_reg[j][w]);
            v_reg[j][w] &= ~nan;
            bad |= nan;
          }
        }
        if constexpr (C == kE4m3)
          if (__ballot(bad != 0) >> (16 * g) & 0xFFFF) ill |= 1u << (16 * (j >> 2) + (j & 3));
      }
    }
    const float vr[2] = {v_scale[0] * kUp, v_scale[1] * kUp};
    const float loudest = __builtin_fmaxf(__builtin_fmaxf(vr[0], vr[1]), kFar);
    v4u pf[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float e[8], sum;
      auto exponentials = [&]() {
        const float off = kBias - m[t];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][j >> 2][j & 3], f[j >> 2], off));
        if (!clean) {
#pragma unroll
          for (int j = 0; j < 8; ++j) e[j] = or_zero(e[j], bit(sees[t], 16 * (j >> 2) + (j & 3)));
        }
        sum = e[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) sum += e[j];
      };
      exponentials();
      if (__any(!(sum * loudest <= kMost))) {  // m moves
        const float loud[2] = {loudness(vr[0]), loudness(vr[1])};
        float top = -__builtin_inff();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          top = __builtin_fmaxf(
              top, or_lowest(__builtin_fmaf(x[t][j >> 2][j & 3], f[j >> 2], loud[j >> 2]),
                             bit(sees[t], 16 * (j >> 2) + (j & 3))));
        top = __builtin_fmaxf(top, __shfl_xor(top, 16, 64));
        top = __builtin_fmaxf(top, __shfl_xor(top, 32, 64));
        const float to = __builtin_fmaxf(m[t], top);
        const float keep = __builtin_amdgcn_exp2f(m[t] - to);
        m[t] = to;
        l[t] *= keep;
#pragma unroll
        for (int u = 0; u < U; ++u) acc[t][u] *= keep;
        exponentials();
      }
      l[t] += sum;
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] *= vr[j >> 2];
      if (!clean) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int at = 16 * (j >> 2) + (j & 3);
          e[j] = __uint_as_float(__float_as_uint(or_zero(e[j], bit(sees[t], at))) |
                                 (bit(sees[t] & ill, at) & 0x7FC00000u));
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pf[t][i] = __builtin_bit_cast(uint32_t, v2h{(_Float16)e[2 * i], (_Float16)e[2 * i + 1]});
    }
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      uint32_t in[4], a[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) in[j] = v_reg[j][w];
      transpose4(in, a);
#pragma unroll
      for (int j = 0; j < 4; ++j) in[j] = v_reg[4 + j][w];
      transpose4(in, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const v4u vf = widen8<kFp16, C>(a[i], b[i]);
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t][4 * w + i] = mfma<kFp16>(vf, pf[t], acc[t][4 * w + i]);
      }
    }
    load_v(st + WAVES);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
    if (sees_nothing<M>(p, col_row[t], col_s[t], col_e[t])) l[t] = 0.f;  // sums of a row that sees nothing
  finish<T, false>(p, s_finish, block, unit * p.R, columns, tile, h, wave, m, l, acc);
}

template <int M, int T, int C, int D>
void launch_narrow(const AttendParams& p, dim3 grid, hipStream_t s) {
  if (p.cols == 16) attend_narrow_kernel<M, T, C, D, 1><<<grid, 256, 0, s>>>(p);
  if (p.cols == 32) attend_narrow_kernel<M, T, C, D, 2><<<grid, 256, 0, s>>>(p);
  // (windows and trees are not planned on 64 columns)
  if constexpr (M == kRange)
    if (p.cols == 64) attend_narrow_kernel<M, T, C, D, 4><<<grid, 256, 0, s>>>(p);
}

}  // namespace

template <int M>
void attend_narrow(const AttendParams& p, dim3 grid, hipStream_t s) {
  dispatch(p, [&](auto t, auto c, auto d) {
    launch_narrow<M, t.value, c.value, d.value>(p, grid, s);
  });
}

}  // namespace mqa
