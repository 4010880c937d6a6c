// Attention over listed positions (see attend_tiles.h for the sums).
#include "attend_tiles.h"

namespace mqa {
namespace {

// A workgroup takes one row and 16 NT HW of the query heads of one key head,
// and one of p.splits parts of the row's list, 32 entries and KW = 4 / HW waves
// at a time. HW waves share 32 entries: each loads its part of their rows (16
// bytes a lane, whole rows next to each other), a step ahead, into registers
// and then into LDS, and every one of them reads all of it for its own 16 NT
// heads, with the products of attend_narrow.h. For 64 heads two waves take 32
// each: with one wave for all, its sums leave room for one wave per SIMD only
// and a gather's latency shows; with four of 16, every code is widened and read
// from LDS four times (4096 rows of 64 heads and 2048 positions, when they were
// compared: 1.14 ms, 666 us, and 594 us for this).
//
// Bound by the gathered bytes where rows share little: 64 x 2 rows of 2048
// positions, 8 key heads of 4 query heads, take 93 us, 5.8 TB/s. With 64 query heads
// on one key head, 4096 rows of 2048 of 65536 positions take 411 to 421 us (eight
// calls after start-up: 482 to 520), 650 to 670 TFLOP/s: of 2.1 GB of gathered codes
// the L2s serve 92% of the requests and 0.23 GB come from beyond them, so that memory
// is not the limit. Vector instructions (widening, which both waves of a pair do
// for every code, and exponentials) take 59% of the cycles or more, the matrix unit
// 26%, and two waves per SIMD overlap them in part.
//
// A step's tokens (slots in the pool) are found by lanes 0 .. 31, an entry
// each, two steps ahead, and go to the other lanes by permutation; scales go
// through LDS, a wave for itself.
template <int T, int C, int D, int NT, int HW>
__global__ __launch_bounds__(256, 2) void attend_list_kernel(AttendParams p) {
  constexpr int KW = 4 / HW;
  constexpr int KC = D / 64;       // 16-byte pieces of a key per lane and product
  constexpr int U = D / 16;        // products per step
  constexpr int PIECES = D / 16;   // 16-byte pieces of a row
  constexpr int GROUP = 64 * HW;   // threads that share 32 entries
  constexpr int EACH = 32 * PIECES / GROUP;  // pieces of 32 keys, and of 32 values, per thread
  constexpr int COLS = 16 * NT * HW, BUFS = HW == 1 ? 1 : 2;
  const KvCache& c = p.c;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, n = lane & 15;
  const int hw = wave % HW, kb = wave / HW, gt = hw * 64 + lane;
  const int64_t block = p.block0 + blockIdx.x;
  const int split = (int)(block % p.splits);
  const int64_t item = block / p.splits;
  const int h = (int)(item % c.kv_heads), tile = (int)(item / c.kv_heads % p.tiles);
  const int row = (int)(item / c.kv_heads / p.tiles);

  __shared__ __align__(16) union {
    struct {
      __align__(16) uint8_t rows[KW][BUFS][64 * D];  // 32 keys, 32 values
      __align__(16) float ks[4][32], vs[4][32], loud[4][32];
    } step;
    Finish<D, NT, HW, KW> finish;
    int used[4];
  } sh;

  int s, e;
  row_range(p, row, s, e);
  v4u q[NT][2 * KC];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int col = tile * COLS + 16 * (NT * hw + t) + n;
    const bool real = col < p.group;
    const uint16_t* src = static_cast<const uint16_t*>(p.q) + row * p.q_row +
                          (h * p.group + (real ? col : 0)) * p.q_head;
#pragma unroll
    for (int k = 0; k < 2 * KC; ++k) {
      q[t][k] = *reinterpret_cast<const v4u*>(src + 64 * (k >> 1) + 16 * g + 8 * (k & 1));
      if (!real) q[t][k] = v4u{0, 0, 0, 0};
    }
  }
  // A row that cannot fill its list (its valid entries come first, but for
  // what a caller wrote himself) ends it at the last entry that names a position.
  int used = p.width;
  if (e - s < p.width) {
    used = 0;
    const int32_t* const list = p.indices + (int64_t)row * p.width;
    for (int i = threadIdx.x; i < p.width; i += 256) {
      const int x = list[i];
      if (x >= 0 && x < e - s) used = i + 1;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) used = max(used, __shfl_xor(used, o, 64));
    if (lane == 0) sh.used[wave] = used;
    __syncthreads();
    used = max(max(sh.used[0], sh.used[1]), max(sh.used[2], sh.used[3]));
    used = __builtin_amdgcn_readfirstlane(used);
    __syncthreads();
  }
  const int steps = (used + 31) / 32;
  const int per_split = ((steps + p.splits - 1) / p.splits + KW - 1) / KW * KW;
  const int step_lo = split * per_split;
  const int rounds = (min(steps, step_lo + per_split) - step_lo + KW - 1) / KW;
  const int step_hi = min(steps, step_lo + per_split);

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

  // entry lane % 32 of the wave's step in a round: its list entry as it is,
  // what it names (-1: nothing), the table entry of that position
  const int32_t* const list = p.indices + (int64_t)row * p.width;
  const int32_t* const table = c.table + (int64_t)(row / p.R) * c.table_stride;
  const int page_mask = (1 << c.page_shift) - 1;
  auto at_of = [&](int round) { return (step_lo + round * KW + kb) * 32 + (lane & 31); };
  auto listed = [&](int round) { return list[min(at_of(round), p.width - 1)]; };
  auto named = [&](int x, int round) {
    return at_of(round) < min(step_hi * 32, used) && x >= 0 && x < e - s ? x : -1;
  };
  auto looked_up = [&](int x) { return table[(x < 0 ? 0 : s + x) >> c.page_shift]; };
  // what a lane loads: piece x = gt + GROUP r of the 32 keys, and of the values
  const int lane_at = 16 * (gt % PIECES);
  const int k_at = code_at(c, 0, h, 0) + lane_at, v_at = code_at(c, 1, h, 0) + lane_at;
  struct Codes {
    v4u k[EACH], v[EACH];
    float ks, vs;
    bool named;
  };
  auto load = [&](Codes& f, int x, int entry) {
    f.named = x >= 0;
    const uint8_t* const page = c.pages + (int64_t)clamp_page(c, entry) * c.page_stride;
    const int slot = x < 0 ? 0 : (s + x) & page_mask;
    const uint64_t token = (uint64_t)(page + slot * D);
#pragma unroll
    for (int r = 0; r < EACH; ++r) {
      const int key = (gt + GROUP * r) / PIECES;
      const uint64_t lo = (uint32_t)__shfl((int)token, key, 64);
      const uint64_t hi = (uint32_t)__shfl((int)(token >> 32), key, 64);
      const uint8_t* const at = (const uint8_t*)(hi << 32 | lo);
      f.k[r] = *reinterpret_cast<const v4u*>(at + k_at);
      f.v[r] = *reinterpret_cast<const v4u*>(at + v_at);
    }
    f.ks = *reinterpret_cast<const float*>(page + scale_at(c, 0, h, slot));
    f.vs = *reinterpret_cast<const float*>(page + scale_at(c, 1, h, slot));
  };
  // byte of piece x of a row in LDS (of 32 rows), 16-byte pieces exchanged so
  // that the lanes of every read touch all banks: 16 rows and one piece of the
  // keys, rows 4 g .. 4 g + 3 of both halves and one piece of the values
  auto k_place = [&](int key, int x) {
    if constexpr (D == 128)
      return (key ^ (key >> 2 & 1)) * D + 16 * (x ^ (key >> 1 & 7));
    else
      return key * D + 16 * (x ^ (key >> 2 & 3));
  };
  auto v_place = [&](int key, int x) {
    if constexpr (D == 128)
      return key * D + 16 * (x ^ ((key >> 1 & 3) | (key >> 2 & 4)));
    else
      return key * D + 16 * (x ^ ((key >> 2 & 1) | (key >> 3 & 2)));
  };
  // (an entry that names no position was read from somewhere: its values become 0)
  auto stage = [&](Codes& f, uint32_t valid, int buf) {
    uint8_t* const to = sh.step.rows[kb][buf];
    if (valid != ~0u) {
#pragma unroll
      for (int r = 0; r < EACH; ++r)
        if (!(valid >> (gt + GROUP * r) / PIECES & 1)) f.v[r] = v4u{0, 0, 0, 0};
    }
#pragma unroll
    for (int r = 0; r < EACH; ++r) {
      const int key = (gt + GROUP * r) / PIECES, x = gt % PIECES;
      *reinterpret_cast<v4u*>(to + k_place(key, x)) = f.k[r];
      *reinterpret_cast<v4u*>(to + 32 * D + v_place(key, x)) = f.v[r];
    }
  };
  auto compute = [&](uint32_t valid, int buf) {
    const bool clean = valid == ~0u;
    const uint8_t* const rows = sh.step.rows[kb][buf];
    v4f x[NT][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int t = 0; t < NT; ++t) x[t][b] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        const v4u w = *reinterpret_cast<const v4u*>(rows + k_place(16 * b + n, g + 4 * k));
        const v4u lo = widen8<T, C>(w[0], w[1]), hi = widen8<T, C>(w[2], w[3]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          x[t][b] = mfma<T>(lo, q[t][2 * k], x[t][b]);
          x[t][b] = mfma<T>(hi, q[t][2 * k + 1], x[t][b]);
        }
      }
    }
    const uint32_t sees = valid >> (4 * g);  // bit 16 b + i: entry 16 b + 4 g + i
    v4f f[2], vr[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f[b] = *reinterpret_cast<const v4f*>(&sh.step.ks[wave][16 * b + 4 * g]);
      vr[b] = *reinterpret_cast<const v4f*>(&sh.step.vs[wave][16 * b + 4 * g]);
    }
    float loudest = kFar;
#pragma unroll
    for (int j = 0; j < 8; ++j) loudest = __builtin_fmaxf(loudest, vr[j >> 2][j & 3]);
    v4u pf[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float e[8], sum;
      auto exponentials = [&]() {
        const float off = kBias - m[t];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][j >> 2][j & 3], f[j >> 2][j & 3], off));
        if (!clean) {
#pragma unroll
          for (int j = 0; j < 8; ++j) e[j] = or_zero(e[j], bit(sees, 16 * (j >> 2) + (j & 3)));
        }
        sum = e[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) sum += e[j];
      };
      exponentials();
      if (__any(!(sum * loudest <= kMost))) {  // m moves
        float top = -__builtin_inff();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float loud = sh.step.loud[wave][16 * (j >> 2) + 4 * g + (j & 3)];
          top = __builtin_fmaxf(
              top, or_lowest(__builtin_fmaf(x[t][j >> 2][j & 3], f[j >> 2][j & 3], loud),
                             bit(sees, 16 * (j >> 2) + (j & 3))));
        }
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
      for (int j = 0; j < 8; ++j) e[j] *= vr[j >> 2][j & 3];  // (0 where nothing is named)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pf[t][i] = __builtin_bit_cast(uint32_t, v2h{(_Float16)e[2 * i], (_Float16)e[2 * i + 1]});
    }
    // A transposing read gives lane n of 16 the bytes n of the eight rows that
    // lanes 2 j and 2 j + 1 point at: the codes of one column and the eight
    // keys whose P the lane holds.
    const int key = 4 * g + (n >> 1 & 3) + 16 * (n >> 3);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      typedef int v2i __attribute__((ext_vector_type(2)));
      const v2i w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (__attribute__((address_space(3))) v2i*)(rows + 32 * D + v_place(key, u) + 8 * (n & 1)));
      const v4u vf = widen8<kFp16, C>(w.x, w.y);
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t][u] = mfma<kFp16>(vf, pf[t], acc[t][u]);
    }
  };

  if (rounds > 0 && s < e) {
    auto sync = [&]() {
      if constexpr (HW > 1)
        __syncthreads();
      else
        __builtin_amdgcn_wave_barrier();
    };
    // a round's scales and which of its entries name positions
    auto take_scales = [&](const Codes& f) {
      const float k = f.named ? f.ks * cs : 0.f, v = f.named ? f.vs : 0.f;
      sh.step.ks[wave][lane & 31] = k;
      sh.step.vs[wave][lane & 31] = v * kUp;
      sh.step.loud[wave][lane & 31] = loudness(v * kUp);
      __builtin_amdgcn_wave_barrier();
    };
    // Loads come back in order: what a later round's addresses wait for is asked
    // for before the next round's codes, so that no one waits for these before
    // they are used (as the compiler placed them otherwise: 149 us, not 123, for
    // 64 x 2 rows of 2048 positions and 8 heads; codes two rounds ahead added
    // nothing to that).
    Codes codes;
    int x = named(listed(0), 0), entry = looked_up(x), x_raw = listed(1);
    auto load_next = [&](int round) {  // codes of `round`; entry of the next, list of the one after
      const int x0 = x, entry0 = entry;
      x = named(x_raw, round + 1);
      entry = looked_up(x);
      x_raw = listed(round + 2);
      load(codes, x0, entry0);
    };
    load_next(0);
    auto round = [&](int i, int buf) {
      const uint32_t valid = (uint32_t)__ballot(codes.named);
      stage(codes, valid, buf);
      take_scales(codes);
      sync();
      load_next(i + 1);
      compute(valid, buf);
      if constexpr (BUFS == 1) __builtin_amdgcn_wave_barrier();
    };
    int i = 0;
    if constexpr (BUFS == 2)  // (two at a time: what LDS addresses add is known)
      for (; i + 1 < rounds; i += 2) {
        round(i, 0);
        round(i + 1, 1);
      }
    for (; i < rounds; ++i) round(i, 0);
  }
  __syncthreads();  // (the steps' memory becomes the sums')
  finish<T, true>(p, sh.finish, block, row, p.group, tile, h, wave, m, l, acc);
}

template <int T, int C, int D>
void launch(const AttendParams& p, dim3 grid, hipStream_t s) {
  if (p.cols == 16) attend_list_kernel<T, C, D, 1, 1><<<grid, 256, 0, s>>>(p);
  if (p.cols == 32) attend_list_kernel<T, C, D, 2, 1><<<grid, 256, 0, s>>>(p);
  if (p.cols == 64) attend_list_kernel<T, C, D, 2, 2><<<grid, 256, 0, s>>>(p);
}

}  // namespace

void attend_list(const AttendParams& p, dim3 grid, hipStream_t s) {
  dispatch(p, [&](auto t, auto c, auto d) { launch<t.value, c.value, d.value>(p, grid, s); });
}

}  // namespace mqa
