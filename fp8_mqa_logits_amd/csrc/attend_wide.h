// Attention over what rows see of the cache for many columns (see attend_tiles.h for
// the sums).
#pragma once

#include "attend_tiles.h"

namespace mqa {
namespace {

// ---------------------------------------------------------------------------
// Many columns: 32 W columns of one request and key head per workgroup, 32 in
// each of its W waves, every wave over all keys of the workgroup's part. Tiles
// of 64 keys pass through LDS once for the workgroup, widened on the way in:
// keys as [key][d], values transposed as [d][key] in the order in which a lane
// holds its scores, both with rows padded by 16 bytes so that 16 lanes of a
// read touch all banks.
//   S^T = K Q^T   32 keys x 32 columns per v_mfma_f32_32x32x16, Q in registers
//   O^T += V^T P^T   P straight from the scores' registers
//
// Half tiles j = 0, 1, .. run as a pipeline inside the wave: the products of
// S(j + 1) and of P(j - 1) V are independent of the exponentials of S(j), so
// that the matrix unit and the vector unit work at the same time. One barrier
// a tile: between the halves of tile i, when the keys of tile i + 1 are in
// LDS; its values follow during the second half and are first read after the
// next barrier.
//
// 4096 rows of 32 heads over 49152 positions of 4 key heads, on several cards: 2.84
// to 2.95 ms in long runs, 1.07 to 1.11 PFLOP/s, 90 to 94% of what a large matrix
// product reaches here (eight calls after start-up: 2.97 to 3.17); two requests of
// 1024 rows packed into 32768 positions of 8 key heads 513 to 547 us, 0.97 to 1.04
// PFLOP/s. By the counters the matrix unit is busy 51% of the cycles, vector
// instructions take 44% or more at four cycles each (exponentials need more), LDS
// is active 37%: two waves per SIMD overlap the first two only in part. When it
// took 3.46 ms, 64 columns a wave, which halve the LDS reads but leave one wave per
// SIMD, took 3.97, and two groups of waves in turn on the matrix and the vector
// unit, which met at too many barriers, 4.46. What the two waves per SIMD spill lies
// outside the plain tiles' loop, but for one reload a tile.
template <int M, int T, int C, int D, int W>
__global__ __launch_bounds__(64 * W, 2) void attend_wide_kernel(AttendParams p) {
  constexpr int THREADS = 64 * W;
  constexpr int KS = D / 16;          // products a half's scores take
  constexpr int DT = D / 32;          // tiles of the output's columns
  // pieces of a tile, EACH of either kind per thread: KB bytes of a key, and VK
  // values' codes of four columns (all threads take the same part, so that the
  // loop has no branch)
  constexpr int KB = 4 * D < THREADS ? 8 : 16, VK = KB / 4;
  constexpr int EACH = 64 * D / KB / THREADS;
  constexpr int COLS = 32 * W;
  const KvCache& c = p.c;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int hh = lane >> 5, n = lane & 31;
  const int64_t block = p.block0 + blockIdx.x;
  const int split = (int)(block % p.splits);
  const int64_t item = block / p.splits;
  const int h = (int)(item % c.kv_heads);
  const int unit = (int)(item / c.kv_heads / p.tiles);
  // the last rows see the most in a causal chunk: they start first
  const int tile = p.tiles - 1 - (int)(item / c.kv_heads % p.tiles);
  const int columns = p.R * p.group;

  constexpr int KROW = 2 * D + 16, VROW = 2 * 64 + 16;  // bytes of a staged key, of a column
  __shared__ __align__(16) uint8_t s_k[2][64 * KROW];
  __shared__ __align__(16) uint8_t s_v[2][D * VROW];
  // of a tile: 8 scales, over and over; keys whose values hold a NaN code. A wave
  // behind the others reads them until the next tile's barrier, one ahead writes
  // two tiles further meanwhile and clears a third: four buffers.
  __shared__ __align__(16) float s_scale[4][256];
  __shared__ uint32_t s_poison[4][2];
  __shared__ Span s_span[W];

  const int row_lo = unit * p.R + tile * COLS / p.group;
  const int last = tile * COLS + COLS < columns ? tile * COLS + COLS : columns;
  const int row_hi = unit * p.R + (last - 1) / p.group;
  Span span = row_span<M>(p, row_lo, row_hi - row_lo + 1, t, THREADS);
  if (lane == 0) s_span[wave] = span;
  if (t < 8) s_poison[t >> 1][t & 1] = 0;
  // the first half adds no values: P = 0 times what is staged "before" them
  for (int x = t; x < D * VROW / 16; x += THREADS)
    reinterpret_cast<v4u*>(s_v[1])[x] = v4u{0, 0, 0, 0};
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) span = join<M>(span, s_span[w]);
  const Walk<M, 64> walk(uniform(span));

  // this lane's column
  int at_col = wave * 32 + n, col_row, col_s, col_e;
  v4u q[KS];
  {
    const int col = tile * COLS + at_col;
    const bool real = col < columns;
    const int row = unit * p.R + (real ? col / p.group : 0);
    const int head = h * p.group + (real ? col % p.group : 0);
    col_row = row;
    row_range(p, row, col_s, col_e);
    const uint16_t* src = static_cast<const uint16_t*>(p.q) + row * p.q_row + head * p.q_head;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      // slot 2 k + hh of a staged key: see stage_k
      const int slot = 2 * k + hh;
      q[k] = *reinterpret_cast<const v4u*>(src + 16 * (slot % (D / 16)) + 8 * (slot / (D / 16)));
      if (!real) q[k] = v4u{0, 0, 0, 0};
    }
  }

  // the part of the keys that this workgroup takes, in tiles of 64: each group of 16
  // keys lies in one block
  const int per_split = (walk.steps + p.splits - 1) / p.splits;
  const int tile_lo = split * per_split;
  const int tiles = min(walk.steps - tile_lo, per_split);
  // Behind the sinks' tiles (kWindow) come the windows', `jump` positions further on.
  const int base = __builtin_amdgcn_readfirstlane(
      (M == kWindow && walk.s_steps > 0 ? walk.s_first : walk.first) + tile_lo * 64);
  const int sink_tiles = M == kWindow ? walk.s_steps - tile_lo : 0;
  const int jump = M == kWindow && walk.s_steps > 0
                       ? walk.first - walk.s_first - walk.s_steps * 64 : 0;
  const int last_pos = M == kWindow ? max(walk.span.hi, walk.span.s_hi) - 1 : 0;
  auto tile_pos = [&](int i) {
    return base + i * 64 + (M == kWindow && i >= sink_tiles ? jump : 0);
  };

  // staging: piece x = t + THREADS r of the keys is KB bytes of key x / (D /
  // KB); of the values, columns 4 (x % (D / 4)) .. + 3 of VK keys from
  // VK (x / (D / 4))
  auto piece = [&](int r) { return t + THREADS * r; };
  auto k_key = [&](int r) { return piece(r) / (D / KB); };
  auto v_key = [&](int r) { return piece(r) / (D / 4) * VK; };
  auto v_d = [&](int r) { return piece(r) % (D / 4) * 4; };
  // What a wave takes lies in one group of 16 keys, so that its page, its
  // addresses (but for an offset that each lane keeps) and its scales are the
  // wave's (3.08 ms, not 3.24, for those 4096 rows on one card). A group outside all
  // rows' ranges is read from the nearest one inside, one between them as it stands
  // (masked later; no branch in the loop). Its table entry is loaded a tile
  // before its use, and only looked at then, by a vector load: a scalar one would
  // have every LDS read in flight waited for.
  static_assert(64 / (D / KB) == 64 / (D / 4) * VK && 64 / (D / KB) <= 16);
  auto group = [&](int r) { return (wave * 64 + THREADS * r) / (D / KB) >> 4; };
  const int* const table = c.table + (int64_t)unit * c.table_stride;
  int zero = 0;
  asm("" : "+v"(zero));
  auto group_pos = [&](int i, int r) {
    if constexpr (M == kWindow)
      return min(tile_pos(i) + 16 * group(r), last_pos) & ~15;
    else
      return min(max(base + i * 64 + 16 * group(r), walk.span.lo), walk.span.hi - 1) & ~15;
  };
  const uint32_t k_lane = (k_key(0) & 15) * D + KB * (t % (D / KB));
  const uint32_t v_lane = (v_key(0) & 15) * D + v_d(0);
  const uint32_t s_lane = (lane & 1) * (scale_at(c, 1, h, 0) - scale_at(c, 0, h, 0));
  uint32_t kreg[EACH][KB / 4], vreg[EACH][VK];
  float sreg[EACH];
  int found[EACH], entry[EACH];
  const uint8_t* page[EACH];
  auto find = [&](int i) {
#pragma unroll
    for (int r = 0; r < EACH; ++r) found[r] = table[(group_pos(i, r) >> c.page_shift) + zero];
  };
  auto look = [&]() {  // (after the loads that may be in flight behind find's)
#pragma unroll
    for (int r = 0; r < EACH; ++r) entry[r] = __builtin_amdgcn_readfirstlane(found[r]);
  };
  auto load_k = [&](int i) {
#pragma unroll
    for (int r = 0; r < EACH; ++r) {
      page[r] = c.pages + (int64_t)clamp_page(c, entry[r]) * c.page_stride;
      const int slot = group_pos(i, r) & ((1 << c.page_shift) - 1);
      typedef uint32_t Piece __attribute__((ext_vector_type(KB / 4)));
      const Piece x = *reinterpret_cast<const Piece*>(page[r] + code_at(c, 0, h, slot) + k_lane);
#pragma unroll
      for (int j = 0; j < KB / 4; ++j) kreg[r][j] = x[j];
      sreg[r] = *reinterpret_cast<const float*>(page[r] + scale_at(c, 0, h, slot) + s_lane);
    }
  };
  auto load_v = [&](int i) {
#pragma unroll
    for (int r = 0; r < EACH; ++r) {
      const int slot = group_pos(i, r) & ((1 << c.page_shift) - 1);
      const uint8_t* const at = page[r] + code_at(c, 1, h, slot);
#pragma unroll
      for (int j = 0; j < VK; ++j)
        vreg[r][j] = *reinterpret_cast<const uint32_t*>(at + (v_lane + j * D));
    }
  };
  auto k_slot = [&](int key, int slot) { return key * KROW + 16 * slot; };
  auto v_slot = [&](int d, int slot) { return d * VROW + 16 * slot; };
  auto inside = [&](int i) { return walk.inside(tile_pos(i)); };
  auto stage_k = [&](int i) {
    uint8_t* const to = s_k[i & 1];
#pragma unroll
    for (int r = 0; r < EACH; ++r) {
      // (the halves of 16 bytes half a row apart: eight lanes write 128 bytes)
#pragma unroll
      for (int j = 0; j < KB / 8; ++j) {
        const int x = piece(r) % (D / KB) * (KB / 8) + j;  // 8 codes
        *reinterpret_cast<v4u*>(to + k_slot(k_key(r), (x & 1) * (D / 16) + (x >> 1))) =
            widen8<T, C>(kreg[r][2 * j], kreg[r][2 * j + 1]);
      }
      s_scale[i & 3][4 * lane + group(r)] = sreg[r];
    }
  };
  // values that no row sees become 0; a NaN code, which some rows may see and
  // others not, becomes 0 too and is put back through the P of the rows that
  // see it (0 * NaN would reach the others)
  auto clean_v = [&](int i) {
    if (inside(i) && inside(i + 1)) return;
    if (t == 0) s_poison[(i + 1) & 3][0] = s_poison[(i + 1) & 3][1] = 0;
    if (inside(i)) return;
#pragma unroll
    for (int r = 0; r < EACH; ++r) {
#pragma unroll
      for (int j = 0; j < VK; ++j) {
        const int key = v_key(r) + j;
        if (i >= tiles || !walk.some(tile_pos(i) + key)) vreg[r][j] = 0;
        if constexpr (C == kE4m3) {
          const uint32_t bad = nan_bytes(vreg[r][j]);
          if (bad) {
            vreg[r][j] &= ~bad;
            atomicOr(&s_poison[i & 3][key >> 5], 1u << (key & 31));
          }
        }
      }
    }
  };
  // keys 16 g + {0..3, 8..11} share slot 2 g, {4..7, 12..15} slot 2 g + 1;
  // column d is row D / 4 (d % 4) + d / 4, so that the lanes of a write, four
  // columns apart, go to neighbouring rows (next to each other in the banks;
  // as rows d they met in four of them, 43% of all LDS cycles)
  auto stage_v = [&](int i) {
#pragma unroll
    for (int r = 0; r < EACH; ++r) {
      const int y = v_key(r) >> 2, slot = 2 * (y >> 2) + (y & 1), half = y >> 1 & 1;
      auto to = [&](int j) {
        return s_v[i & 1] + v_slot(D / 4 * j + v_d(r) / 4, slot) + 8 * half + 2 * (v_key(r) & 3);
      };
      if constexpr (VK == 4) {
        uint32_t a[4];
        transpose4(vreg[r], a);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint2*>(to(j)) = widen4<kFp16, C>(a[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {  // columns j and j + 1 of both keys
          const uint2 w = widen4<kFp16, C>(
              __builtin_amdgcn_perm(vreg[r][1], vreg[r][0], j ? 0x07030602u : 0x05010400u));
          *reinterpret_cast<uint32_t*>(to(j)) = w.x;
          *reinterpret_cast<uint32_t*>(to(j + 1)) = w.y;
        }
      }
    }
  };

  const float cs = p.scale * kLog2e;
  float m = kLowest, l = 0.f;
  v16f acc[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = v16f{};
  struct Prob {
    v4u f[2];  // of the half's two groups of keys
  };
  // of the current tile, per group of 16 keys (the same in all lanes): the
  // factor of the scores; the logarithm + kBias and the inverse of kUp vs
  float fk[4], lv[4], iv[4];
  bool plain = false;  // every row sees every key, and the scales are ordinary

  // lanes 0 .. 3 the groups' keys, 4 .. 7 their values (all at once: 3.18 ms, not
  // 3.34, on one card)
  auto take_scales = [&](int i) {
    const float x = s_scale[i & 3][lane & 7], to_value = x * kUp;
    const float key = x * cs, lg = __builtin_amdgcn_logf(to_value) + kBias;
    const float inv = __builtin_amdgcn_rcpf(to_value);
    auto of = [&](float y, int from) {
      return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(y), from));
    };
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      fk[g] = of(key, g);
      lv[g] = of(lg, 4 + g);
      iv[g] = of(inv, 4 + g);
    }
    plain = (__ballot(to_value >= 0x1p-40f && to_value <= 0x1p40f) & 0xF0) == 0xF0 && inside(i);
  };
  auto scores = [&](v16f& s, int i, int half) {
    const uint8_t* const from = s_k[i & 1] + k_slot(n, hh);
    s = v16f{};
#pragma unroll
    for (int k = 0; k < KS; ++k)
      s = mfma32<T>(*reinterpret_cast<const v4u*>(from + k_slot(32 * half, 2 * k)), q[k], s);
  };
  auto values = [&](const Prob& pr, int i, int half) {
    const uint8_t* const from = s_v[i & 1] + v_slot(n, hh);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int d = 0; d < DT; ++d)
        acc[d] = mfma32<kFp16>(
            *reinterpret_cast<const v4u*>(from + v_slot(32 * d, 2 * (2 * half + k))), pr.f[k],
            acc[d]);
  };
  // bit key_at(e): whether the column sees the key of its score e
  auto seen_keys = [&](int i, int half) {
    return row_bits<M>(p, col_row, tile_pos(i) + 32 * half, col_s, col_e) >> (4 * hh);
  };
  auto key_at = [](int e) { return 8 * (e >> 2) + (e & 3); };
  auto pack = [&](const float* e) {
    v4u f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f[j] = __builtin_bit_cast(uint32_t, v2h{(_Float16)e[2 * j], (_Float16)e[2 * j + 1]});
    return f;
  };
  // scores -> probabilities of one half; of a plain tile's, the largest sum of
  // eight of them: over kMost, m has to move and they are to be formed again
  auto soft = [&](auto is_plain, const v16f& s, Prob& pr, int i, int half) {
    float over = 0.f;
    if constexpr (is_plain.value) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int g = 2 * half + k;
        const float off = lv[g] - m;
        float e[8], sum;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * k + j], fk[g], off));
          sum = j ? sum + e[j] : e[j];
        }
        l = __builtin_fmaf(sum, iv[g], l);
        over = k ? __builtin_fmaxf(over, sum) : sum;
        pr.f[k] = pack(e);
      }
    } else {
      const uint32_t sees = seen_keys(i, half);
      const uint32_t ill = inside(i) ? 0 : sees & (s_poison[i & 3][half] >> (4 * hh));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int g = 2 * half + k;
        const float vr = s_scale[i & 3][4 + g] * kUp;
        float e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t see = bit(sees, key_at(8 * k + j));
          const float x = or_zero(
              __builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * k + j], fk[g], kBias - m)), see);
          l += x;
          e[j] = __uint_as_float(__float_as_uint(or_zero(x * vr, see)) |
                                 (bit(ill, key_at(8 * k + j)) & 0x7FC00000u));
        }
        pr.f[k] = pack(e);
      }
    }
    return over;
  };
  // moves m to a half's loudest weight, where that is above it (to the next integer
  // in plain tiles, where every column has many keys)
  auto settle = [&](auto is_plain, const v16f& s, int i, int half) {
    const uint32_t sees = is_plain.value ? 0 : seen_keys(i, half);
    float top = -__builtin_inff();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int g = 2 * half + (e >> 3);
      const float x = __builtin_fmaf(
          s[e], fk[g], is_plain.value ? lv[g] : __builtin_fmaxf(lv[g] - kTop, kLeast));
      top = __builtin_fmaxf(top, is_plain.value ? x : or_lowest(x, bit(sees, key_at(e))));
    }
    top = __builtin_fmaxf(top, __shfl_xor(top, 32, 64));
    if (is_plain.value) top = __builtin_ceilf(top) - kTop;
    if (!__any(top > m)) return;
    const float to = __builtin_fmaxf(m, top);
    const float keep = __builtin_amdgcn_exp2f(m - to);
    m = to;
    l *= keep;
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[d] *= keep;
  };

  if (tiles > 0) {
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    v16f s0, s1;
    Prob p0, p1;
#pragma unroll
    for (int k = 0; k < 2; ++k) p0.f[k] = p1.f[k] = v4u{0, 0, 0, 0};
    find(0);
    look();
    load_k(0);
    find(1);
    load_v(0);
    look();
    stage_k(0);
    clean_v(0);
    stage_v(0);
    load_k(1);
    find(2);
    load_v(1);
    look();
    __syncthreads();
    // holds the exponentials next to the products (they are used after a branch
    // only, and would be moved behind it)
    auto keep_here = [](Prob& pr, float& x) {
      asm volatile("" : "+v"(pr.f[0]), "+v"(pr.f[1]), "+v"(x));
    };
    // first half: s0 -> p0, scores of the second, values of the last tile's
    // second; keys of the next tile into LDS. Whether p0 is to be formed again.
    auto half0 = [&](auto is_plain, int i) {
      const float before = l;
      scores(s1, i, 1);
      if constexpr (is_plain.value) {
        const float over = soft(is_plain, s0, p0, i, 0);
        values(p1, i - 1, 1);
        stage_k(i + 1);
        load_k(i + 2);
        keep_here(p0, l);
        clean_v(i + 1);
        find(i + 3);
        __syncthreads();
        const bool again = __any(!(over <= kMost));
        if (again) l = before;
        return again;
      } else {
        values(p1, i - 1, 1);
        settle(is_plain, s0, i, 0);
        soft(is_plain, s0, p0, i, 0);
        stage_k(i + 1);
        load_k(i + 2);
        clean_v(i + 1);
        find(i + 3);
        __syncthreads();
        return false;
      }
    };
    // second half: s1 -> p1, scores of the next tile's first, values of this
    // tile's first; values of the next tile into LDS
    auto half1 = [&](auto is_plain, int i) {
      const float before = l;
      scores(s0, i + 1, 0);
      if constexpr (is_plain.value) {
        const float over = soft(is_plain, s1, p1, i, 1);
        values(p0, i, 0);
        stage_v(i + 1);
        load_v(i + 2);
        look();
        keep_here(p1, l);
        const bool again = __any(!(over <= kMost));
        if (again) l = before;
        return again;
      } else {
        values(p0, i, 0);
        settle(is_plain, s1, i, 1);
        soft(is_plain, s1, p1, i, 1);
        stage_v(i + 1);
        load_v(i + 2);
        look();
        return false;
      }
    };
    // The tiles that need nothing but the pipeline run in a loop of their own,
    // whose sums stay in place; it is left where a reference point has to move
    // or a tile needs masks.
    int i = 0;
    take_scales(0);
    scores(s0, 0, 0);
    while (true) {
      if (plain) {
        enum { kFirst, kSecond, kTile } left = kTile;
        while (true) {
          if (half0(yes, i)) {
            left = kFirst;
            break;
          }
          if (half1(yes, i)) {
            left = kSecond;
            break;
          }
          if (++i >= tiles) break;
          take_scales(i);
          if (!plain) break;
        }
        if (i >= tiles) break;
        if (left == kTile) continue;
        if (left == kFirst) {
          settle(yes, s0, i, 0);
          soft(yes, s0, p0, i, 0);
          if (half1(yes, i)) left = kSecond;
        }
        if (left == kSecond) {
          settle(yes, s1, i, 1);
          soft(yes, s1, p1, i, 1);
        }
      } else {
        half0(no, i);
        half1(no, i);
      }
      if (++i >= tiles) break;
      take_scales(i);
    }
    values(p1, tiles - 1, 1);
  }

  const bool direct = p.splits == 1;
  const float both = l + __shfl_xor(l, 32, 64);
  // (sums of a row that sees nothing)
  const float sum = sees_nothing<M>(p, col_row, col_s, col_e) ? 0.f : both;
  const int64_t slot = (((int64_t)unit * p.tiles + tile) * c.kv_heads + h) * p.splits * COLS +
                       (int64_t)split * COLS + at_col;
  asm("" : "+v"(at_col));  // (the row and head are computed anew, not kept in the loop)
  const int col = tile * COLS + at_col;
  if (col >= columns) return;
  const int row = unit * p.R + col / p.group, head = h * p.group + col % p.group;
  if (hh == 0) {
    if (!direct) {
      p.part_ml[2 * slot] = m;
      p.part_ml[2 * slot + 1] = sum;
    } else if (p.lse) {
      p.lse[(int64_t)row * p.heads + head] =
          sum == 0.f ? -__builtin_inff() : (m - kBias) * kLn2 + __builtin_logf(sum);
    }
  }
  // score row x of product d's sums is row 32 d + x of the staged values: four
  // neighbouring columns are in DT products (and halves of them)
  const float by = direct ? 1.f / kUp / sum : 1.f / kUp;
#pragma unroll
  for (int e = 0; e < 4 * DT; ++e) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = sum == 0.f ? 0.f : (DT == 4 ? acc[j][e] : acc[j >> 1][e + 8 * (j & 1)]) * by;
    const int at = 4 * (8 * (e >> 2) + 4 * hh + (e & 3));
    if (direct) {
      const uint32_t x = to_type(v[0], T) | (uint32_t)to_type(v[1], T) << 16;
      const uint32_t y = to_type(v[2], T) | (uint32_t)to_type(v[3], T) << 16;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) +
                                ((int64_t)row * p.heads + head) * D + at) = uint2{x, y};
    } else {
      *reinterpret_cast<float4*>(p.part_o + slot * D + at) = float4{v[0], v[1], v[2], v[3]};
    }
  }
}

template <int M, int T, int C, int D>
void launch_wide(const AttendParams& p, dim3 grid, hipStream_t s) {
  if (p.cols == 128) attend_wide_kernel<M, T, C, D, 4><<<grid, 256, 0, s>>>(p);
  // (windows and trees of heads of 64 are not planned on 256 columns)
  if constexpr (M == kRange || D == 128)
    if (p.cols == 256) attend_wide_kernel<M, T, C, D, 8><<<grid, 512, 0, s>>>(p);
}

}  // namespace

template <int M>
void attend_wide(const AttendParams& p, dim3 grid, hipStream_t s) {
  dispatch(p, [&](auto t, auto c, auto d) { launch_wide<M, t.value, c.value, d.value>(p, grid, s); });
}

}  // namespace mqa
