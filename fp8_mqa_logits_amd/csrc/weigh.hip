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

// The sum of 16 neighbouring lanes' values, in all of them.
__device__ __forceinline__ float sum16(float x) {
  auto add = [&](auto control) {
    x += __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(x), control.value, 0xF, 0xF, false));
  };
  add(std::integral_constant<int, 0xB1>{});   // lane ^ 1
  add(std::integral_constant<int, 0x4E>{});   // lane ^ 2
  add(std::integral_constant<int, 0x141>{});  // the other four of eight
  add(std::integral_constant<int, 0x140>{});  // the other eight
  return x;
}

// Few columns: a wave takes 64 keys, head by head, in the layout of attend_narrow.h's
// scores: lane (g, n) has those of keys 4 g + i of every 16 and column n. Bound by the
// keys' bytes in long contexts, so that reads of several waves a SIMD are what counts.
// Rows of 32 heads over 32 x 32768 positions of 8 key heads of 128: 198 us, 5.4 TB/s of
// keys (the counters see each of them read from memory once); without the next head's keys
// on their way 226, with 32 keys a wave 243.
// SPLIT: the four waves of a workgroup share the keys, each with every fourth head, and
// are joined through LDS; for calls with too few keys to give every wave its own.
template <int T, int C, int D, bool SPLIT>
__global__ __launch_bounds__(256, 3) void weigh_narrow_kernel(WeighParams p) {
  constexpr int KC = D / 64;  // 16-byte pieces of a key per lane
  constexpr int HW = SPLIT ? 4 : 1, KEYS = SPLIT ? 64 : 256;  // of a workgroup
  const AttendParams& a = p.a;
  const KvCache& c = a.c;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, n = lane & 15;
  const int unit = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles;
  const int columns = a.R * a.group;
  __shared__ float s_part[SPLIT ? 4 : 1][64];

  Span span;
  if (a.R == 1) {
    int s, e;
    row_range(a, unit, s, e);
    span = uniform(s < e ? Span{s, e, s, e, 0, 0} : Span{c.cap, 0, 0, c.cap, 0, 0});
  } else {
    span = uniform(row_span<kRange>(a, unit * a.R, a.R, lane, 64));
  }
  const int first = span.lo & ~15;
  const float cs = a.scale * kLog2e;
  const auto* const table = constant(c.table + (int64_t)unit * c.table_stride);

  for (int at = first + tile * KEYS; at < span.hi; at += p.tiles * KEYS) {
    const int pos0 = SPLIT ? at : at + wave * 64;
    float acc[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = 0.f;
    if (pos0 < span.hi) {
      // 16 keys lie in one page and block: their page and scale are scalars (behind the
      // last position that some row sees: the last ones again, masked)
      const uint8_t* page[4];
      int slot[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int pos = min(pos0 + 16 * b, (span.hi - 1) & ~15);
        page[b] = c.pages + (int64_t)clamp_page(c, table[pos >> c.page_shift]) * c.page_stride;
        slot[b] = pos & ((1 << c.page_shift) - 1);
      }
      const bool clean = pos0 >= span.in_lo && pos0 + 64 <= span.in_hi;
      v4u raw[4][KC], q[2 * KC];
      float f[4], lse;
      auto load_k = [&](int b, int h) {
        const uint8_t* const k = page[b] + code_at(c, 0, h, slot[b]) + n * D + 16 * g;
#pragma unroll
        for (int x = 0; x < KC; ++x) raw[b][x] = *reinterpret_cast<const v4u*>(k + 64 * x);
        f[b] = *constant(reinterpret_cast<const float*>(page[b] + scale_at(c, 0, h, slot[b])));
      };
      auto row_of = [&](int col0) {
        return unit * a.R + (col0 + n < columns ? (col0 + n) / a.group : 0);
      };
      auto load_q = [&](int h, int col0) {
        const int row = row_of(col0);
        const int head = h * a.group + (col0 + n < columns ? (col0 + n) % a.group : 0);
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + row * a.q_row + head * a.q_head;
#pragma unroll
        for (int k = 0; k < 2 * KC; ++k)
          q[k] = *reinterpret_cast<const v4u*>(src + 64 * (k >> 1) + 16 * g + 8 * (k & 1));
        lse = p.lse[(int64_t)row * a.heads + head];
      };
      // a head's keys against 16 columns; what is read next takes the registers as soon as
      // they are free: the next columns, or the next head's keys and first columns
      auto step = [&](auto is_last, int h, int col0) {
        const float to = lse * kLog2e, by = lacking(lse, to);
        int s, e;
        row_range(a, row_of(col0), s, e);
        const uint32_t adds =
            col0 + n < columns && s < e && lse != -__builtin_inff() ? ~0u : 0u;
        const int h_next = min(h + HW, c.kv_heads - 1);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float by_block = f[b] * cs;
          v4f x = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < KC; ++k) {
            x = mfma<T>(widen8<T, C>(raw[b][k][0], raw[b][k][1]), q[2 * k], x);
            x = mfma<T>(widen8<T, C>(raw[b][k][2], raw[b][k][3]), q[2 * k + 1], x);
          }
          if (is_last.value) load_k(b, h_next);
          if (b == 3) load_q(is_last.value ? h_next : h, is_last.value ? 0 : col0 + 16);
          const uint32_t sees = clean ? adds : adds & (seen_bits(pos0 + 16 * b, s, e) >> (4 * g));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], by_block, -to)) * by;
            acc[4 * b + i] += or_zero(w, bit(sees, i));
          }
        }
      };
      const int h0 = SPLIT ? wave : 0;
      if (h0 < c.kv_heads) {
#pragma unroll
        for (int b = 0; b < 4; ++b) load_k(b, h0);
        load_q(h0, 0);
      }
      for (int h = h0; h < c.kv_heads; h += HW) {
        int col0 = 0;
        for (; col0 + 16 < columns; col0 += 16) step(std::false_type{}, h, col0);
        step(std::true_type{}, h, col0);
      }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = sum16(acc[j]);
    float* const weights = p.weights + (int64_t)unit * p.width;
    auto put = [&](int key, float sum) {
      const int pos = pos0 + key;
      if (pos >= span.lo && pos < span.hi && pos < p.width) weights[pos] += sum;
    };
    if constexpr (SPLIT) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (n == j) s_part[wave][16 * (j >> 2) + 4 * g + (j & 3)] = acc[j];
      __syncthreads();
      if (wave == 0)
        put(lane, s_part[0][lane] + s_part[1][lane] + s_part[2][lane] + s_part[3][lane]);
      __syncthreads();
    } else {
      // lane (g, n): key 16 (n / 4) + 4 g + n % 4
      float sum = acc[0];
#pragma unroll
      for (int j = 1; j < 16; ++j) sum = n == j ? acc[j] : sum;
      put(16 * (n >> 2) + 4 * g + (n & 3), sum);
    }
  }
}

// Many columns. A column here is a row of one query head; a tile is 32 rows of a head
// (the last ones repeated), and a stage two tiles of one key head's query heads (the last
// one may be empty). weigh_columns_kernel lays out what all keys meet, stage by stage:
// the queries, what the exponentials take of a column, and what a tile sees; and how a
// request's work is cut: its stages into shares so that about p.tiles workgroups have
// work, whatever its span turns out to be.
template <int D>
__global__ __launch_bounds__(256) void weigh_columns_kernel(WeighParams p, int blocks) {
  const AttendParams& a = p.a;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per_head = (a.group * p.row_tiles + 1) / 2;  // stages of a key head
  if ((int)blockIdx.x < a.requests) {
    const int unit = blockIdx.x;
    __shared__ Span s_span[4];
    Span span = row_span<kRange>(a, unit * a.R, a.R, threadIdx.x, 256);
    if (lane == 0) s_span[wave] = span;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < 4; ++w) span = join<kRange>(span, s_span[w]);
    const int first = span.lo & ~15, stages = per_head * a.c.kv_heads;
    const int tiles = span.hi > first ? (span.hi - first + kWeighKeys - 1) / kWeighKeys : 0;
    // shares of a tile for up to kWeighRounds rounds of workgroups, in which a share takes
    // the time of its stages and of a start and an end as long as six
    int shares = 1, best = 0;
    for (int k = 1; k <= kWeighRounds && tiles > 0; ++k) {
      const int n = min(max(k * p.tiles / tiles, 1), stages);
      const int cost = (tiles * n + p.tiles - 1) / p.tiles * ((stages + n - 1) / n + 6);
      if (k > 1 && cost >= best) continue;
      best = cost;
      shares = n;
    }
    p.cut[2 * unit] = int4{first, tiles, shares, 0};
    p.cut[2 * unit + 1] = int4{span.lo, span.hi, 0, 0};
    return;
  }
  const int64_t tiles = (int64_t)a.requests * a.c.kv_heads * per_head * 2;
  for (int64_t x = (int64_t)(blockIdx.x - a.requests) * 4 + wave; x < tiles;
       x += (int64_t)blocks * 4) {
    const int y = (int)(x % (per_head * 2));
    const int64_t key_head = x / (per_head * 2);  // of all requests
    const int unit = (int)(key_head / a.c.kv_heads);
    const bool real = y < a.group * p.row_tiles;
    const int head = (int)(key_head % a.c.kv_heads) * a.group + (real ? y / p.row_tiles : 0);
    const int row0 = real ? y % p.row_tiles * 32 : 0;
    const uint16_t* const q = static_cast<const uint16_t*>(a.q) + head * a.q_head;
    v4u* const to_q = reinterpret_cast<v4u*>(p.queries + x * (32 * D));
#pragma unroll
    for (int r = 0; r < 32 * D / 8 / 64; ++r) {
      const int piece = lane + 64 * r;
      const int row = unit * a.R + min(row0 + piece / (D / 8), a.R - 1);
      to_q[piece] = *reinterpret_cast<const v4u*>(q + row * a.q_row + piece % (D / 8) * 8);
    }
    const int at = row0 + (lane & 31), row = unit * a.R + min(at, a.R - 1);
    const float lse = p.lse[(int64_t)row * a.heads + head];
    int s, e;
    row_range(a, row, s, e);
    const bool adds = real && at < a.R && s < e && lse != -__builtin_inff();
    const float to = lse * kLog2e;
    if (lane < 32)
      p.columns[x * 32 + lane] = adds ? float2{to, lacking(lse, to)} : float2{0.f, 0.f};
    int4 m{adds ? s : a.c.cap, adds ? e : 0, adds ? s : a.c.cap, adds ? e : 0};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      m.x = max(m.x, __shfl_xor(m.x, o, 64));
      m.y = min(m.y, __shfl_xor(m.y, o, 64));
      m.z = min(m.z, __shfl_xor(m.z, o, 64));
      m.w = max(m.w, __shfl_xor(m.w, o, 64));
    }
    if (lane == 0) p.sight[x] = m;
  }
}

// Zeros made here and now: a vector of them would be kept in registers through all loops.
__device__ __forceinline__ v16f fresh_zeros() {
  v16f z;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float x;
    asm volatile("v_mov_b32 %0, 0" : "=v"(x));
    z[e] = x;
  }
  return z;
}

// The lane's number, formed anew: addresses made of it are not kept (and spilled).
__device__ __forceinline__ int lane_again() {
  int lane;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(lane));
  return lane;
}

// A wave holds 64 keys of one key head, widened, in registers as the first operand of
// v_mfma_f32_32x32x16, 512 keys a workgroup. Queries pass through LDS, two tiles of
// columns a stage, so that what is staged meets 512 keys and a wave's traffic per 64 keys
// x 32 columns is one read of the columns from LDS. A workgroup goes from head to head
// in its share of the columns with the same sums; weigh_join_kernel adds the shares up.
//
// A unit: 32 keys x 32 columns. The products of one unit and the exponentials of the one
// before it are independent, so that the matrix and the vector unit work at the same
// time; `late` are the scores whose exponentials are still to be taken. Stages that some
// column sees in part are done unit by unit, with masks.
//
// 2048 rows of 32 heads over 32768 positions of 8 key heads: 552 us with the two small
// launches beside it (9 and 5 us), 0.97 PFLOP/s; by the counters the matrix unit is busy
// 46% of the cycles, vector instructions take 49% or more at four cycles each (exponentials need twice
// that), and two waves per SIMD overlap them in part. When it took 605 us it took 570
// without exponentials and 476 without most products. Steps on the way: keys of a narrow
// workgroup against all columns 2015 us; this layout, a stage's products, then its
// exponentials 742; one unit's products beside another's exponentials 632; in an order
// that alternates them 605; queries laid out beforehand 572; addresses formed anew instead
// of reloaded from scratch 556.
template <int T, int C, int D>
__global__ __launch_bounds__(512, 2) void weigh_wide_kernel(WeighParams p) {
  constexpr int KS = D / 16, COLS = 64, QROW = 2 * D + 16;
  constexpr int EACH = COLS * D / 8 / 512;  // pieces of 8 elements a thread stages
  const AttendParams& a = p.a;
  const KvCache& c = a.c;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int hh = lane >> 5, n = lane & 31;
  const int request = blockIdx.x / p.tiles, g0 = blockIdx.x % p.tiles;
  const int unit_row = request * a.R;
  __shared__ __align__(16) uint8_t s_q[2][COLS * QROW];

  const int4 cut = p.cut[2 * request];
  const int first = __builtin_amdgcn_readfirstlane(cut.x);
  const int tiles = __builtin_amdgcn_readfirstlane(cut.y);
  const int shares = __builtin_amdgcn_readfirstlane(cut.z);
  const int hi = __builtin_amdgcn_readfirstlane(p.cut[2 * request + 1].y);
  const int per_head = (a.group * p.row_tiles + 1) / 2, all = per_head * c.kv_heads;
  const int share = (all + shares - 1) / shares;
  const float cs = a.scale * kLog2e;
  const int32_t* const table = c.table + (int64_t)request * c.table_stride;
  // what lies behind a request's last stage is read (and not used): the workspace goes on
  const v4u* const queries =
      reinterpret_cast<const v4u*>(p.queries + (int64_t)request * all * (COLS * D));
  const float2* const columns = p.columns + (int64_t)request * all * COLS;
  const int* const sight = reinterpret_cast<const int*>(p.sight + (int64_t)request * all * 2);

  v4u q_reg[EACH];
  auto load = [&](int x) {
#pragma unroll
    for (int r = 0; r < EACH; ++r) q_reg[r] = (queries + (int64_t)x * (COLS * D / 8) + 512 * r)[t];
  };
  auto stage = [&](int buf) {
    const int piece = wave * 64 + lane_again();
    uint8_t* const to = s_q[buf] + piece / (D / 8) * QROW + piece % (D / 8) * 16;
#pragma unroll
    for (int r = 0; r < EACH; ++r)
      *reinterpret_cast<v4u*>(to + 512 * r / (D / 8) * QROW) = q_reg[r];
  };
  // of a stage: its lane's column of either tile, and in lanes 0 .. 7 what its tiles see
  struct Known {
    float2 col[2];
    int sight;
  };
  auto know = [&](int x) {
    const float2* const at = columns + (int64_t)x * COLS;
    return Known{{at[n], (at + 32)[n]}, (sight + (int64_t)x * 8)[lane & 7]};
  };

  int count = 0;  // of stages: which buffer
  for (int item = g0; item < tiles * shares; item += p.tiles) {
    const int x_lo = item / tiles * share, x_hi = min(x_lo + share, all);
    const int pos0 = first + item % tiles * kWeighKeys + wave * 64;
    v16f acc[2] = {fresh_zeros(), fresh_zeros()};
    v4u kf[2][KS];
    float f[2][2];
    // piece k of this lane's operands of a tile of columns
    v4u q[KS];
    const uint8_t* q_from;
    auto take_from = [&](int buf, int sub) {
      const int l = lane_again();
      q_from = s_q[buf] + (32 * sub + (l & 31)) * QROW + (l & 32);
    };
    auto take = [&](int k) {
      q[k] = *reinterpret_cast<const v4u*>(q_from + 64 * (k >> 1) + 16 * (k & 1));
    };
    // The products of a unit, s = keys b x q, one at a time, each beside a part of the
    // exponentials of another, pb and pc's keys and column, in the order written (the
    // compiler's own puts products behind products: 632 us for those 2048 rows, 605 in this
    // one). `beside` comes after product k.
    auto unit = [&](v16f& s, int b, const v16f& prev, int pb, const float* pf, const float2& pc,
                    auto beside) {
      constexpr int E = 16 / KS;
      float arg[E], ex[E];
#pragma unroll
      for (int i = 0; i < E; ++i) arg[i] = __builtin_fmaf(prev[i], pf[0], -pc.x);
#pragma unroll
      for (int k = 0; k <= KS; ++k) {
        __builtin_amdgcn_sched_barrier(0);
        if (k < KS) {
          s = mfma32<T>(kf[b][k], q[k], k ? s : v16f{});
          beside(k);
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
          if (k > 0) {
            const int e = (k - 1) * E + i;
            float sum = __builtin_fmaf(ex[i], pc.y, acc[pb][e]);
            asm volatile("" : "+v"(sum));  // (used behind a branch only: it would go there)
            acc[pb][e] = sum;
          }
          if (k < KS) ex[i] = __builtin_amdgcn_exp2f(arg[i]);
          if (k + 1 < KS) {
            const int e = (k + 1) * E + i;
            arg[i] = __builtin_fmaf(prev[e], pf[e >> 3], -pc.x);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto nothing = [](int) {};
    if (x_lo >= x_hi) continue;  // (the join reads no such share)
    load(x_lo);
    stage(count & 1);
    load(x_lo + 1);
    Known known = know(x_lo);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      if (k == 0) take_from(count & 1, 0);
      take(k);
    }
    int x = x_lo;
    Known then;
    auto begin = [&]() {  // of a stage: the next one on its way
      then = know(x + 1);
      stage(~count & 1);  // (the other buffer was last read before the last barrier)
      load(x + 2);
    };
    auto end = [&]() {
      known = then;
      ++x;
      ++count;
    };
    auto word = [&](int i) { return __builtin_amdgcn_readlane(known.sight, i); };
    auto plain = [&]() {  // every column sees every key
      return max(word(0), word(4)) <= pos0 && min(word(1), word(5)) >= pos0 + 64;
    };
    int head_end = x_lo;  // the stage where another key head begins
    while (x < x_hi) {
      if (x == head_end) {
        const int at_head = x / per_head;
        head_end = (at_head + 1) * per_head;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int pos = min(pos0 + 32 * b + n, ((hi - 1) & ~15) + (n & 15));
          const uint8_t* const page =
              c.pages + (int64_t)clamp_page(c, table[pos >> c.page_shift]) * c.page_stride;
          const int slot = pos & ((1 << c.page_shift) - 1);
#pragma unroll
          for (int j = 0; j < KS / 2; ++j) {
            const v4u raw = *reinterpret_cast<const v4u*>(page + code_at(c, 0, at_head, slot) +
                                                          16 * (2 * j + hh));
            kf[b][2 * j] = widen8<T, C>(raw[0], raw[1]);
            kf[b][2 * j + 1] = widen8<T, C>(raw[2], raw[3]);
          }
          const float scale =
              *reinterpret_cast<const float*>(page + scale_at(c, 0, at_head, slot)) * cs;
          f[b][0] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scale), 0));
          f[b][1] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scale), 16));
          __builtin_amdgcn_sched_barrier(0);  // (registers are few)
        }
      }
      if (plain()) {
        // a loop of its own, whose sums stay in place; `late`: the scores whose
        // exponentials are still to be taken (at first none: a factor of 0)
        v16f late = fresh_zeros();
        float2 last{0.f, 0.f};
        float late_f[2] = {0.f, 0.f};
        do {
          const int buf = count & 1;
          v16f s0, s1;
          begin();
          unit(s0, 0, late, 1, late_f, last, nothing);
          unit(s1, 1, s0, 0, f[0], known.col[0], [&](int k) {
            if (k == 0) take_from(buf, 1);
            take(k);
          });
          unit(s0, 0, s1, 1, f[1], known.col[0], nothing);
          __syncthreads();
          unit(late, 1, s0, 0, f[0], known.col[1], [&](int k) {
            if (k == 0) take_from(buf ^ 1, 0);
            take(k);
          });
          last = known.col[1];
          late_f[0] = f[1][0];
          late_f[1] = f[1][1];
          end();
        } while (x < min(x_hi, head_end) && plain());
#pragma unroll
        for (int e = 0; e < 16; ++e)
          acc[1][e] = __builtin_fmaf(
              __builtin_amdgcn_exp2f(__builtin_fmaf(late[e], late_f[e >> 3], -last.x)), last.y,
              acc[1][e]);
        continue;
      }
      const int buf = count & 1;
      begin();
#pragma unroll 1
      for (int sub = 0; sub < 2; ++sub) {
        if (sub) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            if (k == 0) take_from(buf, 1);
            take(k);
          }
        }
        if (word(4 * sub + 3) <= pos0 || word(4 * sub + 2) >= pos0 + 64) continue;
        const float2 col = sub ? known.col[1] : known.col[0];
        int column = n, s, e;
        asm("" : "+v"(column));  // (nothing of this is kept in the other loop)
        const int at = (x % per_head * 2 + sub) % p.row_tiles * 32 + column;
        row_range(a, unit_row + min(at, a.R - 1), s, e);
        if (at >= a.R || col.y == 0.f) s = e = 0;  // (adds nothing)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint32_t sees = seen_bits(pos0 + 32 * b, s, e) >> (4 * hh);
          v16f score = v16f{};
#pragma unroll
          for (int k = 0; k < KS; ++k) score = mfma32<T>(kf[b][k], q[k], score);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float w =
                __builtin_amdgcn_exp2f(__builtin_fmaf(score[i], f[b][i >> 3], -col.x));
            acc[b][i] += or_zero(w * col.y, bit(sees, 8 * (i >> 2) + (i & 3)));
          }
        }
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        if (k == 0) take_from(buf ^ 1, 0);
        take(k);
      }
      end();
    }
    float* const part = p.part + ((int64_t)request * p.slots + item) * kWeighKeys + wave * 64;
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
  const int all = (p.a.group * p.row_tiles + 1) / 2 * p.a.c.kv_heads;  // stages
  const int share = (all + cut.z - 1) / cut.z, shares = (all + share - 1) / share;
  for (int pos = cut.x + (blockIdx.x % blocks) * 256 + (int)threadIdx.x; pos < end;
       pos += blocks * 256) {
    if (pos < span.x) continue;
    const float* part = p.part + (int64_t)unit * p.slots * kWeighKeys + (pos - cut.x);
    float sum = 0.f;
    for (int s = 0; s < shares; ++s) sum += part[(int64_t)s * cut.y * kWeighKeys];
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
      if (p->split)
        weigh_narrow_kernel<t.value, c.value, d.value, true><<<grid, 256, 0, s>>>(*p);
      else
        weigh_narrow_kernel<t.value, c.value, d.value, false><<<grid, 256, 0, s>>>(*p);
    });
    return (int)hipGetLastError();
  }
  const int64_t tiles = (int64_t)p->a.requests * p->a.c.kv_heads *
                        ((p->a.group * (int64_t)p->row_tiles + 1) / 2 * 2);
  const int column_blocks = (int)(tiles < 4 * 4096 ? (tiles + 3) / 4 : 4096);
  dispatch(p->a, [&](auto t, auto c, auto d) {
    weigh_columns_kernel<d.value><<<dim3((unsigned)(p->a.requests + column_blocks)), 256, 0, s>>>(
        *p, column_blocks);
    weigh_wide_kernel<t.value, c.value, d.value><<<grid, 512, 0, s>>>(*p);
  });
  const int cap = p->a.c.cap < p->width ? p->a.c.cap : p->width;
  const int most = (cap + 15 + 255) / 256, want = 2048 / p->a.requests;
  const int blocks = want < 1 ? 1 : want < most ? want : most;
  weigh_join_kernel<<<dim3((unsigned)p->a.requests * blocks), 256, 0, s>>>(*p, blocks);
  return (int)hipGetLastError();
}
