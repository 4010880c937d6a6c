// Attention of query rows over a paged 8-bit key/value cache.
//
//     S_j = scale * ks_j * (q . kc_j)        (kc, vc: codes; ks, vs: block scales)
//     m = max_j S_j,  l = sum_j exp(S_j - m)
//     out = sum_j exp(S_j - m) * vs_j * vc_j / l,   lse = m + ln l
// over the positions j of the row's range, or over its listed positions.
//
// Numbers. Codes of either kind are exact in bf16 and in fp16, so q . kc runs
// on the matrix unit in q's own type with fp32 sums, and the scales come in
// afterwards, in fp32. The probabilities go to the second product in fp16
// whatever q's type (11 bits; bf16's 8 would add an error as large as the
// rounding of a bf16 output), as P = 2^7 exp2(S' - m) vs / vref with S' in
// units of ln 2 and vref the largest value scale met so far: at most 2^15, and
// full precision down to 2^-21 of the row's largest. Reference points move
// lazily: m only when a score passes it by more than 8 (P <= 2^15 until then),
// vref when a larger scale is met; both times the sums are rescaled. l sums the
// fp32 P before its rounding.
#include <type_traits>

#include "attend.h"
#include "launch.h"

namespace mqa {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.4028234e38f;  // m of a column that has seen nothing
constexpr float kLag = 8.f;                // how far scores may pass m
constexpr float kBias = 7.f;               // P = 2^kBias at a score of m
constexpr uint32_t kNone = ~0u;            // token of a key that no row sees

// 4 codes of one dword -> 4 values of the matrix unit's type.
template <int T, int C>
__device__ __forceinline__ uint2 widen4(uint32_t w) {
  if constexpr (C == kE4m3) {
    if constexpr (T == kBf16) {
      return uint2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.f, true))};
    } else {
      return uint2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.f, true))};
    }
  } else if constexpr (T == kBf16) {
    const v2bf a{(__bf16)(float)(int8_t)w, (__bf16)(float)(int8_t)(w >> 8)};
    const v2bf b{(__bf16)(float)(int8_t)(w >> 16), (__bf16)(float)(int8_t)(w >> 24)};
    return uint2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
  } else {
    // the byte as the low mantissa bits of 1024 + (code + 128), exact in fp16
    w ^= 0x80808080u;
    const v2h off{(_Float16)-1152.f, (_Float16)-1152.f};
    const v2h a = __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) + off;
    const v2h b = __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) + off;
    return uint2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
  }
}

template <int T, int C>
__device__ __forceinline__ v4u widen8(uint32_t lo, uint32_t hi) {
  const uint2 a = widen4<T, C>(lo), b = widen4<T, C>(hi);
  return v4u{a.x, a.y, b.x, b.y};
}

template <int T>
__device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
  if constexpr (T == kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

template <int T>
__device__ __forceinline__ v16f mfma32(v4u a, v4u b, v16f c) {
  if constexpr (T == kBf16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Bytes w[i] of four dwords (rows) -> t[b] = bytes b of the four rows.
__device__ __forceinline__ void transpose4(const uint32_t* w, uint32_t* t) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u);  // w0.0 w1.0 w0.1 w1.1
  const uint32_t b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
  const uint32_t d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  t[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  t[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  t[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  t[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// 0xFF in each byte of w that is an e4m3 NaN (0x7F or 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  const uint32_t t = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return (t >> 7) * 0xFFu;
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) x = __builtin_fmaxf(x, __shfl_xor(x, o, 64));
  return x;
}

__device__ __forceinline__ uint16_t to_type(float x, int type) {
  return type == kBf16 ? __builtin_bit_cast(uint16_t, (__bf16)x)
                       : __builtin_bit_cast(uint16_t, (_Float16)x);
}

// A row's range, clamped as the contract says.
__device__ __forceinline__ void row_range(const AttendParams& p, int row, int& s, int& e) {
  s = p.starts[row];
  e = p.ends[row];
  s = s < 0 ? 0 : (s > p.c.cap ? p.c.cap : s);
  e = e < s ? s : (e > p.c.cap ? p.c.cap : e);
}

// Slot of a request's position in the pool: page * page_size + slot.
__device__ __forceinline__ uint32_t token_of(const KvCache& c, int request, int pos) {
  int page = c.table[(int64_t)request * c.table_stride + (pos >> c.page_shift)];
  page = page < 0 ? 0 : (page >= c.num_pages ? c.num_pages - 1 : page);
  return ((uint32_t)page << c.page_shift) + (uint32_t)(pos & ((1 << c.page_shift) - 1));
}

// ---------------------------------------------------------------------------
// Few columns. A column is a (row, query head) pair; the columns of one
// request and key head see the same keys and share a workgroup, 16 NT of them
// at most (lists: the heads of one row). The keys are split over the
// workgroup's four waves and over p.splits workgroups, 32 at a time.
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
// Nothing passes through LDS but a key's token and scales. The tokens are
// looked up two steps ahead, the codes are loaded one step ahead.
//
// Bound by the cache's bytes for few heads a key head, by the two widenings
// for many.
template <int T, int C, int D, int NT, bool LIST>
__global__ __launch_bounds__(256, NT == 4 ? 1 : 2) void attend_narrow_kernel(AttendParams p) {
  constexpr int KC = D / 64;       // 16-byte pieces of a key per lane
  constexpr int U = D / 16;        // products per step and column tile
  constexpr int VW = D / 64;       // dwords of a value per lane
  constexpr int COLS = 16 * NT;
  constexpr int US = U < 8 / NT ? U : 8 / NT;  // products merged per round
  const KvCache& c = p.c;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, n = lane & 15;
  const int64_t block = p.block0 + blockIdx.x;
  const int split = (int)(block % p.splits);
  const int64_t item = block / p.splits;
  const int h = (int)(item % c.kv_heads), tile = (int)(item / c.kv_heads % p.tiles);
  const int unit = (int)(item / c.kv_heads / p.tiles);  // the request, or the row of a list
  const int per_unit = LIST ? 1 : p.R;
  const int request = LIST ? unit / p.R : unit;
  const int columns = per_unit * p.group;        // of the unit

  __shared__ __align__(16) uint32_t s_tok[4][2][32];
  __shared__ __align__(16) float s_ks[4][32], s_vs[4][32];
  __shared__ float s_part[4][US * 16][COLS];
  __shared__ float s_m[4][COLS], s_l[4][COLS];

  // this lane's columns and the tile's range of positions
  const int row_lo = unit * per_unit + tile * COLS / p.group;
  const int last = tile * COLS + COLS < columns ? tile * COLS + COLS : columns;
  const int row_hi = unit * per_unit + (last - 1) / p.group;
  int lo, hi, in_lo, in_hi;  // seen by some row, seen by every row
  {
    const int r = row_lo + lane <= row_hi ? row_lo + lane : row_hi;  // at most COLS rows
    row_range(p, r, in_lo, in_hi);
    const bool some = in_lo < in_hi;  // (rows that see nothing are left out)
    lo = some ? in_lo : c.cap;
    hi = some ? in_hi : 0;
    in_lo = some ? in_lo : 0;
    in_hi = some ? in_hi : c.cap;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      lo = min(lo, __shfl_xor(lo, o, 64));
      hi = max(hi, __shfl_xor(hi, o, 64));
      in_lo = max(in_lo, __shfl_xor(in_lo, o, 64));
      in_hi = min(in_hi, __shfl_xor(in_hi, o, 64));
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    in_lo = __builtin_amdgcn_readfirstlane(in_lo);
    in_hi = __builtin_amdgcn_readfirstlane(in_hi);
  }
  int col_s[NT], col_e[NT];
  v4u q[NT][2 * KC];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int col = tile * COLS + 16 * t + n;
    const bool real = col < columns;
    const int row = unit * per_unit + (real ? col / p.group : 0);
    const int head = h * p.group + (real ? col % p.group : 0);
    row_range(p, row, col_s[t], col_e[t]);
    const uint16_t* src = static_cast<const uint16_t*>(p.q) + row * p.q_row + head * p.q_head;
#pragma unroll
    for (int k = 0; k < 2 * KC; ++k) {
      q[t][k] = *reinterpret_cast<const v4u*>(src + 64 * (k >> 1) + 16 * g + 8 * (k & 1));
      if (!real) q[t][k] = v4u{0, 0, 0, 0};
    }
  }
  // the part of the keys (list entries) that this workgroup takes, in steps
  // of 32 from a multiple of 16, so that a half step lies in one block
  const int first = LIST ? 0 : lo & ~15;
  const int end = LIST ? p.width : hi;
  const int steps = end > first ? (end - first + 31) / 32 : 0;
  const int per_split = ((steps + p.splits - 1) / p.splits + 3) & ~3;
  const int step_lo = split * per_split + wave;
  const int step_hi = steps < (split + 1) * per_split ? steps : (split + 1) * per_split;

  const float cs = p.scale * kLog2e;
  float m[NT], l[NT], vref = 0.f;
  v4f acc[NT][U];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = kLowest;
    l[t] = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) acc[t][u] = v4f{0.f, 0.f, 0.f, 0.f};
  }

  // a key's token (kNone: no row sees it); lanes 32.. repeat lanes 0..31
  auto listed = [&](int st) {
    if constexpr (LIST) {
      const int at = st * 32 + (lane & 31);
      return st < step_hi && at < p.width ? p.indices[(int64_t)unit * p.width + at] : -1;
    } else {
      return 0;
    }
  };
  auto token = [&](int st, int x) -> uint32_t {
    int pos;
    if constexpr (LIST) {
      if (x < 0 || x >= col_e[0] - col_s[0]) return kNone;
      pos = col_s[0] + x;
    } else {
      pos = first + st * 32 + (lane & 31);
      if (st >= step_hi || pos < lo || pos >= hi) return kNone;
    }
    return token_of(c, request, pos);
  };
  const uint8_t* const kbase = c.pages + code_at(c, 0, h, 0);
  const uint8_t* const vbase = c.pages + code_at(c, 1, h, 0);
  const uint32_t slot_mask = (1u << c.page_shift) - 1;
  auto code_offset = [&](uint32_t tok) -> int64_t {
    tok = tok == kNone ? 0u : tok;
    return (int64_t)(tok >> c.page_shift) * c.page_stride + (tok & slot_mask) * D;
  };
  struct Step {
    v4u k[2][KC];
    uint32_t v[8][VW];
    float ks, vs;   // of key lane % 32
    uint32_t tok;   // of key lane % 32
  };
  auto load = [&](Step& s, uint32_t tok, int buf) {
    s.tok = tok;
    s_tok[wave][buf][lane & 31] = tok;
    __builtin_amdgcn_wave_barrier();
    const uint32_t t0 = tok == kNone ? 0u : tok;
    const uint8_t* page = c.pages + (int64_t)(t0 >> c.page_shift) * c.page_stride;
    s.ks = *reinterpret_cast<const float*>(page + scale_at(c, 0, h, t0 & slot_mask));
    s.vs = *reinterpret_cast<const float*>(page + scale_at(c, 1, h, t0 & slot_mask));
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint8_t* at = kbase + code_offset(s_tok[wave][buf][16 * b + n]) + 16 * g;
#pragma unroll
      for (int k = 0; k < KC; ++k) s.k[b][k] = *reinterpret_cast<const v4u*>(at + 64 * k);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const v4u four = *reinterpret_cast<const v4u*>(&s_tok[wave][buf][16 * b + 4 * g]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* at = vbase + code_offset(four[i]) + 4 * VW * n;
        if constexpr (VW == 2) {
          const uint2 x = *reinterpret_cast<const uint2*>(at);
          s.v[4 * b + i][0] = x.x;
          s.v[4 * b + i][1] = x.y;
        } else {
          s.v[4 * b + i][0] = *reinterpret_cast<const uint32_t*>(at);
        }
      }
    }
  };

  auto compute = [&](Step& s, int st, int buf) {
    const bool valid = s.tok != kNone;
    s_ks[wave][lane & 31] = s.ks * cs;
    s_vs[wave][lane & 31] = s.vs;
    __builtin_amdgcn_wave_barrier();
    const int pos0 = first + st * 32;
    const bool clean = __all(valid) && (LIST || (pos0 >= in_lo && pos0 + 32 <= in_hi));
    if (__any(valid && s.vs > vref && s.vs < __builtin_inff())) {
      const float r =  // (at least the least normal number, whose inverse is one)
          __builtin_fmaxf(wave_max(valid && s.vs < __builtin_inff() ? s.vs : 0.f), 0x1p-126f);
      const float keep = vref / r;
      vref = r;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < U; ++u) acc[t][u] *= keep;
    }
    v4f x[NT][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      v4u kf[2 * KC];
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        kf[2 * k] = widen8<T, C>(s.k[b][k][0], s.k[b][k][1]);
        kf[2 * k + 1] = widen8<T, C>(s.k[b][k][2], s.k[b][k][3]);
      }
      const v4f f = *reinterpret_cast<const v4f*>(&s_ks[wave][16 * b + 4 * g]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        v4f a{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2 * KC; ++k) a = mfma<T>(kf[k], q[t][k], a);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[t][b][i] = a[i] * f[i];
      }
    }
    const float inv = vref > 0.f ? 1.f / vref : 0.f;
    v4f vr[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      vr[b] = *reinterpret_cast<const v4f*>(&s_vs[wave][16 * b + 4 * g]);
#pragma unroll
      for (int i = 0; i < 4; ++i) vr[b][i] *= inv;
    }
    uint32_t seen[NT];  // bit 4 b + i
    uint32_t poison = 0;
    if (!clean) {
      uint32_t live = 0;  // keys that some row sees
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const v4u four = *reinterpret_cast<const v4u*>(&s_tok[wave][buf][16 * b + 4 * g]);
#pragma unroll
        for (int i = 0; i < 4; ++i) live |= (four[i] != kNone ? 1u : 0u) << (4 * b + i);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        seen[t] = live;
        if constexpr (!LIST) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int pos = pos0 + 16 * (j >> 2) + 4 * g + (j & 3);
            if (pos < col_s[t] || pos >= col_e[t]) seen[t] &= ~(1u << j);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!(seen[t] >> j & 1)) x[t][j >> 2][j & 3] = -__builtin_inff();
      }
      // values that no row sees become 0; a NaN code, which some rows may
      // see and others not, becomes 0 too and is put back through the P of
      // the rows that see it (0 * NaN would reach the others)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t bad = 0;
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          if (!(live >> j & 1)) s.v[j][w] = 0;
          if constexpr (C == kE4m3) {
            const uint32_t b = nan_bytes(s.v[j][w]);
            s.v[j][w] &= ~b;
            bad |= b;
          }
        }
        if constexpr (C == kE4m3) {
          const uint64_t who = __ballot(bad != 0);
          if (who >> (16 * g) & 0xFFFF) poison |= 1u << j;
        }
      }
    }
    v4u pf[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float top = x[t][0][0];
#pragma unroll
      for (int j = 1; j < 8; ++j) top = __builtin_fmaxf(top, x[t][j >> 2][j & 3]);
      if (__any(top > m[t] + kLag)) {
        top = __builtin_fmaxf(top, __shfl_xor(top, 16, 64));
        top = __builtin_fmaxf(top, __shfl_xor(top, 32, 64));
        const float to = __builtin_fmaxf(m[t], top);
        const float keep = __builtin_amdgcn_exp2f(m[t] - to);
        m[t] = to;
        l[t] *= keep;
#pragma unroll
        for (int u = 0; u < U; ++u) acc[t][u] *= keep;
      }
      float pr[8];
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        pr[j] = __builtin_amdgcn_exp2f(x[t][j >> 2][j & 3] - (m[t] - kBias));
        if (!clean && !(seen[t] >> j & 1)) pr[j] = 0.f;
        sum += pr[j];
        pr[j] *= vr[j >> 2][j & 3];
        if (!clean) {
          if (!(seen[t] >> j & 1)) pr[j] = 0.f;
          else if (poison >> j & 1) pr[j] = __builtin_nanf("");
        }
      }
      l[t] += sum;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pf[t][i] = __builtin_bit_cast(uint32_t, v2h{(_Float16)pr[2 * i], (_Float16)pr[2 * i + 1]});
    }
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      uint32_t in[4], a[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) in[j] = s.v[j][w];
      transpose4(in, a);
#pragma unroll
      for (int j = 0; j < 4; ++j) in[j] = s.v[4 + j][w];
      transpose4(in, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const v4u vf = widen8<kFp16, C>(a[i], b[i]);
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t][4 * w + i] = mfma<kFp16>(vf, pf[t], acc[t][4 * w + i]);
      }
    }
  };

  Step s0, s1;
  int st = step_lo;
  if (st < step_hi) {
    uint32_t tok = token(st, listed(st));
    int x = listed(st + 4);
    load(s0, tok, 0);
    tok = token(st + 4, x);
    x = listed(st + 8);
    while (true) {
      load(s1, tok, 1);
      tok = token(st + 8, x);
      x = listed(st + 12);
      compute(s0, st, 0);
      st += 4;
      if (st >= step_hi) break;
      load(s0, tok, 0);
      tok = token(st + 8, x);
      x = listed(st + 12);
      compute(s1, st, 1);
      st += 4;
      if (st >= step_hi) break;
    }
  }

  // the four waves' sums to one reference point, a round of products at a time
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    l[t] += __shfl_xor(l[t], 16, 64);
    l[t] += __shfl_xor(l[t], 32, 64);
    if (col_s[t] >= col_e[t]) l[t] = 0.f;  // sums of a row that sees nothing
    if (g == 0) {
      s_m[wave][16 * t + n] = m[t];
      s_l[wave][16 * t + n] = l[t];
    }
  }
  __syncthreads();
  float part[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float top = kLowest;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = __builtin_fmaxf(top, s_m[w][16 * t + n]);
    part[t] = __builtin_amdgcn_exp2f(m[t] - top) * vref;
  }
  const int col = threadIdx.x % COLS;  // the column this thread writes
  const int at_col = tile * COLS + col;
  float top = kLowest, sum = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) top = __builtin_fmaxf(top, s_m[w][col]);
#pragma unroll
  for (int w = 0; w < 4; ++w) sum += s_l[w][col] * __builtin_amdgcn_exp2f(s_m[w][col] - top);
  const bool real = at_col < columns;
  const int row = unit * per_unit + (real ? at_col / p.group : 0);
  const int head = h * p.group + (real ? at_col % p.group : 0);
  const bool direct = p.splits == 1;
  const float inv = 1.f / sum;
  const int64_t slot = block * COLS + col;
  if (threadIdx.x < COLS) {
    if (direct) {
      if (real && p.lse)
        p.lse[(int64_t)row * p.heads + head] =
            sum == 0.f ? -__builtin_inff() : (top - kBias) * kLn2 + __builtin_logf(sum);
    } else {
      p.part_ml[2 * slot] = top;
      p.part_ml[2 * slot + 1] = sum;
    }
  }
  for (int u0 = 0; u0 < U; u0 += US) {
    if (u0) __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u < u0 || u >= u0 + US) continue;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s_part[wave][(u - u0) * 16 + 4 * g + i][16 * t + n] = acc[t][u][i] * part[t];
    }
    __syncthreads();
    for (int i = threadIdx.x / COLS; i < US * 16; i += 256 / COLS) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) v += s_part[w][i][col];
      const int d = U * (i & 15) + u0 + (i >> 4);
      if (!direct)
        p.part_o[slot * D + d] = v;
      else if (real)
        static_cast<uint16_t*>(p.out)[((int64_t)row * p.heads + head) * D + d] =
            to_type(sum == 0.f ? 0.f : v * inv, T);
    }
  }
}

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
// next barrier. m and vref only move by powers of two, so that the P in flight
// can be rescaled exactly.
template <int T, int C, int D, int W>
__global__ __launch_bounds__(64 * W, 2) void attend_wide_kernel(AttendParams p) {
  constexpr int THREADS = 64 * W;
  constexpr int KS = D / 16;          // products a half's scores take
  constexpr int DT = D / 32;          // tiles of the output's columns
  constexpr int PIECES = 4 * D;       // 16-byte pieces of a tile's keys; 4 x 4 pieces of its values
  constexpr int EACH = (PIECES + THREADS - 1) / THREADS;  // of each, per thread
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
  __shared__ __align__(16) float s_scale[2][THREADS];  // 8 scales, over and over
  __shared__ uint32_t s_poison[3][2];
  __shared__ int s_range[4][W];

  const int row_lo = unit * p.R + tile * COLS / p.group;
  const int last = tile * COLS + COLS < columns ? tile * COLS + COLS : columns;
  const int row_hi = unit * p.R + (last - 1) / p.group;
  int lo = c.cap, hi = 0, in_lo = 0, in_hi = c.cap;  // seen by some row, seen by every row
  for (int r = row_lo + t; r <= row_hi; r += THREADS) {
    int s, e;
    row_range(p, r, s, e);
    if (s < e) {  // (rows that see nothing are left out)
      lo = min(lo, s);
      hi = max(hi, e);
      in_lo = max(in_lo, s);
      in_hi = min(in_hi, e);
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    lo = min(lo, __shfl_xor(lo, o, 64));
    hi = max(hi, __shfl_xor(hi, o, 64));
    in_lo = max(in_lo, __shfl_xor(in_lo, o, 64));
    in_hi = min(in_hi, __shfl_xor(in_hi, o, 64));
  }
  if (lane == 0) {
    s_range[0][wave] = lo;
    s_range[1][wave] = hi;
    s_range[2][wave] = in_lo;
    s_range[3][wave] = in_hi;
  }
  if (t < 6) s_poison[t >> 1][t & 1] = 0;
  // the first half adds no values: P = 0 times what is staged "before" them
  for (int x = t; x < D * VROW / 16; x += THREADS)
    reinterpret_cast<v4u*>(s_v[1])[x] = v4u{0, 0, 0, 0};
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) {
    lo = min(lo, s_range[0][w]);
    hi = max(hi, s_range[1][w]);
    in_lo = max(in_lo, s_range[2][w]);
    in_hi = min(in_hi, s_range[3][w]);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  in_lo = __builtin_amdgcn_readfirstlane(in_lo);
  in_hi = __builtin_amdgcn_readfirstlane(in_hi);

  // this lane's column
  int at_col = wave * 32 + n, col_s, col_e;
  v4u q[KS];
  {
    const int col = tile * COLS + at_col;
    const bool real = col < columns;
    const int row = unit * p.R + (real ? col / p.group : 0);
    const int head = h * p.group + (real ? col % p.group : 0);
    row_range(p, row, col_s, col_e);
    const uint16_t* src = static_cast<const uint16_t*>(p.q) + row * p.q_row + head * p.q_head;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      q[k] = *reinterpret_cast<const v4u*>(src + 16 * k + 8 * hh);
      if (!real) q[k] = v4u{0, 0, 0, 0};
    }
  }

  // the part of the keys that this workgroup takes, in tiles of 64 from a
  // multiple of 16: each group of 16 keys lies in one block
  const int first = lo & ~15;
  const int all = hi > first ? (hi - first + 63) / 64 : 0;
  const int per_split = (all + p.splits - 1) / p.splits;
  const int tile_lo = split * per_split;
  const int tiles = min(all - tile_lo, per_split);
  const int base = first + tile_lo * 64;

  // staging: piece x = t + THREADS r of the keys is 16 bytes of key x / (D /
  // 16); of the values, columns 4 (x % (D / 4)) .. + 3 of keys 4 y .. 4 y + 3,
  // y = x / (D / 4)
  auto piece = [&](int r) { return t + THREADS * r; };
  auto mine = [&](int r) { return PIECES % THREADS == 0 || piece(r) < PIECES; };
  auto k_key = [&](int r) { return piece(r) / (D / 16); };
  auto v_key = [&](int r) { return piece(r) / (D / 4) * 4; };
  auto v_d = [&](int r) { return piece(r) % (D / 4) * 4; };
  // A group of 16 keys that no row sees is read from the nearest one that some
  // row sees (masked later; no branch in the loop). Its table entry is loaded a
  // tile before its use, and only looked at then.
  const int32_t* const table = c.table + (int64_t)unit * c.table_stride;
  auto group_pos = [&](int i, int g) {
    return min(max(base + i * 64 + 16 * g, lo), hi - 1) & ~15;
  };
  auto group_entry = [&](int i, int g) { return table[group_pos(i, g) >> c.page_shift]; };
  auto page_at = [&](int entry) {
    return c.pages + (int64_t)min(max(entry, 0), c.num_pages - 1) * c.page_stride;
  };
  auto slot_of = [&](int i, int key) {
    return (group_pos(i, key >> 4) + (key & 15)) & ((1 << c.page_shift) - 1);
  };
  v4u kreg[EACH];
  uint32_t vreg[EACH][4];
  float sreg = 0.f;
  int kentry[EACH], ventry[EACH], sentry;
  // (of a workgroup with more threads than pieces, the others read piece 0 too)
  auto k_of = [&](int r) { return mine(r) ? k_key(r) : 0; };
  auto v_of = [&](int r) { return mine(r) ? v_key(r) : 0; };
  auto find_k = [&](int i) {
#pragma unroll
    for (int r = 0; r < EACH; ++r) kentry[r] = group_entry(i, k_of(r) >> 4);
    sentry = group_entry(i, t & 3);
  };
  auto find_v = [&](int i) {
#pragma unroll
    for (int r = 0; r < EACH; ++r) ventry[r] = group_entry(i, v_of(r) >> 4);
  };
  auto load_k = [&](int i) {
#pragma unroll
    for (int r = 0; r < EACH; ++r)
      kreg[r] = *reinterpret_cast<const v4u*>(page_at(kentry[r]) +
                                              code_at(c, 0, h, slot_of(i, k_of(r))) +
                                              16 * (piece(r) % (D / 16)));
    sreg = *reinterpret_cast<const float*>(page_at(sentry) +
                                           scale_at(c, t >> 2 & 1, h, slot_of(i, 16 * (t & 3))));
  };
  auto load_v = [&](int i) {
#pragma unroll
    for (int r = 0; r < EACH; ++r) {
      const uint8_t* at = page_at(ventry[r]) + code_at(c, 1, h, slot_of(i, v_of(r))) + v_d(r);
#pragma unroll
      for (int j = 0; j < 4; ++j) vreg[r][j] = *reinterpret_cast<const uint32_t*>(at + j * D);
    }
  };
  auto k_slot = [&](int key, int slot) { return key * KROW + 16 * slot; };
  auto v_slot = [&](int d, int slot) { return d * VROW + 16 * slot; };
  auto inside = [&](int i) {  // every row sees every key of tile i
    return base + i * 64 >= in_lo && base + i * 64 + 64 <= in_hi;
  };
  auto stage_k = [&](int i) {
    uint8_t* const to = s_k[i & 1];
#pragma unroll
    for (int r = 0; r < EACH; ++r) {
      if (!mine(r)) continue;
      const int x = piece(r) % (D / 16);
      *reinterpret_cast<v4u*>(to + k_slot(k_key(r), 2 * x)) = widen8<T, C>(kreg[r][0], kreg[r][1]);
      *reinterpret_cast<v4u*>(to + k_slot(k_key(r), 2 * x + 1)) =
          widen8<T, C>(kreg[r][2], kreg[r][3]);
    }
    s_scale[i & 1][t] = sreg;
  };
  // values that no row sees become 0; a NaN code, which some rows may see and
  // others not, becomes 0 too and is put back through the P of the rows that
  // see it (0 * NaN would reach the others)
  auto clean_v = [&](int i) {
    if (t == 0) s_poison[(i + 1) % 3][0] = s_poison[(i + 1) % 3][1] = 0;
    if (inside(i)) return;
#pragma unroll
    for (int r = 0; r < EACH; ++r) {
      if (!mine(r)) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = v_key(r) + j, pos = base + i * 64 + key;
        if (i >= tiles || pos < lo || pos >= hi) vreg[r][j] = 0;
        if constexpr (C == kE4m3) {
          const uint32_t bad = nan_bytes(vreg[r][j]);
          if (bad) {
            vreg[r][j] &= ~bad;
            atomicOr(&s_poison[i % 3][key >> 5], 1u << (key & 31));
          }
        }
      }
    }
  };
  // keys 16 g + {0..3, 8..11} share slot 2 g, {4..7, 12..15} slot 2 g + 1
  auto stage_v = [&](int i) {
#pragma unroll
    for (int r = 0; r < EACH; ++r) {
      if (!mine(r)) continue;
      uint32_t a[4];
      transpose4(vreg[r], a);
      const int y = v_key(r) >> 2, slot = 2 * (y >> 2) + (y & 1), half = y >> 1 & 1;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint2*>(s_v[i & 1] + v_slot(v_d(r) + j, slot) + 8 * half) =
            widen4<kFp16, C>(a[j]);
    }
  };

  const float cs = p.scale * kLog2e;
  float m = kLowest, l = 0.f, vref = 0x1p-126f, down = 0x1p126f;  // down = 1 / vref
  v16f acc[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = v16f{};
  struct Prob {
    v4u f[2];  // of the half's two groups of keys
  };
  // of the current tile, per group of 16 keys (the same in all lanes): the
  // factor of the scores; vs / vref, its logarithm + kBias and its inverse
  float fk[4], vr[4], lv[4], iv[4];
  bool plain = false;  // every row sees every key, and the scales are ordinary

  auto uniform = [](float x) {
    return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
  };
  auto rescale_pending = [&](Prob& pr, float keep) {
    const _Float16 k16 = (_Float16)keep;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      pr.f[k] = __builtin_bit_cast(v4u, __builtin_bit_cast(v8h, pr.f[k]) * k16);
  };
  float most = 0.f;
  auto take_scales = [&](int i) {
    const float* s = s_scale[i & 1];
    float vs[4];
    most = 0.f;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      fk[g] = uniform(s[g] * cs);
      vs[g] = uniform(s[4 + g]);
      most = vs[g] < __builtin_inff() ? __builtin_fmaxf(most, vs[g]) : most;
    }
    bool ordinary = true;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      vr[g] = uniform(vs[g] * down);
      lv[g] = uniform(__builtin_amdgcn_logf(vr[g]) + kBias);
      iv[g] = uniform(__builtin_amdgcn_rcpf(vr[g]));
      ordinary = ordinary && vr[g] >= 0x1p-60f && vr[g] <= 1.f;
    }
    plain = __builtin_amdgcn_readfirstlane((int)(ordinary && inside(i)));
  };
  // moves vref where a scale of tile i passes it
  auto settle_scales = [&](int i, Prob& pending) {
    if (most <= vref) return;
    const uint32_t u = __float_as_uint(most);
    const float to = __uint_as_float((u & 0x7FFFFFu) ? (u & 0x7F800000u) + 0x800000u : u);
    const float keep = vref / to;
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[d] *= keep;
    rescale_pending(pending, keep);
    vref = uniform(to);
    down = uniform(1.f / to);
    take_scales(i);
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
  // bit 8 (e / 4) + e % 4: whether the column sees the key of its score e
  auto seen_keys = [&](int i, int half) -> uint32_t {
    const int pos = base + i * 64 + 32 * half;
    const int from = max(col_s - pos, 0), to = min(col_e - pos, 32);
    if (from >= to) return 0u;
    return (~0u << from & ~0u >> (32 - to)) >> (4 * hh);
  };
  // all ones where bit e of such a mask is set
  auto bit = [&](uint32_t mask, int e) -> uint32_t {
    return (uint32_t)__builtin_amdgcn_sbfe((int)mask, 8 * (e >> 2) + (e & 3), 1);
  };
  auto pack = [&](const float* e) {
    v4u f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f[j] = __builtin_bit_cast(uint32_t, v2h{(_Float16)e[2 * j], (_Float16)e[2 * j + 1]});
    return f;
  };
  // scores -> probabilities of one half
  auto soft = [&](auto is_plain, const v16f& s, Prob& pr, int i, int half) {
    if constexpr (is_plain.value) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int g = 2 * half + k;
        const float off = lv[g] - m;
        float e[8], sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * k + j], fk[g], off));
          sum += e[j];
        }
        l = __builtin_fmaf(sum, iv[g], l);
        pr.f[k] = pack(e);
      }
    } else {
      const uint32_t sees = seen_keys(i, half);
      const uint32_t ill = sees & (s_poison[i % 3][half] >> (4 * hh));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int g = 2 * half + k;
        float e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // (masks by bits: what is unseen may be NaN)
          const uint32_t see = bit(sees, 8 * k + j);
          const float x =
              __builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * k + j], fk[g], -(m - kBias)));
          const float y = __uint_as_float(__float_as_uint(x) & see);
          l += y;
          e[j] = __uint_as_float((__float_as_uint(y * vr[g]) & see) |
                                 (bit(ill, 8 * k + j) & 0x7FC00000u));
        }
        pr.f[k] = pack(e);
      }
    }
  };
  // a half's largest score in this lane
  auto largest = [&](auto is_plain, const v16f& s, int i, int half) {
    if constexpr (is_plain.value) {
      float x = s[0], y = s[8];
#pragma unroll
      for (int j = 1; j < 8; ++j) {
        x = __builtin_fmaxf(x, s[j]);
        y = __builtin_fmaxf(y, s[8 + j]);
      }
      return __builtin_fmaxf(x * fk[2 * half], y * fk[2 * half + 1]);
    } else {
      const uint32_t sees = seen_keys(i, half);
      float top = -__builtin_inff();
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t see = bit(sees, e);
        const float x = s[e] * fk[2 * half + (e >> 3)];
        top = __builtin_fmaxf(
            top, __uint_as_float((__float_as_uint(x) & see) | (~see & 0xFF800000u)));
      }
      return top;
    }
  };
  // moves m where a score passes it by more than kLag; `pending`: the P not
  // yet in the sums
  auto passes = [&](float top) { return __any(top > m + kLag); };
  auto settle = [&](float top, Prob& pending) {
    if (!passes(top)) return;
    const float x = __builtin_fmaxf(top, __shfl_xor(top, 32, 64));
    const float to = __builtin_fmaxf(m, __builtin_ceilf(x));
    const float keep = __builtin_amdgcn_exp2f(m - to);
    m = to;
    l *= keep;
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[d] *= keep;
    rescale_pending(pending, keep);
  };

  if (tiles > 0) {
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    v16f s0, s1;
    Prob p0, p1;
#pragma unroll
    for (int k = 0; k < 2; ++k) p0.f[k] = p1.f[k] = v4u{0, 0, 0, 0};
    find_k(0);
    find_v(0);
    load_k(0);
    load_v(0);
    find_k(1);
    find_v(1);
    stage_k(0);
    clean_v(0);
    stage_v(0);
    load_k(1);
    load_v(1);
    find_k(2);
    find_v(2);
    __syncthreads();
    // holds the exponentials next to the products (they are used after a branch
    // only, and would be moved behind it)
    auto keep_here = [](Prob& pr, float& x) {
      asm volatile("" : "+v"(pr.f[0]), "+v"(pr.f[1]), "+v"(x));
    };
    // first half: s0 -> p0, scores of the second, values of the last tile's
    // second; keys of the next tile into LDS. The largest of the scores.
    auto half0 = [&](auto is_plain, int i) {
      scores(s1, i, 1);
      soft(is_plain, s0, p0, i, 0);
      values(p1, i - 1, 1);
      stage_k(i + 1);
      load_k(i + 2);
      const float top = largest(is_plain, s1, i, 1);
      keep_here(p0, l);
      clean_v(i + 1);
      find_k(i + 3);
      __syncthreads();
      return top;
    };
    // second half: s1 -> p1, scores of the next tile's first, values of this
    // tile's first; values of the next tile into LDS
    auto half1 = [&](auto is_plain, int i) {
      scores(s0, i + 1, 0);
      soft(is_plain, s1, p1, i, 1);
      values(p0, i, 0);
      stage_v(i + 1);
      load_v(i + 2);
      keep_here(p1, l);
      find_v(i + 3);
    };
    // The tiles that need nothing but the pipeline run in a loop of their own,
    // whose sums stay in place; it is left where a reference point has to move
    // or a tile needs masks.
    int i = 0;
    take_scales(0);
    settle_scales(0, p0);
    scores(s0, 0, 0);
    settle(largest(no, s0, 0, 0), p0);
    while (true) {
      float top;
      if (plain) {
        bool within = false;
        while (true) {
          top = half0(yes, i);
          if (passes(top)) {
            within = true;
            break;
          }
          half1(yes, i);
          if (++i >= tiles) break;
          take_scales(i);
          if (!plain || most > vref || passes(largest(yes, s0, i, 0))) break;
        }
        if (i >= tiles) break;
        if (!within) {
          settle_scales(i, p1);
          settle(largest(no, s0, i, 0), p1);
          continue;
        }
      } else {
        top = half0(no, i);
      }
      settle(top, p0);
      half1(no, i);
      if (++i >= tiles) break;
      take_scales(i);
      settle_scales(i, p1);
      settle(largest(no, s0, i, 0), p1);
    }
    values(p1, tiles - 1, 1);
  }

  const bool direct = p.splits == 1;
  const float both = l + __shfl_xor(l, 32, 64);
  const float sum = col_s >= col_e ? 0.f : both;  // (sums of a row that sees nothing)
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
  const float by = direct ? vref / sum : vref;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int at = 32 * d + 8 * e + 4 * hh;
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = sum == 0.f ? 0.f : acc[d][4 * e + j] * by;
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

// Joins the splits of a (row, query head), in order: a thread a column of the
// output. A split that saw nothing has l = 0.
template <int T>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendParams p) {
  const int D = p.c.head_dim;
  const int64_t pair = (p.block0 + blockIdx.x) * (256 / D) + threadIdx.x / D;
  if (pair >= (int64_t)p.rows * p.heads) return;
  const int d = threadIdx.x % D;
  const int row = (int)(pair / p.heads), head = (int)(pair % p.heads), h = head / p.group;
  const int per_unit = p.indices ? 1 : p.R;
  const int unit = row / per_unit;
  const int column = row % per_unit * p.group + head % p.group;
  const int64_t item = ((int64_t)unit * p.tiles + column / p.cols) * p.c.kv_heads + h;
  const int64_t first = item * p.splits * p.cols + column % p.cols;
  float top = kLowest;
  for (int s = 0; s < p.splits; ++s)
    top = __builtin_fmaxf(top, p.part_ml[2 * (first + (int64_t)s * p.cols)]);
  float sum = 0.f, v = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const int64_t at = first + (int64_t)s * p.cols;
    const float w = __builtin_amdgcn_exp2f(p.part_ml[2 * at] - top);
    const float ls = p.part_ml[2 * at + 1];
    if (ls == 0.f) continue;
    sum = __builtin_fmaf(ls, w, sum);
    v = __builtin_fmaf(p.part_o[at * D + d], w, v);
  }
  static_cast<uint16_t*>(p.out)[pair * D + d] = to_type(sum == 0.f ? 0.f : v / sum, T);
  if (d == 0 && p.lse)
    p.lse[pair] = sum == 0.f ? -__builtin_inff() : (top - kBias) * kLn2 + __builtin_logf(sum);
}

// A launch's grid stays below 2^32 threads: more workgroups go in several.
template <class Launch>
void in_pieces(AttendParams p, int64_t blocks, Launch launch) {
  constexpr int64_t kMost = 1 << 22;
  for (p.block0 = 0; p.block0 < blocks; p.block0 += kMost)
    launch(p, dim3((unsigned)(blocks - p.block0 < kMost ? blocks - p.block0 : kMost)));
}

template <int T, int C, int D, int NT>
void narrow(const AttendParams& p, dim3 grid, hipStream_t s) {
  if (p.indices)
    attend_narrow_kernel<T, C, D, NT, true><<<grid, 256, 0, s>>>(p);
  else
    attend_narrow_kernel<T, C, D, NT, false><<<grid, 256, 0, s>>>(p);
}

template <int T, int C, int D>
void attend(const AttendParams& all, hipStream_t s) {
  const int64_t units = all.indices ? all.rows : all.requests;
  in_pieces(all, units * all.tiles * all.c.kv_heads * all.splits,
            [&](const AttendParams& p, dim3 grid) {
              if (p.cols == 16) narrow<T, C, D, 1>(p, grid, s);
              if (p.cols == 32) narrow<T, C, D, 2>(p, grid, s);
              if (p.cols == 64) narrow<T, C, D, 4>(p, grid, s);
              if (p.cols == 128) attend_wide_kernel<T, C, D, 4><<<grid, 256, 0, s>>>(p);
              if (p.cols == 256) attend_wide_kernel<T, C, D, 8><<<grid, 512, 0, s>>>(p);
            });
  if (all.splits > 1) {
    const int64_t pairs = (int64_t)all.rows * all.heads, per = 256 / D;
    in_pieces(all, (pairs + per - 1) / per, [&](const AttendParams& p, dim3 grid) {
      attend_join_kernel<T><<<grid, 256, 0, s>>>(p);
    });
  }
}

template <int T, int C>
void attend_dim(const AttendParams& p, hipStream_t s) {
  p.c.head_dim == 64 ? attend<T, C, 64>(p, s) : attend<T, C, 128>(p, s);
}

}  // namespace
}  // namespace mqa

extern "C" int mqa_attend_launch(const mqa::AttendParams* p, hipStream_t s) {
  using namespace mqa;
  const bool e = p->c.codes == kE4m3;
  if (p->dtype == kBf16) e ? attend_dim<kBf16, kE4m3>(*p, s) : attend_dim<kBf16, kInt8>(*p, s);
  if (p->dtype == kFp16) e ? attend_dim<kFp16, kE4m3>(*p, s) : attend_dim<kFp16, kInt8>(*p, s);
  return (int)hipGetLastError();
}
