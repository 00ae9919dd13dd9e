// Attention over the 4-bit cache for many query rows (prompts, long chunks).
//
// A workgroup takes a tile of query rows, 32 for each of its waves, and walks
// over the keys 64 at a time.  The waves expand the 64 keys and values from
// their codes to fp16 into LDS once; then every wave multiplies all 64 with its
// own rows:
//   S^T [64 keys, rows] = K^ Q^T,   O^T [D, rows] += V^^T P^T   (32x32x16)
// As in the rows kernel, the first product's result layout is the second one's
// operand layout, so P stays in registers.  Codes are fetched two tiles ahead
// and expanded one tile ahead, into the other of two buffers.
//
// The expansion costs a wave some 60 to 90 vector instructions per 64 keys, an
// eighth of what it would be for 32 rows alone; the softmax of its 32 rows
// costs 170.  Counters for a prompt of 4096 (32 heads of 128, causal): vector
// unit 55 % busy, matrix unit 38 %; reading the operands from LDS takes as long
// as the products (one 1 KiB operand each).  Rates: 212 us or 650 TFLOP/s there,
// where a library product of 8192^3 reaches 1190; ragged chunks with groups of
// 32 and fp16 results 170 us (twice the products, see below); a window of 4096
// keys at 256 channels 91.5 us (one wave a SIMD, and a quarter to a third of its
// vector instructions only move accumulation registers).
#pragma once

#include "kv4_rows.h"

namespace gq {
namespace kv4 {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTK = 64;   // keys per tile

// As kRoom and kSlack of the rows kernel.  Raising the reference costs more here
// (a prompt of 4096: 199 us without room, 200 with 8 and 7, 204 with 11 and 4), and
// scales of groups take none of the room: all bits down to 2^-22, none below 2^-33.
constexpr float kTileRoom = 8.0f, kTileSlack = 7.0f;

// Waves of a workgroup.  The results of 32 rows take D / 2 registers: up to 128
// channels two waves fit a SIMD, and one's vector work runs beside the other's
// matrix products.
constexpr int tile_waves(int d) { return d > 128 ? 4 : 8; }

template <int D, int NG, bool SYM, bool SPLIT, bool F16>
struct Tile {
  static constexpr int NS = D / 32, SPG = NS / NG;
  static constexpr int NW = tile_waves(D);
  static constexpr int TQ = NW * 32;                  // rows of a workgroup
  static constexpr int KP = D * 2 + 16;               // LDS row of a key: padded, 16 lanes
  static constexpr int VP = kTK * 2 + 16;             //   reading 16 rows hit all banks
  // How the keys go to the matrix cores, exactly either way: as the integers
  // c - z, with a scale per group applied to the scores (SPLIT false), or as
  // x^ / 2^E in two fp16 parts (true).
  static constexpr int kV = kTK * KP * (SPLIT ? 2 : 1);   // the values, behind the keys and their lower parts
  // The rounding of a value to fp16 (2^-11) is far below that of a bf16 result,
  // but as large as that of an fp16 one: F16 adds what it left, as a second part.
  static constexpr int kParts = F16 ? 2 : 1;
  static constexpr int kScale = kV + kParts * D * VP;     // key scales fp16 [NG][2][2][16]
  static constexpr int kEx = kScale + (SPLIT ? 0 : NG * kTK * 2);   // floats {E, 2^-E} of the values' blocks of
  static constexpr int kBuf = kEx + 48;                   //   16, 2^E of the keys'; bytes of one buffer

  // Two buffers, so that one is filled while the other is read; 256 channels in
  // two parts have room for one.
  static constexpr int kBufs = 2 * kBuf <= 160 * 1024 ? 2 : 1;

  f16x8 q[D / 16];
  float A, mref, l;
  f32x16 o[NS];

  // What a wave holds of the next tile: codes and parameters of 16 keys (lane
  // (m, kg): token m) or of 16 values (tokens 4 kg ..).
  struct Codes {
    uint32_t d[NS];
    uint32_t p[NG][4];   // keys: {S | z << 16}; values: {S, S, z, z} pairs
    int pos;             // of the first token
    bool ok;

    __device__ __forceinline__ const uint8_t* start(const Kv4Attn& a, int64_t page, int h, int u) {
      pos = u;
      ok = page >= 0 && page < a.c.n_pages;
      return a.c.cache +
             kv4_block_offset(a.c, ok ? page : 0, h, ok ? u & ((1 << a.c.page_shift) - 1) : 0);
    }
    __device__ __forceinline__ void load_k(const Kv4Attn& a, int64_t page, int h, int u, int m, int kg) {
      const uint8_t* blk = start(a, page, h, u);
      load_dwords<NS>(blk + m * (D / 2) + kg * (4 * NS), d);
      const uint16_t* kp = (const uint16_t*)(blk + 8 * D);
#pragma unroll
      for (int g = 0; g < NG; ++g) p[g][0] = kp[g * 16 + m];
      if constexpr (!SYM) {
#pragma unroll
        for (int g = 0; g < NG; ++g) p[g][1] = kp[16 * NG + m * NG + g];
      }
    }
    __device__ __forceinline__ void load_v(const Kv4Attn& a, int64_t page, int h, int u, int m, int kg) {
      const uint8_t* w = start(a, page, h, u) + 8 * D + a.c.meta;
      load_dwords<NS>(w + kg * (64 * NS) + m * (4 * NS), d);
      const uint8_t* vp = w + 8 * D;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if constexpr (SYM) {
          const uint2 t = *(const uint2*)(vp + g * 32 + kg * 8);
          p[g][0] = t.x; p[g][1] = t.y;
        } else {
          load_dwords<4>(vp + g * 64 + kg * 16, p[g]);
        }
      }
    }
  };

  // Largest value over the wave, as a scalar.
  template <int CTRL>
  static __device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
    const uint32_t u = __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
    return u > v ? u : v;
  }
  static __device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max_dpp<0x140>(max_dpp<0x141>(max_dpp<0x4E>(max_dpp<0xB1>(v))));   // over rows of 16 lanes
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    const uint32_t x = a > b ? a : b, y = c > d ? c : d;
    return x > y ? x : y;
  }

  // Exponent field of the largest of the wave's fp16 scales, and 2^-E for it: E is
  // ten less than its exponent, so that codes times scales reach 2^15, the end of
  // fp16's range, and scales down to 2^-24 of the largest keep their bits beside it
  // (2^-14 with E its exponent).  Subnormal ones, and zeros (rows of zeros), count as
  // the smallest normal one: as 2^0 a block of zeros would set the softmax's reference.
  static __device__ __forceinline__ uint32_t top_exponent(uint32_t top) {
    const uint32_t e = wave_max(top) >> 10;
    return e ? e : 1;
  }
  static __device__ __forceinline__ float pow2_neg(uint32_t e) { return __uint_as_float((152 - e) << 23); }

  // Keys.  Parts: x^ / 2^E as fp16, E from the largest scale of the 16, and what
  // its rounding left, as fp16 too: together x^ to 2^-22 of it and 2^-33 of the
  // largest of the 16.  2^E comes back in the factor of the scores.  Keys that no
  // row sees count as zeros, whatever their memory holds.
  static __device__ __forceinline__ void expand_k(const Nibbles& nib, Codes& c, const Span& sp, uint8_t* buf,
                                                  int blk, int m, int kg) {
    if (!(c.ok && c.pos >= sp.lo && c.pos + 16 <= sp.hi)) {
      const bool live = c.ok && c.pos + m >= sp.lo && c.pos + m < sp.hi;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        c.p[g][0] = live ? c.p[g][0] : 0u;
        if constexpr (!SYM) c.p[g][1] = live ? c.p[g][1] : 0u;
      }
    }
    uint32_t top = 0;
    if constexpr (SPLIT) {
#pragma unroll
      for (int g = 0; g < NG; ++g) top = c.p[g][0] > top ? c.p[g][0] : top;
    }
    float inv = 1.0f;
    if constexpr (SPLIT) {
      const uint32_t e = top_exponent(top);
      inv = pow2_neg(e);
      if (m == 0 && kg == 0) ((float*)(buf + kEx))[8 + blk] = __uint_as_float((102 + e) << 23);
    } else if (kg == 0) {
      // scale of token m: the lanes of one result half take 16 tokens of 32 in
      // the order 8 (i / 4) + 4 half + i % 4
      const int r = (blk & 1) * 16 + m;
      uint16_t* sc = (uint16_t*)(buf + kScale) + (blk >> 1) * 32 + ((r >> 2) & 1) * 16 + (r >> 3) * 4 + (r & 3);
#pragma unroll
      for (int g = 0; g < NG; ++g) sc[g * kTK] = (uint16_t)c.p[g][0];
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f16x2 n1 = {(_Float16)-1032.0f, (_Float16)-1032.0f};
      if constexpr (!SYM) {
        const _Float16 z = __builtin_bit_cast(_Float16, (uint16_t)c.p[g][1]);
        n1 = f16x2{z, z};
      }
      const f16x2 n2 = n1 + (_Float16)960.0f;
      const _Float16 S = (_Float16)(lo_f16(c.p[g][0]) * inv);
      const f16x2 S2 = {S, S};
#pragma unroll
      for (int s = g * SPG; s < (g + 1) * SPG; ++s) {
        const uint32_t d = c.d[s], d8 = d >> 8;
        u32x4 w = {nib.lo(d, n1), nib.hi(d, n2), nib.lo(d8, n1), nib.hi(d8, n2)};
        uint8_t* o = buf + (blk * 16 + m) * KP + s * 64 + kg * 16;
        if constexpr (SPLIT) {
          u32x4 low;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f16x2 k = __builtin_bit_cast(f16x2, (uint32_t)w[i]), h = k * S2;
            w[i] = __builtin_bit_cast(uint32_t, h);
            low[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(k, S2, -h));
          }
          *(u32x4*)(o + kTK * KP) = low;
        }
        *(u32x4*)o = w;
      }
    }
  }

  // Values: x^ / 2^E as fp16 (F16: and what the rounding left), E from the largest
  // scale of the 16: x^ to 2^-11 of it (2^-22) and 2^-33 of the largest of them.
  // 2^E comes back in the exponent of P.
  static __device__ __forceinline__ void expand_v(const Nibbles& nib, Codes& c, const Span& sp, uint8_t* buf, int blk, int m,
                                                  int kg) {
    if (!(c.ok && c.pos >= sp.lo && c.pos + 16 <= sp.hi)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int p = c.pos + 4 * kg + 2 * i;
        const uint32_t live = (c.ok && p >= sp.lo && p < sp.hi ? 0xFFFFu : 0u) |
                              (c.ok && p + 1 >= sp.lo && p + 1 < sp.hi ? 0xFFFF0000u : 0u);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          c.p[g][i] &= live;
          if constexpr (!SYM) c.p[g][2 + i] &= live;
        }
      }
    }
    u16x2 most = {0, 0};
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < 2; ++i) most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, c.p[g][i]));
    const uint32_t top = most[0] > most[1] ? most[0] : most[1];
    const uint32_t e = top_exponent(top);
    const float inv = pow2_neg(e);
    if (m == 0 && kg == 0) {
      float* ex = (float*)(buf + kEx);
      // -inf takes keys that do not exist out of the softmax
      ex[blk] = c.ok ? (float)((int)e - 25) : kNegInf;
      ex[4 + blk] = inv;
    }
    uint8_t* vb = buf + kV + blk * 32 + (kg & 1) * 16 + (kg >> 1) * 8;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f16x2 S2[2], n1[2], n2[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        S2[i] = f16x2{(_Float16)(lo_f16(c.p[g][i]) * inv), (_Float16)(hi_f16(c.p[g][i]) * inv)};
        n1[i] = f16x2{(_Float16)-1032.0f, (_Float16)-1032.0f};
        if constexpr (!SYM) n1[i] = __builtin_bit_cast(f16x2, c.p[g][2 + i]);
        n2[i] = n1[i] + (_Float16)960.0f;
      }
#pragma unroll
      for (int b = g * SPG; b < (g + 1) * SPG; ++b) {
        f16x2 v[2][2], x[2][2];   // channel 2 m or 2 m + 1, token pair
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w = byte_pair<NS>(c.d, 2 * i * NS + b, (2 * i + 1) * NS + b);
          v[0][i] = __builtin_bit_cast(f16x2, nib.lo(w, n1[i]));
          v[1][i] = __builtin_bit_cast(f16x2, nib.hi(w, n2[i]));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint8_t* row = vb + (32 * b + 2 * m + j) * VP;
#pragma unroll
          for (int i = 0; i < 2; ++i) x[j][i] = v[j][i] * S2[i];
          *(uint2*)row = make_uint2(__builtin_bit_cast(uint32_t, x[j][0]), __builtin_bit_cast(uint32_t, x[j][1]));
          if constexpr (F16) {
            const f16x2 r0 = __builtin_elementwise_fma(v[j][0], S2[0], -x[j][0]);
            const f16x2 r1 = __builtin_elementwise_fma(v[j][1], S2[1], -x[j][1]);
            *(uint2*)(row + D * VP) = make_uint2(__builtin_bit_cast(uint32_t, r0), __builtin_bit_cast(uint32_t, r1));
          }
        }
      }
    }
  }

  __device__ __forceinline__ void load_q(const Kv4Attn& a, const Seq& s, int h, int row, int hf) {
    const bool ok = row < s.n * a.r;
    const uint16_t* p = a.q;
    const int tok = div_r(a, row);
    if (ok) p += (int64_t)(s.q0 + tok) * a.q_ts + (int64_t)(h * a.r + row - tok * a.r) * a.q_hs;
    float mx = 0.0f;
#pragma unroll
    for (int st = 0; st < D / 16; ++st) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (ok) v = *(const uint4*)(p + 16 * st + 8 * hf);
      q[st] = __builtin_bit_cast(f16x8, u32x4{v.x, v.y, v.z, v.w});   // raw bits for now
      float x[8];
      widen(a.bf16, q[st], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(x[i]));
    }
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    int e = (int)(__float_as_uint(mx) >> 23) - 127;
    e = e < -112 ? -112 : (e > 127 ? 127 : e);   // 128: infinite or NaN
    const float f = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
    A = a.scale_log2 * __uint_as_float((uint32_t)(127 - 14 + e) << 23);
    // never 0, which would make NaN of a hidden key's -inf; scores times 2^-100 vanish too
    A = fmaxf(A, 0x1p-100f);
#pragma unroll
    for (int st = 0; st < D / 16; ++st) {
      float x[8];
      widen(a.bf16, q[st], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) q[st][i] = (_Float16)(x[i] * f);
    }
    mref = kNegInf;
    l = 0.0f;
#pragma unroll
    for (int d = 0; d < NS; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  }
  static __device__ __forceinline__ void widen(int bf16, f16x8 raw, float (&x)[8]) {
    const u32x4 w = __builtin_bit_cast(u32x4, raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16 ? bf16_to_f32(w[i] & 0xFFFFu) : lo_f16(w[i]);
      x[2 * i + 1] = bf16 ? __uint_as_float(w[i] & 0xFFFF0000u) : hi_f16(w[i]);
    }
  }

  // One tile of 64 keys from position u on: scores, weights, sums.
  //
  // The order is written out, product by product, and held by the scheduling
  // fences (left alone, the scheduler saves registers and waits out the latency
  // of every read of LDS, one read per product): operands are read kAhead
  // products before their use, and the vector work that is independent of a
  // product stands behind it, where it runs beside the matrix unit: the scales
  // of one run of scores beside the next run's products, the exponentials of
  // 16 keys beside the products of the 16 before.
  __device__ __forceinline__ void attend(const Kv4Attn& a, const Seq& s, int row0, int u, const uint8_t* buf,
                                         int n, int hf) {
    constexpr int kAhead = 4;
    f16x8 ring[kAhead];
    f32x16 x[2];
    // products go first where the SIMD's other wave has vector work (2 %)
    __builtin_amdgcn_s_setprio(1);
    if constexpr (SPLIT) {
      // both halves of the keys, their lower parts, then the next channels
      constexpr int kAll = D / 4;
      auto read = [&](int r) {
        return *(const f16x8*)(buf + ((r >> 1 & 1) * kTK + 32 * (r & 1) + n) * KP + (r / 4) * 32 + hf * 16);
      };
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 16; ++i) x[tt][i] = 0.0f;
#pragma unroll
      for (int r = 0; r < kAhead; ++r) ring[r] = read(r);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int r = 0; r < kAll; ++r) {
        x[r & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[r % kAhead], q[r / 4], x[r & 1], 0, 0, 0);
        if (r + kAhead < kAll) ring[r % kAhead] = read(r + kAhead);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      // runs of products with one scale per key: (half of the keys, group)
      constexpr int kRun = 2 * SPG, kRuns = 2 * NG, kAll = kRun * kRuns;
      auto read = [&](int r) {
        const int tt = r / (kRun * NG), st = r % (kRun * NG);
        return *(const f16x8*)(buf + (32 * tt + n) * KP + st * 32 + hf * 16);
      };
      f32x16 acc[2];
      f16x8 sc[2][2];
      // elements from .. to - 1 of run i's scores, scaled
      auto scale = [&](int i, int from, int to) {
        const int tt = i / NG, g = i % NG;
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (e >= from && e < to) {
            float v = __builtin_fmaf((float)sc[i & 1][e >> 3][e & 7], acc[i & 1][e], g == 0 ? 0.0f : x[tt][e]);
            asm volatile("" : "+v"(v));   // here, not where it is used first
            x[tt][e] = v;
          }
      };
#pragma unroll
      for (int r = 0; r < kAhead; ++r) ring[r] = read(r);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < kRuns; ++i) {
        const f16x8* sp = (const f16x8*)(buf + kScale + (i % NG) * (kTK * 2) + (i / NG) * 64 + hf * 32);
        sc[i & 1][0] = sp[0];
        sc[i & 1][1] = sp[1];
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i & 1][e] = 0.0f;
#pragma unroll
        for (int st = 0; st < kRun; ++st) {
          const int r = i * kRun + st;
          acc[i & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[r % kAhead], q[r % (kRun * NG)], acc[i & 1], 0, 0, 0);
          if (r + kAhead < kAll) ring[r % kAhead] = read(r + kAhead);
          if (i > 0) scale(i - 1, 16 * st / kRun, 16 * (st + 1) / kRun);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      scale(kRuns - 1, 0, 16);
    }
    __builtin_amdgcn_s_setprio(0);
    const uint8_t* vb = buf + kV;
    auto read_v = [&](int r) {   // 16 keys, part, channels 32 d ..
      const int b = r / (kParts * NS), d = r % (kParts * NS);
      return *(const f16x8*)(vb + (32 * d + n) * VP + b * 32 + hf * 16);
    };
#pragma unroll
    for (int r = 0; r < kAhead; ++r) ring[r] = read_v(r);
    // per 16 keys, the scores have the factor 2^E of the keys and P that of the values
    const float4 ev = *(const float4*)(buf + kEx), ei = *(const float4*)(buf + kEx + 16);
    const float evv[4] = {ev.x, ev.y, ev.z, ev.w}, eiv[4] = {ei.x, ei.y, ei.z, ei.w};
    const float least = fminf(fminf(ev.x, ev.y), fminf(ev.z, ev.w));
    // whether every row of the wave sees all 64 keys
    const int rows = s.n * a.r;
    const int lastrow = row0 + 32 < rows ? row0 + 31 : rows - 1;
    bool full = u + kTK <= s.kv;
    if (a.causal) full = full && u + kTK - 1 <= s.kv - s.n + div_r(a, row0);
    if (a.window > 0) full = full && u > s.kv - s.n + div_r(a, lastrow) - a.window;
    // and all of them exist: a query that is not finite makes NaN of the zeros that stand there
    full = full && __builtin_amdgcn_readfirstlane(__float_as_uint(least)) != __float_as_uint(kNegInf);
    if (!full) {
      const int pos = s.kv - s.n + div_r(a, row0 + n);
      const int last = a.causal && pos < s.kv - 1 ? pos : s.kv - 1;
      const int first = a.window > 0 ? pos - a.window + 1 : 0;
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = u + 32 * tt + 8 * (i / 4) + 4 * hf + (i & 3);
          x[tt][i] = j <= last && j >= first && evv[2 * tt + i / 8] != kNegInf ? x[tt][i] : kNegInf;
        }
    }
    float Ab[4] = {A, A, A, A};
    if constexpr (SPLIT) {
      const float4 ek = *(const float4*)(buf + kEx + 32);
      Ab[0] *= ek.x; Ab[1] *= ek.y; Ab[2] *= ek.z; Ab[3] *= ek.w;
    }
    float top = kNegInf;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      float t = x[b >> 1][8 * (b & 1)];
#pragma unroll
      for (int i = 1; i < 8; ++i) t = fmaxf(t, x[b >> 1][8 * (b & 1) + i]);
      top = fmaxf(top, __builtin_fmaf(t, Ab[b], evv[b]));
    }
    top -= kTileRoom;
    if (__any(top > mref + kTileSlack)) {
      top = fmaxf(top, __shfl_xor(top, 32));
      const float mn = fmaxf(top, mref);
      const float f = mn == mref ? 1.0f : exp2_hw(mref - mn);
      mref = mn;
      l *= f;
#pragma unroll
      for (int d = 0; d < NS; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= f;
    }
    const float base = mref == kNegInf ? 0.0f : mref;
    f16x8 pw[2];
    float sum[2];
    // weights from .. to - 1 of 16 keys' 8 in this lane.  They are rounded to fp16
    // (2^-11, their sum is not): fp16 results are off by 2.6e-4 where their own
    // rounding alone makes 2.1e-4; a second part would double the second products.
    auto weigh = [&](int b, int from, int to) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= from && i < to) {
          const float e = exp2_hw(__builtin_fmaf(x[b >> 1][8 * (b & 1) + i], Ab[b], evv[b] - base));
          sum[b & 1] = i == 0 ? e : sum[b & 1] + e;
          pw[b & 1][i] = (_Float16)e;
          if (i == 7) l = __builtin_fmaf(sum[b & 1], eiv[b], l);
        }
    };
    weigh(0, 0, 8);
    __builtin_amdgcn_s_setprio(1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int d = 0; d < kParts * NS; ++d) {
        const int r = b * (kParts * NS) + d;
        o[d % NS] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[r % kAhead], pw[b & 1], o[d % NS], 0, 0, 0);
        if (r + kAhead < 4 * kParts * NS) ring[r % kAhead] = read_v(r + kAhead);
        if (b < 3) weigh(b + 1, 8 * d / (kParts * NS), 8 * (d + 1) / (kParts * NS));
        __builtin_amdgcn_sched_barrier(0);
      }
    __builtin_amdgcn_s_setprio(0);
  }

  __device__ __forceinline__ void finish(const Kv4Attn& a, const Seq& s, int h, int qt, int ri, float* part,
                                         int hf) {
    using R = Rows<D, 1, 1, true>;
    const int row = qt * TQ + ri;
    const float L = l + __shfl_xor(l, 32);
    if (row >= s.n * a.r) return;
    if (part) {
#pragma unroll
      for (int d = 0; d < NS; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *(float4*)(part + ri * D + 32 * d + 8 * i + 4 * hf) =
              make_float4(o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]);
      if (hf == 0) {
        part[TQ * D + ri] = mref;
        part[TQ * D + TQ + ri] = L;
      }
      return;
    }
    const int64_t orow = out_row(a, s, h, row);
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int d = 0; d < NS; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *(uint2*)(a.out + orow * D + 32 * d + 8 * i + 4 * hf) =
            make_uint2(R::pack_out(a.bf16, o[d][4 * i] * inv, o[d][4 * i + 1] * inv),
                       R::pack_out(a.bf16, o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv));
    if (a.lse && hf == 0) a.lse[orow] = R::lse_of(mref, L);
  }
};

template <int D, int NG, bool SYM, bool SPLIT, bool F16>
__global__ __launch_bounds__(tile_waves(D) * 64, tile_waves(D) / 4) void kv4_tile_kernel(Kv4Attn a) {
  using T = Tile<D, NG, SYM, SPLIT, F16>;
  constexpr bool kBoth = T::NW == 4;   // a wave expands keys and values of its block; else one of them
  __shared__ __attribute__((aligned(16))) uint8_t smem[T::kBufs * T::kBuf];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, kg = lane >> 4, n = lane & 31, hf = lane >> 5;
  const int blk = wave & 3;            // the 16 keys of a tile that this wave expands
  const bool is_k = wave < 4;
  const int ps = a.c.page_shift;
  T st;
  const Nibbles nib;
  const Share sh = find_share<T::TQ>(a, lane);
  uint32_t at = sh.at;
  int last = -1;
  Cursor cur = sh.cur;
  Seq s{0, 0, 0};
  if (at < sh.end) {
    s = wave_seq(a, cur.b);
    for (;;) {
      const Span sp = get_span<T::TQ>(a, s, cur.qt);
      const int j0 = cur.off, left = (int)(sh.end - at);
      const int j1 = sp.cnt - j0 < left ? sp.cnt : j0 + left;
      const bool starts = j0 == 0, ends = j1 == sp.cnt;
      const int row0 = cur.qt * T::TQ + wave * 32;
      // the run's keys, 64 at a time
      const int64_t cut = tile_start(a, sp, j1);
      const int stop = cut < sp.hi ? (int)cut : sp.hi;
      int u0 = (int)tile_start(a, sp, j0);
      if (u0 < sp.lo) u0 = sp.lo & ~(kTK - 1);
      const PageRow table = page_row(a, cur.b);
      // page of this wave's 16 of the 64 keys from u on, -1 where no row sees them
      auto page_of = [&](int u) -> int64_t {
        const int pos = u + blk * 16;
        return pos < stop && pos + 16 > sp.lo ? table[pos >> ps] : -1;
      };
      typename T::Codes ck, cv;   // a wave that expands one of them uses ck for it
      auto fetch = [&](int64_t page, int u) {
        u += blk * 16;
        if constexpr (kBoth) {
          ck.load_k(a, page, cur.h, u, m, kg);
          cv.load_v(a, page, cur.h, u, m, kg);
        } else if (is_k) {
          ck.load_k(a, page, cur.h, u, m, kg);
        } else {
          ck.load_v(a, page, cur.h, u, m, kg);
        }
      };
      auto expand = [&](uint8_t* buf) {
        if constexpr (kBoth) {
          T::expand_k(nib, ck, sp, buf, blk, m, kg);
          T::expand_v(nib, cv, sp, buf, blk, m, kg);
        } else if (is_k) {
          T::expand_k(nib, ck, sp, buf, blk, m, kg);
        } else {
          T::expand_v(nib, ck, sp, buf, blk, m, kg);
        }
      };
      fetch(page_of(u0), u0);
      st.load_q(a, s, cur.h, row0 + n, hf);   // beside the codes
      expand(smem);
      fetch(page_of(u0 + kTK), u0 + kTK);
      int64_t next = page_of(u0 + 2 * kTK);
      __syncthreads();
      // Codes are fetched a tile before they are expanded.  The waves of keys
      // expand before their products and those of values after: of the two
      // waves of a SIMD one has vector work while the other multiplies.
      for (int u = u0, b = 0; u < stop; u += kTK, b ^= T::kBufs - 1) {
        const bool more = u + kTK < stop;
        auto refill = [&] {
          if (!more) return;
          expand(smem + (b ^ (T::kBufs - 1)) * T::kBuf);
          fetch(next, u + 2 * kTK);
          next = page_of(u + 3 * kTK);
        };
        if (!kBoth && is_k) refill();
        if (row0 < s.n * a.r) st.attend(a, s, row0, u, smem + b * T::kBuf, n, hf);
        if (T::kBufs == 1) __syncthreads();
        if (kBoth || !is_k) refill();
        __syncthreads();
      }
      float* part = nullptr;
      if (!(starts && ends)) {
        part = a.part + ((int64_t)2 * sh.w + (starts ? 1 : 0)) * (T::TQ * (D + 2));
        if (starts) last = sh.worker_with(at + sp.cnt - 1);
      }
      st.finish(a, s, cur.h, cur.qt, wave * 32 + n, part, hf);
      at += j1 - j0;
      if (at >= sh.end) break;
      cur.off = 0;
      const int nqt = row_tiles(a, s, T::TQ);
      if (++cur.qt == nqt) {
        cur.qt = 0;
        if (++cur.h == a.c.hkv) {
          cur.h = 0;
          do { ++cur.b; s = wave_seq(a, cur.b); } while (s.n == 0);
        }
      }
    }
  }
  if (threadIdx.x == 0) leave_meta(a, sh, last, cur, s);
}

template <int D, int NG, bool SYM, bool SPLIT, bool F16>
hipError_t launch_tile_as(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s) {
  using T = Tile<D, NG, SYM, SPLIT, F16>;
  hipLaunchKernelGGL((kv4_tile_kernel<D, NG, SYM, SPLIT, F16>), dim3(a.workers), dim3(T::NW * 64), 0, s, a);
  if (hipError_t e = hipGetLastError()) return e;
  return launch_join<D, T::TQ, 1>(a, p.tile_rows, s);
}

template <int D, int NG>
hipError_t launch_tile(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s) {
  // Several scales a key and two sets of unfinished scores do not fit the
  // registers: two parts are then twice the first products but no scales.
  // Prompts of 4096 and 2048: 128 channels, 1 group 218 us with scales, 246
  // in parts; 4 groups 158 in parts, 560 with scales (which spill).
  constexpr bool kSplit = NG > (D <= 128 ? 2 : 1);
  if (a.bf16)
    return a.c.sym ? launch_tile_as<D, NG, true, kSplit, false>(a, p, s)
                   : launch_tile_as<D, NG, false, kSplit, false>(a, p, s);
  return a.c.sym ? launch_tile_as<D, NG, true, kSplit, true>(a, p, s)
                 : launch_tile_as<D, NG, false, kSplit, true>(a, p, s);
}

}  // namespace kv4
}  // namespace gq
