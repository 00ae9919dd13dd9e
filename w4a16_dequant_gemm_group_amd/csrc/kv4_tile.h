// Attention over the 4-bit cache for many query rows (prompts, long chunks).
//
// A workgroup takes a tile of query rows, 32 for each of its waves, and walks
// over the keys 64 at a time.  The waves expand the 64 keys and values from
// their codes to fp16 into LDS once; then every wave multiplies all 64 with its
// own rows:
//   S^T [64 keys, rows] = K^ Q^T,   O^T [D, rows] += V^^T P^T   (32x32x16)
// As in the rows kernel, the first product's result layout is the second one's
// operand layout, so P stays in registers.  Two buffers: the next tile is
// fetched before and expanded after the products of the present one.
#pragma once

#include "kv4_rows.h"

namespace gq {
namespace kv4 {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTK = 64;   // keys per tile

// Waves of a workgroup.  The results of 32 rows take D / 2 registers: up to 128
// channels two waves fit a SIMD, and one's vector work runs beside the other's
// matrix products.
constexpr int tile_waves(int d) { return d > 128 ? 4 : 8; }

template <int D, int NG, bool SYM>
struct Tile {
  static constexpr int NS = D / 32, SPG = NS / NG;
  static constexpr int NW = tile_waves(D);
  static constexpr int TQ = NW * 32;                  // rows of a workgroup
  static constexpr int KP = D * 2 + 16;               // LDS row of a key: padded, 16 lanes
  static constexpr int VP = kTK * 2 + 16;             //   reading 16 rows hit all banks
  static constexpr int kScale = kTK * KP + D * VP;    // key scales fp16 [NG][2][2][16]
  static constexpr int kEx = kScale + NG * kTK * 2;   // floats {E, 2^-E} of the values' blocks
  static constexpr int kBuf = kEx + 32;               // bytes of one buffer

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

  // Largest of a non-negative value over the wave, as a scalar.
  static __device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    float f = __uint_as_float(v);   // bit patterns of non-negative halfs order as floats do
    f = fmaxf(f, stream_util::dpp_f32<0xB1, 0xF>(f));
    f = fmaxf(f, stream_util::dpp_f32<0x4E, 0xF>(f));
    f = fmaxf(f, stream_util::dpp_f32<0x141, 0xF>(f));
    f = fmaxf(f, stream_util::dpp_f32<0x140, 0xF>(f));
    const uint32_t a = __builtin_amdgcn_readlane(__float_as_uint(f), 0);
    const uint32_t b = __builtin_amdgcn_readlane(__float_as_uint(f), 16);
    const uint32_t c = __builtin_amdgcn_readlane(__float_as_uint(f), 32);
    const uint32_t d = __builtin_amdgcn_readlane(__float_as_uint(f), 48);
    const uint32_t x = a > b ? a : b, y = c > d ? c : d;
    return x > y ? x : y;
  }

  // Keys: the exact integers c - z; their scales wait for the finished scores.
  // Keys that no row sees count as zeros, whatever their memory holds.
  static __device__ __forceinline__ void expand_k(const Nibbles& nib, Codes& c, const Span& sp, uint8_t* buf, int blk, int m,
                                                  int kg) {
    const bool live = c.ok && c.pos + m >= sp.lo && c.pos + m < sp.hi;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f16x2 n1 = {(_Float16)-1032.0f, (_Float16)-1032.0f};
      if constexpr (!SYM) {
        const _Float16 z = __builtin_bit_cast(_Float16, (uint16_t)(live ? c.p[g][1] : 0u));
        n1 = f16x2{z, z};
      }
      const f16x2 n2 = n1 + (_Float16)960.0f;
#pragma unroll
      for (int s = g * SPG; s < (g + 1) * SPG; ++s) {
        const uint32_t d = c.d[s], e = d >> 8;
        const u32x4 w = {nib.lo(d, n1), nib.hi(d, n2), nib.lo(e, n1), nib.hi(e, n2)};
        *(u32x4*)(buf + (blk * 16 + m) * KP + s * 64 + kg * 16) = w;
      }
    }
    // scale of token m: the lanes of one result half take 16 tokens of 32 in
    // the order 8 (i / 4) + 4 half + i % 4
    if (kg == 0) {
      const int r = (blk & 1) * 16 + m;
      uint16_t* sc = (uint16_t*)(buf + kScale) + (blk >> 1) * 32 + ((r >> 2) & 1) * 16 + (r >> 3) * 4 + (r & 3);
#pragma unroll
      for (int g = 0; g < NG; ++g) sc[g * kTK] = live ? (uint16_t)c.p[g][0] : (uint16_t)0;
    }
  }

  // Values: x^ / 2^E as fp16, rounded once (2^-11); E is the exponent of the
  // largest scale of the 16, so that they lie in fp16's normal range whatever
  // the scales are.  2^E comes back in the exponent of P.
  static __device__ __forceinline__ void expand_v(const Nibbles& nib, Codes& c, const Span& sp, uint8_t* buf, int blk, int m,
                                                  int kg) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int p = c.pos + 4 * kg + 2 * i;
      const uint32_t live = (c.ok && p >= sp.lo && p < sp.hi ? 0xFFFFu : 0u) |
                            (c.ok && p + 1 >= sp.lo && p + 1 < sp.hi ? 0xFFFF0000u : 0u);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        c.p[g][i] &= live;
        if constexpr (!SYM) c.p[g][2 + i] &= live;
        const uint32_t x = c.p[g][i] & 0xFFFFu, y = c.p[g][i] >> 16;
        top = x > top ? x : top;
        top = y > top ? y : top;
      }
    }
    top = wave_max(top);
    // exponent field of the largest scale; where all are subnormal they stay
    // as they are
    const uint32_t e = top >> 10;
    const float inv = __uint_as_float((e ? 142 - e : 127) << 23);
    if (m == 0 && kg == 0) {
      float* ex = (float*)(buf + kEx);
      // -inf takes keys that do not exist out of the softmax
      ex[blk] = c.ok ? (e ? (float)((int)e - 15) : 0.0f) : kNegInf;
      ex[4 + blk] = inv;
    }
    uint8_t* vb = buf + kTK * KP + blk * 32 + (kg & 1) * 16 + (kg >> 1) * 8;
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
        uint32_t lo[2], hi[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w = byte_pair<NS>(c.d, 2 * i * NS + b, (2 * i + 1) * NS + b);
          lo[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, nib.lo(w, n1[i])) * S2[i]);
          hi[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, nib.hi(w, n2[i])) * S2[i]);
        }
        *(uint2*)(vb + (32 * b + 2 * m) * VP) = make_uint2(lo[0], lo[1]);
        *(uint2*)(vb + (32 * b + 2 * m + 1) * VP) = make_uint2(hi[0], hi[1]);
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
    e = e < -60 ? -60 : (e > 100 ? 100 : e);
    const float f = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
    A = a.scale_log2 * __uint_as_float((uint32_t)(127 - 14 + e) << 23);
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
  __device__ __forceinline__ void attend(const Kv4Attn& a, const Seq& s, int row0, int u, const uint8_t* buf,
                                         int n, int hf) {
    f32x16 x[2];
#pragma unroll
    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        f32x16 acc;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
#pragma unroll
        for (int st = 2 * g * SPG; st < 2 * (g + 1) * SPG; ++st) {
          const f16x8 kf = *(const f16x8*)(buf + (32 * tt + n) * KP + st * 32 + hf * 16);
          acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, q[st], acc, 0, 0, 0);
        }
        const f16x8* sc = (const f16x8*)(buf + kScale + g * (kTK * 2) + tt * 64 + hf * 32);
        const f16x8 s0 = sc[0], s1 = sc[1];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float S = (float)(i < 8 ? s0[i & 7] : s1[i & 7]);
          x[tt][i] = g == 0 ? S * acc[i] : __builtin_fmaf(S, acc[i], x[tt][i]);
        }
      }
    // whether every row of the wave sees all 64 keys
    const int rows = s.n * a.r;
    const int lastrow = row0 + 32 < rows ? row0 + 31 : rows - 1;
    bool full = u + kTK <= s.kv;
    if (a.causal) full = full && u + kTK - 1 <= s.kv - s.n + div_r(a, row0);
    if (a.window > 0) full = full && u > s.kv - s.n + div_r(a, lastrow) - a.window;
    if (!full) {
      const int pos = s.kv - s.n + div_r(a, row0 + n);
      const int last = a.causal && pos < s.kv - 1 ? pos : s.kv - 1;
      const int first = a.window > 0 ? pos - a.window + 1 : 0;
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = u + 32 * tt + 8 * (i / 4) + 4 * hf + (i & 3);
          x[tt][i] = j <= last && j >= first ? x[tt][i] : kNegInf;
        }
    }
    // per 16 keys, P gets the factor 2^E of their values
    const float4 ev = *(const float4*)(buf + kEx), ei = *(const float4*)(buf + kEx + 16);
    const float evv[4] = {ev.x, ev.y, ev.z, ev.w}, eiv[4] = {ei.x, ei.y, ei.z, ei.w};
    float top = kNegInf;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      float t = x[b >> 1][8 * (b & 1)];
#pragma unroll
      for (int i = 1; i < 8; ++i) t = fmaxf(t, x[b >> 1][8 * (b & 1) + i]);
      top = fmaxf(top, __builtin_fmaf(t, A, evv[b]));
    }
    if (__any(top > mref + kSlack)) {
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
    f16x8 pw[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const float nm = evv[b] - (mref == kNegInf ? 0.0f : mref);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e = exp2_hw(__builtin_fmaf(x[b >> 1][8 * (b & 1) + i], A, nm));
        sum += e;
        pw[b][i] = (_Float16)e;
      }
      l = __builtin_fmaf(sum, eiv[b], l);
    }
    const uint8_t* vb = buf + kTK * KP;
#pragma unroll
    for (int st = 0; st < 4; ++st)
#pragma unroll
      for (int d = 0; d < NS; ++d) {
        const f16x8 vf = *(const f16x8*)(vb + (32 * d + n) * VP + st * 32 + hf * 16);
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, pw[st], o[d], 0, 0, 0);
      }
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

template <int D, int NG, bool SYM>
__global__ __launch_bounds__(tile_waves(D) * 64, tile_waves(D) / 4) void kv4_tile_kernel(Kv4Attn a) {
  using T = Tile<D, NG, SYM>;
  constexpr bool kBoth = T::NW == 4;   // a wave expands keys and values of its block; else one of them
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * T::kBuf];
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
  if (at < sh.end) {
    Seq s = wave_seq(a, cur.b);
    for (;;) {
      const Span sp = get_span<T::TQ>(a, s, cur.qt);
      const int j0 = cur.off, left = (int)(sh.end - at);
      const int j1 = sp.cnt - j0 < left ? sp.cnt : j0 + left;
      const bool starts = j0 == 0, ends = j1 == sp.cnt;
      const int row0 = cur.qt * T::TQ + wave * 32;
      // the run's keys, 64 at a time
      const int64_t cut = (int64_t)(sp.t0 + j1) << a.grain;
      const int stop = cut < sp.hi ? (int)cut : sp.hi;
      int u0 = (sp.t0 + j0) << a.grain;
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
      st.load_q(a, s, cur.h, row0 + n, hf);
      fetch(page_of(u0), u0);
      expand(smem);
      int64_t next = page_of(u0 + kTK);
      __syncthreads();
      for (int u = u0, b = 0; u < stop; u += kTK, b ^= 1) {
        const bool more = u + kTK < stop;
        if (more) {
          fetch(next, u + kTK);
          next = page_of(u + 2 * kTK);
        }
        if (row0 < s.n * a.r) st.attend(a, s, row0, u, smem + b * T::kBuf, n, hf);
        if (more) expand(smem + (b ^ 1) * T::kBuf);
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
  if (threadIdx.x == 0) leave_meta(a, sh, last, cur);
}

template <int D, int NG>
hipError_t launch_tile(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s) {
  if (a.c.sym)
    hipLaunchKernelGGL((kv4_tile_kernel<D, NG, true>), dim3(a.workers), dim3(Tile<D, NG, true>::NW * 64), 0, s, a);
  else
    hipLaunchKernelGGL((kv4_tile_kernel<D, NG, false>), dim3(a.workers), dim3(Tile<D, NG, true>::NW * 64), 0, s, a);
  if (hipError_t e = hipGetLastError()) return e;
  return launch_join<D, Tile<D, NG, true>::TQ, 1>(a, p.tile_rows, s);
}

}  // namespace kv4
}  // namespace gq
