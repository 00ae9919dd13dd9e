// Attention over the 8-bit cache for many query rows (prompts, long chunks): the 4-bit
// cache's scheme (kv4_tile.h) with its query side, split and join.  A workgroup takes 32
// rows for each of its waves and walks over the keys 64 at a time; the waves expand the
// codes of 64 keys and values to fp16 integers into LDS once, then every wave multiplies
// all 64 with its own rows.  Codes are exact as fp16 and a block's scales are the same for
// 16 keys, so both products take one part each: the keys' scale is a factor of 16 scores
// at once, the values' goes into the exponent of the weights.
// Bound by vector work beside the products (57 and 49 % busy): a prompt of 4096 with 32 heads of
// 128 on 8 143 us among other calls (962 TFLOP/s) and 145 to 150 in bursts, 512 queries behind 32 K keys 284 to 295
// (960 to 925).  A key tile
// costs 1.7 / 1.95 / 2.25 us at 64 / 96 / 128 channels, a row tile taken up about five of them.
#include "kv8.h"
#include "kv4_tile.h"
#include <type_traits>

namespace gq {
namespace kv8 {

using namespace kv4;

__device__ __forceinline__ f16x2 pair_lo(uint32_t w) {
  const f16x2 off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
  return __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) + off;
}
__device__ __forceinline__ f16x2 pair_hi(uint32_t w) {
  const f16x2 off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
  return __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) + off;
}
__device__ __forceinline__ uint32_t bits(f16x2 v) { return __builtin_bit_cast(uint32_t, v); }

template <int D>
struct Tile8 : Tile<D, 1, true, false, false> {
  using Base = Tile<D, 1, true, false, false>;
  using Base::A;
  using Base::l;
  using Base::mref;
  using Base::o;
  using Base::q;
  float ltop;      // log2 of the largest value scale so far
  bool steep;
  int full0, full1;   // tiles from positions in between on: every row of the wave sees all 64 keys

  __device__ __forceinline__ void set_full(const Kv4Attn& a, const Seq& s, int row0) {
    const int rows = s.n * a.r, last = row0 + 32 < rows ? row0 + 31 : rows - 1, p = s.kv - s.n;
    full1 = s.kv - kTK;
    if (a.causal) full1 = min(full1, p + div_r(a, row0) - (kTK - 1));
    full0 = a.window > 0 ? p + div_r(a, last) - a.window + 1 : 0;
  }
  static constexpr int NS = D / 32, NW = Base::NW, TQ = Base::TQ, KP = Base::KP, VP = kTK * 2;
  static constexpr int kV = kTK * KP;                 // the values, behind the keys
  static constexpr int kEx = kV + D * VP;             // floats {log2 S_V, 2^40 / S_V, S_K} of the four blocks
  static constexpr int kBuf = kEx + 48;
  static_assert(2 * kBuf <= 160 * 1024, "two tiles in LDS");

  // What a wave holds of the next tile: the codes of 16 keys or 16 values.
  struct Codes {
    uint32_t d[2 * NS];
    float S;
    bool ok;

    // p0, s0: codes and scale of the head's first block of page 0; per: blocks of a page.
    __device__ __forceinline__ void load(const uint8_t* p0, const float* s0, uint32_t per, uint32_t n_pages, int page, int in,
                                         uint32_t lane) {
      ok = (uint32_t)page < n_pages;
      const uint64_t blk = ok ? (uint64_t)(uint32_t)page * per + (uint32_t)in : 0;
      const uint8_t* p = p0 + blk * (32 * D);
#pragma unroll
      for (int s = 0; s + 1 < NS; s += 2) {
        const u32x4 w = *(const u32x4*)(p + 512 * s + 16 * lane);
        d[2 * s] = w.x; d[2 * s + 1] = w.y; d[2 * s + 2] = w.z; d[2 * s + 3] = w.w;
      }
      if constexpr (NS % 2) {
        const uint2 w = *(const uint2*)(p + 512 * (NS - 1) + 8 * lane);
        d[2 * NS - 2] = w.x; d[2 * NS - 1] = w.y;
      }
      S = s0[2 * blk];
    }
  };

  // Where piece p (8 keys, 16 bytes) of a channel's 64 values lies in its row of 128 bytes:
  // turned such that 16 rows next to each other, which are read together, and rows 2 NS
  // apart, which are written together, spread over the banks.
  static __device__ __forceinline__ int piece(int row, int p) { return ((p ^ (row >> 1) ^ (row >> 4)) & 7) * 16; }

  // Keys that no row sees are finite integers all the same, and masked later.
  static __device__ __forceinline__ void expand_k(const Codes& c, uint8_t* buf, int blk, int m, int kg) {
    if (m == 0 && kg == 0) ((float*)(buf + kEx))[8 + blk] = c.ok ? c.S : 1.0f;
#pragma unroll
    for (int s = 0; s < NS; ++s)
      *(u32x4*)(buf + (blk * 16 + m) * KP + s * 64 + kg * 16) =
          u32x4{bits(pair_lo(c.d[2 * s])), bits(pair_hi(c.d[2 * s])), bits(pair_lo(c.d[2 * s + 1])), bits(pair_hi(c.d[2 * s + 1]))};
  }
  static __device__ __forceinline__ void expand_v(const Codes& c, uint8_t* buf, int blk, int m, int kg) {
    if (m == 0 && kg == 0) {
      float* ex = (float*)(buf + kEx);
      // -inf takes keys that do not exist out of the softmax
      const float e = c.ok ? __log2f(c.S) : kNegInf;
      ex[blk] = e;
      ex[4 + blk] = c.ok ? exp2_hw(kKv8Shift - e) : 1.0f;
    }
    uint8_t* vb = buf + kV + (kg >> 1) * 8;
#pragma unroll
    for (int t = 0; t < 2 * NS; ++t) {
      const int row = 2 * NS * m + t;
      *(uint2*)(vb + row * VP + piece(row, 2 * blk + (kg & 1))) = make_uint2(bits(pair_lo(c.d[t])), bits(pair_hi(c.d[t])));
    }
  }

  // The queries as they lie, and then as fp16 times a power of two per row (as Base::load_q
  // does in one go): the first codes come in between.
  __device__ __forceinline__ void fetch_q(const Kv4Attn& a, const Seq& s, int h, int row, int hf) {
    const bool ok = row < s.n * a.r;
    const uint16_t* p = a.q;
    const int tok = div_r(a, row);
    if (ok) p += (int64_t)(s.q0 + tok) * a.q_ts + (int64_t)(h * a.r + row - tok * a.r) * a.q_hs;
#pragma unroll
    for (int st = 0; st < D / 16; ++st) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (ok) v = *(const uint4*)(p + 16 * st + 8 * hf);
      q[st] = __builtin_bit_cast(f16x8, u32x4{v.x, v.y, v.z, v.w});
    }
  }
  __device__ __forceinline__ void take_q(const Kv4Attn& a) {
    float mx = 0.0f;
#pragma unroll
    for (int st = 0; st < D / 16; ++st) {
      float x[8];
      Base::widen(a.bf16, q[st], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(x[i]));
    }
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    int e = (int)(__float_as_uint(mx) >> 23) - 127;
    e = e < -112 ? -112 : (e > 127 ? 127 : e);   // 128: infinite or NaN
    const float f = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
    A = a.scale_log2 * __uint_as_float((uint32_t)(127 - 14 + e) << 23);
    if (mx == 0.0f) A = 1.0f;   // all scores are 0
#pragma unroll
    for (int st = 0; st < D / 16; ++st) {
      float x[8];
      Base::widen(a.bf16, q[st], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) q[st][i] = (_Float16)(x[i] * f);
    }
    // A finite reference below all scores and a scale below all: nothing has to be told apart.
    mref = -0x1.fffffep127f;
    ltop = -100.0f;
    // times a scale of 2^121 beyond fp32, or times one of 2^-40 near 0, which makes NaN of a
    // hidden key's -inf
    steep = __any(!(A >= 0x1p-80f && A < 0x1p6f));
    l = 0.0f;
#pragma unroll
    for (int d = 0; d < NS; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  }

  // Writes the rows: to `part`, or as results (of lanes n and n + 32 each gets 8 channels of
  // two pieces, so that stores are 16 bytes).
  __device__ __forceinline__ void finish(const Kv4Attn& a, const Seq& s, int h, int qt, int ri, float* part, int hf) {
    const int row = qt * TQ + ri;
    const float L = l + __shfl_xor(l, 32);
    if (row >= s.n * a.r) return;
    mref -= kKv8Shift;
    if (part) {
#pragma unroll
      for (int d = 0; d < NS; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *(float4*)(part + ri * D + 32 * d + 8 * i + 4 * hf) =
              make_float4(o[d][4 * i] * kKv8Up, o[d][4 * i + 1] * kKv8Up, o[d][4 * i + 2] * kKv8Up, o[d][4 * i + 3] * kKv8Up);
      if (hf == 0) {
        part[TQ * D + ri] = mref;
        part[TQ * D + TQ + ri] = L;
      }
      return;
    }
    const int64_t orow = out_row(a, s, h, row);
    const float inv = L == 0.0f ? 0.0f : kKv8Up / L;
    uint16_t* const out = a.out + orow * D + 8 * hf;
    auto write = [&](auto bf16) {
#pragma unroll
      for (int d = 0; d < NS; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = pack_result<decltype(bf16)::value>(o[d][i + 2 * j] * inv, o[d][i + 2 * j + 1] * inv);
          const auto x = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
          const auto y = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
          *(uint4*)(out + 32 * d + 2 * i) = make_uint4(x[0], y[0], x[1], y[1]);
        }
    };
    if (a.bf16)
      write(std::true_type{});
    else
      write(std::false_type{});
    if (a.lse && hf == 0) a.lse[orow] = Rows<D, 1, 1, true>::lse_of(mref, L);
  }

  // One tile of 64 keys from position u on, in the written order of kv4_tile.h: operands
  // are read kAhead products before their use, the exponentials of 16 keys stand beside the
  // products of the 16 before.
  __device__ __forceinline__ void attend(const Kv4Attn& a, const Seq& s, int row0, int u, const uint8_t* buf, int n, int hf) {
    constexpr int kAhead = 4;
    f16x8 ring[kAhead];
    f32x16 x[2];
    __builtin_amdgcn_s_setprio(1);
    constexpr int kAll = D / 8;
    auto read = [&](int r) { return *(const f16x8*)(buf + (32 * (r & 1) + n) * KP + (r / 2) * 32 + hf * 16); };
#pragma unroll
    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[tt][i] = 0.0f;
#pragma unroll
    for (int r = 0; r < kAhead; ++r) ring[r] = read(r);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int r = 0; r < kAll; ++r) {
      x[r & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[r % kAhead], q[r / 2], x[r & 1], 0, 0, 0);
      if (r + kAhead < kAll) ring[r % kAhead] = read(r + kAhead);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
    const uint8_t* vb = buf + kV;
    // piece(32 d + n, 2 b + hf) by what d and b change of it: an even number
    const uint8_t* vp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) vp[i] = vb + n * VP + piece(n, 2 * i + hf);
    auto read_v = [&](int r) { return *(const f16x8*)(vp[(r / NS ^ r % NS) & 3] + 32 * (r % NS) * VP); };
#pragma unroll
    for (int r = 0; r < kAhead; ++r) ring[r] = read_v(r);
    const float4 ev = *(const float4*)(buf + kEx), ei = *(const float4*)(buf + kEx + 16), ek = *(const float4*)(buf + kEx + 32);
    const float evv[4] = {ev.x, ev.y, ev.z, ev.w}, ekv[4] = {ek.x, ek.y, ek.z, ek.w};
    float eiv[4] = {ei.x, ei.y, ei.z, ei.w};
    // (Minima and maxima start with a number: two operands that might be signalling NaN cost an
    // instruction more each.)
    const float least = fminf(fminf(fminf(fminf(-kNegInf, ev.x), ev.y), ev.z), ev.w);
    ltop = fmaxf(fmaxf(fmaxf(fmaxf(ltop, ev.x), ev.y), ev.z), ev.w);
    // A block that does not exist, or whose values are 2^80 and more smaller than others.
    const bool odd = __builtin_amdgcn_readfirstlane(least < ltop - 80.0f);
    // A query that is not finite makes NaN of what stands where no block is.
    if (u < full0 || u > full1 || odd) {
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
    float Ab[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) Ab[b] = A * ekv[b];
    if (__builtin_expect(steep, 0)) {
#pragma unroll
      for (int b = 0; b < 4; ++b) Ab[b] = kv8_factor(A, ekv[b]);
    }
    float top = kNegInf;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      float t = kNegInf;   // first: a maximum of two products of the matrix cores costs two more instructions
#pragma unroll
      for (int i = 0; i < 8; ++i) t = fmaxf(t, x[b >> 1][8 * (b & 1) + i]);
      top = fmaxf(top, __builtin_fmaf(t, Ab[b], evv[b]));
    }
    if (__any(top > mref + (kTileRoom + kTileSlack))) {
      top = fmaxf(top, __shfl_xor(top, 32)) - kTileRoom;
      const float mn = fmaxf(top, mref);
      // The far case apart and first: 512 queries behind 32 K keys of 256 channels 378 us otherwise, so 364
      // (357 without it).
      const bool far = moves_far(mref, mn);
      if (__builtin_expect(far, 0)) l = sum_at(l, mref, mn);
      const float f = mn == mref ? 1.0f : exp2_hw(mref - mn);
      l *= far ? 1.0f : f;
      mref = mn;
#pragma unroll
      for (int d = 0; d < NS; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= f;
    }
    // Small values' weights times their scale are nothing to the results, but may be most of
    // the sum, and too small for fp32.
    if (__builtin_expect(odd, 0)) {
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (evv[b] < ltop - 80.0f) {
#pragma unroll
          for (int i = 0; i < 8; ++i) l += exp2_hw(__builtin_fmaf(x[b >> 1][8 * (b & 1) + i], Ab[b], kKv8Shift - mref));
          eiv[b] = 0.0f;
        }
    }
    f16x8 pw[2];
    float sum[2];
    auto weigh = [&](int b, int from, int to) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= from && i < to) {
          const float e = exp2_hw(__builtin_fmaf(x[b >> 1][8 * (b & 1) + i], Ab[b], evv[b] - mref));
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
      for (int d = 0; d < NS; ++d) {
        const int r = b * NS + d;
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[r % kAhead], pw[b & 1], o[d], 0, 0, 0);
        if (r + kAhead < 4 * NS) ring[r % kAhead] = read_v(r + kAhead);
        if (b < 3) weigh(b + 1, 8 * d / NS, 8 * (d + 1) / NS);
        __builtin_amdgcn_sched_barrier(0);
      }
    __builtin_amdgcn_s_setprio(0);
  }
};

template <int D>
__global__ __launch_bounds__(tile_waves(D) * 64, tile_waves(D) / 4) void kv8_tile_kernel(Kv8Attn a) {
  using T = Tile8<D>;
  constexpr bool kBoth = T::NW == 4;   // a wave expands keys and values of its block; else one of them
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * T::kBuf];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, kg = lane >> 4, n = lane & 31, hf = lane >> 5;
  const int blk = wave & 3;            // the 16 keys of a tile that this wave expands
  const bool is_k = wave < 4;
  const int ps = a.c.page_shift;
  T st;
  const Share sh = find_share<T::TQ, true>(a, lane);
  uint32_t at = sh.at;
  int last = -1;
  Cursor cur = sh.cur;
  Seq s{0, 0, 0};
  if (at < sh.end) {
    s = wave_seq(a, cur.b);
    for (;;) {
      const int nqt = row_tiles(a, s, T::TQ), qt = tile_at<true>(cur.qt, nqt);   // cur.qt counts in the turned order
      const Span sp = get_span<T::TQ>(a, s, qt);
      const int j0 = cur.off, left = (int)(sh.end - at);
      const int j1 = sp.cnt - j0 < left ? sp.cnt : j0 + left;
      const bool starts = j0 == 0, ends = j1 == sp.cnt;
      const int row0 = qt * T::TQ + wave * 32;
      // the run's keys, 64 at a time
      const int64_t cut = tile_start(a, sp, j1);
      const int stop = cut < sp.hi ? (int)cut : sp.hi;
      int u0 = (int)tile_start(a, sp, j0);
      if (u0 < sp.lo) u0 = sp.lo & ~(kTK - 1);
      const PageRow table = (PageRow)(a.table + cur.b * a.table_b + cur.h * a.table_h);
      // page of this wave's 16 of the 64 keys from u on, -1 where no row sees them
      auto page_of = [&](int u) -> int {
        const int pos = u + blk * 16;
        return pos < stop && pos + 16 > sp.lo ? table[pos >> ps] : -1;
      };
      typename T::Codes ck, cv;   // a wave that expands one of them uses ck for it
      const int64_t head = (int64_t)cur.h << (ps - 4);
      const bool ckv = !kBoth && !is_k;
      const uint8_t* const codes0 = a.c.cache + head * (32 * D) + (ckv ? 16 * D : 0);
      const float* const scales0 = (const float*)(a.scales + head) + (ckv ? 1 : 0);
      const uint32_t per = (uint32_t)a.c.hkv << (ps - 4), n_pages = (uint32_t)a.c.n_pages;
      auto fetch = [&](int page, int u) {
        const int in = ((u + blk * 16) & ((1 << ps) - 1)) >> 4;
        ck.load(codes0, scales0, per, n_pages, page, in, lane);
        if constexpr (kBoth) cv.load(codes0 + 16 * D, scales0 + 1, per, n_pages, page, in, lane);
      };
      auto expand = [&](uint8_t* buf) {
        if constexpr (kBoth) {
          T::expand_k(ck, buf, blk, m, kg);
          T::expand_v(cv, buf, blk, m, kg);
        } else if (is_k) {
          T::expand_k(ck, buf, blk, m, kg);
        } else {
          T::expand_v(ck, buf, blk, m, kg);
        }
      };
      const int page = page_of(u0);
      st.fetch_q(a, s, cur.h, row0 + n, hf);
      fetch(page, u0);
      st.take_q(a);
      st.set_full(a, s, row0);
      expand(smem);
      fetch(page_of(u0 + kTK), u0 + kTK);
      int next = page_of(u0 + 2 * kTK);
      __syncthreads();
      // Codes are fetched a tile before they are expanded.  The waves of keys
      // expand before their products and those of values after: of the two
      // waves of a SIMD one has vector work while the other multiplies.
      auto step = [&](int u, auto which) {
        constexpr int b = decltype(which)::value;
        const bool more = u + kTK < stop;
        auto refill = [&] {
          if (!more) return;
          const int after = page_of(u + 3 * kTK);   // on its way while the codes are expanded
          expand(smem + (b ^ 1) * T::kBuf);
          fetch(next, u + 2 * kTK);
          next = after;
        };
        if (!kBoth && is_k) refill();
        if (row0 < s.n * a.r) st.attend(a, s, row0, u, smem + b * T::kBuf, n, hf);
        if (kBoth || !is_k) refill();
        __syncthreads();
      };
      for (int u = u0; u < stop; u += 2 * kTK) {
        step(u, std::integral_constant<int, 0>{});
        if (u + kTK < stop) step(u + kTK, std::integral_constant<int, 1>{});
      }
      float* part = nullptr;
      if (!(starts && ends)) {
        part = a.part + ((int64_t)2 * sh.w + (starts ? 1 : 0)) * (T::TQ * (D + 2));
        if (starts) last = sh.worker_with(at + sp.cnt - 1);
      }
      st.finish(a, s, cur.h, qt, wave * 32 + n, part, hf);
      at += j1 - j0;
      if (at >= sh.end) {
        cur.qt = qt;
        break;
      }
      cur.off = 0;
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

template <int D>
hipError_t launch_tile_d(const Kv8Attn& a, const Kv4Plan& p, hipStream_t s) {
  using T = Tile8<D>;
  hipLaunchKernelGGL((kv8_tile_kernel<D>), dim3(a.workers), dim3(T::NW * 64), 0, s, a);
  if (hipError_t e = hipGetLastError()) return e;
  // Workgroups for 64 rows of a row tile go over all of them: where nothing was split, which a
  // causal prompt's order often brings about, four times as many took 1 us more to start and end.
  return launch_join<D, T::TQ, 1, true>(a, p.tile_rows < 64 ? p.tile_rows : 64, s);
}

}  // namespace kv8

hipError_t launch_kv8_tile(const Kv8Attn& a, const Kv4Plan& p, hipStream_t s) {
  switch (a.c.d) {
    case 64: return kv8::launch_tile_d<64>(a, p, s);
    case 96: return kv8::launch_tile_d<96>(a, p, s);
    case 128: return kv8::launch_tile_d<128>(a, p, s);
    default: return kv8::launch_tile_d<256>(a, p, s);
  }
}

}  // namespace gq
