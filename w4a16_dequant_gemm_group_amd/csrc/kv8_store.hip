// Appending keys and values to the 8-bit cache, and reading them back.
//
// Appending: one wave per block of 16 tokens and head, for keys and for values, so
// that the scale of a block is found and its codes are written by one wave, without
// exchange.  A workgroup looks through a run of input rows for the first row of each
// block among them (the first of its sequence, or one at a multiple of 16).  Lanes hold
// the channels in the order of the codes (kv8.h): loads of 16 bytes, those of values change
// places in LDS, codes leave in pieces of 16 bytes that make one run.
// 16 K tokens of 8 heads of 128: 32 us (98 MB read, the keys once more for their bounds, and
// 34 MB written: 4.1 TB/s; bound by loads in flight), without bounds and with the inputs in
// cache 24 to 25; read back in 18.4 (101 MB).  One token 4.6.
#include "kv8.h"
#include "kv8_seq.h"
#include "stream_util.h"

namespace gq {
namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
  const uint32_t u = __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
  return u > v ? u : v;
}
// Largest 16-bit half over the wave, as a scalar.
__device__ __forceinline__ uint32_t wave_max16(uint32_t v) {
  v = (v & 0xFFFFu) > v >> 16 ? v & 0xFFFFu : v >> 16;
  v = max_dpp<0x140>(max_dpp<0x141>(max_dpp<0x4E>(max_dpp<0xB1>(v))));   // over rows of 16 lanes
  const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
  const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
  const uint32_t x = a > b ? a : b, y = c > d ? c : d;
  return x > y ? x : y;
}

// Bits of infinity of a 16-bit type; the bits of absolute values are ordered as they are.
template <bool BF16>
constexpr uint32_t kInf = BF16 ? 0x7F80u : 0x7C00u;

// A pair of values as they count: NaN as 0, infinities as the largest of the type.
template <bool BF16>
__device__ __forceinline__ uint32_t clean(uint32_t w) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h = w >> (16 * i) & 0xFFFFu;
    const uint32_t m = h & 0x7FFFu;
    h = m > kInf<BF16> ? 0u : m == kInf<BF16> ? h - 1 : h;
    r |= h << (16 * i);
  }
  return r;
}

template <bool BF16>
__device__ __forceinline__ float lo_of(uint32_t w) {
  return BF16 ? __uint_as_float(w << 16) : f16_to_f32((uint16_t)(w & 0xFFFFu));
}
template <bool BF16>
__device__ __forceinline__ float hi_of(uint32_t w) {
  return BF16 ? __uint_as_float(w & 0xFFFF0000u) : f16_to_f32((uint16_t)(w >> 16));
}

// Largest absolute value of the wave's pairs, which are cleaned if any is not finite.
template <bool BF16, int N>
__device__ __forceinline__ float largest(uint32_t (&w)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = pk_max(m, w[i] & 0x7FFF7FFFu);
  uint32_t top = wave_max16(m);
  if (top >= kInf<BF16>) {
    m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w[i] = clean<BF16>(w[i]);
      m = pk_max(m, w[i] & 0x7FFF7FFFu);
    }
    top = wave_max16(m);
  }
  return lo_of<BF16>(top);
}

// round(x / S), half to even, plus 128, as the low byte of kMagic + it.  x times the
// rounded 1 / S is off by at most 2^-17 for |x| <= 127 S (and a little), so wherever
// it lies 2^-16 and more from k + 1/2, its rounding is that of the quotient.
constexpr float kMagic = 12582912.0f + 128.0f, kEdge = 0.5f - 0x1p-16f;
// The same exactly: the quotient in fp32 is at most one step off, and only beside
// k + 1/2; the rest x - k S is exact (a multiple of S's ulp below 2 S; where x's own ulp
// is finer, k is 0).
__device__ __forceinline__ float exact_code(float x, float S, float inv) {
  float k = __builtin_rintf(x * inv);
  const float e = __builtin_fmaf(-k, S, x), d = fabsf(e) + fabsf(e);
  const bool odd = ((int)k & 1) != 0;
  const bool off = (d > S) | ((d == S) & odd);
  return k + (off ? __builtin_copysignf(1.0f, e) : 0.0f) + kMagic;
}
__device__ __forceinline__ uint32_t pack4(const float (&t)[4]) {
  const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(t[1]), __float_as_uint(t[0]), 0x0C0C0400u);
  const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(t[3]), __float_as_uint(t[2]), 0x04000C0Cu);
  return lo | hi;
}
// Codes of four values.  Some 5 instructions each, and the exact form only where a value
// of the wave lies beside a border: half of a block's largest always does, so that with one
// test per block nearly every block took it (16 K tokens 36 us, so 28).
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], float S, float inv) {
  float t[4], edge = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = __builtin_fmaf(x[i], inv, kMagic);
    edge = fmaxf(edge, fabsf(__builtin_fmaf(x[i], inv, kMagic - t[i])));
  }
  if (__any(edge >= kEdge)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = exact_code(x[i], S, inv);
  }
  return pack4(t);
}
template <bool BF16>
__device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, float S, float inv) {
  const float x[4] = {lo_of<BF16>(a), hi_of<BF16>(a), lo_of<BF16>(b), hi_of<BF16>(b)};
  return codes4(x, S, inv);
}

// Codes of an older scale: round(q S0 / S1), half to even, as it is exactly: products of
// a code and a scale are exact in binary64, and so is what the rounded quotient leaves.
__device__ __forceinline__ uint32_t requantise(uint32_t w, double s0, double s1, double ratio) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double q = (double)((int)(w >> (8 * i) & 255u) - 128);
    const double k = __builtin_rint(q * ratio);
    const double e = __builtin_fma(-k, s1, q * s0), d = __builtin_fabs(e + e);
    const int n = (int)k;
    const bool off = (d > s1) | ((d == s1) & ((n & 1) != 0));
    r |= (uint32_t)(n + 128 + (off ? (e < 0.0 ? -1 : 1) : 0)) << (8 * i);
  }
  __builtin_amdgcn_sched_barrier(0);   // one after another: few registers, where time does not matter
  return r;
}

// What a wave does to one block: new tokens a .. e - 1 of its 16 (the first one is row
// t of the input), older ones before a; where it lies.
struct Part {
  int64_t t;
  int a, e;
  int64_t page;
  int in_page;
};

__device__ __forceinline__ float block_scale(float mx, float s0) {
  return fmaxf(fmaxf(mx / 127.0f, s0), kKv8Least);
}

// Offset of a lane's dword i of the 2 NS it has of a block's keys (or values).
template <int NS>
__device__ __forceinline__ int code_offset(int i, int lane) {
  return i >= NS / 2 * 4 ? 256 * (NS / 2 * 4) + 8 * lane + 4 * (i & 1) : 1024 * (i / 4) + 16 * lane + 4 * (i & 3);
}
template <int NS>
__device__ __forceinline__ void load_codes(const uint8_t* p, int lane, uint32_t (&w)[2 * NS]) {
#pragma unroll
  for (int i = 0; i + 3 < 2 * NS; i += 4) {
    const uint4 v = *(const uint4*)(p + code_offset<NS>(i, lane));
    w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
  }
  if constexpr (NS % 2) {
    const uint2 v = *(const uint2*)(p + code_offset<NS>(2 * NS - 2, lane));
    w[2 * NS - 2] = v.x; w[2 * NS - 1] = v.y;
  }
}
template <int NS>
__device__ __forceinline__ void store_codes(uint8_t* p, int lane, const uint32_t (&w)[2 * NS]) {
#pragma unroll
  for (int i = 0; i + 3 < 2 * NS; i += 4)
    *(uint4*)(p + code_offset<NS>(i, lane)) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  if constexpr (NS % 2) *(uint2*)(p + code_offset<NS>(2 * NS - 2, lane)) = make_uint2(w[2 * NS - 2], w[2 * NS - 1]);
}

// Keys: a lane holds 8 channels of token m for each of the NS steps.
template <int D>
__device__ __forceinline__ void load_keys(const Kv8Append& a, const Part& p, int h, int lane, uint32_t (&raw)[D / 8]) {
  const int m = lane & 15, kg = lane >> 4;
  const bool fresh = m >= p.a && m < p.e;
  const uint16_t* row = a.k + h * a.k_hs + (p.t + (m - p.a)) * a.k_ts + 8 * kg;
#pragma unroll
  for (int s = 0; s < D / 32; ++s) {
    const uint4 v = fresh ? *(const uint4*)(row + 32 * s) : make_uint4(0, 0, 0, 0);
    raw[4 * s] = v.x; raw[4 * s + 1] = v.y; raw[4 * s + 2] = v.z; raw[4 * s + 3] = v.w;
  }
}
template <int D, bool BF16>
__device__ __forceinline__ void write_keys(const Kv8Append& a, const Part& p, int h, int lane, uint32_t (&raw)[D / 8]) {
  constexpr int NS = D / 32;
  const int m = lane & 15;
  const int64_t blk = kv8_block(p.page, a.c.hkv, h, a.c.page_shift, p.in_page);
  uint8_t* codes = a.c.cache + blk * (32 * D);
  float* scale = (float*)(a.c.scales + blk);
  float s0 = 0.0f;
  uint32_t old[2 * NS];
  if (p.a > 0) {
    s0 = *scale;
    load_codes<NS>(codes, lane, old);
  }
  const float S = block_scale(largest<BF16>(raw), s0), inv = 1.0f / S;
  uint32_t w[2 * NS];
#pragma unroll
  for (int i = 0; i < 2 * NS; ++i) w[i] = codes4<BF16>(raw[2 * i], raw[2 * i + 1], S, inv);
  if (m < p.a) {
#pragma unroll
    for (int i = 0; i < 2 * NS; ++i) w[i] = S == s0 ? old[i] : requantise(old[i], s0, S, (double)s0 / S);
  }
  store_codes<NS>(codes, lane, w);
  if (lane == 0) *scale = S;
}

// Values are loaded as they lie, 8 channels of a token per lane (loads of 4 bytes in the
// order of the codes took 7 us more for 16 K tokens): D / 8 lanes hold a token, 96 channels
// 12 of 16.  Register j of a lane holds the j-th of its tokens.  They pass the caches by, which
// leaves room for the keys, that bounds are made of too (16 K tokens 34 us, so 32).
template <int D>
struct Load {
  static constexpr int P = D == 96 ? 16 : D / 8;   // lanes of a token
  static constexpr int R = 64 / P, N = 16 / R;     // tokens of a load, loads of a block
};
template <int D>
__device__ __forceinline__ void load_values(const Kv8Append& a, const Part& p, int h, int lane, uint32_t (&raw)[4 * Load<D>::N]) {
  using L = Load<D>;
  const int c = lane % L::P;
  const uint16_t* row = a.v + h * a.v_hs + 8 * c;
#pragma unroll
  for (int j = 0; j < L::N; ++j) {
    const int tok = L::R * j + lane / L::P;
    const bool fresh = tok >= p.a && tok < p.e && c < D / 8;
    u32x4 v = {0, 0, 0, 0};
    if (fresh) v = __builtin_nontemporal_load((const u32x4*)(row + (p.t + (tok - p.a)) * a.v_ts));
    raw[4 * j] = v.x; raw[4 * j + 1] = v.y; raw[4 * j + 2] = v.z; raw[4 * j + 3] = v.w;
  }
}
// The codes' own order takes four tokens of a channel in one dword.  They change places
// in LDS: 16 rows (tokens) of D bytes, written as loaded, read as dwords of 4 channels of 4
// tokens, whose bytes are then transposed.
template <int D>
constexpr int kTurnPitch = D + 16;

// What the wave's lanes wrote to LDS before is what they read behind it.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int D, bool BF16>
__device__ __forceinline__ void write_values(const Kv8Append& a, const Part& p, int h, int lane, uint32_t (&raw)[4 * Load<D>::N],
                                             uint8_t* turn) {
  constexpr int NS = D / 32, T = 2 * NS;
  using L = Load<D>;
  const int m = lane & 15, kg = lane >> 4;
  const int64_t blk = kv8_block(p.page, a.c.hkv, h, a.c.page_shift, p.in_page);
  uint8_t* codes = a.c.cache + blk * (32 * D) + 16 * D;
  float* scale = (float*)(a.c.scales + blk) + 1;
  float s0 = 0.0f;
  uint32_t old[T];
  if (p.a > 0) {
    s0 = *scale;
    load_codes<NS>(codes, lane, old);
  }
  const float S = block_scale(largest<BF16>(raw), s0), inv = 1.0f / S;
#pragma unroll
  for (int j = 0; j < L::N; ++j) {
    const uint2 w = make_uint2(codes4<BF16>(raw[4 * j], raw[4 * j + 1], S, inv), codes4<BF16>(raw[4 * j + 2], raw[4 * j + 3], S, inv));
    if (D != 96 || lane % L::P < 12) *(uint2*)(turn + (L::R * j + lane / L::P) * kTurnPitch<D> + 8 * (lane % L::P)) = w;
  }
  wave_fence();
  uint32_t w[T];
  const uint8_t* at = turn + 4 * kg * kTurnPitch<D> + T * m;
  if constexpr (T % 4 == 0) {
    uint32_t x[4][T / 4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int g = 0; g < T / 4; ++g) x[i][g] = ((const uint32_t*)(at + i * kTurnPitch<D>))[g];
#pragma unroll
    for (int g = 0; g < T / 4; ++g) {
      const uint32_t a0 = __builtin_amdgcn_perm(x[1][g], x[0][g], 0x05010400u), a1 = __builtin_amdgcn_perm(x[1][g], x[0][g], 0x07030602u);
      const uint32_t b0 = __builtin_amdgcn_perm(x[3][g], x[2][g], 0x05010400u), b1 = __builtin_amdgcn_perm(x[3][g], x[2][g], 0x07030602u);
      w[4 * g] = __builtin_amdgcn_perm(b0, a0, 0x05040100u);
      w[4 * g + 1] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
      w[4 * g + 2] = __builtin_amdgcn_perm(b1, a1, 0x05040100u);
      w[4 * g + 3] = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
    }
  } else {
#pragma unroll
    for (int t = 0; t < T; t += 2) {
      uint32_t x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = *(const uint16_t*)(at + i * kTurnPitch<D> + t);
      const uint32_t u = x[0] | x[1] << 16, v = x[2] | x[3] << 16;
      w[t] = __builtin_amdgcn_perm(v, u, 0x06040200u);
      w[t + 1] = __builtin_amdgcn_perm(v, u, 0x07050301u);
    }
  }
  wave_fence();
  // which of the lane's four tokens are older ones
  const int older = p.a - 4 * kg;
  if (older > 0) {
    const uint32_t keep = older >= 4 ? 0xFFFFFFFFu : (1u << (8 * older)) - 1u;
#pragma unroll
    for (int i = 0; i < T; ++i) w[i] = ((S == s0 ? old[i] : requantise(old[i], s0, S, (double)s0 / S)) & keep) | (w[i] & ~keep);
  }
  store_codes<NS>(codes, lane, w);
  if (lane == 0) *scale = S;
}

// 16-bit floats as integers of the same order (a pair), and back: the map is its own inverse.
__device__ __forceinline__ uint32_t ordered(uint32_t w) {
  const i16x2 v = __builtin_bit_cast(i16x2, w);
  return w ^ (__builtin_bit_cast(uint32_t, v >> 15) & 0x7FFF7FFFu);
}
__device__ __forceinline__ uint32_t pk_min_i(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(i16x2, a), __builtin_bit_cast(i16x2, b)));
}
__device__ __forceinline__ uint32_t pk_max_i(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(i16x2, a), __builtin_bit_cast(i16x2, b)));
}

// The bounds of one page, by the two waves of a workgroup: D / 8 lanes hold a key.
template <int D, bool BF16>
__device__ __forceinline__ void write_bounds(const Kv8Append& a, int h, int64_t page, int64_t t, int n, bool older,
                                             uint4 (*smem)[2]) {
  constexpr int L = D / 8, R = 64 / L, G = 2 * R;   // lanes of a key, keys of a wave and of both
  constexpr uint32_t kMost = 0x7FFF7FFFu, kLeast = 0x80008000u;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane % L, g = wave * R + lane / L;
  const uint16_t* k = a.k + h * a.k_hs + t * a.k_ts + 8 * c;
  uint32_t lo[4] = {kMost, kMost, kMost, kMost}, hi[4] = {kLeast, kLeast, kLeast, kLeast};
  if (lane < L * R) {
    uint32_t top = 0;
    auto take = [&](uint32_t (&w)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t o = ordered(w[i]);
        lo[i] = pk_min_i(lo[i], o);
        hi[i] = pk_max_i(hi[i], o);
      }
    };
#pragma unroll 4
    for (int j = g; j < n; j += G) {
      const uint4 v = *(const uint4*)(k + j * a.k_ts);
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) top = pk_max(top, w[i] & 0x7FFF7FFFu);
      take(w);
    }
    if ((top & 0xFFFFu) >= kInf<BF16> || top >> 16 >= kInf<BF16>) {
      // some value of this lane is not finite: once more, cleaned
#pragma unroll
      for (int i = 0; i < 4; ++i) { lo[i] = kMost; hi[i] = kLeast; }
      for (int j = g; j < n; j += G) {
        const uint4 v = *(const uint4*)(k + j * a.k_ts);
        uint32_t w[4] = {clean<BF16>(v.x), clean<BF16>(v.y), clean<BF16>(v.z), clean<BF16>(v.w)};
        take(w);
      }
    }
    smem[g * L + c][0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    smem[g * L + c][1] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
  __syncthreads();
  // pair x of the smallest and of the largest
  if (threadIdx.x < D / 2) {
    const int x = threadIdx.x;
    uint32_t* bounds = (uint32_t*)(a.bounds + (page * a.c.hkv + h) * (2 * D));
    uint32_t u = kMost, v = kLeast;
    for (int j = 0; j < G; ++j) {
      u = pk_min_i(u, ((const uint32_t*)&smem[j * L + x / 4][0])[x % 4]);
      v = pk_max_i(v, ((const uint32_t*)&smem[j * L + x / 4][1])[x % 4]);
    }
    if (older) {
      u = pk_min_i(u, ordered(bounds[x]));
      v = pk_max_i(v, ordered(bounds[D / 2 + x]));
    }
    bounds[x] = ordered(u);
    bounds[D / 2 + x] = ordered(v);
  }
  __syncthreads();
}

// The heads of one block, from the workgroup's first one on: the rows of the next head are
// on their way while one's codes are made, and those of the first while its page is looked up.
template <int D, bool BF16, bool KEYS>
__device__ __forceinline__ void write_heads(const Kv8Append& a, const Part& p, int lane, uint8_t* turn) {
  constexpr int N = KEYS ? D / 8 : 4 * Load<D>::N;
  uint32_t raw[N], next[N];
  auto load = [&](int h, uint32_t (&r)[N]) {
    if constexpr (KEYS) load_keys<D>(a, p, h, lane, r);
    else load_values<D>(a, p, h, lane, r);
  };
  load(blockIdx.y, raw);
  if (p.page < 0 || p.page >= a.c.n_pages) return;
  for (int h = blockIdx.y;;) {
    const int hn = h + gridDim.y;
    if (hn < a.c.hkv) load(hn, next);
    if constexpr (KEYS) write_keys<D, BF16>(a, p, h, lane, raw);
    else write_values<D, BF16>(a, p, h, lane, raw, turn);
    if (hn >= a.c.hkv) return;
    h = hn;
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = next[i];
  }
}

// grid.y: heads (or as many of them as run at once); grid.z: bounds, blocks (a wave for keys, a
// wave for values).
template <int D, bool BF16>
__global__ __launch_bounds__(128) void kv8_append_kernel(Kv8Append a) {
  __shared__ uint4 smem[16 * kTurnPitch<D> > 4096 ? 16 * kTurnPitch<D> / 32 : 128][2];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool pages = blockIdx.z + 1 < gridDim.z;   // first, as theirs is the longest chain of loads
  const int ps = a.c.page_shift, unit = pages ? ps : 4, run = pages ? a.page_run : a.run;
  const int64_t cap = a.table_pages << ps;
  // Workgroups go round robin over 8 dies: the blocks of a page to the one where its bounds are
  // made, which reads the same keys (16 K tokens 36 us, so 34).
  uint32_t first = blockIdx.x;
  if (!pages && run == 16) {
    const uint32_t all = 8u << (ps - 4), in = first & (all - 1);
    if (first - in + all <= gridDim.x) first = first - in + ((in & 7) << (ps - 4)) + (in >> 3);
  }
  for (int64_t r0 = (int64_t)first * run; r0 < a.tokens; r0 += (int64_t)gridDim.x * run) {
    const int64_t r1 = r0 + run < a.tokens ? r0 + run : a.tokens;
    int64_t t = r0;
    while (t < r1) {
      const RowSeq s = seq_of_row(a.starts, a.kv_lens, a.batch, a.tokens, t, lane);
      if (s.b < 0) { ++t; continue; }
      const int64_t end = s.first + s.n, p0 = (int64_t)s.kv - s.n;   // position of its first row
      const int32_t* table = a.table + s.b * a.table_pages;
      while (t < end && t < r1) {
        const int64_t pos = p0 + (t - s.first);
        if (pos < 0) { t = t - pos < end ? t - pos : end; continue; }
        if (pos >= cap) { t = end; break; }
        const int in = (int)(pos & ((1 << unit) - 1));
        const int64_t left = end - t, room = (1 << unit) - in;
        const int n = (int)(left < room ? left : room);
        // the first row of its block (page) that the call brings
        if (in == 0 || t == s.first) {
          const int64_t page = table[pos >> ps];
          if (pages) {
            if (page >= 0 && page < a.c.n_pages)
              for (int h = blockIdx.y; h < a.c.hkv; h += gridDim.y) write_bounds<D, BF16>(a, h, page, t, n, in > 0, smem);
          } else {
            const Part p{t, in, in + n, page, (int)(pos & ((1 << ps) - 1))};
            if (wave == 0)
              write_heads<D, BF16, true>(a, p, lane, nullptr);
            else
              write_heads<D, BF16, false>(a, p, lane, (uint8_t*)smem);
          }
        }
        t += n;
      }
    }
  }
}

// Reading back: a lane holds 8 channels of one row's key and value.
template <int D>
__global__ __launch_bounds__(256) void kv8_read_kernel(Kv8Geo c, const int64_t* __restrict__ slots, int64_t tokens,
                                                       void* __restrict__ k, void* __restrict__ v, gq_dtype odt) {
  constexpr int L = D / 8, R = 256 / L, NS = D / 32;
  const int row = threadIdx.x / L, lane = threadIdx.x % L, h = blockIdx.y;
  const int64_t t = (int64_t)blockIdx.x * R + row;
  if (row >= R || t >= tokens) return;
  const int64_t slot = slots[t];
  float kx[8], vx[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) kx[i] = vx[i] = 0.0f;
  if (slot >= 0 && slot < c.n_pages << c.page_shift) {
    const int in = (int)(slot & ((1 << c.page_shift) - 1)), m = in & 15;
    const int64_t blk = kv8_block(slot >> c.page_shift, c.hkv, h, c.page_shift, in);
    const uint8_t* codes = c.cache + blk * (32 * D);
    const int s = lane >> 2, kg = lane & 3;
    const bool odd = NS % 2 && s == NS - 1;
    const uint2 kw = *(const uint2*)(codes + 512 * (s & ~1) + (odd ? 8 : 16) * (kg * 16 + m) + 8 * (s & 1));
    const float2 S = c.scales[blk];
    // channel 8 lane + i is row r of tile t; byte m % 4 of the dword of its four tokens
    const uint8_t* vc = codes + 16 * D;
    const int sh = 8 * (m & 3);
    uint32_t w[8];
    if constexpr (NS % 2 == 0) {
      // the channels lie in one row (64 channels: in two), in tiles by fours
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int ch = 8 * lane + 4 * g, r = ch / (2 * NS), t = ch % (2 * NS);
        const uint4 u = *(const uint4*)(vc + 1024 * (t / 4) + 16 * ((m >> 2) * 16 + r));
        w[4 * g] = u.x; w[4 * g + 1] = u.y; w[4 * g + 2] = u.z; w[4 * g + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int ch = 8 * lane + i, r = ch / (2 * NS), t = ch % (2 * NS), at = (m >> 2) * 16 + r;
        w[i] = *(const uint32_t*)(vc + 1024 * (t / 4) + (t >= 2 * NS / 4 * 4 ? 8 : 16) * at + 4 * (t % 4));
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      vx[i] = (float)((int)(w[i] >> sh & 255u) - 128) * S.y;
      kx[i] = (float)((int)((i < 4 ? kw.x : kw.y) >> (8 * (i & 3)) & 255u) - 128) * S.x;
    }
  }
  const int64_t o = (t * c.hkv + h) * D + 8 * lane;
  if (odt == GQ_F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ((float4*)((float*)k + o))[i] = make_float4(kx[4 * i], kx[4 * i + 1], kx[4 * i + 2], kx[4 * i + 3]);
      ((float4*)((float*)v + o))[i] = make_float4(vx[4 * i], vx[4 * i + 1], vx[4 * i + 2], vx[4 * i + 3]);
    }
    return;
  }
  auto two = [&](float a, float b) {
    return odt == GQ_BF16 ? f32_to_bf16_rne(a) | (uint32_t)f32_to_bf16_rne(b) << 16
                          : stream_util::f32_to_f16_rne(a) | (uint32_t)stream_util::f32_to_f16_rne(b) << 16;
  };
  *(uint4*)((uint16_t*)k + o) = make_uint4(two(kx[0], kx[1]), two(kx[2], kx[3]), two(kx[4], kx[5]), two(kx[6], kx[7]));
  *(uint4*)((uint16_t*)v + o) = make_uint4(two(vx[0], vx[1]), two(vx[2], vx[3]), two(vx[4], vx[5]), two(vx[6], vx[7]));
}

template <int D>
hipError_t append_d(const Kv8Append& a, gq_dtype dt, dim3 grid, hipStream_t s) {
  if (dt == GQ_BF16)
    hipLaunchKernelGGL((kv8_append_kernel<D, true>), grid, dim3(128), 0, s, a);
  else
    hipLaunchKernelGGL((kv8_append_kernel<D, false>), grid, dim3(128), 0, s, a);
  return hipGetLastError();
}

template <int D>
hipError_t read_d(const Kv8Geo& c, const int64_t* slots, int64_t tokens, void* k, void* v, gq_dtype odt, hipStream_t s) {
  constexpr int R = 256 / (D / 8);
  // at most 2^32 threads along the grid's first dimension
  constexpr int64_t kLaunch = (int64_t)1 << 24;
  const int64_t row = (int64_t)c.hkv * D * (odt == GQ_F32 ? 4 : 2);
  for (int64_t t = 0; t < tokens; t += kLaunch) {
    const int64_t n = tokens - t < kLaunch ? tokens - t : kLaunch;
    hipLaunchKernelGGL((kv8_read_kernel<D>), dim3((unsigned)((n + R - 1) / R), c.hkv), dim3(256), 0, s, c, slots + t, n,
                       (uint8_t*)k + t * row, (uint8_t*)v + t * row, odt);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_kv8_append(const Kv8Append& in, gq_dtype dt, hipStream_t s) {
  Kv8Append a = in;
  // A run holds about one block.  Few tokens, or few per sequence: a run each, so
  // that no wave has several blocks to do one after another.
  a.run = a.starts && a.tokens >= 16 * a.batch ? 16 : 1;
  a.page_run = a.run == 1 ? 1 : 1 << a.c.page_shift;
  const int64_t runs = (a.tokens + a.run - 1) / a.run;
  // a workgroup per head until they fill the card
  int heads = a.c.hkv;
  while (heads > 1 && runs * heads > 4096) heads = (heads + 1) / 2;
  const dim3 grid((unsigned)(runs < (1 << 20) ? runs : 1 << 20), heads, a.bounds ? 2 : 1);
  switch (a.c.d) {
    case 64: return append_d<64>(a, dt, grid, s);
    case 96: return append_d<96>(a, dt, grid, s);
    case 128: return append_d<128>(a, dt, grid, s);
    default: return append_d<256>(a, dt, grid, s);
  }
}

hipError_t launch_kv8_read(const Kv8Geo& c, const int64_t* slots, int64_t tokens, void* k, void* v, gq_dtype odt,
                           hipStream_t s) {
  switch (c.d) {
    case 64: return read_d<64>(c, slots, tokens, k, v, odt, s);
    case 96: return read_d<96>(c, slots, tokens, k, v, odt, s);
    case 128: return read_d<128>(c, slots, tokens, k, v, odt, s);
    default: return read_d<256>(c, slots, tokens, k, v, odt, s);
  }
}

}  // namespace gq
