// Appending keys and values to the 8-bit cache, and reading them back.
//
// Appending: one wave per block of 16 tokens and head, for keys and for values, so
// that the scale of a block is found and its codes are written by one wave, without
// exchange.  A workgroup looks through a run of input rows for the first row of each
// block among them (the first of its sequence, or one at a multiple of 16).  Lanes hold
// the channels in the order of the codes (kv8.h): keys in loads of 16 bytes, values of
// four tokens in loads of 4, codes leave in pieces of 16 bytes that make one run.
#include "kv8.h"
#include "kv8_seq.h"
#include "stream_util.h"

namespace gq {
namespace {

using stream_util::dpp_f32;

__device__ __forceinline__ float max2(float a, float b) {
  float r;
  asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

// Largest value over the wave, in every lane.
__device__ __forceinline__ float wave_max(float v) {
  v = max2(v, dpp_f32<0xB1, 0xF>(v));    // quad_perm [1,0,3,2]
  v = max2(v, dpp_f32<0x4E, 0xF>(v));    // quad_perm [2,3,0,1]
  v = max2(v, dpp_f32<0x141, 0xF>(v));   // row_half_mirror: 8 lanes
  v = max2(v, dpp_f32<0x140, 0xF>(v));   // row_mirror: 16 lanes
  v = max2(v, __shfl_xor(v, 16));
  return max2(v, __shfl_xor(v, 32));
}

// A value as it counts: NaN as 0, infinities as the largest of the type.
template <bool BF16>
__device__ __forceinline__ float clean(float x) {
  constexpr float lim = BF16 ? 0x1.FEp127f : 65504.0f;
  return x == x ? __builtin_amdgcn_fmed3f(x, -lim, lim) : 0.0f;
}

template <bool BF16>
__device__ __forceinline__ void widen2(uint32_t w, float& a, float& b) {
  a = clean<BF16>(BF16 ? __uint_as_float(w << 16) : f16_to_f32((uint16_t)(w & 0xFFFFu)));
  b = clean<BF16>(BF16 ? __uint_as_float(w & 0xFFFF0000u) : f16_to_f32((uint16_t)(w >> 16)));
}

// round(x / S), half to even, as it is exactly: the fp32 quotient is at most one step
// off and only beside k + 1/2, and the rest x - k S is exact (a multiple of S's ulp below
// 2 S; where x's own ulp is finer, k is 0).
__device__ __forceinline__ float code_of(float x, float S, float inv) {
  float k = __builtin_rintf(x * inv);
  const float e = __builtin_fmaf(-k, S, x), d = fabsf(e) + fabsf(e);
  const bool odd = ((int)k & 1) != 0;
  if (d > S || (d == S && odd)) k += __builtin_copysignf(1.0f, e);
  return k;
}

template <int BYTE>
__device__ __forceinline__ uint32_t put_code(float k, uint32_t w) {
  return __builtin_amdgcn_cvt_pk_u8_f32(k + 128.0f, BYTE, w);
}
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  return put_code<3>(d, put_code<2>(c, put_code<1>(b, put_code<0>(a, 0u))));
}

// Codes of an older scale: round(q S0 / S1).
__device__ __forceinline__ uint32_t requantise(uint32_t w, double s0, double s1) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = (int)(w >> (8 * i) & 255u) - 128;
    r |= (uint32_t)((int)__builtin_rint((double)q * s0 / s1) + 128) << (8 * i);
  }
  return r;
}

// What a wave does to one block: new tokens a .. e - 1 of its 16 (the first one is row
// t of the input), older ones before a.
struct Part {
  int64_t t;
  int a, e;
};

__device__ __forceinline__ float block_scale(float mx, float s0) {
  return fmaxf(fmaxf(mx / 127.0f, s0), kKv8Least);
}

template <int D, bool BF16>
__device__ __forceinline__ void write_keys(const uint16_t* k, int64_t ts, uint8_t* codes, float* scale, Part p, int lane) {
  constexpr int NS = D / 32;
  const int m = lane & 15, kg = lane >> 4;
  const bool fresh = m >= p.a && m < p.e;
  float x[NS][8], mx = 0.0f;
  uint4 raw[NS];
  const uint16_t* row = k + (p.t + (m - p.a)) * ts + 8 * kg;
#pragma unroll
  for (int s = 0; s < NS; ++s) raw[s] = fresh ? *(const uint4*)(row + 32 * s) : make_uint4(0, 0, 0, 0);
  const float s0 = p.a > 0 ? *scale : 0.0f;
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    widen2<BF16>(raw[s].x, x[s][0], x[s][1]);
    widen2<BF16>(raw[s].y, x[s][2], x[s][3]);
    widen2<BF16>(raw[s].z, x[s][4], x[s][5]);
    widen2<BF16>(raw[s].w, x[s][6], x[s][7]);
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = max2(mx, fabsf(x[s][i]));
  }
  const float S = block_scale(wave_max(mx), s0), inv = 1.0f / S;
  uint32_t w[NS][2];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = code_of(x[s][i], S, inv);
    w[s][0] = pack4(c[0], c[1], c[2], c[3]);
    w[s][1] = pack4(c[4], c[5], c[6], c[7]);
  }
  if (p.a > 0 && m < p.a) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const uint8_t* at = s == NS - 1 && NS % 2 ? codes + 512 * s + 8 * lane : codes + 1024 * (s / 2) + 16 * lane + 8 * (s % 2);
      const uint2 old = *(const uint2*)at;
      w[s][0] = S == s0 ? old.x : requantise(old.x, s0, S);
      w[s][1] = S == s0 ? old.y : requantise(old.y, s0, S);
    }
  }
#pragma unroll
  for (int s = 0; s + 1 < NS; s += 2)
    *(uint4*)(codes + 512 * s + 16 * lane) = make_uint4(w[s][0], w[s][1], w[s + 1][0], w[s + 1][1]);
  if constexpr (NS % 2) *(uint2*)(codes + 512 * (NS - 1) + 8 * lane) = make_uint2(w[NS - 1][0], w[NS - 1][1]);
  if (lane == 0) *scale = S;
}

template <int D, bool BF16>
__device__ __forceinline__ void write_values(const uint16_t* v, int64_t ts, uint8_t* codes, float* scale, Part p, int lane) {
  constexpr int NS = D / 32;
  const int m = lane & 15, kg = lane >> 4;
  uint32_t raw[4][NS];
  float mx = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int tok = 4 * kg + i;
    const bool fresh = tok >= p.a && tok < p.e;
    const uint16_t* row = v + (p.t + (tok - p.a)) * ts + 2 * m;
#pragma unroll
    for (int b = 0; b < NS; ++b) raw[i][b] = fresh ? *(const uint32_t*)(row + 32 * b) : 0u;
  }
  const float s0 = p.a > 0 ? *scale : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int b = 0; b < NS; ++b) {
      float x, y;
      widen2<BF16>(raw[i][b], x, y);
      mx = max2(mx, max2(fabsf(x), fabsf(y)));
    }
  const float S = block_scale(wave_max(mx), s0), inv = 1.0f / S;
  // which of the lane's four tokens are older ones
  const int older = p.a - 4 * kg;
  const uint32_t keep = older <= 0 ? 0u : older >= 4 ? 0xFFFFFFFFu : (1u << (8 * older)) - 1u;
  uint32_t w[2 * NS];
#pragma unroll
  for (int b = 0; b < NS; ++b) {
    float c[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x, y;
      widen2<BF16>(raw[i][b], x, y);
      c[0][i] = code_of(x, S, inv);
      c[1][i] = code_of(y, S, inv);
    }
    w[2 * b] = pack4(c[0][0], c[0][1], c[0][2], c[0][3]);
    w[2 * b + 1] = pack4(c[1][0], c[1][1], c[1][2], c[1][3]);
  }
  if (keep) {
#pragma unroll
    for (int t = 0; t < 2 * NS; ++t) {
      const uint8_t* at = t >= 2 * NS / 4 * 4 ? codes + 1024 * (t / 4) + 8 * lane + 4 * (t % 2)
                                               : codes + 1024 * (t / 4) + 16 * lane + 4 * (t % 4);
      const uint32_t old = *(const uint32_t*)at;
      const uint32_t q = S == s0 ? old : requantise(old, s0, S);
      w[t] = (q & keep) | (w[t] & ~keep);
    }
  }
#pragma unroll
  for (int t = 0; t + 3 < 2 * NS; t += 4)
    *(uint4*)(codes + 256 * t + 16 * lane) = make_uint4(w[t], w[t + 1], w[t + 2], w[t + 3]);
  if constexpr (NS % 2) *(uint2*)(codes + 512 * (NS - 1) + 8 * lane) = make_uint2(w[2 * NS - 2], w[2 * NS - 1]);
  if (lane == 0) *scale = S;
}

__device__ __forceinline__ uint16_t narrow(bool bf16, float f) {
  return bf16 ? (uint16_t)(__float_as_uint(f) >> 16) : stream_util::f32_to_f16_rne(f);   // exact
}

// The bounds of one page, by the two waves of a workgroup: D / 8 lanes hold a key.
template <int D, bool BF16>
__device__ __forceinline__ void write_bounds(const uint16_t* k, int64_t ts, uint16_t* bounds, int64_t t, int n, bool older,
                                             float (*smem)[8]) {
  constexpr int L = D / 8, R = 64 / L, G = 2 * R;   // lanes of a key, keys of a wave and of both
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane % L, g = wave * R + lane / L;
  const bool live = lane < L * R;
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) { lo[i] = __builtin_inff(); hi[i] = -__builtin_inff(); }
  if (live) {
#pragma unroll 4
    for (int j = g; j < n; j += G) {
      const uint4 v = *(const uint4*)(k + (t + j) * ts + 8 * c);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x, y;
        widen2<BF16>(w[i], x, y);
        lo[2 * i] = fminf(lo[2 * i], x);
        hi[2 * i] = fmaxf(hi[2 * i], x);
        lo[2 * i + 1] = fminf(lo[2 * i + 1], y);
        hi[2 * i + 1] = fmaxf(hi[2 * i + 1], y);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      smem[(g * L + c) * 2][i] = lo[i];
      smem[(g * L + c) * 2 + 1][i] = hi[i];
    }
  }
  __syncthreads();
  // smallest of channel x: thread x; largest: thread x again
  for (int x = threadIdx.x; x < D; x += 128) {
    float a = __builtin_inff(), b = -__builtin_inff();
    for (int j = 0; j < G; ++j) {
      a = fminf(a, smem[(j * L + x / 8) * 2][x % 8]);
      b = fmaxf(b, smem[(j * L + x / 8) * 2 + 1][x % 8]);
    }
    if (older) {
      a = fminf(a, BF16 ? bf16_to_f32(bounds[x]) : f16_to_f32(bounds[x]));
      b = fmaxf(b, BF16 ? bf16_to_f32(bounds[D + x]) : f16_to_f32(bounds[D + x]));
    }
    bounds[x] = narrow(BF16, a);
    bounds[D + x] = narrow(BF16, b);
  }
  __syncthreads();
}

// grid.y: heads; grid.z: blocks (a wave for keys, a wave for values), bounds.
template <int D, bool BF16>
__global__ __launch_bounds__(128) void kv8_append_kernel(Kv8Append a) {
  __shared__ float smem[2 * 2 * 64][8];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool pages = blockIdx.z == 1;
  const int h = blockIdx.y, ps = a.c.page_shift, unit = pages ? ps : 4;
  const int64_t cap = a.table_pages << ps;
  for (int64_t r0 = (int64_t)blockIdx.x * a.run; r0 < a.tokens; r0 += (int64_t)gridDim.x * a.run) {
    const int64_t r1 = r0 + a.run < a.tokens ? r0 + a.run : a.tokens;
    int64_t t = r0;
    while (t < r1) {
      const RowSeq s = seq_of_row(a.starts, a.batch, a.tokens, t, lane);
      if (s.b < 0) { ++t; continue; }
      const int64_t end = s.first + s.n, p0 = (int64_t)a.kv_lens[s.b] - s.n;   // position of its first row
      const int32_t* table = a.table + s.b * a.table_pages;
      for (; t < end && t < r1;) {
        const int64_t pos = p0 + (t - s.first);
        if (pos < 0) { t = t - pos < end ? t - pos : end; continue; }
        if (pos >= cap) { t = end; break; }
        const int in = (int)(pos & ((1 << unit) - 1));
        const int64_t left = end - t, room = (1 << unit) - in;
        const int64_t n = left < room ? left : room;
        // the first row of its block (page) that the call brings
        if (in == 0 || t == s.first) {
          const int64_t page = table[pos >> ps];
          if (page >= 0 && page < a.c.n_pages) {
            if (pages) {
              write_bounds<D, BF16>(a.k + h * a.k_hs, a.k_ts, a.bounds + (page * a.c.hkv + h) * (2 * D), t, (int)n, in > 0, smem);
            } else {
              const int64_t blk = kv8_block(page, a.c.hkv, h, ps, (int)(pos & ((1 << ps) - 1)));
              uint8_t* codes = a.c.cache + blk * (32 * D);
              float* scale = (float*)(a.c.scales + blk);
              const Part p{t, in, in + (int)n};
              if (wave == 0)
                write_keys<D, BF16>(a.k + h * a.k_hs, a.k_ts, codes, scale, p, lane);
              else
                write_values<D, BF16>(a.v + h * a.v_hs, a.v_ts, codes + 16 * D, scale + 1, p, lane);
            }
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
    // rows 4 (lane % 4) .. of tiles 2 s, 2 s + 1: both codes of 4 tokens
    const uint8_t* vc = codes + 16 * D + 1024 * (s >> 1) + (odd ? 0 : 8 * (s & 1));
    const int at = (m >> 2) * 16 + 4 * (lane & 3), sh = 8 * (m & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint2 w = *(const uint2*)(vc + (odd ? 8 : 16) * (at + i));
      vx[2 * i] = (float)((int)(w.x >> sh & 255u) - 128) * S.y;
      vx[2 * i + 1] = (float)((int)(w.y >> sh & 255u) - 128) * S.y;
      kx[i] = (float)((int)(kw.x >> (8 * i) & 255u) - 128) * S.x;
      kx[4 + i] = (float)((int)(kw.y >> (8 * i) & 255u) - 128) * S.x;
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
  const int64_t runs = (a.tokens + a.run - 1) / a.run;
  const dim3 grid((unsigned)(runs < (1 << 20) ? runs : 1 << 20), a.c.hkv, a.bounds ? 2 : 1);
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
