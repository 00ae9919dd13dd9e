// Rotary positions.
//
// One pass over the data: 16 bytes of a head's channels per lane (twice that where
// the partners of the pairs lie half a rotation apart).  The angles of a token are
// the same for all of its heads, so a workgroup first makes the table of cosines
// and sines of a few tokens in LDS and then turns all their heads with it: 64
// sines and cosines per token against 40 x 8 pieces of 40 heads of 128.
// An angle is p f in binary64, reduced to a turn there (off by 2^-52 of the angle: 2^-22 at
// a position of 2^30); what fp32 cannot hold of the turn is put back as a small rotation, so
// that cosine and sine are good to about an ulp of 1 besides.
// Bound by memory: 8191 tokens of 40 heads of 128, 168 MB, in 29 us where part of them is in the
// caches and 33 over four inputs in turn (5.0 TB/s; a copy 5.1), 36 a call among other work; one token
// 2.7.  Rows that are no whole pieces of 16 bytes go pair by pair: 40 heads of 80 (105 MB) of which 20 are
// rotated 64 us, all 80 27.
#include "rope.h"
#include "stream_util.h"

namespace gq {
namespace {

constexpr int kThreads = 256;
constexpr int kTable = 512;   // pairs in LDS

template <typename T> struct Elem;
template <> struct Elem<float> {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float f) { return f; }
};
struct Bf16 { uint16_t b; };
struct F16 { uint16_t b; };
template <> struct Elem<Bf16> {
  static __device__ __forceinline__ float get(Bf16 v) { return bf16_to_f32(v.b); }
  static __device__ __forceinline__ Bf16 put(float f) { return Bf16{f == f ? f32_to_bf16_rne(f) : (uint16_t)0x7FC0u}; }
};
template <> struct Elem<F16> {
  static __device__ __forceinline__ float get(F16 v) { return f16_to_f32(v.b); }
  static __device__ __forceinline__ F16 put(float f) { return F16{stream_util::f32_to_f16_rne(f)}; }
};

// E consecutive elements; a piece of 16 bytes is aligned to them.
template <typename T, int E>
struct __attribute__((aligned(sizeof(T) * E == 16 ? 16 : sizeof(T)))) Piece {
  T e[E];
};

// N entries of a table from one whose index is a multiple of N (N a power of two).
template <int N>
struct __attribute__((aligned(N < 4 ? 4 * N : 16))) Row {
  float f[N];
};

template <typename T, int E, bool PAIRS>
__global__ __launch_bounds__(kThreads) void rope_kernel(Rope a) {
  __shared__ __attribute__((aligned(16))) float cs[kTable], sn[kTable];
  using P = Piece<T, E>;
  const int half = a.rot >> 1, work = a.heads * a.items;
  for (int64_t t0 = (int64_t)blockIdx.x * a.tokens_per_group; t0 < a.tokens;
       t0 += (int64_t)gridDim.x * a.tokens_per_group) {
    const int n = (int)(a.tokens - t0 < a.tokens_per_group ? a.tokens - t0 : a.tokens_per_group);
    for (int i = threadIdx.x; i < n * half; i += kThreads) {
      const int t = i / half, j = i - t * half;
      const double turns = (double)a.positions[t0 + t] * a.freqs[j] * 0.15915494309189533577;
      const double r = turns - rint(turns);
      const float f = (float)r;
      const float rest = (float)(r - (double)f) * 6.28318530717958647693f;
      float s, c;
      sincospif(2.0f * f, &s, &c);
      cs[i] = __builtin_fmaf(-s, rest, c) * a.amplitude;
      sn[i] = __builtin_fmaf(c, rest, s) * a.amplitude * a.sign;
    }
    __syncthreads();
    // piece p of head h of token t: the first by division, the next by steps with carry
    const int first = blockIdx.y * kThreads + threadIdx.x, step = gridDim.y * kThreads;
    int t = first / work, h = (first - t * work) / a.items, p = first - t * work - h * a.items;
    const int dt = step / work, dh = (step - dt * work) / a.items, dp = step - dt * work - dh * a.items;
    auto next = [&] {
      p += dp;
      h += dh;
      t += dt;
      if (p >= a.items) { p -= a.items; ++h; }
      if (h >= a.heads) { h -= a.heads; ++t; }
    };
    for (; t < n; next()) {
      const uint8_t* x = a.x + (t0 + t) * a.x_ts + h * a.x_hs;
      uint8_t* o = a.out + (t0 + t) * a.out_ts + h * a.out_hs;
      if (p >= a.pair_items) {
        const int c = a.rot + (p - a.pair_items) * E;
        *(P*)(o + c * (int)sizeof(T)) = *(const P*)(x + c * (int)sizeof(T));
        continue;
      }
      if constexpr (PAIRS) {
        // neighbours: E / 2 pairs in one piece
        const int c = p * E, at = t * half + c / 2;
        const P v = *(const P*)(x + c * (int)sizeof(T));
        const Row<E / 2> cr = *(const Row<E / 2>*)(cs + at), sr = *(const Row<E / 2>*)(sn + at);
        P y;
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
          const float u = Elem<T>::get(v.e[2 * k]), w = Elem<T>::get(v.e[2 * k + 1]);
          const float co = cr.f[k], si = sr.f[k];
          y.e[2 * k] = Elem<T>::put(__builtin_fmaf(u, co, -(w * si)));
          y.e[2 * k + 1] = Elem<T>::put(__builtin_fmaf(w, co, u * si));
        }
        *(P*)(o + c * (int)sizeof(T)) = y;
      } else {
        const int c = p * E, at = t * half + c;
        const P v = *(const P*)(x + c * (int)sizeof(T)), w = *(const P*)(x + (c + half) * (int)sizeof(T));
        const Row<E> cr = *(const Row<E>*)(cs + at), sr = *(const Row<E>*)(sn + at);
        P y, z;
#pragma unroll
        for (int k = 0; k < E; ++k) {
          const float u = Elem<T>::get(v.e[k]), q = Elem<T>::get(w.e[k]);
          const float co = cr.f[k], si = sr.f[k];
          y.e[k] = Elem<T>::put(__builtin_fmaf(u, co, -(q * si)));
          z.e[k] = Elem<T>::put(__builtin_fmaf(q, co, u * si));
        }
        *(P*)(o + c * (int)sizeof(T)) = y;
        *(P*)(o + (c + half) * (int)sizeof(T)) = z;
      }
    }
    __syncthreads();   // the table is free again
  }
}

template <typename T, int E, bool PAIRS>
hipError_t launch(Rope& r, hipStream_t s) {
  r.pair_items = PAIRS ? r.rot / E : r.rot / (2 * E);
  r.items = r.pair_items + (r.tail ? (r.d - r.rot) / E : 0);
  const int half = r.rot / 2;
  // Few tokens: one a workgroup, its heads over as many workgroups as give every
  // thread one piece.  Many: enough tokens that the table costs little.
  r.tokens_per_group = 1;
  while (r.tokens_per_group < 4 && 2 * r.tokens_per_group * half <= kTable &&
         r.tokens / (2 * r.tokens_per_group) >= 4 * num_cus())
    r.tokens_per_group *= 2;
  const int64_t gx = (r.tokens + r.tokens_per_group - 1) / r.tokens_per_group;
  int64_t gy = 1;
  if (gx < 4 * num_cus()) gy = ((int64_t)r.heads * r.items + kThreads - 1) / kThreads;
  if (gy > 64) gy = 64;
  const unsigned groups = (unsigned)(gx < (1 << 17) ? gx : 1 << 17);
  hipLaunchKernelGGL((rope_kernel<T, E, PAIRS>), dim3(groups, (unsigned)gy), dim3(kThreads), 0, s, r);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_typed(const gq_rope_args& a, Rope& r, hipStream_t s) {
  constexpr int E = 16 / (int)sizeof(T);
  const uint64_t mis = (uint64_t)(uintptr_t)r.x | (uint64_t)(uintptr_t)r.out | (uint64_t)r.x_ts | (uint64_t)r.x_hs |
                       (uint64_t)r.out_ts | (uint64_t)r.out_hs;
  // whole pieces of 16 bytes, else pair by pair
  const bool wide = mis % 16 == 0 && r.d % E == 0 && r.rot % (a.interleaved ? E : 2 * E) == 0;
  if (a.interleaved) {
    if (wide) return launch<T, E, true>(r, s);
    return launch<T, 2, true>(r, s);
  }
  if (wide) return launch<T, E, false>(r, s);
  return launch<T, 1, false>(r, s);
}

}  // namespace

hipError_t launch_rope(const gq_rope_args& a, hipStream_t s) {
  const int64_t size = a.dtype == GQ_F32 ? 4 : 2;
  Rope r;
  r.x = (const uint8_t*)a.x;
  r.out = (uint8_t*)a.out;
  r.x_ts = a.x_token_stride * size;
  r.x_hs = a.x_head_stride * size;
  r.out_ts = a.out_token_stride * size;
  r.out_hs = a.out_head_stride * size;
  r.positions = a.positions;
  r.freqs = a.freqs;
  r.tokens = a.tokens;
  r.heads = (int32_t)a.heads;
  r.d = a.head_dim;
  r.rot = a.rot_dim;
  r.amplitude = a.amplitude;
  r.sign = a.inverse ? -1.0f : 1.0f;
  r.tail = a.out != a.x && a.rot_dim < a.head_dim;
  switch (a.dtype) {
    case GQ_F32: return launch_typed<float>(a, r, s);
    case GQ_F16: return launch_typed<F16>(a, r, s);
    default: return launch_typed<Bf16>(a, r, s);
  }
}

}  // namespace gq
