// Writing keys and values into the 4-bit cache, and reading them back.
//
// Both are one pass over the data and bound by it.  A lane holds 8 consecutive
// channels of one (token, head) row: 16 bytes of 16-bit values, one dword of
// codes; D / 8 lanes make a row (padded to 16 for D = 96).  A workgroup takes
// the same head of consecutive tokens, so that the pieces of 16 bytes that a
// token leaves in the value order are completed by the same workgroup, in the
// L2 cache, for consecutive slots.
#include "kv4.h"
#include "stream_util.h"

namespace gq {
namespace {

using stream_util::dpp_f32;

constexpr int kThreads = 256;

template <int D>
struct Row {
  static constexpr int kLanes = D / 8;                  // lanes that hold channels
  static constexpr int kPitch = D == 96 ? 16 : D / 8;   // lanes per row
  static constexpr int kRows = kThreads / kPitch;       // rows per pass of a workgroup
};

// Largest value over the lanes of a group of g channels (g / 8 lanes; the 12
// of g = 96 lie in a row of 16 whose last 4 hold zeros, which the callers'
// ranges include).
__device__ __forceinline__ float group_max(float v, int g) {
  v = fmaxf(v, dpp_f32<0xB1, 0xF>(v));    // quad_perm [1,0,3,2]
  v = fmaxf(v, dpp_f32<0x4E, 0xF>(v));    // quad_perm [2,3,0,1]
  if (g > 32) v = fmaxf(v, dpp_f32<0x141, 0xF>(v));   // row_half_mirror: 8 lanes
  if (g > 64) v = fmaxf(v, dpp_f32<0x140, 0xF>(v));   // row_mirror: 16 lanes
  if (g > 128) v = fmaxf(v, __shfl_xor(v, 16));
  return v;
}

// fp16 scale of a range r >= 0 cut into n steps, as the storage contract has
// it: r / n in binary64, rounded once.  r / n is taken in fp32 first (relative
// error below 2^-22): if the values 2^-21 to either side round to the same
// fp16, so does the exact one.  Otherwise (about one in 2^10) binary64 decides.
__device__ __forceinline__ uint16_t group_scale(float hi, float lo, double n, float inv_n) {
  const float r = hi - lo;
  const float v = r * inv_n;
  const uint16_t a = __builtin_bit_cast(uint16_t, (_Float16)(v * (1.0f - 0x1p-21f)));
  const uint16_t b = __builtin_bit_cast(uint16_t, (_Float16)(v * (1.0f + 0x1p-21f)));
  if (a == b && a != 0 && a < 0x7C00u) return a;
  const double rd = (double)hi - (double)lo;
  return rd > 0.0 ? scale_to_f16(rd / n) : (uint16_t)0x3C00u;   // 1.0: an all-zero group
}

// round(x / S), half to even, for a 16-bit float x and an fp16 S: the quotient
// of two 11-bit numbers is either k + 1/2 exactly or at least 2^-14 away from
// it, so an fp32 quotient good to a few units in the last place decides every
// case but the ties; one residual step (exact by FMA) makes those exact.
// |x / S| beyond 64 is only ever clamped: it is cut there.
__device__ __forceinline__ float div_round(float x, float S, float inv) {
  float q = __builtin_amdgcn_fmed3f(x * inv, -64.0f, 64.0f);
  q = __builtin_fmaf(__builtin_fmaf(-q, S, x), inv, q);
  return __builtin_rintf(q);
}

template <int D>
__global__ __launch_bounds__(kThreads) void kv4_write_kernel(
    const uint16_t* __restrict__ k, int64_t k_ts, int64_t k_hs, const uint16_t* __restrict__ v,
    int64_t v_ts, int64_t v_hs, int bf16, int64_t tokens, const int64_t* __restrict__ slots,
    Kv4Geo c) {
  constexpr int NS = D / 32, P = Row<D>::kPitch, L = Row<D>::kLanes;
  __shared__ uint32_t sv[kThreads];
  const int is_v = blockIdx.z;
  const int head = blockIdx.y;
  const int lane = threadIdx.x % P;
  const int row = threadIdx.x / P;
  const int64_t t = (int64_t)blockIdx.x * Row<D>::kRows + row;
  const bool live = t < tokens && lane < L;
  uint4 raw = make_uint4(0, 0, 0, 0);
  int64_t slot = -1;
  if (live) {
    const uint16_t* p = is_v ? v + t * v_ts + head * v_hs : k + t * k_ts + head * k_hs;
    raw = *(const uint4*)(p + lane * 8);
    slot = slots[t];
  }
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16 ? bf16_to_f32(w[i] & 0xFFFFu) : f16_to_f32((uint16_t)(w[i] & 0xFFFFu));
    x[2 * i + 1] = bf16 ? __uint_as_float(w[i] & 0xFFFF0000u) : f16_to_f32((uint16_t)(w[i] >> 16));
  }
  float hi = 0.0f, lo = 0.0f;
  if (c.sym) {
#pragma unroll
    for (int i = 0; i < 8; ++i) hi = fmaxf(hi, fabsf(x[i]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) { hi = fmaxf(hi, x[i]); lo = fmaxf(lo, -x[i]); }
    lo = group_max(lo, c.g);
  }
  hi = group_max(hi, c.g);
  const uint16_t sh = c.sym ? group_scale(hi, 0.0f, 7.0, 1.0f / 7.0f)
                            : group_scale(hi, -lo, 15.0, 1.0f / 15.0f);
  const float S = f16_to_f32(sh);
  const float inv = __builtin_amdgcn_rcpf(S);
  // the zero point, and the range of round(x / S) that keeps codes in 0..15
  const float z = c.sym ? 8.0f : fminf(fmaxf(div_round(lo, S, inv), 0.0f), 15.0f);
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    q[i] = (uint32_t)fminf(fmaxf(div_round(x[i], S, inv) + z, 0.0f), 15.0f);

  const int64_t page = slot >> c.page_shift;
  const bool ok = live && slot >= 0 && page < c.n_pages;
  const int tp = (int)(slot & ((1 << c.page_shift) - 1));
  uint8_t* blk = c.cache + (ok ? kv4_block_offset(c, page, head, tp) : 0);
  if (is_v) blk += 8 * D + c.meta;
  const int ts = tp & 15;
  if (ok && (lane * 8) % c.g == 0) {   // first lane of a group: its parameters
    const int gi = lane * 8 / c.g;
    const uint16_t zh = __builtin_bit_cast(uint16_t, (_Float16)z);
    uint16_t* m = (uint16_t*)(blk + 8 * D);
    if (c.sym) {
      m[gi * 16 + ts] = sh;
    } else if (is_v) {
      m += gi * 32 + (ts >> 2) * 8 + (ts & 3);
      m[0] = sh;
      m[4] = zh;
    } else {
      m[gi * 16 + ts] = sh;
      m[16 * c.ng + ts * c.ng + gi] = zh;
    }
  }
  if (!is_v) {
    // nibbles 0, 4, 1, 5, 2, 6, 3, 7
    const uint32_t d = q[0] | q[1] << 16 | q[2] << 4 | q[3] << 20 | q[4] << 8 | q[5] << 24 |
                       q[6] << 12 | q[7] << 28;
    if (ok) *(uint32_t*)(blk + ts * (D / 2) + ((lane & 3) * NS + (lane >> 2)) * 4) = d;
    return;
  }
  // natural packed dword (bytes 4 lane .. of the row) -> bytes (m, b)
  sv[threadIdx.x] = q[0] | q[1] << 4 | q[2] << 8 | q[3] << 12 | q[4] << 16 | q[5] << 20 |
                    q[6] << 24 | q[7] << 28;
  __syncthreads();
  if (!ok) return;
  const uint8_t* rowb = (const uint8_t*)(sv + row * P);
  uint8_t* quad = blk + (ts >> 2) * (64 * NS) + (ts & 3) * NS;
  for (int m = lane; m < 16; m += L) {
    uint8_t* o = quad + m * (4 * NS);
    if (NS == 2) {
      *(uint16_t*)o = (uint16_t)(rowb[m] | rowb[16 + m] << 8);
    } else if (NS == 3) {
#pragma unroll
      for (int b = 0; b < 3; ++b) o[b] = rowb[16 * b + m];
    } else {
#pragma unroll
      for (int i = 0; i < NS / 4; ++i)
        ((uint32_t*)o)[i] = rowb[64 * i + m] | rowb[64 * i + 16 + m] << 8 |
                            rowb[64 * i + 32 + m] << 16 | (uint32_t)rowb[64 * i + 48 + m] << 24;
    }
  }
}

template <int D>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(Kv4Geo c, const int64_t* __restrict__ slots,
                                                          int64_t tokens, void* __restrict__ k,
                                                          void* __restrict__ v, gq_dtype odt) {
  constexpr int NS = D / 32, P = Row<D>::kPitch, L = Row<D>::kLanes;
  const int is_v = blockIdx.z;
  const int head = blockIdx.y;
  const int lane = threadIdx.x % P;
  const int64_t t = (int64_t)blockIdx.x * Row<D>::kRows + threadIdx.x / P;
  if (t >= tokens || lane >= L) return;
  const int64_t slot = slots[t];
  const int64_t page = slot >> c.page_shift;
  const bool ok = slot >= 0 && page < c.n_pages;
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = 0.0f;
  if (ok) {
    const int tp = (int)(slot & ((1 << c.page_shift) - 1));
    const uint8_t* blk = c.cache + kv4_block_offset(c, page, head, tp);
    if (is_v) blk += 8 * D + c.meta;
    const int ts = tp & 15;
    const int gi = lane * 8 / c.g;
    const uint16_t* m = (const uint16_t*)(blk + 8 * D);
    float S, z = 8.0f;
    if (c.sym) {
      S = f16_to_f32(m[gi * 16 + ts]);
    } else if (is_v) {
      m += gi * 32 + (ts >> 2) * 8 + (ts & 3);
      S = f16_to_f32(m[0]);
      z = f16_to_f32(m[4]);
    } else {
      S = f16_to_f32(m[gi * 16 + ts]);
      z = f16_to_f32(m[16 * c.ng + ts * c.ng + gi]);
    }
    uint32_t q[8];
    if (!is_v) {
      const uint32_t d = *(const uint32_t*)(blk + ts * (D / 2) + ((lane & 3) * NS + (lane >> 2)) * 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = (d >> (4 * ((i >> 1) + 4 * (i & 1)))) & 15u;
    } else {
      // bytes 4 lane .. 4 lane + 3 of the row: m = 4 (lane % 4) + i, b = lane / 4
      const uint8_t* o = blk + (ts >> 2) * (64 * NS) + (ts & 3) * NS + (lane & 3) * (16 * NS) + (lane >> 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b = o[i * 4 * NS];
        q[2 * i] = b & 15u;
        q[2 * i + 1] = b >> 4;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = S * ((float)q[i] - z);   // exact: 11 bits times 5
  }
  const int64_t o = (t * c.hkv + head) * D + lane * 8;
  void* out = is_v ? v : k;
  if (odt == GQ_F32) {
    float4* p = (float4*)((float*)out + o);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = odt == GQ_BF16 ? f32_to_bf16_rne(x[2 * i]) : stream_util::f32_to_f16_rne(x[2 * i]);
      const uint32_t b =
          odt == GQ_BF16 ? f32_to_bf16_rne(x[2 * i + 1]) : stream_util::f32_to_f16_rne(x[2 * i + 1]);
      h[i] = a | (b << 16);
    }
    *(uint4*)((uint16_t*)out + o) = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

template <int D>
dim3 grid_of(int64_t tokens, int heads) {
  return dim3((unsigned)((tokens + Row<D>::kRows - 1) / Row<D>::kRows), (unsigned)heads, 2);
}

}  // namespace

hipError_t launch_kv4_write(const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts,
                            int64_t v_hs, gq_dtype dt, int64_t tokens, const int64_t* slots,
                            const Kv4Geo& c, hipStream_t s) {
#define GQ_KV4_WRITE(D)                                                                        \
  hipLaunchKernelGGL(kv4_write_kernel<D>, grid_of<D>(tokens, c.hkv), dim3(kThreads), 0, s,     \
                     (const uint16_t*)k, k_ts, k_hs, (const uint16_t*)v, v_ts, v_hs,           \
                     (int)(dt == GQ_BF16), tokens, slots, c)
  if (c.d == 64) GQ_KV4_WRITE(64);
  else if (c.d == 96) GQ_KV4_WRITE(96);
  else if (c.d == 128) GQ_KV4_WRITE(128);
  else GQ_KV4_WRITE(256);
#undef GQ_KV4_WRITE
  return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4Geo& c, const int64_t* slots, int64_t tokens, void* k, void* v,
                           gq_dtype odt, hipStream_t s) {
#define GQ_KV4_READ(D)                                                                            \
  hipLaunchKernelGGL(kv4_read_kernel<D>, grid_of<D>(tokens, c.hkv), dim3(kThreads), 0, s, c, slots, \
                     tokens, k, v, odt)
  if (c.d == 64) GQ_KV4_READ(64);
  else if (c.d == 96) GQ_KV4_READ(96);
  else if (c.d == 128) GQ_KV4_READ(128);
  else GQ_KV4_READ(256);
#undef GQ_KV4_READ
  return hipGetLastError();
}

}  // namespace gq
