// Writing keys and values into the 4-bit cache, and reading them back.
//
// Both are one pass over the data.  A lane holds 8 consecutive channels of one
// (token, head) row, of its key and of its value: 16 bytes of 16-bit values, one
// dword of codes each; D / 8 lanes make a row (padded to 16 for D = 96).  Key and
// value in one lane share the slot and the address and keep twice the loads
// under way.  A workgroup takes the same head of consecutive tokens, so that the
// pieces of 16 bytes that a token leaves in the value order are completed by
// the same workgroup, in the L2 cache, for consecutive slots.
//
// 16 K tokens of 8 heads of 128: written in 21 us (86 MB, 4.1 TB/s; bound by
// vector instructions, 22 per pair of values), read back in 17 us; 64 K tokens
// read back in 80 to 86 us (340 MB, 4.2 TB/s; a copy reaches 5.0).  All tokens of one
// head before the next, or all heads of a token first, measured level.
#include "kv4.h"
#include "stream_util.h"

namespace gq {
namespace {

using stream_util::dpp_f32;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

template <int D>
struct Row {
  static constexpr int kLanes = D / 8;                  // lanes that hold channels
  static constexpr int kPitch = D == 96 ? 16 : D / 8;   // lanes per row
  static constexpr int kRows = kThreads / kPitch;       // rows per pass of a workgroup
};

// The larger of two, in one instruction: fmaxf first quiets its operands.
__device__ __forceinline__ float max2(float a, float b) {
  float r;
  asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

// Largest value over the lanes of a group of g channels (g / 8 lanes; the 12
// of g = 96 lie in a row of 16 whose last 4 hold zeros, which the callers'
// ranges include).
__device__ __forceinline__ float group_max(float v, int g) {
  v = max2(v, dpp_f32<0xB1, 0xF>(v));    // quad_perm [1,0,3,2]
  v = max2(v, dpp_f32<0x4E, 0xF>(v));    // quad_perm [2,3,0,1]
  if (g > 32) v = max2(v, dpp_f32<0x141, 0xF>(v));   // row_half_mirror: 8 lanes
  if (g > 64) v = max2(v, dpp_f32<0x140, 0xF>(v));   // row_mirror: 16 lanes
  if (g > 128) v = max2(v, __shfl_xor(v, 16));
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

// round(x / S), half to even, for a 16-bit float x and an fp16 S, held in
// lo .. hi (integers), as 1.5 2^23 + the result: the quotient of two 11-bit
// numbers is either k + 1/2 exactly or at least 2^-14 away from it, so an fp32
// quotient good to a few units in the last place decides every case but the
// ties; one residual step (exact by FMA) makes those exact.  The sum rounds.
__device__ __forceinline__ float div_round(float x, float S, float inv, float lo, float hi) {
  float q = x * inv;
  q = __builtin_fmaf(__builtin_fmaf(-q, S, x), inv, q);
  return __builtin_amdgcn_fmed3f(q, lo, hi) + 12582912.0f;
}

template <bool BF16>
__device__ __forceinline__ void widen(uint4 raw, float (&x)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = BF16 ? __uint_as_float(w[i] << 16) : f16_to_f32((uint16_t)(w[i] & 0xFFFFu));
    x[2 * i + 1] = BF16 ? __uint_as_float(w[i] & 0xFFFF0000u) : f16_to_f32((uint16_t)(w[i] >> 16));
  }
}

struct Quant {
  uint16_t S;       // fp16 bits
  int z;            // zero point (8: symmetric)
  uint32_t codes;   // nibble at[i] is channel i's
};

// 8 channels of a row, the lanes of a group together.  at: where each code goes
// in the dword, 4 bits each from the lowest.
template <bool SYM>
__device__ __forceinline__ Quant quantise(float (&x)[8], int g, uint32_t at) {
  constexpr bool sym = SYM;
  float hi = 0.0f, lo = 0.0f;
  if (sym) {
#pragma unroll
    for (int i = 0; i < 8; ++i) hi = max2(hi, fabsf(x[i]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) { hi = max2(hi, x[i]); lo = max2(lo, -x[i]); }
    lo = group_max(lo, g);
  }
  hi = group_max(hi, g);
  Quant r;
  r.S = sym ? group_scale(hi, 0.0f, 7.0, 1.0f / 7.0f) : group_scale(hi, -lo, 15.0, 1.0f / 15.0f);
  if (r.S == 0x7BFFu) {
    // a saturated scale: infinities become finite, beyond any code all the same
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __builtin_amdgcn_fmed3f(x[i], -4194304.0f, 4194304.0f);
    lo = fminf(lo, 4194304.0f);
  }
  const float S = f16_to_f32(r.S);
  const float inv = __builtin_amdgcn_rcpf(S);
  const float zf = sym ? 8.0f : div_round(lo, S, inv, 0.0f, 15.0f) - 12582912.0f;
  r.z = (int)zf;
  // the bits of 1.5 2^23 + n are 0x4B400000 + n: shifted sums of them leave the
  // codes and a constant
  uint32_t sum = (uint32_t)r.z * 0x11111111u, extra = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t sh = (at >> (4 * i)) & 15u;
    sum += __float_as_uint(div_round(x[i], S, inv, -zf, 15.0f - zf)) << (4 * sh);
    extra += 0x4B400000u << (4 * sh);
  }
  r.codes = sum - extra;
  // a group of zeros stands for them whatever its scale is; kept as 0, it does
  // not pass for a group of large values where attention looks at the scales
  if (hi + lo == 0.0f) r.S = 0;
  return r;
}

template <int D, bool SYM, bool BF16>
__global__ __launch_bounds__(kThreads) void kv4_write_kernel(
    const uint16_t* __restrict__ k, int64_t k_ts, int64_t k_hs, const uint16_t* __restrict__ v,
    int64_t v_ts, int64_t v_hs, int64_t tokens, const int64_t* __restrict__ slots,
    Kv4Geo c) {
  constexpr int NS = D / 32, P = Row<D>::kPitch, L = Row<D>::kLanes;
  __shared__ uint32_t sv[kThreads];
  const int head = blockIdx.y;
  const int lane = threadIdx.x % P;
  const int row = threadIdx.x / P;
  const int64_t t = (int64_t)blockIdx.x * Row<D>::kRows + row;
  uint4 kr = make_uint4(0, 0, 0, 0), vr = kr;
  int64_t slot = -1;
  if (t < tokens && lane < L) {
    kr = *(const uint4*)(k + t * k_ts + head * k_hs + lane * 8);
    vr = *(const uint4*)(v + t * v_ts + head * v_hs + lane * 8);
    slot = slots[t];
  }
  float x[8];
  widen<BF16>(kr, x);
  const Quant qk = quantise<SYM>(x, c.g, 0x73625140u);
  widen<BF16>(vr, x);
  const Quant qv = quantise<SYM>(x, c.g, 0x76543210u);
  // natural order (bytes 4 lane .. of the row) -> bytes (m, b)
  sv[threadIdx.x] = qv.codes;
  __syncthreads();
  const int64_t page = slot >> c.page_shift;
  if (slot < 0 || page >= c.n_pages) return;
  const int tp = (int)(slot & ((1 << c.page_shift) - 1));
  uint8_t* blk = c.cache + kv4_block_offset(c, page, head, tp);
  uint8_t* blv = blk + 8 * D + c.meta;
  const int ts = tp & 15;
  *(uint32_t*)(blk + ts * (D / 2) + ((lane & 3) * NS + (lane >> 2)) * 4) = qk.codes;
  const uint8_t* rowb = (const uint8_t*)(sv + row * P);
  uint8_t* quad = blv + (ts >> 2) * (64 * NS) + (ts & 3) * NS;
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
  if ((lane * 8) % c.g == 0) {   // first lane of a group: its parameters
    const int gi = lane * 8 / c.g;
    uint16_t* mk = (uint16_t*)(blk + 8 * D);
    uint16_t* mv = (uint16_t*)(blv + 8 * D);
    mk[gi * 16 + ts] = qk.S;
    if (SYM) {
      mv[gi * 16 + ts] = qv.S;
    } else {
      mk[16 * c.ng + ts * c.ng + gi] = kv4_zero_bits(qk.z);
      mv += gi * 32 + (ts >> 2) * 8 + (ts & 3);
      mv[0] = qv.S;
      mv[4] = kv4_zero_bits(qv.z);
    }
  }
}

// U rows per lane: the loads of all of them are under way together.
template <int D, int U>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(Kv4Geo c, const int64_t* __restrict__ slots,
                                                          int64_t tokens, void* __restrict__ k,
                                                          void* __restrict__ v, gq_dtype odt) {
  constexpr int NS = D / 32, P = Row<D>::kPitch, L = Row<D>::kLanes;
  constexpr int kPieces = (16 + L - 1) / L;        // pieces (m, all b) of a value row per lane
  __shared__ uint32_t sv[U][kThreads];
  const int head = blockIdx.y;
  const int lane = threadIdx.x % P;
  const int row = threadIdx.x / P;
  const int64_t t0 = (int64_t)blockIdx.x * (U * Row<D>::kRows) + row;
  int64_t slot[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = t0 + u * Row<D>::kRows;
    slot[u] = t < tokens && lane < L ? slots[t] : -1;
  }
  uint32_t kc[U], vw[U][kPieces][(NS + 3) / 4];
  // 0 (S) times anything: a slot out of range reads as zeros
  uint16_t S[U][2], z[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t page = slot[u] >> c.page_shift;
    kc[u] = 0;
    S[u][0] = S[u][1] = 0;
    z[u][0] = z[u][1] = kv4_zero_bits(8);
    if (slot[u] < 0 || page >= c.n_pages) continue;
    const int tp = (int)(slot[u] & ((1 << c.page_shift) - 1));
    const uint8_t* blk = c.cache + kv4_block_offset(c, page, head, tp);
    const uint8_t* blv = blk + 8 * D + c.meta;
    const int ts = tp & 15;
    const int gi = lane * 8 / c.g;
    kc[u] = *(const uint32_t*)(blk + ts * (D / 2) + ((lane & 3) * NS + (lane >> 2)) * 4);
    const uint8_t* quad = blv + (ts >> 2) * (64 * NS) + (ts & 3) * NS;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int m = lane + i * L;
      if (16 % L != 0 && m >= 16) continue;
      const uint8_t* o = quad + m * (4 * NS);
      if (NS == 2) {
        vw[u][i][0] = *(const uint16_t*)o;
      } else if (NS == 3) {
        vw[u][i][0] = o[0] | o[1] << 8 | (uint32_t)o[2] << 16;
      } else {
#pragma unroll
        for (int j = 0; j < NS / 4; ++j) vw[u][i][j] = ((const uint32_t*)o)[j];
      }
    }
    const uint16_t* mk = (const uint16_t*)(blk + 8 * D);
    const uint16_t* mv = (const uint16_t*)(blv + 8 * D);
    S[u][0] = mk[gi * 16 + ts];
    if (c.sym) {
      S[u][1] = mv[gi * 16 + ts];
    } else {
      z[u][0] = mk[16 * c.ng + ts * c.ng + gi];
      mv += gi * 32 + (ts >> 2) * 8 + (ts & 3);
      S[u][1] = mv[0];
      z[u][1] = mv[4];
    }
  }
  // bytes (m, b) -> natural order, byte 16 b + m of the row
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint8_t* rowb = (uint8_t*)(sv[u] + row * P);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int m = lane + i * L;
      if (lane >= L || m >= 16) continue;
#pragma unroll
      for (int b = 0; b < NS; ++b) rowb[16 * b + m] = (uint8_t)(vw[u][i][b / 4] >> (8 * (b % 4)));
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = t0 + u * Row<D>::kRows;
    if (t >= tokens || lane >= L) break;
    const uint32_t vc = sv[u][threadIdx.x];
    const int64_t o = (t * c.hkv + head) * D + lane * 8;
#pragma unroll
    for (int is_v = 0; is_v < 2; ++is_v) {
      const float Sf = f16_to_f32(S[u][is_v]), nz = -kv4_zero(z[u][is_v]) * Sf;
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = is_v ? i : (i >> 1) + 4 * (i & 1);         // nibble of channel i
        const uint32_t q = ((is_v ? vc : kc[u]) >> (at & 1 ? 4 : 0)) & 0x0F0F0F0Fu;
        x[i] = __builtin_fmaf(Sf, (float)(q >> (8 * (at >> 1)) & 0xFFu), nz);   // exact: 11 bits times 5
      }
      void* out = is_v ? v : k;
      if (odt == GQ_F32) {
        float4* p = (float4*)((float*)out + o);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
      } else {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (odt == GQ_BF16)
            h[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)x[2 * i], (__bf16)x[2 * i + 1]});
          else
            h[i] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)x[2 * i], (_Float16)x[2 * i + 1]});
        }
        *(uint4*)((uint16_t*)out + o) = make_uint4(h[0], h[1], h[2], h[3]);
      }
    }
  }
}

template <int D>
dim3 grid_of(int64_t tokens, int heads, int u) {
  const int64_t n = u * Row<D>::kRows;
  return dim3((unsigned)((tokens + n - 1) / n), (unsigned)heads);
}

}  // namespace

hipError_t launch_kv4_write(const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts,
                            int64_t v_hs, gq_dtype dt, int64_t tokens, const int64_t* slots,
                            const Kv4Geo& c, hipStream_t s) {
#define GQ_KV4_WRITE(D, SYM, BF16)                                                                       \
  hipLaunchKernelGGL((kv4_write_kernel<D, SYM, BF16>), grid_of<D>(tokens, c.hkv, 1), dim3(kThreads), 0, s, \
                     (const uint16_t*)k, k_ts, k_hs, (const uint16_t*)v, v_ts, v_hs, tokens, slots, c)
#define GQ_KV4_WRITE_D(D)                                      \
  if (c.sym && dt == GQ_BF16) GQ_KV4_WRITE(D, true, true);     \
  else if (c.sym) GQ_KV4_WRITE(D, true, false);                \
  else if (dt == GQ_BF16) GQ_KV4_WRITE(D, false, true);        \
  else GQ_KV4_WRITE(D, false, false)
  switch (c.d) {
    case 64: GQ_KV4_WRITE_D(64); break;
    case 96: GQ_KV4_WRITE_D(96); break;
    case 128: GQ_KV4_WRITE_D(128); break;
    default: GQ_KV4_WRITE_D(256); break;
  }
#undef GQ_KV4_WRITE_D
#undef GQ_KV4_WRITE
  return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4Geo& c, const int64_t* slots, int64_t tokens, void* k, void* v,
                           gq_dtype odt, hipStream_t s) {
  // Four rows per lane where 16-bit results and what they are made of pass the 256 MB
  // that the card's last cache holds (8 heads of 128, 57 K tokens 77 -> 70 us, 131 K 179
  // -> 155; 4 heads of 256 197 -> 153); up to there one row is as fast or faster (8 heads
  // of 64, 33 K tokens 17.0 against 18.5), for fp32 results beyond it too (156 against 167).
  const int64_t bytes = tokens * c.hkv * (4 * c.d + c.sb / 16);
  const bool many = odt != GQ_F32 && bytes >= (int64_t)1 << 28;
#define GQ_KV4_READ(D)                                                                                \
  if (many)                                                                                           \
    hipLaunchKernelGGL((kv4_read_kernel<D, 4>), grid_of<D>(tokens, c.hkv, 4), dim3(kThreads), 0, s, c, \
                       slots, tokens, k, v, odt);                                                     \
  else                                                                                                \
    hipLaunchKernelGGL((kv4_read_kernel<D, 1>), grid_of<D>(tokens, c.hkv, 1), dim3(kThreads), 0, s, c, \
                       slots, tokens, k, v, odt)
  switch (c.d) {
    case 64: GQ_KV4_READ(64); break;
    case 96: GQ_KV4_READ(96); break;
    case 128: GQ_KV4_READ(128); break;
    default: GQ_KV4_READ(256); break;
  }
#undef GQ_KV4_READ
  return hipGetLastError();
}

}  // namespace gq
