// The 8-bit key/value cache: byte order and the declarations shared by the kernels
// that write it, read it, attend over it and choose its pages.
//
// Codes first: page by page, head by head, page_size / 16 blocks of 16 tokens, each
// 32 D bytes (D channels, NS = D / 32): keys, then values.  A code q is stored as
// q + 128 (1 .. 255), which as the low byte of the fp16 0x6400 is 1024 + 128 + q.
// Behind all codes the scales: {keys', values'} fp32 of every block, in the same order.
// Both code orders are those in which the 16x16x32 matrix product takes its first
// operand, whose lane l (m = l % 16, kg = l / 16) holds row m and 8 consecutive k, in
// pieces of 16 bytes a lane, so that reads of a wave are one run:
//   keys (row = token, k = channel): steps s of 32 channels in pairs p = s / 2; lane l
//     has 16 bytes at 1024 p + 16 l, channels 32 s + 8 kg .. of token m for both steps.
//     A last step without a partner (96 channels): 8 bytes at 1024 p + 8 l.
//   values (row = channel, k = token): T = D / 16 tiles t of 16 channels; row m of tile t is
//     channel T m + t.  Tiles in fours: lane l has 16 bytes at 1024 (t / 4) + 16 l, for
//     each tile the tokens 4 kg .. 4 kg + 3 of its row.  Two tiles left (96 channels):
//     8 bytes at 1024 + 8 l.
#pragma once

#include "gq_internal.h"
#include "gq_kv8.h"
#include "kv4.h"

namespace gq {

constexpr float kKv8Least = 0x1p-40f;   // least scale of a block

struct Kv8Geo {
  uint8_t* cache;
  float2* scales;       // {keys', values'} by block
  int64_t n_pages;
  int32_t hkv, d;
  int32_t page_shift;   // log2(page_size)
};

// Number of the block of (page, head, token in the page): its codes lie at 32 d times it.
__device__ __forceinline__ int64_t kv8_block(int64_t page, int hkv, int head, int page_shift, int token) {
  return ((page * hkv + head) << (page_shift - 4)) + (token >> 4);
}

// Append: what the kernel gets.
struct Kv8Append {
  Kv8Geo c;
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_ts, k_hs, v_ts, v_hs;   // elements
  int64_t tokens;
  const int32_t* table;
  int64_t batch, table_pages;
  const int32_t* kv_lens;
  const int32_t* starts;            // or nullptr: one token per sequence
  uint16_t* bounds;                 // or nullptr
  int32_t run, page_run;            // tokens that a workgroup looks through, for blocks and for bounds
};

hipError_t launch_kv8_append(const Kv8Append& a, gq_dtype dt, hipStream_t s);
hipError_t launch_kv8_read(const Kv8Geo& c, const int64_t* slots, int64_t tokens, void* k, void* v, gq_dtype odt,
                           hipStream_t s);

// Attention: what the kernels get besides what those of the 4-bit cache do, whose
// split over workgroups, join and query side they share (kv4_rows.h, kv4_tile.h).
struct Kv8Attn : Kv4Attn {
  const float2* scales;
  int64_t table_b, table_h;         // page_table entries from a sequence, and a head, to the next
};

// A weight p without its value scale S_V of 2^-40 .. 2^121 spans more than fp32 does where
// p S_V has to be near 2^11.  So the sums hold p 2^40: at most 2^95, at least 2^-70 for the
// heaviest key, with room for those far lighter; the results, which hold p S_V, get the
// factor when they are done, and the reference of both is 40 less.  A reference that rises from
// the smallest scale to the largest moves by more than fp32 holds: the sums follow it by move_sum.
constexpr float kKv8Shift = 40.0f, kKv8Up = 0x1p40f, kKv8Down = 0x1p-40f;

// Factor of the scores of a block: what a row's queries and the block's keys were divided
// by.  Never 0, which would make NaN of a hidden key's -inf, nor infinite, of a score of 0.
__device__ __forceinline__ float kv8_factor(float A, float sk) {
  return __builtin_amdgcn_fmed3f(A * sk, 0x1p-120f, 0x1.fffffep127f);
}

// Two results as 16 bits, nearest-even.
template <bool BF16>
__device__ __forceinline__ uint32_t pack_result(float a, float b) {
  if constexpr (BF16) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
  } else {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
  }
}

// Waves per SIMD of the rows kernel: as many workgroups as fit the LDS of a compute unit.
constexpr int kv8_rows_waves(int d, int nq) {
  if (d == 64) return nq > 1 ? 3 : 4;   // four with two row tiles spill
  return d == 96 ? 3 : d == 128 ? 2 : 1;
}

struct Kv8Plan : Kv4Plan {
  bool once;   // rows kernel: codes pass the caches by
};
Kv8Plan kv8_plan(const gq_kv8_attention_args& a);
hipError_t launch_kv8_rows(const Kv8Attn& a, const Kv8Plan& p, hipStream_t s);
hipError_t launch_kv8_tile(const Kv8Attn& a, const Kv4Plan& p, hipStream_t s);

// Choice of pages: what the kernels get.
struct Kv8Select {
  const uint16_t* q;
  int64_t q_ts, q_hs, q_tokens;
  int32_t hq, r, hkv, d, page_shift;
  const uint16_t* bounds;
  int64_t n_pages;
  const int32_t* table;
  int64_t batch, table_pages;
  const int32_t* kv_lens;
  const int32_t* q_starts;
  int64_t most;                     // pages that lengths are held to
  int32_t keep, first, last;
  int32_t* pages;
  int32_t* lens;
  double* scores;                   // [q_tokens][hkv][most]
};

hipError_t launch_kv8_select(const Kv8Select& a, gq_dtype dt, hipStream_t s);

}  // namespace gq
