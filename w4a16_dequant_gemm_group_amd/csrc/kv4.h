// The 4-bit key/value cache: byte order of a page and the declarations shared
// by the kernels that write it, read it and attend over it.
//
// A page holds, head by head, page_size / 16 sub-blocks of 16 tokens.  One
// sub-block of D channels in NG groups (NS = D / 32):
//   key codes    16 rows (tokens) of D / 2 bytes
//   key params   S fp16 [NG][16 tokens], then (asymmetric) z fp16 [16 tokens][NG]
//   value codes  [4 token quads][16 m][4 tokens][NS] bytes
//   value params S fp16 [NG][16 tokens] (symmetric), or [NG][4 token quads] of
//                {S of 4 tokens, z of 4 tokens} fp16
// A group of zeros has S = 0.  A zero point z (an integer 0 .. 15) is kept as
// -(1024 + z), what a code takes on as fp16 bits 0x6400 | c is short of c - z by.
// Both code orders are those in which the 16x16x32 matrix product takes its first
// operand, whose lane (m = lane % 16, kg = lane / 16) holds row m and 8
// consecutive k:
//   keys (row = token, k = channel): channel dword w = 4 s + kg (channels
//     32 s + 8 kg ..) is stored at dword kg * NS + s, so a lane's operands of
//     all NS steps are NS consecutive dwords, and step s covers the channels of
//     one block of 32, inside one group.  Inside a dword channel j of 8 sits at
//     nibble {0, 4, 1, 5, 2, 6, 3, 7}[j], so that the masks 0x000F000F and
//     0x00F000F0 (and both again after a shift by 8) give the pairs (0, 1),
//     (2, 3), (4, 5), (6, 7) as 16-bit halves.  The zero points of a lane's
//     token lie together; scales are applied to results, whose lanes hold the
//     tokens 4 kg .. 4 kg + 3.
//   values (row = channel, k = token): byte (m, b) of a token holds channels
//     32 b + 2 m (low nibble) and 32 b + 2 m + 1; the four tokens of a quad
//     stand next to each other.  A byte belongs to one token: writing a token
//     touches no byte of another one.
#pragma once

#include "gq_internal.h"
#include "gq_kv.h"

namespace gq {

struct Kv4Geo {
  uint8_t* cache;
  int64_t n_pages;
  int32_t hkv, d, g, ng, sym;
  int32_t page_shift;   // log2(page_size)
  uint32_t meta;        // bytes of one parameter section: 16 * ng * (sym ? 2 : 4)
  uint32_t sb;          // bytes of a sub-block: 2 * (8 d + meta)
};

// A zero point as it is stored, and back.
__device__ __forceinline__ uint16_t kv4_zero_bits(int z) { return (uint16_t)(0xE400u | (uint32_t)z); }
__device__ __forceinline__ float kv4_zero(uint16_t b) { return -1024.0f - f16_to_f32(b); }

// Byte offset of the sub-block that holds `slot` for `head`.
__device__ __forceinline__ int64_t kv4_block_offset(const Kv4Geo& c, int64_t page, int head,
                                                    int token_in_page) {
  return ((page * c.hkv + head) << (c.page_shift - 4)) * (int64_t)c.sb +
         (int64_t)(token_in_page >> 4) * c.sb;
}

hipError_t launch_kv4_write(const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts,
                            int64_t v_hs, gq_dtype dt, int64_t tokens, const int64_t* slots,
                            const Kv4Geo& c, hipStream_t s);
hipError_t launch_kv4_read(const Kv4Geo& c, const int64_t* slots, int64_t tokens, void* k, void* v,
                           gq_dtype odt, hipStream_t s);

// Attention: what the kernels get.
struct Kv4Attn {
  Kv4Geo c;
  const uint16_t* q;
  int64_t q_ts, q_hs, q_tokens;
  int32_t hq, r;                     // query heads, query heads per kv head
  uint32_t r_mul, r_shift;           // n / r = (2 n * r_mul >> 32) >> r_shift for n < 2^31
  int32_t bf16;                      // 1: bf16 q and out, 0: fp16
  const int32_t* table;
  int64_t batch, table_pages;
  const int32_t* kv_lens;
  const int32_t* q_starts;           // or nullptr: one query per sequence
  int32_t causal, window;
  float scale_log2;                  // scale * log2(e)
  uint16_t* out;
  float* lse;
  // the split over workgroups
  int32_t workers;                   // workgroups of a split launch
  int32_t grain;                     // log2 of the keys of a tile of the split
  int32_t over;                      // what a row tile costs besides its keys, in such tiles
  int32_t few;                       // few row tiles per sequence: lanes share the sequences
  int32_t grid_q;                    // row tiles in an unsplit launch's grid
  int32_t* meta;                     // [workers][8] which row tiles were left open
  float* part;                       // [2 * workers][rows][D + 2] partial results
};

// Waves per SIMD of the rows kernel (d channels in ng groups, nq tiles of 16 rows),
// which limits their registers.  16 sequences of 8192 keys, 8 key/value heads, with
// as many as here / one fewer: 128 channels 35 / 39 us, in 4 groups 43 / 48 (though
// with two row tiles 30 registers spill: 69 / 88); 256 channels 60 / 69, in 4 groups
// 70 / 86, in 8 groups one wave: 106, two spill 50 registers in the loop, 117.
constexpr int kv4_rows_waves(int d, int ng, int nq) {
  if (d * nq > 256 || ng > 4) return 1;
  return d > 128 || nq > 1 ? 2 : 3;
}

struct Kv4Plan {
  bool tile;           // the kernel for many rows; else the rows kernel
  bool split;
  int nq;              // rows kernel: 16-row query tiles per workgroup
  int workers;         // workgroups when split
  int grid_q;          // row tiles per (sequence, head) when not split
  int tile_rows;       // rows of a row tile, as far as max_q_len tells
  int grain;           // log2 of the keys of a tile of the split
  bool few;            // few row tiles per sequence
  size_t ws_bytes;
};

Kv4Plan kv4_plan(const gq_kv4_attention_args& a);
hipError_t launch_kv4_attention(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s);

// one translation unit per head_dim
hipError_t launch_kv4_rows_64(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s);
hipError_t launch_kv4_rows_96(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s);
hipError_t launch_kv4_rows_128(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s);
hipError_t launch_kv4_rows_256(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s);
hipError_t launch_kv4_tile_64(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s);
hipError_t launch_kv4_tile_96(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s);
hipError_t launch_kv4_tile_128(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s);
hipError_t launch_kv4_tile_256(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s);

}  // namespace gq
