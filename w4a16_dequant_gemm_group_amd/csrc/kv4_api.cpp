// C ABI of the 4-bit key/value cache (gq_kv.h): argument validation, the launch
// plan of the attention, and dispatch.  Validation runs on the host before any
// HIP call, as in gq_api.cpp.
#include <algorithm>
#include <cmath>

#include "kv4.h"

namespace gq {
namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Taking up a row tile and writing it out costs about as much as two tiles of
// keys (measured for prompts: 6.5 us, a tile of 64 keys 2.8 us).
constexpr int kOverhead = 2;

constexpr int64_t kMaxTokens = (int64_t)1 << 30;
// Tokens of one launch of the storage kernels: at 8 rows per workgroup of 256
// threads at least, 2^29 threads along the grid's first dimension (2^32 is the end).
constexpr int64_t kLaunchTokens = (int64_t)1 << 24;

gq_status check_layout(const gq_kv4_layout& y) {
  if (y.kv_heads < 1 || y.kv_heads > 65535 || y.head_dim < 1) return GQ_ERR_INVALID_ARG;
  if (y.page_size < 16 || y.page_size > 1024 || (y.page_size & (y.page_size - 1)) != 0)
    return GQ_ERR_INVALID_ARG;
  if (y.symmetric != 0 && y.symmetric != 1) return GQ_ERR_INVALID_ARG;
  if (y.group_size < 32 || y.group_size % 32 != 0 || y.head_dim % y.group_size != 0)
    return GQ_ERR_INVALID_ARG;
  if (y.head_dim != 64 && y.head_dim != 96 && y.head_dim != 128 && y.head_dim != 256)
    return GQ_ERR_UNSUPPORTED;
  return GQ_OK;
}

// Bytes of 16 tokens of one head.
uint32_t params_bytes(const gq_kv4_layout& y) {
  return 16u * (uint32_t)(y.head_dim / y.group_size) * (y.symmetric ? 2u : 4u);
}
uint32_t block_bytes(const gq_kv4_layout& y) { return 2u * (8u * (uint32_t)y.head_dim + params_bytes(y)); }

// Also that every offset into the cache fits 63 bits.
gq_status check_cache(int64_t n_pages, const gq_kv4_layout& y) {
  if (gq_status s = check_layout(y)) return s;
  if (n_pages < 1 || n_pages > INT32_MAX) return GQ_ERR_INVALID_ARG;
  const int64_t page = (int64_t)y.kv_heads * (y.page_size / 16) * block_bytes(y);
  if (n_pages > INT64_MAX / page) return GQ_ERR_INVALID_ARG;
  return GQ_OK;
}

Kv4Geo geometry(const uint8_t* cache, int64_t n_pages, const gq_kv4_layout& y) {
  Kv4Geo c;
  c.cache = const_cast<uint8_t*>(cache);
  c.n_pages = n_pages;
  c.hkv = y.kv_heads;
  c.d = y.head_dim;
  c.g = y.group_size;
  c.ng = y.head_dim / y.group_size;
  c.sym = y.symmetric;
  c.page_shift = __builtin_ctz((unsigned)y.page_size);
  c.meta = params_bytes(y);
  c.sb = block_bytes(y);
  return c;
}

gq_status from_hip(hipError_t e) { return e == hipSuccess ? GQ_OK : GQ_ERR_HIP; }

// Strides in elements: rows of 16-byte pieces, far from overflowing 64 bits.
gq_status check_strides(int64_t ts, int64_t hs) {
  constexpr int64_t lim = (int64_t)1 << 40;
  if (ts < -lim || ts > lim || hs < -lim || hs > lim) return GQ_ERR_INVALID_ARG;
  if (ts % 8 != 0 || hs % 8 != 0) return GQ_ERR_MISALIGNED;
  return GQ_OK;
}

// What the sizes and options of an attention call have to satisfy.
gq_status check_attention(const gq_kv4_attention_args& a) {
  if (gq_status s = check_cache(a.n_pages, a.layout)) return s;
  if (a.dtype != GQ_BF16 && a.dtype != GQ_F16)
    return a.dtype == GQ_F32 ? GQ_ERR_UNSUPPORTED : GQ_ERR_INVALID_ARG;
  if (a.q_heads < 1 || a.q_heads % a.layout.kv_heads != 0 || a.q_heads / a.layout.kv_heads > 64)
    return GQ_ERR_INVALID_ARG;
  if (a.q_tokens < 0 || a.q_tokens * a.q_heads > kMaxTokens || a.q_tokens > kMaxTokens)
    return GQ_ERR_INVALID_ARG;
  if (a.batch < 0 || a.batch > (1 << 24) || a.table_pages < 0) return GQ_ERR_INVALID_ARG;
  if (a.table_pages > kMaxTokens / a.layout.page_size) return GQ_ERR_INVALID_ARG;
  if (a.max_q_len < 0 || a.max_kv_len < 0 || a.max_q_len > kMaxTokens || a.max_kv_len > kMaxTokens)
    return GQ_ERR_INVALID_ARG;
  if ((a.causal != 0 && a.causal != 1) || a.window < 0 || (a.window > 0 && !a.causal))
    return GQ_ERR_INVALID_ARG;
  if (!(a.scale > 0.0f) || !std::isfinite(a.scale)) return GQ_ERR_INVALID_ARG;
  return GQ_OK;
}

}  // namespace

Kv4Plan kv4_plan(const gq_kv4_attention_args& a) {
  const int d = a.layout.head_dim, r = a.q_heads / a.layout.kv_heads;
  const int64_t rows = std::max<int64_t>(1, a.max_q_len) * r;
  Kv4Plan p;
  p.workers = 0;
  p.ws_bytes = 0;
  p.nq = rows <= 16 ? 1 : 2;
  p.tile = rows > 32;
  const int tq = p.tile ? (d > 128 ? 128 : 256) : 16 * p.nq;    // rows of a row tile
  p.grid_q = (int)((rows + tq - 1) / tq);
  p.tile_rows = (int)std::min<int64_t>(rows, tq);
  // lanes that share the sequences walk over the row tiles of each, lanes that
  // share the row tiles walk over the sequences (a load and a scan for each)
  p.few = p.grid_q <= 8 * std::min<int64_t>(a.batch, 64);
  // The kernels count tiles in 32 bits: a coarser grain where there might be
  // more (never more than q_tokens sequences have rows, so it ends).
  const int64_t cap = a.table_pages * a.layout.page_size;
  const int64_t row_tiles = (a.q_tokens * r / tq + std::min(a.batch, a.q_tokens)) * a.layout.kv_heads;
  p.grain = p.tile ? 6 : 7;
  while (p.grain < 30 && row_tiles * ((cap >> p.grain) + 1 + kOverhead) >= INT32_MAX) ++p.grain;
  // counted up to 2^24: so many row tiles are split and take all workgroups in any case
  constexpr int64_t kMany = (int64_t)1 << 24;
  const int64_t segs = std::min(kMany, std::min(kMany, a.batch * a.layout.kv_heads) * p.grid_q);
  const int64_t tiles = segs * (kOverhead + ((a.max_kv_len + (1 << p.grain) - 1) >> p.grain));
  // One workgroup per row tile, without the second kernel, as long as that is faster
  // than the split, which spreads few row tiles over the card.  Equal lengths of 512 /
  // 1024 keys, one against split: 8 row tiles of 128 channels 9.9 : 11.0 / 14.0 : 11.3
  // us, 64 of 256 channels 14.6 : 17.6 / 21.2 : 21.3, 128 of 128 channels 10.2 : 13.8 /
  // 14.4 : 16.5, 512 14.6 : 21.7 / 22 : 31.  Of more row tiles it would be faster for
  // longer (512: 4096 keys), but one long sequence among short ones runs alone then.
  // (A launch takes fewer than 2^32 threads.)
  p.split = p.tile || a.max_kv_len > std::min<int64_t>(1024, 512 + 8 * segs) || segs >= kMany;
  if (p.split) {
    // as many workgroups (a wave on each SIMD) as run at once
    const int64_t want = (int64_t)num_cus() * (p.tile ? 1 : kv4_rows_waves(d, d / a.layout.group_size, p.nq));
    p.workers = (int)std::max<int64_t>(8, std::min(tiles, want) & ~(int64_t)7);
    p.ws_bytes = (size_t)p.workers * 32 + (size_t)p.workers * 2 * tq * (d + 2) * sizeof(float);
  }
  return p;
}

hipError_t launch_kv4_attention(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s) {
  if (p.tile) {
    switch (a.c.d) {
      case 64: return launch_kv4_tile_64(a, p, s);
      case 96: return launch_kv4_tile_96(a, p, s);
      case 128: return launch_kv4_tile_128(a, p, s);
      default: return launch_kv4_tile_256(a, p, s);
    }
  }
  switch (a.c.d) {
    case 64: return launch_kv4_rows_64(a, p, s);
    case 96: return launch_kv4_rows_96(a, p, s);
    case 128: return launch_kv4_rows_128(a, p, s);
    default: return launch_kv4_rows_256(a, p, s);
  }
}

}  // namespace gq

using namespace gq;

extern "C" {

gq_status gq_kv4_cache_bytes(int64_t n_pages, gq_kv4_layout layout, size_t* bytes) {
  if (!bytes) return GQ_ERR_INVALID_ARG;
  *bytes = 0;
  if (gq_status s = check_cache(n_pages, layout)) return s;
  const Kv4Geo c = geometry(nullptr, n_pages, layout);
  *bytes = (size_t)n_pages * layout.kv_heads * (layout.page_size / 16) * c.sb;
  return GQ_OK;
}

gq_status gq_kv4_write(const void* k, int64_t k_token_stride, int64_t k_head_stride,
                       const void* v, int64_t v_token_stride, int64_t v_head_stride,
                       gq_dtype dtype, int64_t tokens, const int64_t* slots, uint8_t* cache,
                       int64_t n_pages, gq_kv4_layout layout, void* stream) {
  if (gq_status s = check_cache(n_pages, layout)) return s;
  if (dtype != GQ_BF16 && dtype != GQ_F16)
    return dtype == GQ_F32 ? GQ_ERR_UNSUPPORTED : GQ_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > kMaxTokens) return GQ_ERR_INVALID_ARG;
  if (tokens == 0) return GQ_OK;
  if (!k || !v || !slots || !cache) return GQ_ERR_INVALID_ARG;
  if (gq_status s = check_strides(k_token_stride, k_head_stride)) return s;
  if (gq_status s = check_strides(v_token_stride, v_head_stride)) return s;
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache) || ((uintptr_t)slots & 7u))
    return GQ_ERR_MISALIGNED;
  hipStream_t s = (hipStream_t)stream;
  if (gq_status st = check_device(s)) return st;
  const Kv4Geo c = geometry(cache, n_pages, layout);
  for (int64_t t = 0; t < tokens; t += kLaunchTokens)
    if (hipError_t e = launch_kv4_write((const uint16_t*)k + t * k_token_stride, k_token_stride, k_head_stride,
                                        (const uint16_t*)v + t * v_token_stride, v_token_stride, v_head_stride,
                                        dtype, std::min(tokens - t, kLaunchTokens), slots + t, c, s))
      return from_hip(e);
  return GQ_OK;
}

gq_status gq_kv4_read(const uint8_t* cache, int64_t n_pages, gq_kv4_layout layout,
                      const int64_t* slots, int64_t tokens, void* k, void* v, gq_dtype out_dtype,
                      void* stream) {
  if (gq_status s = check_cache(n_pages, layout)) return s;
  if (out_dtype != GQ_F32 && out_dtype != GQ_F16 && out_dtype != GQ_BF16) return GQ_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > kMaxTokens) return GQ_ERR_INVALID_ARG;
  if (tokens == 0) return GQ_OK;
  if (!k || !v || !slots || !cache) return GQ_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache) || ((uintptr_t)slots & 7u))
    return GQ_ERR_MISALIGNED;
  hipStream_t s = (hipStream_t)stream;
  if (gq_status st = check_device(s)) return st;
  const Kv4Geo c = geometry(cache, n_pages, layout);
  const int64_t row = (int64_t)layout.kv_heads * layout.head_dim * (out_dtype == GQ_F32 ? 4 : 2);
  for (int64_t t = 0; t < tokens; t += kLaunchTokens)
    if (hipError_t e = launch_kv4_read(c, slots + t, std::min(tokens - t, kLaunchTokens), (uint8_t*)k + t * row,
                                       (uint8_t*)v + t * row, out_dtype, s))
      return from_hip(e);
  return GQ_OK;
}

gq_status gq_kv4_attention_workspace_size(const gq_kv4_attention_args* args, size_t* bytes) {
  if (!args || !bytes) return GQ_ERR_INVALID_ARG;
  *bytes = 0;
  if (gq_status s = check_attention(*args)) return s;
  if (args->batch == 0 || args->q_tokens == 0) return GQ_OK;
  probe_device();
  *bytes = kv4_plan(*args).ws_bytes;
  return GQ_OK;
}

gq_status gq_kv4_attention(const gq_kv4_attention_args* args, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!args) return GQ_ERR_INVALID_ARG;
  const gq_kv4_attention_args& a = *args;
  if (gq_status s = check_attention(a)) return s;
  if (a.batch == 0 || a.q_tokens == 0) return GQ_OK;
  if (!a.q || !a.cache || !a.kv_lens || !a.out) return GQ_ERR_INVALID_ARG;
  if (!a.page_table && a.table_pages > 0) return GQ_ERR_INVALID_ARG;
  if (!a.q_starts && a.q_tokens < a.batch) return GQ_ERR_INVALID_ARG;
  if (gq_status s = check_strides(a.q_token_stride, a.q_head_stride)) return s;
  if (!aligned16(a.q) || !aligned16(a.cache) || !aligned16(a.out)) return GQ_ERR_MISALIGNED;
  if (((uintptr_t)a.page_table & 3u) || ((uintptr_t)a.kv_lens & 3u) || ((uintptr_t)a.q_starts & 3u) ||
      ((uintptr_t)a.lse & 3u))
    return GQ_ERR_MISALIGNED;
  probe_device();   // the split depends on the device's compute-unit count
  const Kv4Plan p = kv4_plan(a);
  if (p.ws_bytes > 0 && (!workspace || workspace_bytes < p.ws_bytes)) return GQ_ERR_INVALID_ARG;
  if (p.ws_bytes > 0 && !aligned16(workspace)) return GQ_ERR_MISALIGNED;
  hipStream_t s = (hipStream_t)stream;
  if (gq_status st = check_device(s)) return st;
  Kv4Attn k;
  k.c = geometry(a.cache, a.n_pages, a.layout);
  k.q = (const uint16_t*)a.q;
  k.q_ts = a.q_token_stride;
  k.q_hs = a.q_head_stride;
  k.q_tokens = a.q_tokens;
  k.hq = a.q_heads;
  k.r = a.q_heads / a.layout.kv_heads;
  k.bf16 = a.dtype == GQ_BF16;
  k.table = a.page_table;
  k.batch = a.batch;
  k.table_pages = a.table_pages;
  k.kv_lens = a.kv_lens;
  k.q_starts = a.q_starts;
  k.causal = a.causal;
  // a window longer than any sequence hides nothing
  k.window = a.window > kMaxTokens ? 0 : a.window;
  k.scale_log2 = a.scale * 1.4426950408889634f;
  k.out = (uint16_t*)a.out;
  k.lse = a.lse;
  k.r_shift = 0;
  while ((1 << k.r_shift) < k.r) ++k.r_shift;
  k.r_mul = (uint32_t)((((uint64_t)1 << (31 + k.r_shift)) + k.r - 1) / k.r);
  k.workers = p.workers;
  k.grain = p.grain;
  k.over = kOverhead;
  k.few = p.few;
  k.grid_q = p.grid_q;
  k.meta = (int32_t*)workspace;
  k.part = p.split ? (float*)((uint8_t*)workspace + (size_t)p.workers * 32) : nullptr;
  return from_hip(launch_kv4_attention(k, p, s));
}

}  // extern "C"
