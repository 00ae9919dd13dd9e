// C ABI of the 8-bit key/value cache (gq_kv8.h): argument validation, the launch
// plan of the attention, and dispatch.  Validation runs on the host before any
// HIP call, as in gq_api.cpp.
#include <algorithm>
#include <cmath>

#include "kv8.h"

namespace gq {
namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// What a row tile costs besides its keys, in tiles of keys: a prompt of 4096 at 128 channels
// with 2 / 3 / 4 / 5 / 6 / 8 213 / 205 / 196 / 191 / 192 / 194 us, at 256 151 / 137 / 137 / 136 / 139 / 142,
// chunks of 1010 tokens there 57 / 55 / 55 / 59 / 58 / 58, before row tiles were dealt in turn and
// their ends became cheaper; 3 to 6 are within 2 % of each other since.
constexpr int overhead(int d, bool tile) { return !tile ? 2 : d > 128 ? 3 : 5; }
constexpr int64_t kMaxTokens = (int64_t)1 << 30;
constexpr int64_t kMaxBatch = 1 << 24;

gq_status check_layout(const gq_kv8_layout& y) {
  if (y.kv_heads < 1 || y.kv_heads > 65535 || y.head_dim < 32 || y.head_dim % 32 != 0) return GQ_ERR_INVALID_ARG;
  if (y.page_size < 16 || y.page_size > 1024 || (y.page_size & (y.page_size - 1)) != 0) return GQ_ERR_INVALID_ARG;
  if (y.head_dim != 64 && y.head_dim != 96 && y.head_dim != 128 && y.head_dim != 256) return GQ_ERR_UNSUPPORTED;
  return GQ_OK;
}

int64_t blocks_per_page(const gq_kv8_layout& y) { return (int64_t)y.kv_heads * (y.page_size / 16); }
int64_t block_bytes(const gq_kv8_layout& y) { return 32 * (int64_t)y.head_dim + 8; }

// Also that every offset into the cache fits 62 bits.
gq_status check_cache(int64_t n_pages, const gq_kv8_layout& y) {
  if (gq_status s = check_layout(y)) return s;
  if (n_pages < 1 || n_pages > INT32_MAX) return GQ_ERR_INVALID_ARG;
  if (n_pages >= ((int64_t)1 << 62) / (blocks_per_page(y) * block_bytes(y))) return GQ_ERR_INVALID_ARG;
  return GQ_OK;
}

Kv8Geo geometry(const uint8_t* cache, int64_t n_pages, const gq_kv8_layout& y) {
  Kv8Geo c;
  c.cache = const_cast<uint8_t*>(cache);
  c.scales = (float2*)(c.cache + n_pages * blocks_per_page(y) * 32 * y.head_dim);
  c.n_pages = n_pages;
  c.hkv = y.kv_heads;
  c.d = y.head_dim;
  c.page_shift = __builtin_ctz((unsigned)y.page_size);
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

gq_status check_dtype(gq_dtype t) {
  if (t == GQ_BF16 || t == GQ_F16) return GQ_OK;
  return t == GQ_F32 ? GQ_ERR_UNSUPPORTED : GQ_ERR_INVALID_ARG;
}

// Sizes of a call with queries.
gq_status check_queries(int64_t q_tokens, int32_t q_heads, const gq_kv8_layout& y, int64_t batch, int64_t table_pages,
                        int64_t max_kv_len) {
  if (q_heads < 1 || q_heads % y.kv_heads != 0 || q_heads / y.kv_heads > 64) return GQ_ERR_INVALID_ARG;
  if (q_tokens < 0 || q_tokens > kMaxTokens || q_tokens * q_heads > kMaxTokens) return GQ_ERR_INVALID_ARG;
  if (batch < 0 || batch > kMaxBatch || table_pages < 0 || table_pages > kMaxTokens / y.page_size) return GQ_ERR_INVALID_ARG;
  if (max_kv_len < 0 || max_kv_len > kMaxTokens) return GQ_ERR_INVALID_ARG;
  return GQ_OK;
}

gq_status check_attention(const gq_kv8_attention_args& a) {
  if (gq_status s = check_cache(a.n_pages, a.layout)) return s;
  if (gq_status s = check_dtype(a.dtype)) return s;
  if (gq_status s = check_queries(a.q_tokens, a.q_heads, a.layout, a.batch, a.table_pages, a.max_kv_len)) return s;
  if (a.max_q_len < 0 || a.max_q_len > kMaxTokens) return GQ_ERR_INVALID_ARG;
  if (a.head_tables != 0 && a.head_tables != 1) return GQ_ERR_INVALID_ARG;
  if ((a.causal != 0 && a.causal != 1) || a.window < 0 || (a.window > 0 && !a.causal)) return GQ_ERR_INVALID_ARG;
  if (!(a.scale > 0.0f) || !std::isfinite(a.scale)) return GQ_ERR_INVALID_ARG;
  return GQ_OK;
}

gq_status check_select(const gq_kv8_select_args& a) {
  if (gq_status s = check_cache(a.n_pages, a.layout)) return s;
  if (gq_status s = check_dtype(a.dtype)) return s;
  if (gq_status s = check_queries(a.q_tokens, a.q_heads, a.layout, a.batch, a.table_pages, a.max_kv_len)) return s;
  if (a.keep < 1 || a.keep > 65536 || a.first < 0 || a.last < 1 || a.last > a.keep || a.first > a.keep - a.last)
    return GQ_ERR_INVALID_ARG;
  const int64_t lists = a.q_tokens * a.layout.kv_heads;
  if (lists >= ((int64_t)1 << 31) || lists * a.keep >= ((int64_t)1 << 40)) return GQ_ERR_INVALID_ARG;
  return GQ_OK;
}

// Pages that a length can have.
int64_t most_pages(const gq_kv8_select_args& a) {
  const int64_t n = (a.max_kv_len + a.layout.page_size - 1) / a.layout.page_size;
  return std::min(n, a.table_pages);
}
size_t select_bytes(const gq_kv8_select_args& a) {
  return (size_t)a.q_tokens * a.layout.kv_heads * (size_t)most_pages(a) * sizeof(double);
}

}  // namespace

Kv8Plan kv8_plan(const gq_kv8_attention_args& a) {
  const int d = a.layout.head_dim, r = a.q_heads / a.layout.kv_heads;
  const int64_t rows = std::max<int64_t>(1, a.max_q_len) * r;
  Kv8Plan p;
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
  const int over = overhead(d, p.tile);
  while (p.grain < 30 && row_tiles * ((cap >> p.grain) + 1 + over) >= INT32_MAX) ++p.grain;
  // counted up to 2^24: so many row tiles are split and take all workgroups in any case
  constexpr int64_t kMany = (int64_t)1 << 24;
  const int64_t segs = std::min(kMany, std::min(kMany, a.batch * a.layout.kv_heads) * p.grid_q);
  const int64_t tiles = segs * (over + ((a.max_kv_len + (1 << p.grain) - 1) >> p.grain));
  // One workgroup per row tile, without the second kernel, as long as that is faster than
  // the split, which spreads few row tiles over the card.  Equal lengths, one against split, us:
  //   8 row tiles of 128 channels, 512 / 768 keys 9.4 : 11.2 / 10.9 : 11.1; 160, 2048 keys 22.0 : 25.7
  //   4 of 64, 768 / 2048 keys 8.9 : 11.1 / 14.6 : 11.7; 80, 2048 keys 15.3 : 16.6
  //   2 of 256, 256 / 512 keys 11.1 : 13.5 / 15.3 : 13.8; 128, 1024 / 2048 keys 26.2 : 27.3 / 41 : 36
  // Of more row tiles it would be faster for longer (512 of 128 channels: 4096 keys), but one
  // long sequence among short ones runs alone then.
  const int64_t alone = d == 64 ? 960 + 14 * segs : d == 256 ? 360 + 7 * segs : 600 + 8 * segs;
  // Codes that are read once, and are more than stays in the caches beside all else until they
  // are read again, pass them by.  Without / with, us: 64 sequences of up to 8191 keys of 8 heads
  // of 128 120.5 / 109.7, 131071 keys of one 65.0 / 58.7, 16 of 8000 75.1 / 68.6 (262 MB); but
  // 32 of 8000 with one head (65 MB) 31.8 / 34.2, 4 of 500 14.7 / 15.3.  Chosen pages are often
  // those of the queries beside (head_tables: 40 queries of 16 sequences 28.5 / 29.2).
  const int64_t seen = a.window > 0 ? std::min<int64_t>(a.max_kv_len, (int64_t)a.window + a.max_q_len) : a.max_kv_len;
  p.once = !a.head_tables && (double)a.batch * (double)seen * a.layout.kv_heads * 2.0 * d > (double)(1 << 27);
  p.split = p.tile || a.max_kv_len > std::min<int64_t>(2048, alone) || segs >= kMany;
  if (p.split) {
    // as many workgroups (a wave on each SIMD) as run at once
    const int64_t want = (int64_t)num_cus() * (p.tile ? 1 : kv8_rows_waves(d, p.nq));
    p.workers = (int)std::max<int64_t>(8, std::min(tiles, want) & ~(int64_t)7);
    p.ws_bytes = (size_t)p.workers * 32 + (size_t)p.workers * 2 * tq * (d + 2) * sizeof(float);
  }
  return p;
}

}  // namespace gq

using namespace gq;

extern "C" {

gq_status gq_kv8_cache_bytes(int64_t n_pages, gq_kv8_layout layout, size_t* bytes) {
  if (!bytes) return GQ_ERR_INVALID_ARG;
  *bytes = 0;
  if (gq_status s = check_cache(n_pages, layout)) return s;
  *bytes = (size_t)(n_pages * blocks_per_page(layout) * block_bytes(layout));
  return GQ_OK;
}

gq_status gq_kv8_append(const gq_kv8_append_args* args, void* stream) {
  if (!args) return GQ_ERR_INVALID_ARG;
  const gq_kv8_append_args& a = *args;
  if (gq_status s = check_cache(a.n_pages, a.layout)) return s;
  if (gq_status s = check_dtype(a.dtype)) return s;
  if (a.tokens < 0 || a.tokens > kMaxTokens || a.batch < 0 || a.batch > kMaxBatch || a.table_pages < 0 ||
      a.table_pages > kMaxTokens / a.layout.page_size)
    return GQ_ERR_INVALID_ARG;
  if (a.tokens == 0 || a.batch == 0) return GQ_OK;
  if (!a.starts && a.tokens < a.batch) return GQ_ERR_INVALID_ARG;
  if (!a.k || !a.v || !a.cache || !a.kv_lens) return GQ_ERR_INVALID_ARG;
  if (!a.page_table && a.table_pages > 0) return GQ_ERR_INVALID_ARG;
  if (gq_status s = check_strides(a.k_token_stride, a.k_head_stride)) return s;
  if (gq_status s = check_strides(a.v_token_stride, a.v_head_stride)) return s;
  if (!aligned16(a.k) || !aligned16(a.v) || !aligned16(a.cache) || !aligned16(a.bounds)) return GQ_ERR_MISALIGNED;
  if (!aligned4(a.page_table) || !aligned4(a.kv_lens) || !aligned4(a.starts)) return GQ_ERR_MISALIGNED;
  hipStream_t s = (hipStream_t)stream;
  if (gq_status st = check_device(s)) return st;
  Kv8Append k;
  k.c = geometry(a.cache, a.n_pages, a.layout);
  k.k = (const uint16_t*)a.k;
  k.v = (const uint16_t*)a.v;
  k.k_ts = a.k_token_stride;
  k.k_hs = a.k_head_stride;
  k.v_ts = a.v_token_stride;
  k.v_hs = a.v_head_stride;
  k.tokens = a.starts ? a.tokens : a.batch;
  k.table = a.page_table;
  k.batch = a.batch;
  k.table_pages = a.table_pages;
  k.kv_lens = a.kv_lens;
  k.starts = a.starts;
  k.bounds = (uint16_t*)a.bounds;
  return from_hip(launch_kv8_append(k, a.dtype, s));
}

gq_status gq_kv8_read(const uint8_t* cache, int64_t n_pages, gq_kv8_layout layout,
                      const int64_t* slots, int64_t tokens, void* k, void* v, gq_dtype out_dtype,
                      void* stream) {
  if (gq_status s = check_cache(n_pages, layout)) return s;
  if (out_dtype != GQ_F32 && out_dtype != GQ_F16 && out_dtype != GQ_BF16) return GQ_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > kMaxTokens) return GQ_ERR_INVALID_ARG;
  if (tokens == 0) return GQ_OK;
  if (!k || !v || !slots || !cache) return GQ_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache) || ((uintptr_t)slots & 7u)) return GQ_ERR_MISALIGNED;
  hipStream_t s = (hipStream_t)stream;
  if (gq_status st = check_device(s)) return st;
  return from_hip(launch_kv8_read(geometry(cache, n_pages, layout), slots, tokens, k, v, out_dtype, s));
}

gq_status gq_kv8_attention_workspace_size(const gq_kv8_attention_args* args, size_t* bytes) {
  if (!args || !bytes) return GQ_ERR_INVALID_ARG;
  *bytes = 0;
  if (gq_status s = check_attention(*args)) return s;
  if (args->batch == 0 || args->q_tokens == 0) return GQ_OK;
  probe_device();
  *bytes = kv8_plan(*args).ws_bytes;
  return GQ_OK;
}

gq_status gq_kv8_attention(const gq_kv8_attention_args* args, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!args) return GQ_ERR_INVALID_ARG;
  const gq_kv8_attention_args& a = *args;
  if (gq_status s = check_attention(a)) return s;
  if (a.batch == 0 || a.q_tokens == 0) return GQ_OK;
  if (!a.q || !a.cache || !a.kv_lens || !a.out) return GQ_ERR_INVALID_ARG;
  if (!a.page_table && a.table_pages > 0) return GQ_ERR_INVALID_ARG;
  if (!a.q_starts && a.q_tokens < a.batch) return GQ_ERR_INVALID_ARG;
  if (gq_status s = check_strides(a.q_token_stride, a.q_head_stride)) return s;
  if (!aligned16(a.q) || !aligned16(a.cache) || !aligned16(a.out)) return GQ_ERR_MISALIGNED;
  if (!aligned4(a.page_table) || !aligned4(a.kv_lens) || !aligned4(a.q_starts) || !aligned4(a.lse)) return GQ_ERR_MISALIGNED;
  probe_device();   // the split depends on the device's compute-unit count
  const Kv8Plan p = kv8_plan(a);
  if (p.ws_bytes > 0 && (!workspace || workspace_bytes < p.ws_bytes)) return GQ_ERR_INVALID_ARG;
  if (p.ws_bytes > 0 && !aligned16(workspace)) return GQ_ERR_MISALIGNED;
  hipStream_t s = (hipStream_t)stream;
  if (gq_status st = check_device(s)) return st;
  const Kv8Geo c = geometry(a.cache, a.n_pages, a.layout);
  Kv8Attn k{};
  k.c.cache = c.cache;
  k.c.n_pages = c.n_pages;
  k.c.hkv = c.hkv;
  k.c.d = c.d;
  k.c.page_shift = c.page_shift;
  k.scales = c.scales;
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
  k.table_h = a.head_tables ? a.table_pages : 0;
  k.table_b = a.head_tables ? a.table_pages * a.layout.kv_heads : a.table_pages;
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
  k.over = overhead(c.d, p.tile);
  k.few = p.few;
  k.grid_q = p.grid_q;
  k.meta = (int32_t*)workspace;
  k.part = p.split ? (float*)((uint8_t*)workspace + (size_t)p.workers * 32) : nullptr;
  return from_hip(p.tile ? launch_kv8_tile(k, p, s) : launch_kv8_rows(k, p, s));
}

gq_status gq_kv8_select_workspace_size(const gq_kv8_select_args* args, size_t* bytes) {
  if (!args || !bytes) return GQ_ERR_INVALID_ARG;
  *bytes = 0;
  if (gq_status s = check_select(*args)) return s;
  *bytes = select_bytes(*args);
  return GQ_OK;
}

gq_status gq_kv8_select(const gq_kv8_select_args* args, void* workspace, size_t workspace_bytes,
                        void* stream) {
  if (!args) return GQ_ERR_INVALID_ARG;
  const gq_kv8_select_args& a = *args;
  if (gq_status s = check_select(a)) return s;
  if (a.q_tokens == 0) return GQ_OK;
  if (!a.q || !a.bounds || !a.pages || !a.lens || (!a.kv_lens && a.batch > 0)) return GQ_ERR_INVALID_ARG;
  if (!a.page_table && a.table_pages > 0 && a.batch > 0) return GQ_ERR_INVALID_ARG;
  if (!a.q_starts && a.q_tokens < a.batch) return GQ_ERR_INVALID_ARG;
  if (gq_status s = check_strides(a.q_token_stride, a.q_head_stride)) return s;
  if (!aligned16(a.q) || !aligned16(a.bounds)) return GQ_ERR_MISALIGNED;
  if (!aligned4(a.page_table) || !aligned4(a.kv_lens) || !aligned4(a.q_starts) || !aligned4(a.pages) || !aligned4(a.lens))
    return GQ_ERR_MISALIGNED;
  const size_t need = select_bytes(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return GQ_ERR_INVALID_ARG;
  if (need > 0 && !aligned16(workspace)) return GQ_ERR_MISALIGNED;
  hipStream_t s = (hipStream_t)stream;
  if (gq_status st = check_device(s)) return st;
  Kv8Select k;
  k.q = (const uint16_t*)a.q;
  k.q_ts = a.q_token_stride;
  k.q_hs = a.q_head_stride;
  k.q_tokens = a.q_tokens;
  k.hq = a.q_heads;
  k.r = a.q_heads / a.layout.kv_heads;
  k.hkv = a.layout.kv_heads;
  k.d = a.layout.head_dim;
  k.page_shift = __builtin_ctz((unsigned)a.layout.page_size);
  k.bounds = (const uint16_t*)a.bounds;
  k.n_pages = a.n_pages;
  k.table = a.page_table;
  k.batch = a.batch;
  k.table_pages = a.table_pages;
  k.kv_lens = a.kv_lens;
  k.q_starts = a.q_starts;
  k.most = most_pages(a);
  k.keep = a.keep;
  k.first = a.first;
  k.last = a.last;
  k.pages = a.pages;
  k.lens = a.lens;
  k.scores = (double*)workspace;
  return from_hip(launch_kv8_select(k, a.dtype, s));
}

}  // extern "C"
