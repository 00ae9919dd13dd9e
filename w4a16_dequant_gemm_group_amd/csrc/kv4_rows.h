// Attention over the 4-bit cache for few query rows per key/value head (single
// tokens, a few tokens to verify), and the pieces that every attention kernel
// of the cache shares: row tiles, the split of the key axis, the join.
//
// A query row is one (token, query head) pair; the r query heads that share a
// key/value head are rows of the same tile, so keys and values are read once
// for all of them.  Row tile qt of a sequence holds its rows qt * TQ ..; row i
// is token i / r, head kvh * r + i % r.
#pragma once

#include "kv4.h"
#include "stream_util.h"

namespace gq {
namespace kv4 {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;            // waves per workgroup
constexpr int kUnit = 32;            // tokens a wave takes at once (two sub-blocks)
constexpr int kTile = kWaves * kUnit;  // tokens of a key tile, the grain of the split
constexpr int kMetaInts = 8;
constexpr float kNegInf = -__builtin_inff();
// The running reference of the softmax lies kRoom powers of two below the largest
// score and is raised only when a score exceeds that by kSlack more: the largest
// weight is 2^11 to 2^15 as fp16, so weights keep all their bits down to 2^-25 of
// it and vanish below 2^-36.  With the largest at 1 and less room, what many light
// keys add up to beside a heavy one was lost (4096 keys 18 nats behind: all of it).
constexpr float kRoom = 11.0f, kSlack = 4.0f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// A sum of weights l that follows its reference from `from` up to `to`, f = 2^(from - to): the
// product of what this returns.  References that hold scales which lie up to 2^161 apart (the
// 8-bit cache's) can move so far that f is below fp32, and l f still worth keeping.  Then whole
// and broken powers of two are taken apart, which also keeps the bits that from - to would lose.
struct Moved {
  float l, f;
};

__device__ __forceinline__ bool moves_far(float from, float to) {
  return from - to < -100.0f && from - to > -300.0f;   // beyond it nothing is left
}

__device__ __forceinline__ Moved move_sum(float l, float from, float to, float f) {
  if (!moves_far(from, to)) return Moved{l, f};
  const float u = __builtin_rintf(from), v = __builtin_rintf(to);
  return Moved{__builtin_ldexpf(l * exp2_hw((from - u) - (to - v)), (int)(u - v)), 1.0f};
}

// The same, done.
__device__ __forceinline__ float sum_at(float l, float from, float to) {
  const Moved m = move_sum(l, from, to, exp2_hw(from - to));
  return m.l * m.f;
}

struct Seq {
  int q0, n, kv;   // first query row of q, queries, keys
};

__device__ __forceinline__ Seq get_seq(const Kv4Attn& a, int64_t b) {
  Seq s;
  if (a.q_starts) {
    const int64_t lim = a.q_tokens;
    int64_t x = a.q_starts[b], y = a.q_starts[b + 1];
    x = x < 0 ? 0 : (x > lim ? lim : x);
    y = y < x ? x : (y > lim ? lim : y);
    s.q0 = (int)x;
    s.n = (int)(y - x);
  } else {
    s.q0 = (int)b;
    s.n = 1;
  }
  const int64_t cap = a.table_pages << a.c.page_shift;
  int64_t kv = a.kv_lens[b];
  kv = kv < 0 ? 0 : (kv > cap ? cap : kv);
  s.kv = (int)kv;
  return s;
}

// The sequence b that the whole wave works on, in scalar registers.
__device__ __forceinline__ Seq wave_seq(const Kv4Attn& a, int64_t b) {
  Seq s = get_seq(a, b);
  s.q0 = __builtin_amdgcn_readfirstlane(s.q0);
  s.n = __builtin_amdgcn_readfirstlane(s.n);
  s.kv = __builtin_amdgcn_readfirstlane(s.kv);
  return s;
}

// n / r, the query heads per key/value head, for n < 2^31.
__device__ __forceinline__ int div_r(const Kv4Attn& a, int n) {
  return (int)(__umulhi(2u * (uint32_t)n, a.r_mul) >> a.r_shift);
}
__device__ __forceinline__ int row_tiles(const Kv4Attn& a, const Seq& s, int tq) {
  return (s.n * a.r + tq - 1) / tq;
}

// Row of `out` and `lse` that row `row` of a sequence's rows of head h is.
__device__ __forceinline__ int64_t out_row(const Kv4Attn& a, const Seq& s, int h, int row) {
  const int tok = div_r(a, row);
  return (int64_t)(s.q0 + tok) * a.hq + h * a.r + row - tok * a.r;
}

// The keys that row tile qt can see: positions lo .. hi - 1, in tiles of 2^grain
// keys from tile t0 on.  cnt: these tiles after `over` that hold no keys and
// stand for the work that a row tile is besides (a row without keys is written
// too), so that the split evens out both.
struct Span {
  int p0, p1;   // positions of the first and last query
  int lo, hi, t0, cnt;
};

template <int TQ>
__device__ __forceinline__ Span get_span(const Kv4Attn& a, const Seq& s, int qt) {
  const int rows = s.n * a.r;
  const int last = (qt + 1) * TQ < rows ? (qt + 1) * TQ - 1 : rows - 1;
  Span p;
  p.p0 = s.kv - s.n + div_r(a, qt * TQ);
  p.p1 = s.kv - s.n + div_r(a, last);
  p.hi = a.causal ? (p.p1 + 1 < s.kv ? p.p1 + 1 : s.kv) : s.kv;
  p.hi = p.hi < 0 ? 0 : p.hi;
  p.lo = a.window > 0 && p.p0 - a.window + 1 > 0 ? p.p0 - a.window + 1 : 0;
  p.t0 = p.lo >> a.grain;
  const int t1 = (p.hi + (1 << a.grain) - 1) >> a.grain;
  p.cnt = a.over + (t1 > p.t0 ? t1 - p.t0 : 0);
  return p;
}
// Position where tile j of a span begins.
__device__ __forceinline__ int64_t tile_start(const Kv4Attn& a, const Span& sp, int j) {
  return (int64_t)(sp.t0 + (j > a.over ? j - a.over : 0)) << a.grain;
}

// The i-th row tile of n in the order that the split goes through them: as they are,
// or (TURN) the last, the first, the last but one, ... so that under a causal mask any
// two next to each other hold about the same number of keys, and runs of equal work end
// at their borders.
template <bool TURN>
__device__ __forceinline__ int tile_at(int i, int n) {
  if constexpr (!TURN) return i;
  return i & 1 ? i >> 1 : n - 1 - (i >> 1);
}

// Where the split stands: sequence, head, row tile, and the key tiles of the
// row tile that lie before.
struct Cursor {
  int b, h, qt, off;
};

__device__ __forceinline__ uint32_t wave_scan(uint32_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  return v;
}
__device__ __forceinline__ uint32_t lane_of(uint32_t v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// Key tiles of one head over all row tiles of a sequence; lanes share the row
// tiles.  With `find`: the row tile that holds tile number i.
template <int TQ, bool TURN>
__device__ __forceinline__ uint32_t seq_tiles(const Kv4Attn& a, const Seq& s, int lane, bool find, uint32_t i,
                                              Cursor* cur) {
  const int nqt = row_tiles(a, s, TQ);
  uint32_t base = 0;
  for (int q = 0; q < nqt; q += 64) {
    const uint32_t v = q + lane < nqt ? get_span<TQ>(a, s, tile_at<TURN>(q + lane, nqt)).cnt : 0;
    const uint32_t sc = wave_scan(v, lane);
    if (find) {
      const uint64_t hit = __ballot(base + sc > i);
      if (hit) {
        const int l = __builtin_ctzll(hit);
        cur->qt = q + l;
        cur->off = (int)(i - base - lane_of(sc - v, l));
        return 0;
      }
    }
    base += lane_of(sc, 63);
  }
  return base;
}

// All key tiles of the call, in the order sequence, head, row tile, key tile,
// are cut into one run per worker, as equal as whole tiles allow.
struct Share {
  uint32_t total, at, end;   // tiles of the call; this worker's
  int busy;                  // workers that have any
  int w;                     // this one's number
  Cursor cur;                // where tile `at` is

  // The worker numbers are dealt such that each of the 8 dies (workgroups go
  // round robin over them) works on neighbouring runs: its L2 cache sees
  // neighbouring keys.
  __device__ __forceinline__ void cut(const Kv4Attn& a) {
    busy = total < (uint32_t)a.workers ? (int)total : a.workers;
    const int per_die = (busy + 7) >> 3, x = blockIdx.x >> 3;
    w = (blockIdx.x & 7) * per_die + x;
    at = end = 0;
    if (x >= per_die || w >= busy) return;
    const uint32_t q = total / busy, m = total % busy;   // the first m have one more
    at = q * w + (w < (int)m ? w : m);
    end = at + q + (w < (int)m ? 1 : 0);
  }
  // the worker that has tile i
  __device__ __forceinline__ int worker_with(uint32_t i) const {
    const uint32_t q = total / busy, m = total % busy, big = (q + 1) * m;
    return (int)(i < big ? i / (q + 1) : m + (i - big) / q);
  }
};

template <int TQ, bool TURN = false>
__device__ __forceinline__ Share find_share(const Kv4Attn& a, int lane) {
  Share sh{};
  sh.cur = Cursor{0, 0, 0, 0};
  const int batch = (int)a.batch, heads = a.c.hkv;
  uint32_t base = 0;
  if (a.few) {
    uint32_t v = 0, sc = 0;
    auto scan = [&](int b0) {
      v = 0;
      if (b0 + lane < batch) {
        const Seq s = get_seq(a, b0 + lane);
        const int nqt = row_tiles(a, s, TQ);
        for (int q = 0; q < nqt; ++q) v += get_span<TQ>(a, s, q).cnt;
      }
      sc = wave_scan(v, lane);
    };
    for (int b0 = 0; b0 < batch; b0 += 64) {
      scan(b0);
      base += lane_of(sc, 63);
    }
    sh.total = base * heads;
    sh.cut(a);
    if (sh.at == sh.end) return sh;
    base = 0;
    for (int b0 = 0;; b0 += 64) {
      if (batch > 64) scan(b0);
      const uint64_t hit = __ballot((base + sc) * heads > sh.at);
      if (hit) {
        const int l = __builtin_ctzll(hit);
        const uint32_t per = lane_of(v, l);
        const uint32_t i = sh.at - (base + lane_of(sc - v, l)) * heads;
        sh.cur.b = b0 + l;
        sh.cur.h = (int)(i / per);
        seq_tiles<TQ, TURN>(a, wave_seq(a, sh.cur.b), lane, true, i % per, &sh.cur);
        return sh;
      }
      base += lane_of(sc, 63);
    }
  }
  if (batch == 1) {
    // one sequence: its lengths are loaded once, and up to 64 row tiles scanned once
    const Seq s = wave_seq(a, 0);
    const int nqt = row_tiles(a, s, TQ);
    const uint32_t v = lane < nqt ? get_span<TQ>(a, s, tile_at<TURN>(lane, nqt)).cnt : 0, sc = wave_scan(v, lane);
    const uint32_t per = nqt <= 64 ? lane_of(sc, 63) : seq_tiles<TQ, TURN>(a, s, lane, false, 0, nullptr);
    sh.total = per * heads;
    sh.cut(a);
    if (sh.at == sh.end) return sh;
    sh.cur.h = (int)(sh.at / per);
    const uint32_t i = sh.at % per;
    if (nqt <= 64) {
      const int l = __builtin_ctzll(__ballot(sc > i));
      sh.cur.qt = l;
      sh.cur.off = (int)(i - lane_of(sc - v, l));
    } else {
      seq_tiles<TQ, TURN>(a, s, lane, true, i, &sh.cur);
    }
    return sh;
  }
  for (int b = 0; b < batch; ++b) base += seq_tiles<TQ, TURN>(a, wave_seq(a, b), lane, false, 0, nullptr);
  sh.total = base * heads;
  sh.cut(a);
  if (sh.at == sh.end) return sh;
  base = 0;
  for (int b = 0;; ++b) {
    const Seq s = wave_seq(a, b);
    const uint32_t per = seq_tiles<TQ, TURN>(a, s, lane, false, 0, nullptr), i = sh.at - base * heads;
    if (i < per * heads) {
      sh.cur.b = b;
      sh.cur.h = (int)(i / per);
      seq_tiles<TQ, TURN>(a, s, lane, true, i % per, &sh.cur);
      return sh;
    }
    base += per;
  }
}

// What the join has to know of a worker: the row tile that it left open (last:
// the last of the workers after it that hold the rest), or none (last < 0).
__device__ __forceinline__ void leave_meta(const Kv4Attn& a, const Share& sh, int last, const Cursor& cur,
                                           const Seq& s) {
  if ((int)blockIdx.x >= sh.busy) a.meta[(int64_t)blockIdx.x * kMetaInts] = -1;   // a number nobody has
  if (sh.at == sh.end) return;
  int4* mt = (int4*)(a.meta + (int64_t)sh.w * kMetaInts);
  mt[0] = make_int4(last, cur.h, cur.qt, 0);
  mt[1] = make_int4(s.q0, s.n, 0, 0);
}

// A row of the page table, which no kernel writes: read through the scalar
// unit, so that the loads of the keys are not waited for along with it.
typedef const int32_t __attribute__((address_space(4))) * PageRow;
__device__ __forceinline__ PageRow page_row(const Kv4Attn& a, int64_t b) {
  return (PageRow)(a.table + b * a.table_pages);
}

// 16 bytes per lane from p + voff to LDS at lds + 16 * lane, without registers
// between.  The wait for it is the caller's (wait_dma).
__device__ __forceinline__ void dma16(const uint8_t* p, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(voff), "s"(p)
               : "memory", "m0");
}
// Until at most N of the wave's loads are under way.
template <int N>
__device__ __forceinline__ void wait_dma() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
// Until the wave's reads of LDS have arrived: what they read may be overwritten.
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// N dwords from a 4-byte (N = 1, 3) or 8 / 16-byte aligned address.
template <int N>
__device__ __forceinline__ void load_dwords(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 v = ((const u32x4*)p)[i];
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const uint2 v = *(const uint2*)p;
    w[0] = v.x; w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = ((const uint32_t*)p)[i];
  }
}

// What a wave reads of one sub-block.  Keys: codes of its operand token m, the
// scales of its result tokens 4 kg .. 4 kg + 3 (pairs of halfs), the zero points
// of token m.  Values: codes, scales and zero points of its operand tokens 4 kg ...
template <int D, int NG, bool SYM>
struct KeyBlock {
  static constexpr int NS = D / 32;
  uint32_t c[NS], s[NG][2], z[(NG + 1) / 2];

  __device__ __forceinline__ void load(const uint8_t* blk, uint32_t m, uint32_t kg) {
    load_dwords<NS>(blk + m * (D / 2) + kg * (4 * NS), c);
    const uint8_t* p = blk + 8 * D;
#pragma unroll
    for (int g = 0; g < NG; ++g) load_dwords<2>(p + g * 32 + kg * 8, s[g]);
    if constexpr (!SYM) {
      const uint8_t* zp = p + 32 * NG + m * (2 * NG);
      if constexpr (NG % 2 == 0) {
        load_dwords<NG / 2>(zp, z);
      } else {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint32_t h = ((const uint16_t*)zp)[g];
          z[g / 2] = g & 1 ? z[g / 2] | h << 16 : h;
        }
      }
    }
  }
};

template <int D, int NG, bool SYM>
struct ValueBlock {
  static constexpr int NS = D / 32;
  // Three groups and more: a group's zero points are read when it is multiplied;
  // all of them at once spill (24 rows at 4 groups 56 us, so 44).
  static constexpr bool kLate = !SYM && NG > 2;
  uint32_t c[NS], s[NG][2], z[SYM || kLate ? 1 : NG][2];

  __device__ __forceinline__ void load(const uint8_t* w, uint32_t m, uint32_t kg) {
    load_dwords<NS>(w + kg * (64 * NS) + m * (4 * NS), c);
    const uint8_t* pv = w + 8 * D;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if constexpr (SYM) {
        load_dwords<2>(pv + g * 32 + kg * 8, s[g]);
      } else if constexpr (kLate) {
        load_dwords<2>(pv + g * 64 + kg * 16, s[g]);
      } else {
        uint32_t t[4];
        load_dwords<4>(pv + g * 64 + kg * 16, t);
        s[g][0] = t[0]; s[g][1] = t[1];
        z[g][0] = t[2]; z[g][1] = t[3];
      }
    }
  }
};

__device__ __forceinline__ float lo_f16(uint32_t w) { return f16_to_f32((uint16_t)(w & 0xFFFFu)); }
__device__ __forceinline__ float hi_f16(uint32_t w) { return f16_to_f32((uint16_t)(w >> 16)); }

// Half i of a dword array, as float.
template <int N>
__device__ __forceinline__ float half_of(const uint32_t (&w)[N], int i) {
  return i & 1 ? hi_f16(w[i >> 1]) : lo_f16(w[i >> 1]);
}

// Byte i of a dword array next to byte j: {i, 0, j, 0}.
template <int N>
__device__ __forceinline__ uint32_t byte_pair(const uint32_t (&w)[N], int i, int j) {
  const uint32_t sel = (uint32_t)(i & 3) | 0x0C000C00u | (uint32_t)(4 + (j & 3)) << 16;
  return __builtin_amdgcn_perm(w[j >> 2], w[i >> 2], sel);
}

// A pair of codes, masked in place, to fp16 c - z.  lo: nibbles at bits 0..3 of
// each half, where 0x6400 | c is 1024 + c; hi: at bits 4..7, where 0x5400 | c is
// 64 + c.  n: -(1024 + z) as it is stored, or -(64 + z).  Every step is exact.
// The masks live in vector registers and the exponents in scalar ones: an
// instruction takes one scalar and no literal besides, so mask and exponent
// as constants would make two of each and-or.
struct Nibbles {
  uint32_t mlo, mhi, elo, ehi;
  __device__ __forceinline__ Nibbles() : mlo(0x000F000Fu), mhi(0x00F000F0u), elo(0x64006400u), ehi(0x54005400u) {
    asm("" : "+v"(mlo), "+v"(mhi));
    asm("" : "+s"(elo), "+s"(ehi));
  }
  __device__ __forceinline__ uint32_t lo(uint32_t w, f16x2 n) const {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, (w & mlo) | elo) + n);
  }
  __device__ __forceinline__ uint32_t hi(uint32_t w, f16x2 n) const {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, (w & mhi) | ehi) + n);
  }
};

__device__ __forceinline__ f16x8 frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const u32x4 v = {a, b, c, d};
  return __builtin_bit_cast(f16x8, v);
}

// The rows kernel.  Each wave takes 32 keys at a time on its own, straight from
// memory to registers, with two products of the matrix cores:
//   S^T [keys, rows] = codes_K [keys, D] Q^T     (16x16x32, one step per 32 channels)
//   O^T [D, rows]   += codes_V^T [D, keys] P^T   (one step per 32 keys)
// The result layout of the first (lane = row, registers = 4 keys) is the operand
// layout of the second, so P never leaves its lane.
//
// Codes enter as the exact fp16 integers c - z.  (As subnormals c 2^-24, two of
// them for one AND, they would be exact too, but the products are aligned by
// the operands' exponent fields: measured errors of 2^-14 of a code.)
// What bounds it: vector instructions, most of them the expansion of the codes.
// Of a unit of 32 keys at 128 channels 176 of some 300 make the operands of its 16
// products; counters show the vector unit 70 to 76 % busy, the matrix unit 10 %,
// and no byte fetched twice.  151 MB of one sequence of 128 K keys pass in 35.5 us
// (4.2 TB/s; a copy reaches 5.0), 332 MB of 64 ragged ones in 79 us (4.2; 94 to 99
// where passes follow each other for milliseconds).
// Q becomes fp16 with a power of two per row that puts its largest element
// near 2^14: exact for fp16 and bf16 elements down to 2^-29 of the largest.
// So the scores are exact up to fp32 sums: s = sum_g S_g ((codes - z) . q).
// P' = p S_V goes to the matrix cores as fp16, one operand per group; it is
// rounded once (2^-11; `rest` below keeps what that leaves where it would show most,
// in fp16 results of the fewest rows: elsewhere a second part would double the second
// products, and in bf16 results it is an eighth of their own rounding).
// The reference that the exponentials subtract is the running maximum of score +
// log2 S_V, so that P' itself, not p, is what lies in fp16's range; a weight whose
// scale in one group is far below the largest of its groups has that much less of
// the room above.
template <int D, int NG, int NQ, bool SYM>
struct Rows {
  static constexpr int NS = D / 32, SPG = NS / NG, TQ = 16 * NQ;
  static constexpr int DH = D > 128 ? 128 : D;       // columns of a join pass
  static constexpr int kSmemRow = DH + 4;
  static constexpr int kSmemFloats = kWaves * 16 * kSmemRow + 2 * kWaves * 16;
  static constexpr int kSub = 2 * (8 * D + 16 * NG * (SYM ? 2 : 4));   // bytes of a sub-block
  static constexpr int kLoads = 2 * ((kSub + 1023) / 1024);            // wave-wide loads of a unit
  // two units per wave, later the waves' results
  static constexpr int kSmem = kWaves * 4 * kSub > 4 * kSmemFloats ? kWaves * 4 * kSub : 4 * kSmemFloats;

  f16x8 q[NQ][NS];
  float A[NQ];                      // score factor
  f32x4 o[NQ][2 * NS];
  float mref[NQ], l[NQ];
  // fp16 outputs of at most 8 rows: lanes 8 .. 15 of a tile hold the same rows
  // once more and carry what the rounding of p S_V to fp16 left, so that it
  // costs an fp16 result no accuracy.  The columns would be idle otherwise.
  bool rest;
  Nibbles nib;
  // The workgroups of a compute unit have equal work, but a SIMD serves its
  // oldest wave first: without more, the first of three ended at 21 us, the
  // others, ever fewer waves to hide their loads, at 26 and 32 (one token over
  // 128 K keys).  So a wave begins with the highest priority and steps down
  // with every quarter of its work: whoever is behind is served first.
  int left = 0, next = -1, quarter = 0;   // tiles left, those at which to step down
  __device__ __forceinline__ void begin_share(uint32_t tiles) {
    left = __builtin_amdgcn_readfirstlane((int)tiles);
    quarter = (left >> 2) + 1;
    next = left - quarter;
    __builtin_amdgcn_s_setprio(3);
  }
  __device__ __forceinline__ void tile_done() {
    left = __builtin_amdgcn_readfirstlane(left - 1);
    if (left != next) return;
    next = __builtin_amdgcn_readfirstlane(next - quarter);
    if (left > 2 * quarter) __builtin_amdgcn_s_setprio(2);
    else if (left > quarter) __builtin_amdgcn_s_setprio(1);
    else __builtin_amdgcn_s_setprio(0);
  }

  __device__ __forceinline__ int row_of_lane() const { return threadIdx.x & (rest ? 7 : 15); }

  __device__ __forceinline__ void load_q(const Kv4Attn& a, const Seq& s, int h, int qt, int m, int kg) {
    const int rows = s.n * a.r;
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      const int row = qt * TQ + nq * 16 + row_of_lane(), tok = div_r(a, row);
      float x[NS][8];
      float mx = 0.0f;
      const bool ok = row < rows;
      const uint16_t* p = a.q;
      if (ok) p += (int64_t)(s.q0 + tok) * a.q_ts + (int64_t)(h * a.r + row - tok * a.r) * a.q_hs;
#pragma unroll
      for (int st = 0; st < NS; ++st) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (ok) v = *(const uint4*)(p + 32 * st + 8 * kg);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[st][2 * i] = a.bf16 ? bf16_to_f32(w[i] & 0xFFFFu) : lo_f16(w[i]);
          x[st][2 * i + 1] = a.bf16 ? __uint_as_float(w[i] & 0xFFFF0000u) : hi_f16(w[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(x[st][i]));
      }
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      int e = (int)(__float_as_uint(mx) >> 23) - 127;   // exponent of the largest
      e = e < -112 ? -112 : (e > 127 ? 127 : e);   // 128: infinite or NaN
      const float f = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
      A[nq] = a.scale_log2 * __uint_as_float((uint32_t)(127 - 14 + e) << 23);   // / f
#pragma unroll
      for (int st = 0; st < NS; ++st)
#pragma unroll
        for (int i = 0; i < 8; ++i) q[nq][st][i] = (_Float16)(x[st][i] * f);
    }
  }

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      mref[nq] = kNegInf;
      l[nq] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2 * NS; ++i) o[nq][i] = f32x4{0, 0, 0, 0};
    }
  }

  // x = K^ q of 32 keys, without the row's factor A.
  __device__ __forceinline__ void scores(const KeyBlock<D, NG, SYM> (&kb)[2], float (&x)[NQ][2][4]) const {
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x4 acc[NQ];
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) acc[nq] = f32x4{0, 0, 0, 0};
        f16x2 n1 = {(_Float16)-1032.0f, (_Float16)-1032.0f};
        if constexpr (!SYM) {
          const _Float16 z = __builtin_bit_cast(_Float16, (uint16_t)(kb[t].z[g / 2] >> (16 * (g & 1))));
          n1 = f16x2{z, z};
        }
        const f16x2 n2 = n1 + (_Float16)960.0f;
#pragma unroll
        for (int st = g * SPG; st < (g + 1) * SPG; ++st) {
          const uint32_t d = kb[t].c[st], e = d >> 8;
          const f16x8 w = frag(nib.lo(d, n1), nib.hi(d, n2), nib.lo(e, n1), nib.hi(e, n2));
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq)
            acc[nq] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, q[nq][st], acc[nq], 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float S = half_of(kb[t].s[g], i);
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq)
            x[nq][t][i] = __builtin_fmaf(S, acc[nq][i], g == 0 ? 0.0f : x[nq][t][i]);
        }
      }
  }

  // Keys that no row of the tile sees: whatever their memory holds counts as
  // value scale 0 and a finite zero point (their scores are dropped in `weights`).
  static __device__ __forceinline__ void clear_unseen(const Span& sp, int u, bool ok0, bool ok1,
                                                      ValueBlock<D, NG, SYM> (&vb)[2], int kg) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t live[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int pos = u + 16 * t + 4 * kg + 2 * i;
        const bool ok = t ? ok1 : ok0;
        live[i] = (ok && pos >= sp.lo && pos < sp.hi ? 0xFFFFu : 0u) |
                  (ok && pos + 1 >= sp.lo && pos + 1 < sp.hi ? 0xFFFF0000u : 0u);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          vb[t].s[g][i] &= live[i];
          if constexpr (!SYM && !ValueBlock<D, NG, SYM>::kLate) vb[t].z[g][i] &= live[i];
        }
    }
  }

  // Scores to weights p = 2^(x A - mref); `masked` where some row does not see
  // all 32 keys from position u on.  ok0 / ok1: the sub-blocks that exist.
  __device__ __forceinline__ void weights(const Kv4Attn& a, const Seq& s, int qt, int u, bool masked, bool ok0,
                                          bool ok1, const ValueBlock<D, NG, SYM> (&vb)[2], float (&x)[NQ][2][4],
                                          int kg) {
    // log2 of the largest value scale of each key, within a tenth: the bits of
    // a non-negative half count powers of two in steps of 1 / 1024.  As the low
    // half of 2^23 + bits they are a float at once.
    float lv[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        u16x2 b = __builtin_bit_cast(u16x2, vb[t].s[0][i]);
#pragma unroll
        for (int g = 1; g < NG; ++g) b = __builtin_elementwise_max(b, __builtin_bit_cast(u16x2, vb[t].s[g][i]));
        const uint32_t w = __builtin_bit_cast(uint32_t, b);
        const float f0 = __uint_as_float(__builtin_amdgcn_perm(0x4B000000u, w, 0x07060100u));
        const float f1 = __uint_as_float(__builtin_amdgcn_perm(0x4B000000u, w, 0x07060302u));
        lv[t][2 * i] = __builtin_fmaf(f0, 1.0f / 1024.0f, -8207.0f - kRoom);
        lv[t][2 * i + 1] = __builtin_fmaf(f1, 1.0f / 1024.0f, -8207.0f - kRoom);
      }
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      float y[2][4];
      uint32_t hide = 0;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[t][i] = __builtin_fmaf(x[nq][t][i], A[nq], lv[t][i]);
      if (masked) {
        const int tok = div_r(a, qt * TQ + nq * 16 + row_of_lane());
        const int pos = s.kv - s.n + tok;
        const int last = a.causal && pos < s.kv - 1 ? pos : s.kv - 1;
        const int first = a.window > 0 ? pos - a.window + 1 : 0;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = u + 16 * t + 4 * kg + i;
            const bool seen = (t ? ok1 : ok0) && j <= last && j >= first;
            hide |= seen ? 0u : 1u << (4 * t + i);
            y[t][i] = seen ? y[t][i] : kNegInf;
          }
      }
      float top = kNegInf;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, y[t][i]);
      if (__any(top > mref[nq] + kSlack)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float mn = fmaxf(top, mref[nq]);
        const float c = mn == mref[nq] ? 1.0f : exp2_hw(mref[nq] - mn);
        mref[nq] = mn;
        l[nq] *= c;
#pragma unroll
        for (int i = 0; i < 2 * NS; ++i) o[nq][i] *= c;
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[nq][t][i] = exp2_hw(__builtin_fmaf(x[nq][t][i], A[nq], -mref[nq]));
      if (masked) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[nq][t][i] = hide >> (4 * t + i) & 1u ? 0.0f : x[nq][t][i];
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) l[nq] += x[nq][t][i];
    }
  }

  // o += V^^T p.  blk: the unit in LDS; masked: it may hold memory of any content.
  __device__ __forceinline__ void values(const ValueBlock<D, NG, SYM> (&vb)[2], const float (&p)[NQ][2][4],
                                         const uint8_t* blk, bool masked, uint32_t kg) {
    constexpr bool kLate = ValueBlock<D, NG, SYM>::kLate;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      uint32_t zl[2][2];
      if constexpr (kLate) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          load_dwords<2>(blk + kSub / 2 + t * kSub + 8 * D + g * 64 + kg * 16 + 8, zl[t]);
          if (masked) {   // any finite one will do beside a scale of 0
#pragma unroll
            for (int i = 0; i < 2; ++i) zl[t][i] = (zl[t][i] & 0x000F000Fu) | 0xE400E400u;
          }
        }
      }
      f16x8 pw[NQ];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float S = half_of(vb[t].s[g], i);
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq) pw[nq][4 * t + i] = (_Float16)__builtin_fmaf(p[nq][t][i], S, 0.0f);
        }
      if (rest) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float S = half_of(vb[t].s[g], i);
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) {
              const _Float16 h = pw[nq][4 * t + i];
              const _Float16 d = (_Float16)__builtin_fmaf(p[nq][t][i], S, -(float)h);
              pw[nq][4 * t + i] = (threadIdx.x & 8) != 0 ? d : h;
            }
          }
      }
      f16x2 n1[4], n2[4];   // by token pair
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        n1[i] = SYM ? f16x2{(_Float16)-1032.0f, (_Float16)-1032.0f}
                : kLate ? __builtin_bit_cast(f16x2, zl[i >> 1][i & 1])
                        : __builtin_bit_cast(f16x2, vb[i >> 1].z[SYM || kLate ? 0 : g][i & 1]);
        n2[i] = n1[i] + (_Float16)960.0f;
      }
#pragma unroll
      for (int b = g * SPG; b < (g + 1) * SPG; ++b) {
        uint32_t w[4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          w[2 * t] = byte_pair<NS>(vb[t].c, b, NS + b);
          w[2 * t + 1] = byte_pair<NS>(vb[t].c, 2 * NS + b, 3 * NS + b);
        }
        const f16x8 ev = frag(nib.lo(w[0], n1[0]), nib.lo(w[1], n1[1]), nib.lo(w[2], n1[2]), nib.lo(w[3], n1[3]));
        const f16x8 od = frag(nib.hi(w[0], n2[0]), nib.hi(w[1], n2[1]), nib.hi(w[2], n2[2]), nib.hi(w[3], n2[3]));
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
          o[nq][2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ev, pw[nq], o[nq][2 * b], 0, 0, 0);
          o[nq][2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(od, pw[nq], o[nq][2 * b + 1], 0, 0, 0);
        }
      }
    }
  }

  // Key tiles j0 .. j1 - 1 of the span.  A wave's units pass through LDS, two
  // at a time: a sub-block is one contiguous piece there as in the cache, and
  // loads that need no registers leave those to more waves.  Load by load into
  // registers, each with half a unit's work to arrive, 64 ragged sequences
  // (groups of 32) took 130 us where this takes 110 (89 with the split evened
  // out, 79 with late zero points), one token over 128 K keys 45 against 39 (36
  // with the steps of priority).
  __device__ __forceinline__ void keys(const Kv4Attn& a, const Seq& s, const Span& sp, int64_t b, int h,
                                       int qt, int j0, int j1, uint8_t* smem, int wave, int m, int kg) {
    const PageRow row = page_row(a, b);
    const int ps = a.c.page_shift;
    int u = (int)tile_start(a, sp, j0);
    const int64_t cut = tile_start(a, sp, j1);
    const int end = cut < sp.hi ? (int)cut : sp.hi;
    if (u < sp.lo) u = sp.lo & ~(kTile - 1);   // only the first tile can hold keys before the span
    u += wave * kUnit;
    if (u + kUnit <= sp.lo) u += kTile;
    rest = NQ == 1 && !a.bf16 && s.n * a.r <= 8;
    reset();
    if (u >= end) return;
    const uint32_t voff = (threadIdx.x & 63) * 16u;
    uint8_t* const own = smem + wave * (4 * kSub);
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_offset(own));
    // pages of the sub-blocks of a unit, -1 where no row sees keys of one
    struct Pages { int32_t p[2]; };
    auto pages = [&](int u) {
      Pages r = {{-1, -1}};
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int pos = u + 16 * t;
        if (pos < end && pos + 16 > sp.lo) r.p[t] = row[pos >> ps];
      }
      return r;
    };
    // bit t: sub-block t exists
    auto fetch = [&](const Pages& pg, int u, int buf) -> int {
      int ok = 0;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int pos = u + 16 * t;
        const int64_t page = pg.p[t];
        const bool is = page >= 0 && page < a.c.n_pages;
        ok |= is ? 1 << t : 0;
        // one that does not is read from the first page; its keys are not seen
        const uint8_t* p = a.c.cache + kv4_block_offset(a.c, is ? page : 0, h, is ? pos & ((1 << ps) - 1) : 0);
        const uint32_t dst = lds + (2 * buf + t) * kSub;
#pragma unroll
        for (int i = 0; i < kSub; i += 1024) {
          if (i + 1024 <= kSub)
            dma16(p + i, voff, dst + i);
          else if (voff < (uint32_t)(kSub - i))
            dma16(p + i, voff, dst + i);
        }
      }
      return ok;
    };
    const Pages first = pages(u);
    Pages next = pages(u + kTile);
    int ok = fetch(first, u, 0), oknext = 0;
    if (u + kTile < end) oknext = fetch(next, u + kTile, 1);
    load_q(a, s, h, qt, m, kg);
    for (int buf = 0;; buf ^= 1) {
      const int un = u + kTile;
      next = pages(un + kTile);
      if (un < end)
        wait_dma<kLoads>();
      else
        wait_dma<0>();
      // every row sees every key: all before the first query's position and
      // inside the last one's window
      bool full = ok == 3 && u + kUnit <= s.kv;
      if (a.causal) full = full && u + kUnit - 1 <= sp.p0;
      if (a.window > 0) full = full && u > sp.p1 - a.window;
      const uint8_t* blk = own + buf * (2 * kSub);
      float x[NQ][2][4];
      {
        KeyBlock<D, NG, SYM> kb[2];
        kb[0].load(blk, m, kg);
        kb[1].load(blk + kSub, m, kg);
        scores(kb, x);
      }
      ValueBlock<D, NG, SYM> vb[2];
      vb[0].load(blk + kSub / 2, m, kg);
      vb[1].load(blk + kSub / 2 + kSub, m, kg);
      if (!full) clear_unseen(sp, u, ok & 1, ok & 2, vb, kg);
      weights(a, s, qt, u, !full, ok & 1, ok & 2, vb, x, kg);
      values(vb, x, blk, !full, kg);
      tile_done();
      if (un >= end) break;
      u = un;
      ok = oknext;
      if (un + kTile < end) {
        wait_lds();
        oknext = fetch(next, un + kTile, buf);
      }
    }
  }

  // Joins the four waves' results and writes the rows: to `out` (part null) or,
  // unnormalized with their statistics, to a partial slot.
  __device__ __forceinline__ void finish(const Kv4Attn& a, const Seq& s, int h, int qt, float* part,
                                         float* smem, int wave, int m, int kg) {
    const int rows = s.n * a.r;
    float* so = smem;
    float* sm = smem + kWaves * 16 * kSmemRow;
    float* sl = sm + kWaves * 16;
    if (rest) {
#pragma unroll
      for (int i = 0; i < 2 * NS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[0][i][e] += __shfl_xor(o[0][i][e], 8);
    }
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      float lt = l[nq];
      lt += __shfl_xor(lt, 16);
      lt += __shfl_xor(lt, 32);
      // the reference is the same in the four lanes of a row unless the row
      // has seen nothing; the waves' references differ
      for (int half = 0; half < D / DH; ++half) {
        __syncthreads();
        if (kg == 0) {
          sm[wave * 16 + m] = mref[nq];
          sl[wave * 16 + m] = lt;
        }
#pragma unroll
        for (int bb = 0; bb < DH / 32; ++bb) {
#pragma unroll
          for (int hb = 0; hb < D / DH; ++hb) {
            if (hb != half) continue;
            const int b = hb * (DH / 32) + bb;
            const f32x4 e = o[nq][2 * b], d = o[nq][2 * b + 1];
            float4* dst = (float4*)(so + (wave * 16 + m) * kSmemRow + 32 * bb + 8 * kg);
            dst[0] = make_float4(e[0], d[0], e[1], d[1]);
            dst[1] = make_float4(e[2], d[2], e[3], d[3]);
          }
        }
        __syncthreads();
        constexpr int C = DH / 16;               // columns per thread
        const int rr = threadIdx.x >> 4, c0 = (threadIdx.x & 15) * C;
        const int row = qt * TQ + nq * 16 + rr;
        if (row < rows) {
          float M = kNegInf;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) M = fmaxf(M, sm[w * 16 + rr]);
          float L = 0.0f, acc[C];
#pragma unroll
          for (int i = 0; i < C; ++i) acc[i] = 0.0f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) {
            const float mw = sm[w * 16 + rr];
            const float f = mw == kNegInf ? 0.0f : exp2_hw(mw - M);
            L = __builtin_fmaf(f, sl[w * 16 + rr], L);
#pragma unroll
            for (int i = 0; i < C; ++i)
              acc[i] = __builtin_fmaf(f, so[(w * 16 + rr) * kSmemRow + c0 + i], acc[i]);
          }
          if (part) {
            float* po = part + (nq * 16 + rr) * D + half * DH + c0;
#pragma unroll
            for (int i = 0; i < C; ++i) po[i] = acc[i];
            if ((threadIdx.x & 15) == 0 && half == 0) {
              part[TQ * D + nq * 16 + rr] = M;
              part[TQ * D + TQ + nq * 16 + rr] = L;
            }
          } else {
            const int64_t orow = out_row(a, s, h, row);
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
            uint16_t* po = a.out + orow * D + half * DH + c0;
#pragma unroll
            for (int i = 0; i < C; i += 2) {
              const float v0 = acc[i] * inv, v1 = acc[i + 1] * inv;
              *(uint32_t*)(po + i) = pack_out(a.bf16, v0, v1);
            }
            if (a.lse && (threadIdx.x & 15) == 0 && half == 0) a.lse[orow] = lse_of(M, L);
          }
        }
      }
    }
  }

  static __device__ __forceinline__ float lse_of(float M, float L) {
    // kRoom moved from one term to the other, exactly: both are smaller so
    return L == 0.0f ? kNegInf : (M + kRoom + __log2f(L * (1.0f / (1 << (int)kRoom)))) * 0.69314718055994531f;
  }
  static __device__ __forceinline__ uint32_t pack_out(int bf16, float a, float b) {
    if (bf16) return bf16_bits(a) | (uint32_t)bf16_bits(b) << 16;
    return stream_util::f32_to_f16_rne(a) | (uint32_t)stream_util::f32_to_f16_rne(b) << 16;
  }
  // nearest-even bf16; NaN stays NaN
  static __device__ __forceinline__ uint16_t bf16_bits(float f) {
    return f == f ? f32_to_bf16_rne(f) : (uint16_t)0x7FC0u;
  }
};

template <int D, int NG, int NQ, bool SYM>
__global__ __launch_bounds__(kWaves * 64, kv4_rows_waves(D, NG, NQ)) void kv4_rows_kernel(Kv4Attn a) {
  using R = Rows<D, NG, NQ, SYM>;
  __shared__ __attribute__((aligned(16))) uint8_t smem[R::kSmem];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, kg = lane >> 4;
  R st;
  const bool split = a.workers > 0;
  Share sh{};
  Cursor cur{};
  if (split) {
    sh = find_share<R::TQ>(a, lane);
    cur = sh.cur;
    st.begin_share(sh.end - sh.at);
  } else {
    // one workgroup per (sequence, head, row tile)
    const int id = blockIdx.x, bh = id / a.grid_q;
    cur.qt = id % a.grid_q;
    cur.h = bh % a.c.hkv;
    cur.b = bh / a.c.hkv;
    cur.off = 0;
  }
  uint32_t at = sh.at;
  int last = -1;
  Seq s = wave_seq(a, cur.b);
  int nqt = row_tiles(a, s, R::TQ);
  while (split ? at < sh.end : cur.qt < nqt) {
    const Span sp = get_span<R::TQ>(a, s, cur.qt);
    const int j0 = cur.off, left = (int)(sh.end - at);
    const int j1 = !split || sp.cnt - j0 < left ? sp.cnt : j0 + left;
    const bool starts = j0 == 0, ends = j1 == sp.cnt;
    st.keys(a, s, sp, cur.b, cur.h, cur.qt, j0, j1, smem, wave, m, kg);
    float* part = nullptr;
    if (!(starts && ends)) {
      part = a.part + ((int64_t)2 * sh.w + (starts ? 1 : 0)) * (R::TQ * (D + 2));
      if (starts) last = sh.worker_with(at + sp.cnt - 1);
    }
    st.finish(a, s, cur.h, cur.qt, part, (float*)smem, wave, m, kg);
    __syncthreads();   // the results have been read: the buffers are free again
    if (!split) {
      cur.qt += a.grid_q;
      continue;
    }
    at += j1 - j0;
    if (at >= sh.end) break;
    // the next row tile, head, sequence that has rows
    cur.off = 0;
    if (++cur.qt == nqt) {
      cur.qt = 0;
      if (++cur.h == a.c.hkv) {
        cur.h = 0;
        do { ++cur.b; s = wave_seq(a, cur.b); } while (s.n == 0);
        nqt = row_tiles(a, s, R::TQ);
      }
    }
  }
  if (split && threadIdx.x == 0) leave_meta(a, sh, last, cur, s);
}

// Joins the partial results of the row tiles that were split: 4 to 6 us for
// single tokens (latency: two dependent loads, then the partials), 12.5 us for a
// prompt of 4096 (464 partials of 232 of its 512 row tiles, 62 MB).  Worker w left
// its last row tile open: the workers after it, up to `last`, hold the rest.
// One workgroup per worker and RW rows at a time: D / 4 threads hold a row, PG
// such sets take every PG-th partial of it (many partials of few rows for
// single tokens, few of many rows for prompts).  FAR: where references
// lie far apart the sum of weights is made once more at the end, by move_sum.
template <int D, int TQ, int PG, bool FAR>
__global__ __launch_bounds__(256) void kv4_join_kernel(Kv4Attn a) {
  constexpr int QD = D / 4, RW = 256 / (QD * PG);
  constexpr int64_t kSlot = TQ * (D + 2);
  __shared__ float4 so[RW][PG][QD];
  __shared__ float sm[RW][PG], sl[RW][PG], sn[FAR ? RW : 1][PG];
  const int w = blockIdx.x;
  const int4* mt = (const int4*)(a.meta + (int64_t)w * kMetaInts);
  const int4 open = mt[0], seq = mt[1];
  const int last = open.x, h = open.y, qt = open.z;
  if (last < 0) return;
  const Seq s{seq.x, seq.y, 0};
  const int left = s.n * a.r - qt * TQ, rows = left < TQ ? left : TQ;
  const int tid = threadIdx.x;
  const int rw = tid / (QD * PG), pg = tid / QD % PG, qd = tid % QD;
  for (int r0 = blockIdx.y * RW; r0 < rows; r0 += gridDim.y * RW) {
    const int ri = r0 + rw;      // row within the tile
    const bool mine = rw < RW && ri < rows;
    float M = kNegInf, L = 0.0f, low = -kNegInf;   // low: the lowest reference that has a sum
    float4 acc = make_float4(0, 0, 0, 0);
    if (mine) {
      auto add = [&](int c) {
        const float* p = a.part + (2 * (int64_t)c + (c == w ? 1 : 0)) * kSlot;
        const float mc = p[TQ * D + ri], lc = p[TQ * D + TQ + ri];
        const float4 v = *(const float4*)(p + ri * D + qd * 4);
        const float mn = fmaxf(M, mc);
        const float f0 = M == kNegInf ? 0.0f : exp2_hw(M - mn);
        // NaN statistics (a non-finite query) come with reference -inf: kept
        const float f1 = mc == kNegInf ? 0.0f : exp2_hw(mc - mn);
        if constexpr (FAR) low = lc == 0.0f ? low : fminf(low, mc);
        M = mn;
        L = __builtin_fmaf(L, f0, lc * f1);
        acc.x = acc.x * f0 + v.x * f1;
        acc.y = acc.y * f0 + v.y * f1;
        acc.z = acc.z * f0 + v.z * f1;
        acc.w = acc.w * f0 + v.w * f1;
      };
#pragma unroll 4
      for (int c = w + pg; c <= last; c += PG) add(c);
    }
    if constexpr (PG > 1) {
      if (mine) {
        so[rw][pg][qd] = acc;
        if (qd == 0) {
          sm[rw][pg] = M;
          sl[rw][pg] = L;
          if constexpr (FAR) sn[rw][pg] = low;
        }
      }
      __syncthreads();
      if (mine && pg == 0) {
        M = kNegInf;
#pragma unroll
        for (int i = 0; i < PG; ++i) M = fmaxf(M, sm[rw][i]);
        L = 0.0f;
        acc = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < PG; ++i) {
          const float f = sm[rw][i] == kNegInf ? 0.0f : exp2_hw(sm[rw][i] - M);
          const float4 v = so[rw][i][qd];
          if constexpr (FAR) low = fminf(low, sn[rw][i]);
          L += f * sl[rw][i];
          acc.x += f * v.x;
          acc.y += f * v.y;
          acc.z += f * v.z;
          acc.w += f * v.w;
        }
      }
      __syncthreads();
    }
    if (mine && pg == 0) {
      if constexpr (FAR) {
        if (low - M < -100.0f) {
          L = 0.0f;
#pragma unroll 1
          for (int c = w; c <= last; ++c) {
            const float* p = a.part + (2 * (int64_t)c + (c == w ? 1 : 0)) * kSlot + TQ * D + ri;
            L += sum_at(p[TQ], p[0], M);
          }
        }
      }
      using R = Rows<D, 1, 1, true>;
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      const int row = qt * TQ + ri;
      const int64_t orow = out_row(a, s, h, row);
      *(uint2*)(a.out + orow * D + qd * 4) = make_uint2(R::pack_out(a.bf16, acc.x * inv, acc.y * inv),
                                                        R::pack_out(a.bf16, acc.z * inv, acc.w * inv));
      if (a.lse && qd == 0) a.lse[orow] = R::lse_of(M, L);
    }
  }
}

template <int D, int TQ, int PG, bool FAR = false>
hipError_t launch_join(const Kv4Attn& a, int rows, hipStream_t s) {
  constexpr int RW = 256 / (D / 4 * PG);
  hipLaunchKernelGGL((kv4_join_kernel<D, TQ, PG, FAR>), dim3(a.workers, (rows + RW - 1) / RW), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int D, int NG, int NQ, bool SYM>
hipError_t launch_rows(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s) {
  const int64_t n = p.split ? a.workers : (int64_t)p.grid_q * a.c.hkv * a.batch;
  hipLaunchKernelGGL((kv4_rows_kernel<D, NG, NQ, SYM>), dim3((unsigned)n), dim3(kWaves * 64), 0, s, a);
  if (hipError_t e = hipGetLastError()) return e;
  return p.split ? launch_join<D, 16 * NQ, 256 / (D / 4)>(a, p.tile_rows, s) : hipSuccess;
}

template <int D, int NG>
hipError_t launch_rows_any(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s) {
  if (p.nq == 1) return a.c.sym ? launch_rows<D, NG, 1, true>(a, p, s) : launch_rows<D, NG, 1, false>(a, p, s);
  return a.c.sym ? launch_rows<D, NG, 2, true>(a, p, s) : launch_rows<D, NG, 2, false>(a, p, s);
}

}  // namespace kv4

}  // namespace gq
