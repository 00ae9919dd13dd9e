// Attention over the 8-bit cache for few query rows per key/value head (single
// tokens, a few tokens to verify).  The row tiles, the split of the key axis, the
// query side and the join are those of the 4-bit cache (kv4_rows.h), and so are the two
// products:
//   S^T [keys, rows] = codes_K [keys, D] Q^T,   O^T [D, rows] += codes_V^T [D, keys] P^T
// Codes enter as exact fp16 integers: a byte under 0x64 is 1024 + 128 + q, one addition
// for two codes takes the offset away.  A block's scale is the same for all results of a
// lane, so keys cost one factor per block, and P' = p S_V, rounded to fp16 once, one
// product per weight.
// Bound by memory: 64 sequences of up to 8191 keys, 8 heads of 128 with 4 query heads each,
// 88 us (531 MB at 6.0 TB/s); 131071 keys of one sequence 48 (5.6 TB/s); 201 keys 8.0, a chain
// of loads.
#include "kv8.h"
#include "kv4_rows.h"

namespace gq {
namespace kv8 {

using namespace kv4;

// Bytes of a dword as two pairs of fp16 integers -127 .. 127.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  const f16x2 off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) + off);
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  const f16x2 off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) + off);
}
__device__ __forceinline__ f16x8 codes8(uint32_t a, uint32_t b) {
  return frag(codes_lo(a), codes_hi(a), codes_lo(b), codes_hi(b));
}

// 4 bytes per lane from p to LDS at lds + 4 * lane, of the lanes that are active.
__device__ __forceinline__ void dma4(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" : : "s"(lds), "v"(p) : "memory", "m0");
}

// dma16 of bytes that are not read again soon.
__device__ __forceinline__ void dma16_once(const uint8_t* p, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt" : : "s"(lds), "v"(voff), "s"(p) : "memory", "m0");
}

// NW waves a workgroup: kWaves, or twice that where a compute unit has one alone.  ONCE: codes
// pass the caches by.
template <int D, int NQ, int NW, bool ONCE>
struct Rows8 : Rows<D, 1, NQ, true> {
  using Base = Rows<D, 1, NQ, true>;
  using Base::A;
  using Base::l;
  using Base::mref;
  using Base::o;
  using Base::q;
  using Base::rest;
  static constexpr int NS = D / 32, TQ = 16 * NQ;
  static constexpr int kSub = 32 * D;                 // bytes of a block's codes
  static constexpr int kUnitLds = 2 * kSub + 64;      // two blocks and their scales, padded
  static constexpr int kLoads = 2 * (kSub / 1024) + 1;   // wave-wide loads of a unit
  static constexpr int kStep = NW * kUnit;            // keys that a workgroup takes at once
  static constexpr int kSmem = NW * 2 * kUnitLds;
  static constexpr int kRow = D + 4;                  // floats of a row of results
  static_assert(4 * NW * (16 * kRow + 2 * 16) <= kSmem, "the results of all waves take the place of their units");

  // x = codes . q of 32 keys, without the row's factor A and the block's scale.
  __device__ __forceinline__ void scores(const uint8_t* blk, uint32_t lane, float (&x)[NQ][2][4]) const {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* c = blk + t * kSub;
      f32x4 acc[NQ];
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) acc[nq] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s + 1 < NS; s += 2) {
        const u32x4 w = *(const u32x4*)(c + 512 * s + 16 * lane);
        const f16x8 k0 = codes8(w.x, w.y), k1 = codes8(w.z, w.w);
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
          acc[nq] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, q[nq][s], acc[nq], 0, 0, 0);
          acc[nq] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, q[nq][s + 1], acc[nq], 0, 0, 0);
        }
      }
      if constexpr (NS % 2) {
        const uint2 w = *(const uint2*)(c + 512 * (NS - 1) + 8 * lane);
        const f16x8 k0 = codes8(w.x, w.y);
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
          acc[nq] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, q[nq][NS - 1], acc[nq], 0, 0, 0);
      }
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[nq][t][i] = acc[nq][i];
    }
  }

  // Scores to weights p = 2^(x A S_K - mref + 40); `masked` where some row does not see
  // all 32 keys from position u on.  ok: bit t, block t exists.  The reference is the
  // running maximum of score + log2 S_V less the room, so that P' = p S_V 2^-40 is what lies in
  // fp16's range (kKv8Shift).
  __device__ __forceinline__ void weights(const Kv4Attn& a, const Seq& s, int qt, int u, bool masked, int ok,
                                          const float (&sk)[2], const float (&sv)[2], float (&x)[NQ][2][4], int kg) {
    float lv[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) lv[t] = __log2f(sv[t]) - kRoom;
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      const float f[2] = {kv8_factor(A[nq], sk[0]), kv8_factor(A[nq], sk[1])};
      uint32_t hide = 0;
      float top = kNegInf;
      if (masked) {
        const int tok = div_r(a, qt * TQ + nq * 16 + this->row_of_lane());
        const int pos = s.kv - s.n + tok;
        const int last = a.causal && pos < s.kv - 1 ? pos : s.kv - 1;
        const int first = a.window > 0 ? pos - a.window + 1 : 0;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = u + 16 * t + 4 * kg + i;
            const bool seen = (ok >> t & 1) && j <= last && j >= first;
            hide |= seen ? 0u : 1u << (4 * t + i);
            top = fmaxf(top, seen ? __builtin_fmaf(x[nq][t][i], f[t], lv[t]) : kNegInf);
          }
      } else {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, __builtin_fmaf(x[nq][t][i], f[t], lv[t]));
      }
      if (__any(top > mref[nq] + kSlack)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float mn = fmaxf(top, mref[nq]);
        const float c = mn == mref[nq] ? 1.0f : exp2_hw(mref[nq] - mn);
        const Moved lm = move_sum(l[nq], mref[nq], mn, c);
        mref[nq] = mn;
        l[nq] = lm.l * lm.f;
#pragma unroll
        for (int i = 0; i < 2 * NS; ++i) o[nq][i] *= c;
      }
      const float base = kKv8Shift - mref[nq];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[nq][t][i] = exp2_hw(__builtin_fmaf(x[nq][t][i], f[t], base));
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

  // o += codes_V^T P'.
  __device__ __forceinline__ void values(const uint8_t* blk, const float (&sv)[2], const float (&p)[NQ][2][4],
                                         uint32_t lane) {
    f16x8 pw[NQ];
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = p[nq][t][i] * (sv[t] * kKv8Down);
          _Float16 h = (_Float16)e;
          if (rest) {
            const _Float16 d = (_Float16)(e - (float)h);
            h = (threadIdx.x & 8) != 0 ? d : h;
          }
          pw[nq][4 * t + i] = h;
        }
    const uint8_t* v0 = blk + kSub / 2;
    auto tile = [&](int i, uint32_t w0, uint32_t w1) {
      const f16x8 v = codes8(w0, w1);
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) o[nq][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pw[nq], o[nq][i], 0, 0, 0);
    };
#pragma unroll
    for (int g = 0; g + 3 < 2 * NS; g += 4) {
      const u32x4 a = *(const u32x4*)(v0 + 256 * g + 16 * lane), b = *(const u32x4*)(v0 + kSub + 256 * g + 16 * lane);
      tile(g, a.x, b.x);
      tile(g + 1, a.y, b.y);
      tile(g + 2, a.z, b.z);
      tile(g + 3, a.w, b.w);
    }
    if constexpr (NS % 2) {
      const uint2 a = *(const uint2*)(v0 + 512 * (NS - 1) + 8 * lane), b = *(const uint2*)(v0 + kSub + 512 * (NS - 1) + 8 * lane);
      tile(2 * NS - 2, a.x, b.x);
      tile(2 * NS - 1, a.y, b.y);
    }
  }

  // Joins the waves' results and writes the rows, as Rows::finish does with the other
  // order of channels (a lane's 2 D / 8 results of a row are consecutive ones), all channels
  // at once: the units leave room for them (256 channels in two halves: 0.6 us more), and with
  // all threads of eight waves (with half of them 0.3 us more).
  __device__ __forceinline__ void finish(const Kv4Attn& a, const Seq& s, int h, int qt, float* part, float* smem, int wave,
                                         int m, int kg) {
    constexpr int T = 2 * NS;
    const int rows = s.n * a.r;
    float* so = smem;
    float* sm = smem + NW * 16 * kRow;
    float* sl = sm + NW * 16;
    if (rest) {
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[0][i][e] += __shfl_xor(o[0][i][e], 8);
    }
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
#pragma unroll
      for (int i = 0; i < T; ++i) o[nq][i] *= kKv8Up;
      mref[nq] -= kKv8Shift;
      float lt = l[nq];
      lt += __shfl_xor(lt, 16);
      lt += __shfl_xor(lt, 32);
      __syncthreads();
      if (kg == 0) {
        sm[wave * 16 + m] = mref[nq];
        sl[wave * 16 + m] = lt;
      }
      // channels 4 T kg .. : i T + t of them is element i of tile t
      float4* dst = (float4*)(so + (wave * 16 + m) * kRow + 4 * T * kg);
#pragma unroll
      for (int c = 0; c < 4 * T; c += 4)
        dst[c / 4] = make_float4(o[nq][c % T][c / T], o[nq][(c + 1) % T][(c + 1) / T], o[nq][(c + 2) % T][(c + 2) / T],
                                 o[nq][(c + 3) % T][(c + 3) / T]);
      __syncthreads();
      constexpr int TR = D % (8 * NW) == 0 ? 4 * NW : 16, C = D / TR;   // threads of a row, channels of a thread
      const int rr = threadIdx.x / TR, c0 = threadIdx.x % TR * C;
      const int row = qt * TQ + nq * 16 + rr;
      if (rr < 16 && row < rows) {
        float M = kNegInf;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, sm[w * 16 + rr]);
        float L = 0.0f, low = -kNegInf, acc[C];   // low: the lowest reference that has a sum
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float mw = sm[w * 16 + rr], lw = sl[w * 16 + rr];
          const float f = mw == kNegInf ? 0.0f : exp2_hw(mw - M);
          low = lw == 0.0f ? low : fminf(low, mw);
          L = __builtin_fmaf(f, lw, L);
#pragma unroll
          for (int i = 0; i < C; ++i) acc[i] = __builtin_fmaf(f, so[(w * 16 + rr) * kRow + c0 + i], acc[i]);
        }
        if (low - M < -100.0f) {
          // once more, apart: with move_sum in the loop above short contexts took 0.1 us more
          L = 0.0f;
#pragma unroll 1
          for (int w = 0; w < NW; ++w) L += sum_at(sl[w * 16 + rr], sm[w * 16 + rr], M);
        }
        if (part) {
          float* po = part + (nq * 16 + rr) * D + c0;
#pragma unroll
          for (int i = 0; i < C; ++i) po[i] = acc[i];
          if (c0 == 0) {
            part[TQ * D + nq * 16 + rr] = M;
            part[TQ * D + TQ + nq * 16 + rr] = L;
          }
        } else {
          const int64_t orow = out_row(a, s, h, row);
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          uint32_t* po = (uint32_t*)(a.out + orow * D + c0);
#pragma unroll
          for (int i = 0; i < C; i += 2)
            po[i / 2] = a.bf16 ? pack_result<true>(acc[i] * inv, acc[i + 1] * inv) : pack_result<false>(acc[i] * inv, acc[i + 1] * inv);
          if (a.lse && c0 == 0) a.lse[orow] = Base::lse_of(M, L);
        }
      }
    }
  }

  // Key tiles j0 .. j1 - 1 of the span: as in the 4-bit kernel a wave's units of 32 keys
  // pass through LDS, two at a time, by loads that need no registers.
  __device__ __forceinline__ void keys(const Kv8Attn& a, const Seq& s, const Span& sp, int64_t b, int h, int qt, int j0,
                                       int j1, uint8_t* smem, int wave, int m, int kg) {
    const PageRow row = (PageRow)(a.table + b * a.table_b + h * a.table_h);
    const int ps = a.c.page_shift;
    const uint32_t lane = threadIdx.x & 63;
    int u = (int)tile_start(a, sp, j0);
    const int64_t cut = tile_start(a, sp, j1);
    const int end = cut < sp.hi ? (int)cut : sp.hi;
    if (u < sp.lo) u = sp.lo & ~(kTile - 1);   // only the first tile can hold keys before the span
    u += wave * kUnit;
    if (u + kUnit <= sp.lo) u += kStep;
    rest = NQ == 1 && !a.bf16 && s.n * a.r <= 8;
    this->reset();
    if (u >= end) return;
    uint8_t* const own = smem + wave * (2 * kUnitLds);
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_offset(own));
    struct Pages { int32_t p[2]; };
    // pages of the blocks of a unit, -1 where no row sees keys of one
    auto pages = [&](int u) {
      Pages r = {{-1, -1}};
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int pos = u + 16 * t;
        if (pos < end && pos + 16 > sp.lo) r.p[t] = row[pos >> ps];
      }
      return r;
    };
    // bit t: block t exists; one that does not is read from the first page
    auto fetch = [&](const Pages& pg, int u, int buf) -> int {
      int ok = 0;
      int64_t blk[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int pos = u + 16 * t;
        const int64_t page = pg.p[t];
        const bool is = page >= 0 && page < a.c.n_pages;
        ok |= is ? 1 << t : 0;
        blk[t] = kv8_block(is ? page : 0, a.c.hkv, h, ps, is ? pos & ((1 << ps) - 1) : 0);
        const uint8_t* p = a.c.cache + blk[t] * kSub;
        const uint32_t dst = lds + buf * kUnitLds + t * kSub;
#pragma unroll
        for (int i = 0; i < kSub; i += 1024) ONCE ? dma16_once(p + i, lane * 16u, dst + i) : dma16(p + i, lane * 16u, dst + i);
      }
      if (lane < 4) dma4((const float*)(a.scales + (lane & 2 ? blk[1] : blk[0])) + (lane & 1), lds + buf * kUnitLds + 2 * kSub);
      return ok;
    };
    const Pages first = pages(u);
    Pages next = pages(u + kStep);
    int ok = fetch(first, u, 0), oknext = 0;
    if (u + kStep < end) oknext = fetch(next, u + kStep, 1);
    this->load_q(a, s, h, qt, m, kg);
    for (int buf = 0;; buf ^= 1) {
      const int un = u + kStep;
      next = pages(un + kStep);
      if (un < end)
        wait_dma<kLoads>();
      else
        wait_dma<0>();
      // every row sees every key: all before the first query's position and
      // inside the last one's window
      bool full = ok == 3 && u + kUnit <= s.kv;
      if (a.causal) full = full && u + kUnit - 1 <= sp.p0;
      if (a.window > 0) full = full && u > sp.p1 - a.window;
      const uint8_t* blk = own + buf * kUnitLds;
      const float4 sc = *(const float4*)(blk + 2 * kSub);
      // what stands where no block is counts as 1
      const float sk[2] = {ok & 1 ? sc.x : 1.0f, ok & 2 ? sc.z : 1.0f}, sv[2] = {ok & 1 ? sc.y : 1.0f, ok & 2 ? sc.w : 1.0f};
      float x[NQ][2][4];
      scores(blk, lane, x);
      weights(a, s, qt, u, !full, ok, sk, sv, x, kg);
      values(blk, sv, x, lane);
      this->tile_done();
      if (un >= end) break;
      u = un;
      ok = oknext;
      if (un + kStep < end) {
        wait_lds();
        oknext = fetch(next, un + kStep, buf);
      }
    }
  }
};

template <int D, int NQ, int NW, bool ONCE>
__global__ __launch_bounds__(NW * 64, NW > kWaves ? 2 : kv8_rows_waves(D, NQ)) void kv8_rows_kernel(Kv8Attn a) {
  using R = Rows8<D, NQ, NW, ONCE>;
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

// Eight waves where all workgroups run at once with them and their units fit in LDS: of 8
// sequences' heads 1024 keys 12.7 us, so 14.2, 2048 keys 18.8 : 22.9 (vector instructions of one
// compute unit); 128 keys 7.2 : 6.7.
constexpr int64_t kLds = 160 * 1024;
template <int D, int NQ>
constexpr bool kWide = Rows8<D, NQ, 2 * kWaves, true>::kSmem <= kLds && D * NQ <= 128;

template <int D, int NQ, bool ONCE>
hipError_t launch_rows(const Kv8Attn& a, const Kv8Plan& p, hipStream_t s) {
  const int64_t n = p.split ? a.workers : (int64_t)p.grid_q * a.c.hkv * a.batch;
  if constexpr (kWide<D, NQ>) {
    if (!p.split && n * Rows8<D, NQ, 2 * kWaves, ONCE>::kSmem <= (int64_t)num_cus() * kLds) {
      hipLaunchKernelGGL((kv8_rows_kernel<D, NQ, 2 * kWaves, ONCE>), dim3((unsigned)n), dim3(2 * kWaves * 64), 0, s, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((kv8_rows_kernel<D, NQ, kWaves, ONCE>), dim3((unsigned)n), dim3(kWaves * 64), 0, s, a);
  if (hipError_t e = hipGetLastError()) return e;
  return p.split ? launch_join<D, 16 * NQ, 256 / (D / 4), true>(a, p.tile_rows, s) : hipSuccess;
}

template <int D>
hipError_t launch_rows_d(const Kv8Attn& a, const Kv8Plan& p, hipStream_t s) {
  if (p.once) return p.nq == 1 ? launch_rows<D, 1, true>(a, p, s) : launch_rows<D, 2, true>(a, p, s);
  return p.nq == 1 ? launch_rows<D, 1, false>(a, p, s) : launch_rows<D, 2, false>(a, p, s);
}

}  // namespace kv8

hipError_t launch_kv8_rows(const Kv8Attn& a, const Kv8Plan& p, hipStream_t s) {
  switch (a.c.d) {
    case 64: return kv8::launch_rows_d<64>(a, p, s);
    case 96: return kv8::launch_rows_d<96>(a, p, s);
    case 128: return kv8::launch_rows_d<128>(a, p, s);
    default: return kv8::launch_rows_d<256>(a, p, s);
  }
}

}  // namespace gq
