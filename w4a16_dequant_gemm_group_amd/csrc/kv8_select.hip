// Choosing the pages of the 8-bit cache that a query reads.
//
// The first kernel scores all pages of every (query, key/value head), the second takes
// the best and writes them in order.  A score is a sum of D exact products (16-bit
// factors) in binary64: whatever the order of its terms, it is off by 2^-52 or so, and the
// choice is the one that the formula makes.
// sum_d max(q_d min_d, q_d max_d) = sum_d q_d (q_d > 0 ? max_d : min_d).
// Bound by latency: 2048 pages of 8 heads of 128 are scored in 6.6 us (8.4 MB) and chosen in 5.9;
// 40 queries over 16 sequences of up to 1000 pages, 4 heads of 64, in 12.7 (vector work, 60 %
// busy) and 5.8.
#include "kv8.h"
#include "kv8_seq.h"

namespace gq {
namespace {

constexpr int kThreads = 256, kGroupWaves = kThreads / 64;
constexpr int kPasses = 4;      // pages that a lane has under way

template <bool BF16>
__device__ __forceinline__ float wide(uint32_t h) {
  return BF16 ? __uint_as_float(h << 16) : f16_to_f32((uint16_t)h);
}

// The pages of a query: 0 .. n - 1 of its row, the last of them up to `in` keys.
struct Query {
  int b;      // sequence; < 0: none
  int n, in;
};

__device__ __forceinline__ Query find_query(const Kv8Select& a, int64_t t, int lane) {
  Query q{-1, 0, 0};
  const RowSeq s = seq_of_row(a.q_starts, a.kv_lens, a.batch, a.q_tokens, t, lane);
  if (s.b < 0) return q;
  const int64_t cap = a.most << a.page_shift;
  int64_t kv = s.kv;
  kv = kv > cap ? cap : kv;
  const int64_t p = kv - s.n + (t - s.first);
  if (p < 0) return q;
  q.b = s.b;
  q.n = (int)(p >> a.page_shift) + 1;
  q.in = (int)(p & ((1 << a.page_shift) - 1)) + 1;
  return q;
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (uint32_t)b, CTRL, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sum over the P lanes of a page (D / 8, for 96 channels 16 of which 4 add zeros), in
// all of them.
template <int P>
__device__ __forceinline__ double page_sum(double v) {
  v += dpp_f64<0xB1>(v);      // quad_perm [1,0,3,2]
  v += dpp_f64<0x4E>(v);      // quad_perm [2,3,0,1]
  v += dpp_f64<0x141>(v);     // row_half_mirror: 8 lanes
  if constexpr (P > 8) v += dpp_f64<0x140>(v);   // row_mirror: 16 lanes
  if constexpr (P > 16) v += __shfl_xor(v, 16);
  return v;
}

// Eight channels of a query row, as they lie and widened.
template <bool BF16>
__device__ __forceinline__ void widen8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = wide<BF16>(w[k] & 0xFFFFu);
    x[2 * k + 1] = wide<BF16>(w[k] >> 16);
  }
}

// A wave scores kPasses x R pages: P lanes hold 8 channels each of a page's bounds and
// of the query heads, which are taken one after another.
template <int D, bool BF16>
__global__ __launch_bounds__(kThreads) void kv8_score_kernel(Kv8Select a, int64_t lists, int chunks) {
  constexpr int P = D == 96 ? 16 : D / 8, R = 64 / P;        // lanes of a page, pages of a wave at once
  constexpr int kPages = kGroupWaves * R * kPasses;          // pages of a workgroup
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane % P, g = lane / P;
  const bool live = c < D / 8;
  for (int64_t id = blockIdx.x; id < lists * chunks; id += gridDim.x) {
    // the first pages of all lists, then the next ones: workgroups that find no pages (in
    // lists shorter than the longest) come last, and those that do spread evenly
    const int64_t chunk = id / lists, list = id - chunk * lists, t = list / a.hkv;
    const int h = (int)(list - t * a.hkv), p0 = (int)chunk * kPages;
    // the first head's channels are on their way while the sequence is looked up
    const uint16_t* q = a.q + t * a.q_ts + (int64_t)h * a.r * a.q_hs + 8 * c;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (live) raw = *(const uint4*)q;
    const Query qu = find_query(a, t, lane);
    // all of few pages are taken, whatever their scores
    if (qu.n <= a.keep || p0 + wave * R >= qu.n) continue;
    const int32_t* table = a.table + qu.b * a.table_pages;
    int at[kPasses];
    bool is[kPasses];
    uint4 lo[kPasses], hi[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      at[i] = p0 + (i * kGroupWaves + wave) * R + g;
      const int64_t page = at[i] < qu.n ? table[at[i]] : -1;
      is[i] = page >= 0 && page < a.n_pages;
      lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
      if (is[i] && live) {
        const uint16_t* bd = a.bounds + (page * a.hkv + h) * (2 * D) + 8 * c;
        lo[i] = *(const uint4*)bd;
        hi[i] = *(const uint4*)(bd + D);
      }
    }
    double best[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) best[i] = -__builtin_inf();
    for (int head = 0;;) {
      float x[8];
      widen8<BF16>(raw, x);
      // where a channel is negative, in pairs: there the smallest counts
      typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
      uint32_t neg[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) neg[k] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(i16x2, neg[k]) >> 15);
      if (++head < a.r && live) raw = *(const uint4*)(q + head * a.q_hs);
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const uint32_t lw[4] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w}, hw[4] = {hi[i].x, hi[i].y, hi[i].z, hi[i].w};
        double s = 0.0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t w = (lw[k / 2] & neg[k / 2]) | (hw[k / 2] & ~neg[k / 2]);
          s = __builtin_fma((double)x[k], (double)wide<BF16>(k & 1 ? w >> 16 : w & 0xFFFFu), s);
        }
        s = page_sum<P>(s);
        best[i] = fmax(best[i], s);   // of a sum that is NaN the other
      }
      if (head >= a.r) break;
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      if (c == 0 && at[i] < qu.n) a.scores[list * a.most + at[i]] = is[i] ? best[i] + 0.0 : -__builtin_inf();
  }
}

// Scores as integers of the same order.
__device__ __forceinline__ uint64_t key_of(double s) {
  const uint64_t b = __builtin_bit_cast(uint64_t, s);
  return b >> 63 ? ~b : b | 1ull << 63;
}

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t dpp_or_0(uint32_t v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
// Sums over the lanes up to this one.
__device__ __forceinline__ uint32_t wave_sums(uint32_t v) {
  v += dpp_or_0<0x111>(v);        // row_shr 1, 2, 4, 8
  v += dpp_or_0<0x112>(v);
  v += dpp_or_0<0x114>(v);
  v += dpp_or_0<0x118>(v);
  v += dpp_or_0<0x142, 0xA>(v);   // row_bcast 15, 31
  return v + dpp_or_0<0x143, 0xC>(v);
}
// Smallest over a row of 16 lanes, in every lane, and over the wave, as a scalar.
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  v = min(v, dpp_or_0<0xB1>(v));
  v = min(v, dpp_or_0<0x4E>(v));
  v = min(v, dpp_or_0<0x141>(v));
  return min(v, dpp_or_0<0x140>(v));
}
__device__ __forceinline__ uint32_t wave_min(uint32_t v) {
  v = row_min(v);
  const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
  const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
  return min(min(a, b), min(c, d));
}
// Sum over a row of 16 lanes, in every lane.
__device__ __forceinline__ uint32_t row_sum(uint32_t v) {
  v += dpp_or_0<0xB1>(v);
  v += dpp_or_0<0x4E>(v);
  v += dpp_or_0<0x141>(v);
  return v + dpp_or_0<0x140>(v);
}

constexpr int kSort = 1024, kSortWaves = kSort / 64;   // threads of a workgroup that chooses
constexpr int kHeld = 8;                               // scores that a thread keeps in registers

// One workgroup per (query, head).  The score that the last page taken has is found
// digit by digit, from the range of the scores down (of the upper halves of their bits: both
// reductions in 64 bits took 0.8 us more): a histogram of 256 steps, then of the step that it
// falls into, until that step holds as many pages as are still needed, or one score alone, of
// whose pages the earliest are taken.  A thread has a run of pages; HELD: their scores and
// numbers stay in registers, else they are read again each time.
template <bool HELD>
__global__ __launch_bounds__(kSort) void kv8_choose_kernel(Kv8Select a, int64_t lists) {
  __shared__ __attribute__((aligned(16))) uint32_t bins[2][256];
  __shared__ uint32_t edge[2][kSortWaves];          // upper half of the smallest key, and complement of that of the largest
  __shared__ uint32_t sums[2][kSortWaves];
  __shared__ uint32_t found[3];                     // step, pages above it, pages in it
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int64_t list = blockIdx.x; list < lists; list += gridDim.x) {
    const int64_t t = list / a.hkv;
    const int h = (int)(list - t * a.hkv);
    const Query qu = find_query(a, t, lane);
    int32_t* out = a.pages + list * a.keep;
    const int32_t* table = a.table + (qu.b < 0 ? 0 : qu.b) * a.table_pages;
    const int taken = qu.n < a.keep ? qu.n : a.keep;
    if (tid == 0 && h == 0) a.lens[t] = taken > 0 ? ((taken - 1) << a.page_shift) + qu.in : 0;
    for (int i = taken + tid; i < a.keep; i += kSort) out[i] = -1;
    if (qu.n <= a.keep) {
      for (int i = tid; i < taken; i += kSort) out[i] = table[i];
      continue;
    }
    for (int i = tid; i < a.first; i += kSort) out[i] = table[i];
    for (int i = tid; i < a.last; i += kSort) out[a.keep - a.last + i] = table[qu.n - a.last + i];
    const int n = qu.n - a.first - a.last;       // candidates, from page `first` on
    uint32_t need = (uint32_t)(a.keep - a.first - a.last);
    if (need == 0) continue;
    const double* score = a.scores + list * a.most + a.first;
    const int run = (n + kSort - 1) / kSort, i0 = tid * run;
    const int mine = i0 >= n ? 0 : (i0 + run < n ? run : n - i0);
    uint64_t held[kHeld];
    int entry[kHeld];
    if constexpr (HELD) {
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        held[j] = j < mine ? key_of(score[i0 + j]) : 0;
        entry[j] = j < mine ? table[a.first + i0 + j] : 0;
      }
    }
    auto each = [&](auto&& f) {
      if constexpr (HELD) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
          if (j < mine) f(j, held[j]);
      } else {
        for (int j = 0; j < mine; ++j) f(j, key_of(score[i0 + j]));
      }
    };
    uint32_t least = ~0u, most = ~0u;            // of the complements
    each([&](int, uint64_t k) {
      least = min(least, (uint32_t)(k >> 32));
      most = min(most, ~(uint32_t)(k >> 32));
    });
    least = wave_min(least);
    most = wave_min(most);
    __syncthreads();                             // the list before is done with what is shared
    if (lane == 0) {
      edge[0][wave] = least;
      edge[1][wave] = most;
    }
    if (tid < 256) bins[0][tid] = 0;
    __syncthreads();
    static_assert(kSortWaves == 16, "a lane of a row per wave");
    least = row_min(edge[0][lane & 15]);
    most = row_min(edge[1][lane & 15]);
    // pages with lo <= key <= hi: `need` of them are taken, with more than hi: all
    uint64_t lo = (uint64_t)least << 32, hi = (uint64_t)~most << 32 | ~0u;
    int shift = 64 - __builtin_clzll((hi - lo) | 1) - 8;
    shift = shift < 0 ? 0 : shift;
    for (int b = 0;; b ^= 1) {
      each([&](int, uint64_t k) {
        if (k >= lo && k <= hi) atomicAdd(&bins[b][(uint32_t)((k - lo) >> shift)], 1u);
      });
      __syncthreads();
      if (wave == 0) {
        // lane l: steps 255 - 4 l down to 252 - 4 l
        const uint4 v = *(const uint4*)&bins[b][252 - 4 * lane];
        const uint32_t c[4] = {v.w, v.z, v.y, v.x};
        const uint32_t own = v.x + v.y + v.z + v.w;
        uint32_t above = wave_sums(own) - own;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (above < need && above + c[i] >= need) {
            found[0] = 255 - 4 * lane - i;
            found[1] = above;
            found[2] = c[i];
          }
          above += c[i];
        }
      } else if (tid < 320) {
        bins[b ^ 1][tid - 64] = 0;
      }
      __syncthreads();
      need -= found[1];
      lo += (uint64_t)found[0] << shift;
      const uint64_t rest = ((uint64_t)1 << shift) - 1;
      hi = hi - lo < rest ? hi : lo + rest;      // lo + rest may be beyond 64 bits: +infinity lies near their end
      if (found[2] == need || shift == 0) break;
      shift = shift < 8 ? 0 : shift - 8;
    }
    // how many of the thread's pages lie above, how many in the step
    uint32_t above = 0, step = 0;
    each([&](int, uint64_t k) {
      above += k > hi;
      step += (k >= lo) & (k <= hi);
    });
    uint32_t u = wave_sums(above), v = wave_sums(step);
    if (lane == 63) {
      sums[0][wave] = u;
      sums[1][wave] = v;
    }
    __syncthreads();
    const bool before = (lane & 15) < wave;
    u += row_sum(before ? sums[0][lane & 15] : 0u) - above;
    v += row_sum(before ? sums[1][lane & 15] : 0u) - step;
    uint32_t at = a.first + u + (v < need ? v : need);
    each([&](int j, uint64_t k) {
      bool take = k > hi;
      if ((k >= lo) & (k <= hi)) take = v++ < need;
      if (take) out[at++] = HELD ? entry[j] : table[a.first + i0 + j];
    });
  }
}

template <int D>
hipError_t score_d(const Kv8Select& a, gq_dtype dt, hipStream_t s) {
  constexpr int P = D == 96 ? 16 : D / 8, kPages = kGroupWaves * (64 / P) * kPasses;
  const int64_t lists = a.q_tokens * a.hkv;
  const int chunks = (int)((a.most + kPages - 1) / kPages);
  const int64_t n = lists * chunks;
  const dim3 grid((unsigned)(n < (1 << 22) ? n : 1 << 22));
  if (dt == GQ_BF16)
    hipLaunchKernelGGL((kv8_score_kernel<D, true>), grid, dim3(kThreads), 0, s, a, lists, chunks);
  else
    hipLaunchKernelGGL((kv8_score_kernel<D, false>), grid, dim3(kThreads), 0, s, a, lists, chunks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv8_select(const Kv8Select& a, gq_dtype dt, hipStream_t s) {
  if (a.most > a.keep) {
    hipError_t e;
    switch (a.d) {
      case 64: e = score_d<64>(a, dt, s); break;
      case 96: e = score_d<96>(a, dt, s); break;
      case 128: e = score_d<128>(a, dt, s); break;
      default: e = score_d<256>(a, dt, s); break;
    }
    if (e) return e;
  }
  const int64_t lists = a.q_tokens * a.hkv;
  const dim3 grid((unsigned)(lists < (1 << 21) ? lists : 1 << 21));   // fewer than 2^32 threads
  if (a.most <= kSort * kHeld)
    hipLaunchKernelGGL(kv8_choose_kernel<true>, grid, dim3(kSort), 0, s, a, lists);
  else
    hipLaunchKernelGGL(kv8_choose_kernel<false>, grid, dim3(kSort), 0, s, a, lists);
  return hipGetLastError();
}

}  // namespace gq
