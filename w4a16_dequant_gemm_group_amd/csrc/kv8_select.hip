// Choosing the pages of the 8-bit cache that a query reads.
//
// The first kernel scores all pages of every (query, key/value head), the second takes
// the best and writes them in order.  A score is a sum of D exact products (16-bit
// factors) in binary64: whatever the order of its terms, it is off by 2^-52 or so, and the
// choice is the one that the formula makes.
// sum_d max(q_d min_d, q_d max_d) = sum_d q_d (q_d > 0 ? max_d : min_d).
#include "kv8.h"
#include "kv8_seq.h"

namespace gq {
namespace {

constexpr int kThreads = 256, kGroupWaves = kThreads / 64;
constexpr int kPasses = 4;      // pages that a lane has under way
constexpr int kLdsKeys = 7168;  // pages whose scores are kept in LDS while they are sorted out

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

// Sum over the lanes of a page (D / 8, for 96 channels 16 of which 4 add zeros), in
// all of them.
template <int P>
__device__ __forceinline__ double page_sum(double v) {
#pragma unroll
  for (int d = 1; d < P; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

template <int D, bool BF16>
__global__ __launch_bounds__(kThreads) void kv8_score_kernel(Kv8Select a, int64_t lists, int chunks) {
  constexpr int P = D == 96 ? 16 : D / 8, R = 64 / P;        // lanes of a page, pages of a wave at once
  constexpr int kPages = kGroupWaves * R * kPasses;          // pages of a workgroup
  extern __shared__ __attribute__((aligned(16))) float sq[];   // [r][D]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane % P, g = lane / P;
  for (int64_t id = blockIdx.x; id < lists * chunks; id += gridDim.x) {
    const int64_t list = id / chunks, t = list / a.hkv;
    const int h = (int)(list - t * a.hkv), p0 = (int)(id - list * chunks) * kPages;
    const Query qu = find_query(a, t, lane);
    // all of few pages are taken, whatever their scores
    if (qu.n <= a.keep || p0 >= qu.n) continue;
    const uint16_t* q = a.q + t * a.q_ts + (int64_t)h * a.r * a.q_hs;
    __syncthreads();
    for (int i = threadIdx.x; i < a.r * (D / 8); i += kThreads) {
      const int head = i / (D / 8), at = i - head * (D / 8);
      const uint4 v = *(const uint4*)(q + head * a.q_hs + 8 * at);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sq[head * D + 8 * at + 2 * k] = wide<BF16>(w[k] & 0xFFFFu);
        sq[head * D + 8 * at + 2 * k + 1] = wide<BF16>(w[k] >> 16);
      }
    }
    __syncthreads();
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
      if (is[i] && c < D / 8) {
        const uint16_t* bd = a.bounds + (page * a.hkv + h) * (2 * D) + 8 * c;
        lo[i] = *(const uint4*)bd;
        hi[i] = *(const uint4*)(bd + D);
      }
    }
    double best[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) best[i] = -__builtin_inf();
    for (int head = 0; head < a.r; ++head) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = c < D / 8 ? sq[head * D + 8 * c + k] : 0.0f;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const uint32_t lw[4] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w}, hw[4] = {hi[i].x, hi[i].y, hi[i].z, hi[i].w};
        double s = 0.0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t w = x[k] > 0.0f ? hw[k / 2] : lw[k / 2];
          s = __builtin_fma((double)x[k], (double)wide<BF16>(k & 1 ? w >> 16 : w & 0xFFFFu), s);
        }
        s = page_sum<P>(s);
        best[i] = s > best[i] ? s : best[i];
      }
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

// Exclusive sum over the workgroup; total: of all.
__device__ __forceinline__ uint64_t group_scan(uint64_t v, uint64_t* smem, uint64_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint64_t s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t u = __shfl_up(s, d);
    if (lane >= d) s += u;
  }
  __syncthreads();
  if (lane == 63) smem[wave] = s;
  __syncthreads();
  uint64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kGroupWaves; ++w) {
    if (w < wave) before += smem[w];
    total += smem[w];
  }
  return before + s - v;
}

// One workgroup per (query, head).  The score that the last page taken has is found
// digit by digit, from the range of the scores down: a histogram of 256 steps, then of
// the step that it falls into, until that step holds as many pages as are still needed,
// or one score alone, of whose pages the earliest are taken.
__global__ __launch_bounds__(kThreads) void kv8_choose_kernel(Kv8Select a, int64_t lists) {
  extern __shared__ __attribute__((aligned(16))) uint64_t keys[];
  __shared__ uint64_t sums[kGroupWaves];
  __shared__ uint32_t bins[256];
  __shared__ uint64_t edge[2];      // smallest and largest key
  __shared__ uint32_t found[3];     // step, pages above it, pages in it
  const int tid = threadIdx.x, lane = tid & 63;
  for (int64_t list = blockIdx.x; list < lists; list += gridDim.x) {
    const int64_t t = list / a.hkv;
    const int h = (int)(list - t * a.hkv);
    const Query qu = find_query(a, t, lane);
    int32_t* out = a.pages + list * a.keep;
    const int32_t* table = a.table + (qu.b < 0 ? 0 : qu.b) * a.table_pages;
    const int taken = qu.n < a.keep ? qu.n : a.keep;
    if (tid == 0 && h == 0) a.lens[t] = taken > 0 ? ((taken - 1) << a.page_shift) + qu.in : 0;
    for (int i = taken + tid; i < a.keep; i += kThreads) out[i] = -1;
    if (qu.n <= a.keep) {
      for (int i = tid; i < taken; i += kThreads) out[i] = table[i];
      continue;
    }
    const int n = qu.n - a.first - a.last;       // candidates, from page `first` on
    uint32_t need = (uint32_t)(a.keep - a.first - a.last);
    const double* score = a.scores + list * a.most + a.first;
    const bool lds = n <= kLdsKeys;
    auto key = [&](int i) { return lds ? keys[i] : key_of(score[i]); };
    __syncthreads();
    if (tid == 0) {
      edge[0] = ~0ull;
      edge[1] = 0;
    }
    uint64_t least = ~0ull, most = 0;
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t k = key_of(score[i]);
      if (lds) keys[i] = k;
      least = k < least ? k : least;
      most = k > most ? k : most;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint64_t u = __shfl_xor(least, d), w = __shfl_xor(most, d);
      least = u < least ? u : least;
      most = w > most ? w : most;
    }
    __syncthreads();
    if (lane == 0) {
      atomicMin((unsigned long long*)&edge[0], (unsigned long long)least);
      atomicMax((unsigned long long*)&edge[1], (unsigned long long)most);
    }
    __syncthreads();
    // pages with lo <= key <= hi: `need` of them are taken, with more than hi: all
    uint64_t lo = edge[0], hi = edge[1];
    int shift = 64 - __builtin_clzll((hi - lo) | 1) - 8;
    shift = shift < 0 ? 0 : shift;
    bool all = need == 0;           // none at all: the step is empty
    if (all) { lo = ~0ull; hi = ~0ull; }
    while (!all) {
      bins[tid] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += kThreads) {
        const uint64_t k = key(i);
        if (k >= lo && k <= hi) atomicAdd(&bins[(uint32_t)((k - lo) >> shift)], 1u);
      }
      __syncthreads();
      const uint32_t mine = bins[255 - tid];
      uint64_t total;
      const uint32_t above = (uint32_t)group_scan(mine, sums, total);
      if (above < need && above + mine >= need) {
        found[0] = 255 - tid;
        found[1] = above;
        found[2] = mine;
      }
      __syncthreads();
      need -= found[1];
      lo += (uint64_t)found[0] << shift;
      const uint64_t top = lo + (((uint64_t)1 << shift) - 1);
      hi = top < hi ? top : hi;
      all = found[2] == need;
      if (shift == 0) break;
      shift = shift < 8 ? 0 : shift - 8;
    }
    // a run of candidates per thread: how many above, how many in the step
    const int run = (n + kThreads - 1) / kThreads, i0 = tid * run, i1 = i0 + run < n ? i0 + run : n;
    uint64_t mine = 0;
    const bool none = a.keep == a.first + a.last;
    if (!none) {
      for (int i = i0; i < i1; ++i) {
        const uint64_t k = key(i);
        mine += (uint64_t)(k > hi) + ((uint64_t)(k >= lo && k <= hi) << 32);
      }
    }
    uint64_t total;
    const uint64_t before = group_scan(mine, sums, total);
    uint32_t in_step = (uint32_t)(before >> 32);
    uint32_t at = (uint32_t)before + (in_step < need ? in_step : need);
    if (!none) {
      for (int i = i0; i < i1; ++i) {
        const uint64_t k = key(i);
        bool take = k > hi;
        if (k >= lo && k <= hi) take = in_step++ < need;
        if (take) out[a.first + at++] = table[a.first + i];
      }
    }
    for (int i = tid; i < a.first; i += kThreads) out[i] = table[i];
    for (int i = tid; i < a.last; i += kThreads) out[a.keep - a.last + i] = table[qu.n - a.last + i];
    __syncthreads();
  }
}

template <int D>
hipError_t score_d(const Kv8Select& a, gq_dtype dt, hipStream_t s) {
  constexpr int P = D == 96 ? 16 : D / 8, kPages = kGroupWaves * (64 / P) * kPasses;
  const int64_t lists = a.q_tokens * a.hkv;
  const int chunks = (int)((a.most + kPages - 1) / kPages);
  const int64_t n = lists * chunks;
  const dim3 grid((unsigned)(n < (1 << 22) ? n : 1 << 22));
  const unsigned lds = (unsigned)(a.r * D * sizeof(float));
  if (dt == GQ_BF16)
    hipLaunchKernelGGL((kv8_score_kernel<D, true>), grid, dim3(kThreads), lds, s, a, lists, chunks);
  else
    hipLaunchKernelGGL((kv8_score_kernel<D, false>), grid, dim3(kThreads), lds, s, a, lists, chunks);
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
  const unsigned lds = a.most > a.keep ? (unsigned)((a.most < kLdsKeys ? a.most : kLdsKeys) * sizeof(uint64_t)) : 0;
  hipLaunchKernelGGL(kv8_choose_kernel, dim3((unsigned)(lists < (1 << 22) ? lists : 1 << 22)), dim3(kThreads), lds, s, a, lists);
  return hipGetLastError();
}

}  // namespace gq
