// C ABI of the rotary positions (gq_rope.h): argument validation, which runs on the
// host before any HIP call, and the frequencies.
#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "rope.h"

using namespace gq;

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 40;

bool bad_stride(int64_t s) { return s < -kMaxStride || s > kMaxStride; }

// Whether rows of d elements, `tokens` x `heads` of them at these strides, overlap.  The stride of
// a dimension of one element is never walked.
bool rows_overlap(int64_t tokens, int64_t heads, int64_t token_stride, int64_t head_stride, int64_t d) {
  const int64_t t = std::llabs(token_stride), h = std::llabs(head_stride);
  if ((tokens > 1 && t < d) || (heads > 1 && h < d)) return true;
  if (tokens < 2 || heads < 2) return false;
  // one dimension inside a step of the other: nearly every layout
  if ((heads - 1) * h + d <= t || (h - d) / t >= tokens - 1) return false;
  // else rows i tokens and j heads apart (in either direction): for each j the nearest i
  for (int64_t j = 1; j < heads; ++j) {
    const int64_t x = j * h;
    for (int64_t i = x / t; i <= x / t + 1; ++i)
      if (i >= 1 && i < tokens && std::llabs(x - i * t) < d) return true;
  }
  return false;
}

gq_status check_scaling(const gq_rope_scaling& s) {
  if (s.kind < GQ_ROPE_NONE || s.kind > GQ_ROPE_YARN) return GQ_ERR_INVALID_ARG;
  if (s.kind == GQ_ROPE_NONE) return GQ_OK;
  if (!(s.factor >= 1.0) || !std::isfinite(s.factor)) return GQ_ERR_INVALID_ARG;
  if (s.kind == GQ_ROPE_LINEAR) return GQ_OK;
  if (!(s.original_length > 0.0) || !std::isfinite(s.original_length)) return GQ_ERR_INVALID_ARG;
  if (!(s.low > 0.0) || !(s.high > s.low) || !std::isfinite(s.high)) return GQ_ERR_INVALID_ARG;
  return GQ_OK;
}

double unit(double t) { return t < 0.0 ? 0.0 : (t > 1.0 ? 1.0 : t); }

}  // namespace

extern "C" {

gq_status gq_rope_frequencies(int64_t rot_dim, double base, gq_rope_scaling s, double* freqs,
                              double* amplitude) {
  if (rot_dim < 2 || rot_dim > 1024 || rot_dim % 2 != 0) return GQ_ERR_INVALID_ARG;
  if (!(base > 1.0) || !std::isfinite(base) || !freqs || !amplitude) return GQ_ERR_INVALID_ARG;
  if (gq_status st = check_scaling(s)) return st;
  constexpr double kTurn = 6.28318530717958647693;
  const double rot = (double)rot_dim;
  *amplitude = 1.0;
  double lo = 0.0, hi = 1.0;
  if (s.kind == GQ_ROPE_YARN) {
    auto index = [&](double n) {
      return rot * std::log(s.original_length / (kTurn * n)) / (2.0 * std::log(base));
    };
    lo = std::max(0.0, std::min(std::floor(index(s.high)), rot - 1.0));
    hi = std::max(lo + 0.001, std::min(std::ceil(index(s.low)), rot - 1.0));
    *amplitude = 0.1 * std::log(s.factor) + 1.0;
  }
  for (int64_t i = 0; i < rot_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * (double)i / rot);
    double t = 1.0;   // share of f, the rest of f / s
    if (s.kind == GQ_ROPE_LINEAR) t = 0.0;
    if (s.kind == GQ_ROPE_WAVELENGTH) t = unit((s.original_length * f / kTurn - s.low) / (s.high - s.low));
    if (s.kind == GQ_ROPE_YARN) t = 1.0 - unit(((double)i - lo) / (hi - lo));
    freqs[i] = s.kind == GQ_ROPE_NONE ? f : (1.0 - t) * (f / s.factor) + t * f;
  }
  return GQ_OK;
}

gq_status gq_rope(const gq_rope_args* args, void* stream) {
  if (!args) return GQ_ERR_INVALID_ARG;
  const gq_rope_args& a = *args;
  if (a.dtype != GQ_BF16 && a.dtype != GQ_F16 && a.dtype != GQ_F32) return GQ_ERR_INVALID_ARG;
  if (a.tokens < 0 || a.tokens > ((int64_t)1 << 30) || a.heads < 0 || a.heads > 65536) return GQ_ERR_INVALID_ARG;
  if (a.head_dim < 2 || a.head_dim > 1024 || a.head_dim % 2 != 0) return GQ_ERR_INVALID_ARG;
  if (a.rot_dim < 2 || a.rot_dim > a.head_dim || a.rot_dim % 2 != 0) return GQ_ERR_INVALID_ARG;
  if (!std::isfinite(a.amplitude)) return GQ_ERR_INVALID_ARG;
  if ((a.interleaved != 0 && a.interleaved != 1) || (a.inverse != 0 && a.inverse != 1)) return GQ_ERR_INVALID_ARG;
  if (bad_stride(a.x_token_stride) || bad_stride(a.x_head_stride) || bad_stride(a.out_token_stride) ||
      bad_stride(a.out_head_stride))
    return GQ_ERR_INVALID_ARG;
  if (a.tokens == 0 || a.heads == 0) return GQ_OK;
  if (!a.x || !a.out || !a.positions || !a.freqs) return GQ_ERR_INVALID_ARG;
  if (rows_overlap(a.tokens, a.heads, a.out_token_stride, a.out_head_stride, a.head_dim)) return GQ_ERR_INVALID_ARG;
  if (a.x == a.out && ((a.tokens > 1 && a.x_token_stride != a.out_token_stride) ||
                       (a.heads > 1 && a.x_head_stride != a.out_head_stride)))
    return GQ_ERR_INVALID_ARG;
  const uintptr_t elem = a.dtype == GQ_F32 ? 3u : 1u;
  if (((uintptr_t)a.x & elem) || ((uintptr_t)a.out & elem) || ((uintptr_t)a.positions & 7u) || ((uintptr_t)a.freqs & 7u))
    return GQ_ERR_MISALIGNED;
  hipStream_t s = (hipStream_t)stream;
  if (gq_status st = check_device(s)) return st;
  return launch_rope(a, s) == hipSuccess ? GQ_OK : GQ_ERR_HIP;
}

}  // extern "C"
