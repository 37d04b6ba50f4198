// aq_grid.hpp -- the affine grid of one group, shared by the kernels that
// quantize (weights and cache rows): bias = the group minimum rounded down to
// fp16, scale = the smallest fp16 whose grid reaches the group maximum, codes
// = the nearest grid points, ties to the even code.  Every decision is an
// exact comparison (aq_quant.hip states why binary64 holds them exactly).
#pragma once

#include "aq_device.hpp"

namespace aq {

__device__ __forceinline__ double h2d(uint16_t h) { return (double)f16_to_f32(h); }

// next binary16 pattern towards -infinity
__device__ __forceinline__ uint16_t f16_next_down(uint16_t h) {
  if (h == 0) return 0x8001u;
  return (h & 0x8000u) ? (uint16_t)(h + 1) : (uint16_t)(h - 1);
}

// largest binary16 value <= f; -0 is returned as +0
__device__ __forceinline__ uint16_t f16_round_down(float f) {
  uint16_t h = f32_to_f16_rne(f);  // nearest; at most one step above f
  if (f16_to_f32(h) > f) h = f16_next_down(h);
  return h == 0x8000u ? (uint16_t)0 : h;
}

// the same for a binary64 value: rounding to binary32 and then to binary16
// preserves the order against every binary16 value, so the result is again
// the answer or one step above it
__device__ __forceinline__ uint16_t f16_round_down_d(double x) {
  uint16_t h = f32_to_f16_rne((float)x);
  if (h2d(h) > x) h = f16_next_down(h);
  return h == 0x8000u ? (uint16_t)0 : h;
}

// smallest binary16 s >= 0 with b + L*s >= top (exact test in binary64)
__device__ __forceinline__ uint16_t f16_scale_up(double b, double top, int L) {
  if (b >= top) return 0;
  const float t = (float)(top - b) / (float)L;  // candidate, within a step of the answer
  uint16_t s = f32_to_f16_rne(t);
  if (s > 0x7BFFu) s = 0x7BFFu;
#pragma unroll
  for (int it = 0; it < 3; ++it)
    if (s < 0x7BFFu && b + L * h2d(s) < top) ++s;
#pragma unroll
  for (int it = 0; it < 3; ++it)
    if (s > 0 && b + L * h2d((uint16_t)(s - 1)) >= top) --s;
  return s;
}

// nearest grid index, ties to even.  mid(j) = b + (j + 1/2) s separates j, j+1.
// The binary32 estimate t = (w - b) * rcp(s) of the real (w - b) / s has a
// relative error below 2^-22 (one rounding in the subtraction, at most one
// unit in the last place in v_rcp_f32, one in the product), so below 2^-14
// absolutely for t <= 255: when t is farther than 2^-10 from every
// half-integer, rint(t) clamped to [0, L] is already the answer; only the
// rest take the exact binary64 tests.
__device__ __forceinline__ uint32_t nearest_code(float w, double b, double s, float bf, float rs,
                                                 int L) {
  if (s == 0.0) return 0;
  const float t = (w - bf) * rs;
  const float r = __builtin_rintf(t);
  int q = (int)r;  // candidate, within one of the answer (saturating conversion)
  q = q < 0 ? 0 : (q > L ? L : q);
  if (__builtin_fabsf(t - r) <= 0.5f - 0x1p-10f) return (uint32_t)q;
  const double wd = (double)w;
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    if (q > 0) {
      const double mid = b + ((double)q - 0.5) * s;
      if (wd < mid || (wd == mid && (q & 1))) --q;
    }
  }
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    if (q < L) {
      const double mid = b + ((double)q + 0.5) * s;
      if (wd > mid || (wd == mid && (q & 1))) ++q;
    }
  }
  return (uint32_t)q;
}

}  // namespace aq
