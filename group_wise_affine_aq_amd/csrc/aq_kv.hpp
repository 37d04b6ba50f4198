// aq_kv.hpp -- rows of the paged cache: their place, and writing them quantized
// (shared by the kernels that append, and that turn keys as they append).
#pragma once

#include "aq_grid.hpp"
#include "aq_internal.hpp"

namespace aq {
namespace {

// Row number in the cache of (slot, head), row 0 and `there` false outside the
// cache.  Int: uint32_t where the cache's rows can be counted in 31 bits; the
// page is then slot * magic / 2^32, magic = floor(2^32 / page_size) + 1, which
// is at most one too large (slot < 2^32), else int64_t.
template <typename Int>
__device__ __forceinline__ Int cache_row(const KvCache &c, uint32_t magic, int64_t slot, int h,
                                         bool &there) {
  there = slot >= 0 && slot < c.num_pages * c.page_size;
  const Int s = there ? (Int)slot : 0, size = (Int)c.page_size;
  Int page;
  if constexpr (sizeof(Int) == 4) {
    page = __umulhi(s, magic);
    page = page * size > s ? page - 1 : page;
  } else {
    page = s / size;
  }
  const Int row = (page * (Int)c.kv_heads + (Int)h) * size + (s - page * size);
  return there ? row : 0;
}

// lo and hi over the partner lanes; hi keeps a NaN
template <int CTRL>
__device__ __forceinline__ void spread(float &lo, float &hi) {
  lo = __builtin_fminf(lo, dpp_f<CTRL>(lo));
  hi = __builtin_elementwise_maximum(hi, dpp_f<CTRL>(hi));
}

// The group's scale: the least fp16 s >= 0 with b + L s >= top, in binary32.
// top - b is d + e exactly (two-sum; |e| <= ulp(d) / 2).  L s has at most 19
// bits and is exact; near d it is a multiple of ulp(d) away from it and the
// difference is exact, elsewhere its sign is.  So L s >= d + e is L s - d >= e.
__device__ __forceinline__ uint16_t scale_up(float b, float top, float L, float inv_L) {
  const float d = top - b, bb = top - d, e = (top - (d + bb)) + (bb - b);
  uint32_t s = f32_to_f16_rne(d * inv_L);  // the answer or next to it
  if (s > 0x7BFFu) s = 0x7BFFu;
  auto reaches = [&](uint32_t h) { return __builtin_fmaf(L, f16_to_f32((uint16_t)h), -d) >= e; };
  const uint32_t below = s ? s - 1 : 0, above = s < 0x7BFFu ? s + 1 : s;
  s = reaches(below) ? below : (reaches(s) ? s : above);
  return (uint16_t)s;
}

// The code of w exactly: 2 (w - b) against (2 j + 1) s (at most 20 bits),
// w - b = d + e as above, equality for the even code.
__device__ __forceinline__ uint32_t exact_code(float w, float b, float s, float rs, float L) {
  const float d = w - b, bb = w - d, e = (w - (d + bb)) + (bb - b);
  const float j = __builtin_floorf(d * rs);
  const float x = __builtin_fmaf(2.f * j + 1.f, s, -2.f * d) - 2.f * e;  // midpoint - w, doubled
  const bool odd = ((int)j & 1) != 0;
  return (uint32_t)__builtin_fminf(x < 0.f || (x == 0.f && odd) ? j + 1.f : j, L);
}

// The codes of N values of one group, packed.  t = (w - b) * rcp(s) is in
// [0, L] with an error below 2^-22 L (a rounding each in the subtraction and
// the product, a unit in the last place in v_rcp_f32), so unless it is nearer
// than 2^-21 (L + 1) to a half its rounded value is the code: the low bits of
// t + 1.5 * 2^23.  Values that near are mostly exact ties, about one in 2000 of
// 16-bit values, so the exact comparisons are taken four values at a time.
template <int BITS, int N>
__device__ __forceinline__ void pack_codes(const float *w, float b, float s, float rs,
                                           uint32_t *word) {
  constexpr float L = (1 << BITS) - 1, kRound = 12582912.f;
  constexpr int PER = 32 / BITS, PART = 4;
  constexpr uint32_t kBits = 0x4B400000u;  // kRound's
#pragma unroll
  for (int i = 0; i < N / PER; ++i) {
    word[i] = 0;
#pragma unroll
    for (int p = 0; p < PER; p += PART) {
      float far = 0.f;
      uint32_t sum = 0, bias = 0;
#pragma unroll
      for (int j = p; j < p + PART; ++j) {
        const float t = (w[i * PER + j] - b) * rs, r = t + kRound;
        far = __builtin_fmaxf(far, __builtin_fabsf(t - (r - kRound)));
        sum += __builtin_bit_cast(uint32_t, r) << (j * BITS);
        bias += kBits << (j * BITS);
      }
      sum -= bias;
      if (far > 0.5f - 0x1p-21f * (L + 1.f)) {
        sum = 0;
#pragma unroll
        for (int j = p; j < p + PART; ++j) sum |= exact_code(w[i * PER + j], b, s, rs, L) << (j * BITS);
      }
      word[i] += sum;
    }
  }
}

// 32 values of a row, from `o` on, quantized and written: codes, and the scale
// and bias of the group that begins there.  A row's threads are head_dim / 32
// neighbouring lanes; all lanes of a wave call this together.
template <int BITS, typename Int>
__device__ __forceinline__ void write_row_part(const KvCache &c, uint32_t magic, int64_t slot, int h,
                                               bool is_v, bool active, int o, float *w) {
  constexpr int E = 32;
  const int D = c.head_dim;
  // (maximum keeps a NaN, the minimum of the others stands beside it)
  float lo = w[0], hi = w[0];
#pragma unroll
  for (int i = 1; i < E; ++i) {
    lo = __builtin_fminf(lo, w[i]);
    hi = __builtin_elementwise_maximum(hi, w[i]);
  }
  if (!(lo >= -65504.f && hi <= 65504.f)) {  // rare: past fp16's range, or NaN
#pragma unroll
    for (int i = 0; i < E; ++i) w[i] = __builtin_amdgcn_fmed3f(w[i], -65504.f, 65504.f);
    lo = __builtin_amdgcn_fmed3f(lo, -65504.f, 65504.f);
    if (hi == hi) hi = __builtin_amdgcn_fmed3f(hi, -65504.f, 65504.f);
  }
  // a group is 1, 2 or 4 lanes of a quad
  if (c.group_size >= 64) spread<0xB1>(lo, hi);
  if (c.group_size >= 128) spread<0x4E>(lo, hi);
  const bool nan = hi != hi;
  constexpr float L = (1 << BITS) - 1;
  uint16_t b16 = f16_round_down(lo);
  const float b = f16_to_f32(b16);
  uint16_t s16 = nan || b >= hi ? 0 : scale_up(b, hi, L, 1.f / L);
  const float s = f16_to_f32(s16);
  const float rs = s16 ? __builtin_amdgcn_rcpf(s) : 0.f;
  uint32_t word[E * BITS / 32];
  pack_codes<BITS, E>(w, b, s, rs, word);
  if (s16 == 0)
#pragma unroll
    for (int i = 0; i < E * BITS / 32; ++i) word[i] = 0;
  if (nan) b16 = 0x7E00u;
  bool there;
  const int64_t at = cache_row<Int>(c, magic, slot, h, there);
  if (!active || !there) return;
  uint32_t *dst = reinterpret_cast<uint32_t *>(is_v ? c.v_codes : c.k_codes) + at * (D * BITS / 32) + o * BITS / 32;
#pragma unroll
  for (int i = 0; i < E * BITS / 32; i += 4)
    *reinterpret_cast<uint4 *>(dst + i) = make_uint4(word[i], word[i + 1], word[i + 2], word[i + 3]);
  if ((o & (c.group_size - 1)) == 0) {
    const int64_t gi = at * (D / c.group_size) + o / c.group_size;
    (is_v ? c.v_scales : c.k_scales)[gi] = s16;
    (is_v ? c.v_biases : c.k_biases)[gi] = b16;
  }
}

inline bool narrow(const KvCache &c) {
  return c.num_pages * c.page_size <= 0x7FFFFFFF / c.kv_heads;
}
inline uint32_t magic_of(const KvCache &c) { return (uint32_t)(0x100000000ull / (uint32_t)c.page_size) + 1; }

}  // namespace
}  // namespace aq
