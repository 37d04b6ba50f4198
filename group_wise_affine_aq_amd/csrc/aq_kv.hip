// aq_kv.hip -- writing keys and values into the paged cache, quantized as they
// are written, and reading rows of it back (gfx950).
//
// A cache row is one token's head_dim values in one head, K or V, in the
// weight format: groups of G along the row, each with the bias, scale and
// codes that aq_grid.hpp defines (the cache row of a token is bit for bit what
// the weight quantizer makes of it).  Values are clamped to fp16's finite
// range before that, since bias and scale are fp16, and a group that holds a
// NaN is stored as scale 0, bias NaN: NaN reaches the reader, and the integer
// codes stay finite.
//
// Both kernels move bytes and are bound by HBM at prompt size and by launch
// latency at decode size: append reads 2 bytes a value and writes bits/8 +
// 4/G, read does the reverse.  A workgroup takes consecutive tokens of one
// head: consecutive tokens mostly lie in consecutive places, so its cache side
// is one run of whole lines, scales too, and its other side rows of head_dim
// 16-bit values, whole lines as well.  (Taken in the order of the 16-bit rows,
// all heads of a token, every line of codes was fetched by two XCDs and every
// line of scales by four: 112 us for 65536 tokens of 8 heads of 128, 4 bits to
// bf16, against 78.)  Row addresses are 64-bit, a cache is larger than
// 4 GiB; row numbers are in 32 bits where they fit, which spares 64-bit
// divisions and products of every row.
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

// E values per thread: a row's threads are D/E lanes (1 << shift), a group's G/E
template <int XDT, int BITS, typename Int>
__global__ __launch_bounds__(256) void kv_append_kernel(KvCache c, int64_t T, int shift,
                                                        uint32_t magic,
                                                        const void *__restrict__ k,
                                                        const void *__restrict__ v,
                                                        int64_t k_stride, int64_t v_stride,
                                                        const int64_t *__restrict__ slots) {
  constexpr int E = BITS == 16 ? 8 : 32;
  const int D = c.head_dim, h = blockIdx.x % (unsigned)c.kv_heads;
  int64_t t = (int64_t)(blockIdx.x / (unsigned)c.kv_heads) * (256 >> shift) + (threadIdx.x >> shift);
  const bool active = t < T;
  if (!active) t = T - 1;  // whole rows are inactive together; keep loads in bounds
  const int o = ((int)threadIdx.x & ((1 << shift) - 1)) * E;
  const bool is_v = blockIdx.y != 0;
  const int64_t e = t * (is_v ? v_stride : k_stride) + (int64_t)h * D + o;
  const void *x = is_v ? v : k;
  void *codes = is_v ? c.v_codes : c.k_codes;
  const int64_t slot = slots[t];

  if constexpr (BITS == 16) {
    const uint4 w = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(x) + e);
    bool there;
    const int64_t at = cache_row<Int>(c, magic, slot, h, there);
    if (!active || !there) return;
    *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(codes) + at * D + o) = w;
  } else {
    float w[E];
    load32<XDT>(x, e, w);
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
    uint32_t *dst = reinterpret_cast<uint32_t *>(codes) + at * (D * BITS / 32) + o * BITS / 32;
#pragma unroll
    for (int i = 0; i < E * BITS / 32; i += 4)
      *reinterpret_cast<uint4 *>(dst + i) = make_uint4(word[i], word[i + 1], word[i + 2], word[i + 3]);
    if ((o & (c.group_size - 1)) == 0) {
      const int64_t gi = at * (D / c.group_size) + o / c.group_size;
      (is_v ? c.v_scales : c.k_scales)[gi] = s16;
      (is_v ? c.v_biases : c.k_biases)[gi] = b16;
    }
  }
}

// 8 values per thread and row, so that a wave stores whole kilobytes; U rows
// per thread, all their loads ahead of the first store
// STREAM: the rows go past the caches
template <int BITS, int ODT, bool STREAM, typename Int>
__global__ __launch_bounds__(256) void kv_read_kernel(KvCache c, int64_t T, int shift,
                                                      uint32_t magic,
                                                      const int64_t *__restrict__ slots,
                                                      void *__restrict__ k, void *__restrict__ v) {
  constexpr int U = 4, W = BITS == 16 ? 4 : BITS / 4;
  const int D = c.head_dim, h = blockIdx.x % (unsigned)c.kv_heads, step = 256 >> shift;
  const int64_t t0 = (int64_t)(blockIdx.x / (unsigned)c.kv_heads) * (U * step) + (threadIdx.x >> shift);
  const bool is_v = blockIdx.y != 0;
  const uint32_t *codes = reinterpret_cast<const uint32_t *>(is_v ? c.v_codes : c.k_codes);
  const uint16_t *scales = is_v ? c.v_scales : c.k_scales, *biases = is_v ? c.v_biases : c.k_biases;
  const int o = ((int)threadIdx.x & ((1 << shift) - 1)) * 8;
  // rows outside the cache read its first row: no branch between the loads
  int64_t slot[U], at[U];
  bool there[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = t0 + u * step;
    slot[u] = slots[t < T ? t : T - 1];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) at[u] = cache_row<Int>(c, magic, slot[u], h, there[u]);
  uint32_t word[U][W];
  uint16_t s16[U], b16[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t *src = codes + (at[u] * D + o) * BITS / 32;
    if constexpr (W == 4) {
      const uint4 x = *reinterpret_cast<const uint4 *>(src);
      word[u][0] = x.x, word[u][1] = x.y, word[u][2] = x.z, word[u][3] = x.w;
    } else if constexpr (W == 2) {
      const uint2 x = *reinterpret_cast<const uint2 *>(src);
      word[u][0] = x.x, word[u][1] = x.y;
    } else {
      word[u][0] = *src;
    }
    s16[u] = b16[u] = 0;
    if constexpr (BITS != 16) {
      const int64_t gi = at[u] * (D / c.group_size) + o / c.group_size;
      s16[u] = scales[gi];
      b16[u] = (biases ? biases : scales)[gi];
    }
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = t0 + u * step;
    if (t >= T) return;
    float w[8];
    if constexpr (BITS == 16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint16_t x = (uint16_t)(word[u][i >> 1] >> (16 * (i & 1)));
        w[i] = c.dtype == X_F16 ? f16_to_f32(x) : bf16_to_f32(x);
      }
    } else {
      const float s = f16_to_f32(s16[u]), b = biases ? f16_to_f32(b16[u]) : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = __builtin_fmaf((float)((word[u][i * BITS / 32] >> (i * BITS % 32)) & ((1 << BITS) - 1)), s, b);
    }
    if (!there[u])
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 0.f;
    store8<ODT, STREAM>(is_v ? v : k, (t * c.kv_heads + h) * D + o, w);
  }
}

bool narrow(const KvCache &c) {
  return c.num_pages * c.page_size <= 0x7FFFFFFF / c.kv_heads;
}
uint32_t magic_of(const KvCache &c) { return (uint32_t)(0x100000000ull / (uint32_t)c.page_size) + 1; }

// workgroups of `tokens` tokens of one head
dim3 grid_of(const KvCache &c, int64_t T, int tokens) {
  return dim3((unsigned)((T + tokens - 1) / tokens * c.kv_heads), 2);
}

template <typename Int>
hipError_t append(const void *k, const void *v, int x_dtype, int64_t T, int64_t k_stride,
                  int64_t v_stride, const int64_t *slots, const KvCache &c, hipStream_t s) {
  const int shift = __builtin_ctz((unsigned)(c.head_dim / (c.bits == 16 ? 8 : 32)));
  const dim3 grid = grid_of(c, T, 256 >> shift), block(256);
#define AQ_A(X, B) hipLaunchKernelGGL((kv_append_kernel<X, B, Int>), grid, block, 0, s, c, T, shift, magic_of(c), k, v, k_stride, v_stride, slots)
  if (c.bits == 16) AQ_A(X_F16, 16);
  else if (c.bits == 8 && x_dtype == X_F16) AQ_A(X_F16, 8);
  else if (c.bits == 8) AQ_A(X_BF16, 8);
  else if (x_dtype == X_F16) AQ_A(X_F16, 4);
  else AQ_A(X_BF16, 4);
#undef AQ_A
  return hipGetLastError();
}

template <typename Int>
hipError_t read(const int64_t *slots, int64_t T, const KvCache &c, void *k, void *v, int out_dtype,
                hipStream_t s) {
  const int shift = __builtin_ctz((unsigned)(c.head_dim / 8));
  const dim3 grid = grid_of(c, T, 4 * (256 >> shift)), block(256);
  // Rows that the chip's caches could not hold until they are used go past
  // them, from half the last cache's 256 MB on (4 bits to bf16: 268 MB of rows
  // 54 against 75 us, with a torch sum of both after it 132 against 139; at
  // 34 MB 8.4 against 10.5 us, but with the sum 23.9 against 23.0).
  const int64_t bytes = 2 * T * c.kv_heads * c.head_dim * (out_dtype == X_F32 ? 4 : 2);
  const bool stream = bytes > (128 << 20);
#define AQ_R(B, O)                                                                           \
  do {                                                                                       \
    if (stream)                                                                              \
      hipLaunchKernelGGL((kv_read_kernel<B, O, true, Int>), grid, block, 0, s, c, T, shift,  \
                         magic_of(c), slots, k, v);                                          \
    else                                                                                     \
      hipLaunchKernelGGL((kv_read_kernel<B, O, false, Int>), grid, block, 0, s, c, T, shift, \
                         magic_of(c), slots, k, v);                                          \
  } while (0)
#define AQ_RB(B)                                  \
  if (out_dtype == X_F32) AQ_R(B, X_F32);         \
  else if (out_dtype == X_F16) AQ_R(B, X_F16);    \
  else AQ_R(B, X_BF16);
  if (c.bits == 16) { AQ_RB(16) } else if (c.bits == 8) { AQ_RB(8) } else { AQ_RB(4) }
#undef AQ_RB
#undef AQ_R
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const void *k, const void *v, int x_dtype, int64_t T, int64_t k_stride,
                            int64_t v_stride, const int64_t *slots, const KvCache &c,
                            hipStream_t s) {
  return narrow(c) ? append<uint32_t>(k, v, x_dtype, T, k_stride, v_stride, slots, c, s)
                      : append<int64_t>(k, v, x_dtype, T, k_stride, v_stride, slots, c, s);
}

hipError_t launch_kv_read(const int64_t *slots, int64_t T, const KvCache &c, void *k, void *v,
                          int out_dtype, hipStream_t s) {
  return narrow(c) ? read<uint32_t>(slots, T, c, k, v, out_dtype, s)
                      : read<int64_t>(slots, T, c, k, v, out_dtype, s);
}

}  // namespace aq
