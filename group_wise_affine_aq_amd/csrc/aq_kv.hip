// aq_kv.hip -- writing keys and values into the paged cache, quantized as they
// are written, and reading rows of it back (gfx950).
//
// A cache row is one token's head_dim values in one head, K or V, in the
// weight format: groups of G along the row, each with the bias, scale and
// codes that aq_grid.hpp gives (the cache row of a token is bit for bit what
// the weight quantizer makes of it).  Values are clamped to fp16's finite
// range before that, since bias and scale are fp16, and a group that holds a
// NaN is stored as scale 0, bias NaN: NaN reaches the reader, and the integer
// codes stay finite.
//
// Both kernels move bytes and are bound by HBM at prompt size and by launch
// latency at decode size: append reads 2 bytes a value and writes bits/8 +
// 4/G, read does the reverse.  One thread per 8 values: 16 bytes of 16-bit
// values, 4 or 8 bytes of codes, so a row of 128 is 16 lanes on either side
// and every load and store of a wave covers whole 64-byte segments.  Page
// addresses are 64-bit (a cache is larger than 4 GiB), offsets inside a page
// 32-bit.
#include "aq_grid.hpp"
#include "aq_internal.hpp"

namespace aq {
namespace {

__device__ __forceinline__ float clamp_f16(float v) {
  return __builtin_fminf(__builtin_fmaxf(v, -65504.f), 65504.f);
}

// element offset of (slot, head) in an array of `width` elements per row, or
// -1 outside the cache
__device__ __forceinline__ int64_t row_offset(const KvCache &c, int64_t slot, int h, int width) {
  if (slot < 0 || slot >= c.num_pages * c.page_size) return -1;
  const int64_t page = slot / c.page_size;
  const int at = (int)(slot - page * c.page_size);
  return ((page * c.kv_heads + h) * c.page_size + at) * width;
}

template <int XDT, int BITS>
__global__ __launch_bounds__(256) void kv_append_kernel(KvCache c, const void *__restrict__ k,
                                                        const void *__restrict__ v, int64_t rows,
                                                        int64_t k_stride, int64_t v_stride,
                                                        const int64_t *__restrict__ slots) {
  const int D = c.head_dim, lanes = D >> 3;
  const int64_t total = rows * lanes;
  int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const bool active = idx < total;
  if (!active) idx = total - 1;  // whole rows are inactive together; keep loads in bounds
  const int64_t r = idx / lanes;
  const int o = (int)(idx - r * lanes) * 8;
  const int64_t t = r / c.kv_heads;
  const int h = (int)(r - t * c.kv_heads);
  const bool is_v = blockIdx.y != 0;
  const int64_t e = t * (is_v ? v_stride : k_stride) + (int64_t)h * D + o;
  const void *x = is_v ? v : k;
  void *codes = is_v ? c.v_codes : c.k_codes;
  const int64_t slot = slots[t];

  if constexpr (BITS == 16) {
    const uint4 w = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(x) + e);
    const int64_t at = row_offset(c, slot, h, D);
    if (!active || at < 0) return;
    *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(codes) + at + o) = w;
  } else {
    float w[8];
    load8<XDT>(x, e, w);
    float lo = 65504.f, hi = -65504.f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      nan |= w[i] != w[i];
      w[i] = clamp_f16(w[i]);
      lo = __builtin_fminf(lo, w[i]);
      hi = __builtin_fmaxf(hi, w[i]);
    }
    if (nan) hi = __builtin_inff();  // past every clamped value: marks the whole group
    const int glanes = c.group_size >> 3;
    for (int d = 1; d < glanes; d <<= 1) {
      lo = __builtin_fminf(lo, __shfl_xor(lo, d));
      hi = __builtin_fmaxf(hi, __shfl_xor(hi, d));
    }
    constexpr int L = (1 << BITS) - 1;
    nan = hi > 65504.f;
    uint16_t b16 = f16_round_down(lo);
    const double b = h2d(b16);
    uint16_t s16 = f16_scale_up(b, (double)hi, L);
    if (nan) s16 = 0;
    const double s = h2d(s16);
    const float bf = (float)b;
    const float rs = s16 ? __builtin_amdgcn_rcpf((float)s) : 0.f;
    uint32_t word[BITS / 4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      word[i * BITS / 32] |= nearest_code(w[i], b, s, bf, rs, L) << (i * BITS % 32);
    if (nan) b16 = 0x7E00u;
    const int64_t at = row_offset(c, slot, h, 1);
    if (!active || at < 0) return;
    uint32_t *dst = reinterpret_cast<uint32_t *>(codes) + at * (D * BITS / 32) + o * BITS / 32;
    if constexpr (BITS == 8)
      *reinterpret_cast<uint2 *>(dst) = make_uint2(word[0], word[1]);
    else
      *dst = word[0];
    if ((o & (c.group_size - 1)) == 0) {
      const int64_t gi = at * (D / c.group_size) + o / c.group_size;
      (is_v ? c.v_scales : c.k_scales)[gi] = s16;
      (is_v ? c.v_biases : c.k_biases)[gi] = b16;
    }
  }
}

template <int BITS, int ODT>
__global__ __launch_bounds__(256) void kv_read_kernel(KvCache c, const int64_t *__restrict__ slots,
                                                      int64_t rows, void *__restrict__ k,
                                                      void *__restrict__ v) {
  const int D = c.head_dim, lanes = D >> 3;
  const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (idx >= rows * lanes) return;
  const int64_t r = idx / lanes;
  const int o = (int)(idx - r * lanes) * 8;
  const int64_t t = r / c.kv_heads;
  const int h = (int)(r - t * c.kv_heads);
  const bool is_v = blockIdx.y != 0;
  const void *codes = is_v ? c.v_codes : c.k_codes;
  const int64_t at = row_offset(c, slots[t], h, 1);
  float w[8] = {};
  if (at >= 0) {
    if constexpr (BITS == 16) {
      if (c.dtype == X_F16)
        load8<X_F16>(codes, at * D + o, w);
      else
        load8<X_BF16>(codes, at * D + o, w);
    } else {
      const uint32_t *src = reinterpret_cast<const uint32_t *>(codes) + at * (D * BITS / 32) + o * BITS / 32;
      uint32_t word[BITS / 4];
      if constexpr (BITS == 8) {
        const uint2 u = *reinterpret_cast<const uint2 *>(src);
        word[0] = u.x;
        word[1] = u.y;
      } else {
        word[0] = *src;
      }
      const int64_t gi = at * (D / c.group_size) + o / c.group_size;
      const float s = f16_to_f32((is_v ? c.v_scales : c.k_scales)[gi]);
      const uint16_t *biases = is_v ? c.v_biases : c.k_biases;
      const float b = biases ? f16_to_f32(biases[gi]) : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = __builtin_fmaf((float)((word[i * BITS / 32] >> (i * BITS % 32)) & ((1 << BITS) - 1)), s, b);
    }
  }
  store8<ODT>(is_v ? v : k, r * D + o, w);
}

}  // namespace

hipError_t launch_kv_append(const void *k, const void *v, int x_dtype, int64_t T, int64_t k_stride,
                            int64_t v_stride, const int64_t *slots, const KvCache &c,
                            hipStream_t s) {
  const int64_t rows = T * c.kv_heads;
  const dim3 grid((unsigned)((rows * (c.head_dim >> 3) + 255) / 256), 2), block(256);
#define AQ_A(X, B) hipLaunchKernelGGL((kv_append_kernel<X, B>), grid, block, 0, s, c, k, v, rows, k_stride, v_stride, slots)
  if (c.bits == 16) AQ_A(X_F16, 16);
  else if (c.bits == 8 && x_dtype == X_F16) AQ_A(X_F16, 8);
  else if (c.bits == 8) AQ_A(X_BF16, 8);
  else if (x_dtype == X_F16) AQ_A(X_F16, 4);
  else AQ_A(X_BF16, 4);
#undef AQ_A
  return hipGetLastError();
}

hipError_t launch_kv_read(const int64_t *slots, int64_t T, const KvCache &c, void *k, void *v,
                          int out_dtype, hipStream_t s) {
  const int64_t rows = T * c.kv_heads;
  const dim3 grid((unsigned)((rows * (c.head_dim >> 3) + 255) / 256), 2), block(256);
#define AQ_R(B, O) hipLaunchKernelGGL((kv_read_kernel<B, O>), grid, block, 0, s, c, slots, rows, k, v)
#define AQ_RB(B)                                  \
  if (out_dtype == X_F32) AQ_R(B, X_F32);         \
  else if (out_dtype == X_F16) AQ_R(B, X_F16);    \
  else AQ_R(B, X_BF16);
  if (c.bits == 16) { AQ_RB(16) } else if (c.bits == 8) { AQ_RB(8) } else { AQ_RB(4) }
#undef AQ_RB
#undef AQ_R
  return hipGetLastError();
}

}  // namespace aq
