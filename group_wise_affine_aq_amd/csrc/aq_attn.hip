// aq_attn.hip -- attention of each sequence's newest tokens over the paged,
// quantized key-value cache (gfx950).
//
//   out = sum_t p_t v_t,  p = softmax_t(scale * q . k_t),  t <= len - L + i
//
// in one pass over the tokens with the running maximum m and sum l of the
// softmax: a token with score s rescales what was summed by exp(m - m'),
// m' = max(m, s), and adds exp(s - m').
//
// One workgroup per query row (token and head): its four waves take every
// fourth token, each lane head_dim/64 neighbouring values; the waves' partial
// (m, l, o) are joined through LDS at the end.
#include "aq_device.hpp"
#include "aq_internal.hpp"

namespace aq {
namespace {

// value d of the row at element offset `row` (in rows) of one code array
template <int BITS>
__device__ __forceinline__ float row_value(const KvCache &c, const void *codes,
                                           const uint16_t *scales, const uint16_t *biases,
                                           int64_t row, int d) {
  if constexpr (BITS == 16) {
    const uint16_t u = reinterpret_cast<const uint16_t *>(codes)[row * c.head_dim + d];
    return c.dtype == X_F16 ? f16_to_f32(u) : bf16_to_f32(u);
  } else {
    const uint32_t w = reinterpret_cast<const uint32_t *>(
        codes)[row * (c.head_dim * BITS / 32) + d * BITS / 32];
    const int64_t g = row * (c.head_dim / c.group_size) + d / c.group_size;
    const float q = (float)((w >> (d * BITS % 32)) & ((1 << BITS) - 1));
    return __builtin_fmaf(q, f16_to_f32(scales[g]), biases ? f16_to_f32(biases[g]) : 0.f);
  }
}

template <int BITS, int DPL>  // values per lane: head_dim / 64
__global__ __launch_bounds__(256) void attn_rows_kernel(AttnArgs a, KvCache c) {
  __shared__ float part[4][64 * DPL + 2];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t row = blockIdx.x;  // (b * L + i) * q_heads + h
  const int64_t tok = row / a.q_heads;
  const int h = (int)(row - tok * a.q_heads);
  const int b = (int)(tok / a.L), i = (int)(tok - (int64_t)b * a.L);
  const int j = h / (a.q_heads / c.kv_heads);
  int64_t len = a.lengths[b];
  const int64_t cap = a.max_pages * c.page_size;
  len = len < 0 ? 0 : (len > cap ? cap : len);
  const int64_t sees = len - a.L + 1 + i;

  const uint16_t *q = reinterpret_cast<const uint16_t *>(a.q) + tok * a.q_stride + (int64_t)h * (64 * DPL);
  float qv[DPL], o[DPL];
#pragma unroll
  for (int e = 0; e < DPL; ++e) {
    const uint16_t u = q[lane * DPL + e];
    qv[e] = a.x_dtype == X_F16 ? f16_to_f32(u) : bf16_to_f32(u);
    o[e] = 0.f;
  }
  float m = -__builtin_inff(), l = 0.f;
  for (int64_t t = wave; t < sees; t += 4) {
    const int64_t p = t / c.page_size;
    const int page = a.page_table[b * a.max_pages + p];
    if (page < 0 || page >= c.num_pages) continue;
    const int64_t at = ((int64_t)page * c.kv_heads + j) * c.page_size + (t - p * c.page_size);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < DPL; ++e)
      s = __builtin_fmaf(qv[e], row_value<BITS>(c, c.k_codes, c.k_scales, c.k_biases, at, lane * DPL + e), s);
    s = wave_sum(s) * a.scale;
    const float m2 = __builtin_fmaxf(m, s);
    const float keep = m == m2 ? 1.f : __expf(m - m2), w = __expf(s - m2);
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < DPL; ++e)
      o[e] = o[e] * keep + w * row_value<BITS>(c, c.v_codes, c.v_scales, c.v_biases, at, lane * DPL + e);
    m = m2;
  }
#pragma unroll
  for (int e = 0; e < DPL; ++e) part[wave][lane * DPL + e] = o[e];
  if (lane == 0) {
    part[wave][64 * DPL] = m;
    part[wave][64 * DPL + 1] = l;
  }
  __syncthreads();
  if (wave != 0) return;
  float top = -__builtin_inff(), total = 0.f, sum[DPL] = {};
  for (int w = 0; w < 4; ++w) top = __builtin_fmaxf(top, part[w][64 * DPL]);
  for (int w = 0; w < 4; ++w) {
    if (part[w][64 * DPL + 1] == 0.f) continue;  // a wave that saw no token
    const float keep = __expf(part[w][64 * DPL] - top);
    total += part[w][64 * DPL + 1] * keep;
#pragma unroll
    for (int e = 0; e < DPL; ++e) sum[e] += part[w][lane * DPL + e] * keep;
  }
  uint16_t *out = reinterpret_cast<uint16_t *>(a.out) + row * (64 * DPL);
#pragma unroll
  for (int e = 0; e < DPL; ++e) {
    const float y = total == 0.f ? 0.f : sum[e] / total;
    out[lane * DPL + e] = a.x_dtype == X_F16 ? f32_to_f16_rne(y) : f32_to_bf16_rne(y);
  }
}

}  // namespace

int64_t attn_workspace_bytes(int64_t, int, int, int, int) { return 16; }

hipError_t launch_paged_attention(const AttnArgs &a, const KvCache &c, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.B * a.L * a.q_heads)), block(256);
#define AQ_T(B, D) hipLaunchKernelGGL((attn_rows_kernel<B, D>), grid, block, 0, s, a, c)
#define AQ_TB(B)                          \
  if (c.head_dim == 64) AQ_T(B, 1);       \
  else if (c.head_dim == 128) AQ_T(B, 2); \
  else AQ_T(B, 4);
  if (c.bits == 16) { AQ_TB(16) } else if (c.bits == 8) { AQ_TB(8) } else { AQ_TB(4) }
#undef AQ_TB
#undef AQ_T
  return hipGetLastError();
}

}  // namespace aq
