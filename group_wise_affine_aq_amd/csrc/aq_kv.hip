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
#include "aq_kv.hpp"

namespace aq {
namespace {

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
  const int64_t slot = slots[t];

  if constexpr (BITS == 16) {
    void *codes = is_v ? c.v_codes : c.k_codes;
    const uint4 w = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(x) + e);
    bool there;
    const int64_t at = cache_row<Int>(c, magic, slot, h, there);
    if (!active || !there) return;
    *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(codes) + at * D + o) = w;
  } else {
    float w[E];
    load32<XDT>(x, e, w);
    write_row_part<BITS, Int>(c, magic, slot, h, is_v, active, o, w);
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
