// aq_rope.hip -- rotary positions: rows of queries and keys turned by their
// token's angles, keys written into the paged cache as they are turned (gfx950).
//
// Pair i of a token at position p is turned by a = p f_i.  The angle is a
// binary64 product and is reduced by multiples of pi/2 in two parts of 53 bits,
// so positions of any size keep their angle (in binary32 the product alone is
// off by 2^-24 a, 0.06 at a million); sine and cosine of what remains are their
// Taylor sums to degree 15, below 2^-48.  They are computed once per token and
// pair into LDS and serve all heads.  Each product and sum of the turn is
// rounded to binary32 by itself: the keys that are quantized are the same bits
// on any way there.
//
// A workgroup takes 2^tb neighbouring tokens and all heads of its side, queries
// or keys and values.  A thread turns 8 pairs, 16 values, of one token in every
// `phases`-th head, so it holds its token's cosines in registers.  Turned keys
// go to the cache's quantizer (aq_kv.hpp) through LDS, neighbouring tokens of one head
// together, which mostly lie in one run of the cache.
//
// Bound: HBM at prompt size, launch latency at decode size.  8191 tokens of 32 + 8
// heads of 128: rows alone 168 MB in 33 us (5.1 TB/s), written at 4 bits 178 MB in
// 39 us (4.6 TB/s).  64 tokens: rows alone 2.9 us; written at 8 bits 6.9, where the
// quantizer, two rounds of 32 of the 256 threads, waits for the angles.
#include "aq_kv.hpp"

namespace aq {
namespace {

constexpr int kThreads = 256;
constexpr int kKeyBytes = 16384;  // turned keys on their way to the quantizer

// cosine and sine of p f, times factor
__device__ __forceinline__ float2 cos_sin(int p, float f, double factor) {
  const double a = (double)p * (double)f;
  const double n = __builtin_rint(a * 0.63661977236758134308);       // 2 / pi
  double r = __builtin_fma(n, -1.57079632679489655800, a);           // pi / 2, its first 53 bits
  r = __builtin_fma(n, -6.12323399573676603587e-17, r);              // and the next
  const double x = r * r;
  // -1/3!, 1/5!, ... and -1/2!, 1/4!, ...
  double s = -7.64716373181981647590e-13, c = -1.14707455977297247139e-11;
  s = __builtin_fma(s, x, 1.60590438368216145994e-10);
  s = __builtin_fma(s, x, -2.50521083854417187751e-08);
  s = __builtin_fma(s, x, 2.75573192239858906526e-06);
  s = __builtin_fma(s, x, -1.98412698412698412698e-04);
  s = __builtin_fma(s, x, 8.33333333333333333333e-03);
  s = __builtin_fma(s, x, -1.66666666666666666667e-01);
  s = __builtin_fma(s * x, r, r);
  c = __builtin_fma(c, x, 2.08767569878680989792e-09);
  c = __builtin_fma(c, x, -2.75573192239858906526e-07);
  c = __builtin_fma(c, x, 2.48015873015873015873e-05);
  c = __builtin_fma(c, x, -1.38888888888888888889e-03);
  c = __builtin_fma(c, x, 4.16666666666666666667e-02);
  c = __builtin_fma(c, x, -5.00000000000000000000e-01);
  c = __builtin_fma(c, x, 1.0);
  const int quarter = (int)(n - 4.0 * __builtin_floor(n * 0.25));
  const double u = quarter & 1 ? s : c, v = quarter & 1 ? c : s;
  return make_float2((float)((quarter == 1 || quarter == 2 ? -u : u) * factor),
                     (float)((quarter & 2 ? -v : v) * factor));
}

template <int XDT>
__device__ __forceinline__ float value(uint32_t w, int i) {
  const uint16_t x = (uint16_t)(w >> (16 * i));
  return XDT == X_F16 ? f16_to_f32(x) : bf16_to_f32(x);
}
template <int XDT>
__device__ __forceinline__ uint32_t pair(float a, float b) {
  if constexpr (XDT == X_F16)
    return __builtin_bit_cast(uint32_t, half2v{(_Float16)a, (_Float16)b});
  else
    return __builtin_bit_cast(uint32_t, bf16x2v{(__bf16)a, (__bf16)b});
}

struct Turned { float x, y; };
__device__ __forceinline__ Turned turn(float a, float b, float c, float s) {
#pragma clang fp contract(off)
  const float ac = a * c, bs = b * s, bc = b * c, as = a * s;
  return {ac - bs, bc + as};
}

// 16 values of one head: two runs of 8
struct Part { uint32_t w[2][4]; };

__device__ __forceinline__ Part load_part(const uint16_t *row, int o0, int o1) {
  const uint4 a = *reinterpret_cast<const uint4 *>(row + o0), b = *reinterpret_cast<const uint4 *>(row + o1);
  return {{{a.x, a.y, a.z, a.w}, {b.x, b.y, b.z, b.w}}};
}
__device__ __forceinline__ void store_part(uint16_t *row, int o0, int o1, const Part &p) {
  *reinterpret_cast<uint4 *>(row + o0) = make_uint4(p.w[0][0], p.w[0][1], p.w[0][2], p.w[0][3]);
  *reinterpret_cast<uint4 *>(row + o1) = make_uint4(p.w[1][0], p.w[1][1], p.w[1][2], p.w[1][3]);
}

// (values past the rotary part keep their bits: on = false)
template <int XDT, bool INTER>
__device__ __forceinline__ Part turn_part(const Part &p, const float *c, const float *s, bool on) {
  Part y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (INTER) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const Turned t = turn(value<XDT>(p.w[j][i], 0), value<XDT>(p.w[j][i], 1), c[4 * j + i], s[4 * j + i]);
        y.w[j][i] = pair<XDT>(t.x, t.y);
      }
    } else {
      const Turned t = turn(value<XDT>(p.w[0][i], 0), value<XDT>(p.w[1][i], 0), c[2 * i], s[2 * i]);
      const Turned u = turn(value<XDT>(p.w[0][i], 1), value<XDT>(p.w[1][i], 1), c[2 * i + 1], s[2 * i + 1]);
      y.w[0][i] = pair<XDT>(t.x, u.x);
      y.w[1][i] = pair<XDT>(t.y, u.y);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) y.w[j][i] = on ? y.w[j][i] : p.w[j][i];
  return y;
}

// BITS 0: no cache (rows only), else the cache's.  gridDim.y = 2: queries, then keys and
// values; 1: all of them
template <int XDT, int BITS, bool INTER, typename Int>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, KvCache c, uint32_t magic,
                                                        int tb, int unit_shift) {
  constexpr bool QUANT = BITS == 4 || BITS == 8;
  extern __shared__ float2 table[];  // [tokens][half]
  __shared__ __align__(16) uint16_t keys[QUANT ? kKeyBytes / 2 : 8];
  const int D = a.head_dim, half = a.rotary >> 1, tokens = 1 << tb;
  const int64_t t0 = (int64_t)blockIdx.x << tb;
  for (int i = threadIdx.x; i < half << tb; i += kThreads) {
    const int64_t t = t0 + i / half;
    table[i] = cos_sin(a.positions[t < a.T ? t : a.T - 1], a.freqs[i % half], a.factor);
  }
  __syncthreads();

  const int unit = threadIdx.x & ((1 << unit_shift) - 1);
  const int local = (threadIdx.x >> unit_shift) & (tokens - 1);
  const int phase = threadIdx.x >> (unit_shift + tb), phases = kThreads >> (unit_shift + tb);
  const bool active = t0 + local < a.T, on = unit * 16 < a.rotary;
  const int64_t t = active ? t0 + local : a.T - 1;
  const int o0 = on && !INTER ? 8 * unit : 16 * unit, o1 = on && !INTER ? half + 8 * unit : 16 * unit + 8;
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = table[local * half + (on ? 8 * unit + i : 0)];
    cs[i] = x.x, sn[i] = x.y;
  }

  constexpr int U = 4;  // heads whose loads are under way at once
  const bool both = gridDim.y == 1;
  if (blockIdx.y == 0) {
    const uint16_t *src = a.q + t * a.q_stride;
    uint16_t *dst = a.q_out + t * a.q_out_stride;
    for (int h0 = phase; h0 < a.q_heads; h0 += U * phases) {
      Part p[U];
#pragma unroll
      for (int x = 0; x < U; ++x) {
        const int h = h0 + x * phases;
        p[x] = load_part(src + (int64_t)(h < a.q_heads ? h : h0) * D, o0, o1);
      }
#pragma unroll
      for (int x = 0; x < U; ++x) {
        const int h = h0 + x * phases;
        if (active && h < a.q_heads)
          store_part(dst + (int64_t)h * D, o0, o1, turn_part<XDT, INTER>(p[x], cs, sn, on));
      }
    }
  }
  if (!both && blockIdx.y == 0) return;

  const uint16_t *src = a.k + t * a.k_stride;
  if constexpr (!QUANT) {
    // rows as they are: to k_out, into a 16-bit cache with the values beside them
    bool there = false;
    Int row0 = 0;
    if constexpr (BITS == 16) row0 = cache_row<Int>(c, magic, a.slots[t], 0, there);
    for (int h0 = phase; h0 < a.kv_heads; h0 += U * phases) {
      Part p[U], v[U];
#pragma unroll
      for (int x = 0; x < U; ++x) {
        const int h = h0 + x * phases, hh = h < a.kv_heads ? h : h0;
        p[x] = load_part(src + (int64_t)hh * D, o0, o1);
        if constexpr (BITS == 16)
          v[x] = load_part(a.v + t * a.v_stride + (int64_t)hh * D, 16 * unit, 16 * unit + 8);
      }
#pragma unroll
      for (int x = 0; x < U; ++x) {
        const int h = h0 + x * phases;
        if (!active || h >= a.kv_heads) continue;
        const Part y = turn_part<XDT, INTER>(p[x], cs, sn, on);
        if (a.k_out) store_part(a.k_out + t * a.k_out_stride + (int64_t)h * D, o0, o1, y);
        if constexpr (BITS == 16) {
          if (!there) continue;
          const int64_t at = ((int64_t)row0 + (int64_t)h * c.page_size) * D;
          store_part(reinterpret_cast<uint16_t *>(c.k_codes) + at, o0, o1, y);
          store_part(reinterpret_cast<uint16_t *>(c.v_codes) + at, 16 * unit, 16 * unit + 8, v[x]);
        }
      }
    }
  } else {
    // as many heads at a time as the buffer holds; within it token by token of a head
    const int at_once = kKeyBytes / 2 / D >> tb;
    for (int first = 0; first < a.kv_heads; first += at_once) {
      const int n = a.kv_heads - first < at_once ? a.kv_heads - first : at_once;
      __syncthreads();  // the last round's readers are done
      for (int h0 = phase; h0 < n; h0 += U * phases) {
        Part p[U];
#pragma unroll
        for (int x = 0; x < U; ++x) {
          const int h = h0 + x * phases;
          p[x] = load_part(src + (int64_t)(first + (h < n ? h : h0)) * D, o0, o1);
        }
#pragma unroll
        for (int x = 0; x < U; ++x) {
          const int h = h0 + x * phases;
          if (h >= n) continue;
          const Part y = turn_part<XDT, INTER>(p[x], cs, sn, on);
          store_part(keys + ((h << tb) + local) * D, o0, o1, y);
          if (a.k_out && active) store_part(a.k_out + t * a.k_out_stride + (int64_t)(first + h) * D, o0, o1, y);
        }
      }
      __syncthreads();
      // 32 values a thread
      const int part_shift = unit_shift - 1, rows = n << tb, per = kThreads >> part_shift;
      const int o = ((int)threadIdx.x & ((1 << part_shift) - 1)) * 32;
      auto write = [&](bool is_v) {
        for (int r0 = 0; r0 < rows; r0 += per) {
          const int r = r0 + (int)(threadIdx.x >> part_shift), row = r < rows ? r : rows - 1, h = row >> tb;
          const int64_t mine = t0 + (row & (tokens - 1)), tt = mine < a.T ? mine : a.T - 1;
          float w[32];
          if (is_v)
            load32<XDT>(a.v, tt * a.v_stride + (int64_t)(first + h) * D + o, w);
          else
            load32<XDT>(keys, row * D + o, w);
          write_row_part<BITS, Int>(c, magic, a.slots[tt], first + h, is_v, r < rows && mine < a.T, o, w);
        }
      };
      write(false);
      write(true);
    }
  }
}

template <int BITS, typename Int>
hipError_t launch(const RopeArgs &a, const KvCache &c, hipStream_t s) {
  const int unit_shift = __builtin_ctz((unsigned)a.head_dim / 16);
  int tb = 0;
  while (tb < 4 && (a.T >> (tb + 1)) >= 512) ++tb;
  const int64_t blocks = (a.T + (1 << tb) - 1) >> tb;
  const dim3 grid((unsigned)blocks, a.q_heads && a.kv_heads ? 2 : 1);
  const unsigned lds = (unsigned)(a.rotary / 2 * sizeof(float2)) << tb;
  const uint32_t magic = BITS ? magic_of(c) : 0;
#define AQ_R(X, I) hipLaunchKernelGGL((rope_kernel<X, BITS, I, Int>), grid, dim3(kThreads), lds, s, a, c, magic, tb, unit_shift)
  if (a.x_dtype == X_F16) {
    if (a.interleaved) AQ_R(X_F16, true); else AQ_R(X_F16, false);
  } else {
    if (a.interleaved) AQ_R(X_BF16, true); else AQ_R(X_BF16, false);
  }
#undef AQ_R
  return hipGetLastError();
}

template <typename Int>
hipError_t launch_bits(const RopeArgs &a, const KvCache &c, hipStream_t s) {
  if (c.bits == 16) return launch<16, Int>(a, c, s);
  return c.bits == 8 ? launch<8, Int>(a, c, s) : launch<4, Int>(a, c, s);
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a, const KvCache *c, hipStream_t s) {
  if (!c) return launch<0, uint32_t>(a, KvCache{}, s);
  return narrow(*c) ? launch_bits<uint32_t>(a, *c, s) : launch_bits<int64_t>(a, *c, s);
}

}  // namespace aq
