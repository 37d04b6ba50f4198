// aq_attn.hip -- attention of each sequence's newest tokens over the paged,
// quantized key-value cache (gfx950).
//
//   out = sum_t p_t v_t,  p = softmax_t(scale * q . k_t),  t <= len - L + i
//
// in one pass over the tokens with the running maximum m and sum l of the
// softmax: a tile of tokens with largest score m' > m rescales what was summed
// by exp(m - m') and adds exp(s - m').  The codes are never expanded into
// memory; with k = s code + b in each group g of G values of a row
//
//   q . k_t = sum_g s_tg (sum_{d in g} q_d code_td) + b_tg (sum_{d in g} q_d)
//   sum_t p_t v_td = sum_t (p_t s_tg) (code_td - c) + p_t (b_tg + c s_tg),
//
// both inner sums are products of integer codes and run on the matrix cores,
// scales and biases are applied to their results or to the weights.
//
// Matrix layout (v_mfma_f32_16x16x32).  The queries that share a key head --
// L tokens times the heads of the group -- are the 16 columns of a tile, the
// tokens (S^T = K q^T) and then the values (O^T = V^T p^T) its rows.  The
// result layout of S^T gives a lane one column and tokens 4h .. 4h+3 of each
// 16 (h = lane / 16); 32 tokens are two such results, and those 8 weights are
// one lane's part of the second product's operand, the tokens' order in k being
// free as long as V follows it: no weight crosses lanes, and the running
// maximum and sum of a column are registers of its lanes.
//
//  * Codes enter as fp16 bit patterns: an integer q <= 1023 in the low bits is
//    the fp16 subnormal q * 2^-24, exact in the matrix cores, so unpacking is
//    one byte permute (8 bits) or a mask (4 bits; the odd nibbles are masked
//    in place, 16 times too large, and the query or the result is scaled by
//    1/16) per pair.  2^24 goes into factors that are there anyway.
//  * Queries are scaled by a power of two per row so that their largest value
//    lies in [256, 512) and rounded to fp16: exact for fp16 and bf16 down to
//    2^-18 of the row's largest value.
//  * Weights p s are rounded to fp16 (2^-11 relative) for the second product.
//    They are kept 2^6 (8 bits) or 2^2 (4 bits) times too large, as far as
//    the largest possible scale of a group allows (131008 / 255, / 15), which
//    keeps small ones out of fp16's subnormals; l has the same factor.  The
//    rounded weight multiplies code - c, c the middle code, rather than the
//    code: the rounding then weighs with the value's distance from its group's
//    middle, not from its minimum.  code - c is not formed; -c times the sum of
//    the rounded weights is added in binary32.
//  * bits = 16: the pages' values are the operands.  A bf16 weight would lose
//    8 bits more than the output rounds off, so it is split in two bf16 parts,
//    two products per tile.
//
// Work division.  All tokens of all (sequence, key head, slice of 16 NT query
// rows) form one line of 128-token blocks that the workgroups cut evenly, so
// a batch of ragged lengths and one long sequence load the chip alike and the
// launch does not depend on the lengths.  In a block each of the four waves
// takes 32 tokens; the waves' (m, l, o) are joined through LDS.  A piece that
// does not cover its unit goes to the workspace; the workgroup that finishes
// last among a unit's pieces joins them, in the pieces' order whoever comes
// last, so results do not depend on timing.
//
// Bound: HBM, the codes, scales and biases read once.  At 8 bits a tile of 32
// tokens x 128 values is 8.7 KB and costs about 240 vector and 16 matrix
// instructions; four waves a CU would take 36 bytes a clock at that rate where
// HBM gives a CU about 9.
#include "aq_device.hpp"
#include "aq_internal.hpp"

namespace aq {
namespace {

typedef _Float16 f16x8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

constexpr int kBlock = 128;       // tokens per block: 4 waves of 32
constexpr int kMaxGrid = 1024;    // arrival counters in the workspace
constexpr float kNegInf = -__builtin_inff();

// `bytes` bytes at a uniform address; reads past them give zeros, without a
// memory access
typedef __amdgpu_buffer_rsrc_t Span;
__device__ __forceinline__ Span span(const void *base, int64_t off, int bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(base) + off;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(((uint64_t)hi << 32) | lo), 0,
                                           bytes, 0x00020000);
}
template <int BYTES>
__device__ __forceinline__ void fetch(uint32_t *to, Span from, int off) {
  if constexpr (BYTES % 16 == 0) {
#pragma unroll
    for (int w = 0; w < BYTES / 4; w += 4) {
      const u32x4v x = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(from, off + 4 * w, 0, 0));
#pragma unroll
      for (int i = 0; i < 4; ++i) to[w + i] = x[i];
    }
  } else if constexpr (BYTES == 8) {
    const u32x2v x = __builtin_bit_cast(u32x2v, __builtin_amdgcn_raw_buffer_load_b64(from, off, 0, 0));
    to[0] = x[0], to[1] = x[1];
  } else if constexpr (BYTES == 4) {
    to[0] = __builtin_amdgcn_raw_buffer_load_b32(from, off, 0, 0);
  } else if constexpr (BYTES == 2) {
    to[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(from, off, 0, 0);
  } else {
    static_assert(BYTES == 1, "");
    to[0] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(from, off, 0, 0);
  }
}

// a value and its partner's, 16 or 32 lanes away (xor), in either order
struct Pair { float a, b; };
__device__ __forceinline__ Pair with16(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t x = r[0], y = r[1];
  return {__builtin_bit_cast(float, x), __builtin_bit_cast(float, y)};
}
__device__ __forceinline__ Pair with32(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t x = r[0], y = r[1];
  return {__builtin_bit_cast(float, x), __builtin_bit_cast(float, y)};
}
// over the four lanes of a column (a + b is b + a: all four get the same bits)
__device__ __forceinline__ float quarters_sum(float v) {
  const Pair x = with16(v), y = with32(x.a + x.b);
  return y.a + y.b;
}
__device__ __forceinline__ float quarters_max(float v) {
  const Pair x = with16(v), y = with32(__builtin_fmaxf(x.a, x.b));
  return __builtin_fmaxf(y.a, y.b);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// the lane's number, recomputed where it stands: addresses made from it are
// not carried through the token loop, which needs the registers
__device__ __forceinline__ int lane_here() {
  int l = threadIdx.x & 63;
  asm volatile("" : "+v"(l));
  return l;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  return __builtin_bit_cast(uint32_t, half2v{(_Float16)a, (_Float16)b});
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2v{(__bf16)a, (__bf16)b});
}
// The products of 8 weights p with fp16 scales, rounded once, straight to fp16
// pairs (the compiler would convert the scales, multiply and convert back: 5
// instructions a pair for these 2).  Scale j is the half SEL0 (even j) or SEL1
// (odd j) of word w[j].  The compiler does not see the instructions, so the
// waits that it would put around them are here: one state after a v_exp_f32
// before its result is read, two before the matrix cores read a result; the
// low and high half of a pair are written four instructions apart.
template <int SEL0, int SEL1>
__device__ __forceinline__ u32x4v scaled_weights(const float *p, const uint32_t (&w)[8]) {
  uint32_t a, b, c, d;
#define AQ_LO(D, P, W, S) "v_fma_mixlo_f16 " D ", " P ", " W ", 0 op_sel:[0," S ",0] op_sel_hi:[0,1,0]\n\t"
#define AQ_HI(D, P, W, S) "v_fma_mixhi_f16 " D ", " P ", " W ", 0 op_sel:[0," S ",0] op_sel_hi:[0,1,0]\n\t"
#define AQ_MIX(S0, S1)                                                                      \
  asm("s_nop 0\n\t" AQ_LO("%0", "%4", "%12", S0) AQ_LO("%1", "%6", "%14", S0)               \
          AQ_LO("%2", "%8", "%16", S0) AQ_LO("%3", "%10", "%18", S0)                        \
              AQ_HI("%0", "%5", "%13", S1) AQ_HI("%1", "%7", "%15", S1)                     \
                  AQ_HI("%2", "%9", "%17", S1) AQ_HI("%3", "%11", "%19", S1) "s_nop 1"      \
      : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d)                                              \
      : "v"(p[0]), "v"(p[1]), "v"(p[2]), "v"(p[3]), "v"(p[4]), "v"(p[5]), "v"(p[6]),        \
        "v"(p[7]), "v"(w[0]), "v"(w[1]), "v"(w[2]), "v"(w[3]), "v"(w[4]), "v"(w[5]),        \
        "v"(w[6]), "v"(w[7]))
  if constexpr (SEL0 == 0 && SEL1 == 0)
    AQ_MIX("0", "0");
  else if constexpr (SEL0 == 1)
    AQ_MIX("1", "1");
  else
    AQ_MIX("0", "1");
#undef AQ_MIX
#undef AQ_HI
#undef AQ_LO
  return u32x4v{a, b, c, d};
}
__device__ __forceinline__ float half_at(uint32_t w, int i) {  // fp16 i (0, 1) of a word
  return (float)__builtin_bit_cast(half2v, w)[i];
}

template <bool BF>
__device__ __forceinline__ f32x4v mfma(u32x4v a, u32x4v b, f32x4v c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8v, a),
                                                   __builtin_bit_cast(bf16x8v, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8v, a),
                                                  __builtin_bit_cast(f16x8v, b), c, 0, 0, 0);
}

struct Params {
  const void *q;
  int64_t q_stride;
  const void *kc, *ks, *kb, *vc, *vs, *vb;
  const int32_t *table, *lengths;
  void *out;
  float *parts;       // two pieces per workgroup
  uint32_t *arrived;  // one counter per workgroup, zero between calls
  int64_t max_pages, num_pages;
  uint32_t page_subs, page_magic;  // page_size / 16 and floor(2^32 / that) + 1
  int kv_heads, group, L, B, slices, x_dtype;
  float scale;
};

// the 16-token unit s of a sequence -> its page (the estimate is at most one
// too large: s (magic d - 2^32) / (d 2^32) < 1)
__device__ __forceinline__ uint32_t page_of(const Params &p, uint32_t s) {
  if (p.page_subs == 1) return s;
  uint32_t n = __umulhi(s, p.page_magic);
  return n * p.page_subs > s ? n - 1 : n;
}

__device__ __forceinline__ int clamped_length(const Params &p, int b) {
  const int64_t cap = p.max_pages * p.page_subs * 16;
  const int n = p.lengths[b];
  return n < 0 ? 0 : (n > cap ? (int)cap : n);
}

// ---- one wave's state over a segment of tokens -------------------------------------
// BITS 4, 8 or 16; BF: operands are bf16 (bits = 16 with a bf16 cache); G is
// head_dim for 16 bits.
template <int BITS, bool BF, int D, int G, int NT>
struct Wave {
  static constexpr bool QUANT = BITS != 16;
  static constexpr int NG = QUANT ? D / G : 1;   // groups of a row
  static constexpr int NKS = QUANT ? G / 32 : 1; // products of 32 values per group
  static constexpr int KS = D / 32;
  static constexpr int RB = D * BITS / 8;        // bytes of a row of codes
  // a lane's keys: per group a run of G/4 codes in pieces of at most 16 bytes
  static constexpr int RUNB = QUANT ? G / 4 * BITS / 8 : 16;
  static constexpr int PIECE = RUNB < 16 ? RUNB : 16;
  static constexpr int NP = RUNB / PIECE;
  static constexpr int CP = QUANT ? PIECE * 8 / BITS : 8;  // codes per piece
  static constexpr int KW = D * BITS / 128;      // words of keys per 16 tokens
  // a lane's values: per token and group D/16 (G/16) neighbouring codes
  static constexpr int VN = G / 16;
  static constexpr int VB = VN * BITS / 8;       // bytes
  static constexpr int VW = VB < 4 ? 1 : VB / 4; // words
  static constexpr int SW = (NG * 4 + 1) / 2;    // words of 4 tokens' scales
  static constexpr int NR = NT * D / 4;          // result registers
  static constexpr float CENTRE = BITS == 8 ? 128.f : 8.f;
  static constexpr float UP = BITS == 8 ? 6.f : (BITS == 4 ? 2.f : 0.f);

  struct Scales { uint32_t s[2][SW], b[2][SW]; };
  struct Keys { uint32_t c[2][KW]; Scales g; };
  struct Values { uint32_t c[8][NG][VW]; Scales g; };

  u32x4v q[NT][KS];
  float qsum[NT][NG], C[NT];
  int vis[NT];      // tokens the column sees
  float m[NT], l[NT], bacc[NT][NG];
  f32x4v o[NT][NG][VN];

  // The 16 tokens at rows[sub]; there[sub]: whether their page is (if not,
  // zeros, and nothing is read)
  static __device__ __forceinline__ void load_scales(Scales &g, const void *s, const void *b,
                                                     int sub, int64_t row, bool there, int h) {
    const int bytes = there ? 16 * NG * 2 : 0;
    fetch<NG * 8>(g.s[sub], span(s, row * (NG * 2), bytes), h * (NG * 8));
    // without bias arrays every bias is +0
    fetch<NG * 8>(g.b[sub], span(b ? b : s, row * (NG * 2), b ? bytes : 0), h * (NG * 8));
  }

  static __device__ __forceinline__ void load_keys(Keys &k, const Params &p, const int64_t *rows,
                                                   const bool *there, int lane) {
    const int t = lane & 15, h = lane >> 4;
    constexpr int PIECES = QUANT ? NG * NP : KS;
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const Span codes = span(p.kc, rows[sub] * RB, there[sub] ? 16 * RB : 0);
#pragma unroll
      for (int i = 0; i < PIECES; ++i)  // a piece every 4 lanes' worth along the row
        fetch<PIECE>(k.c[sub] + i * (PIECE / 4), codes, t * RB + h * PIECE + i * 4 * PIECE);
      if constexpr (QUANT) load_scales(k.g, p.ks, p.kb, sub, rows[sub], there[sub], h);
    }
  }

  static __device__ __forceinline__ void load_values(Values &v, const Params &p,
                                                     const int64_t *rows, const bool *there,
                                                     int lane) {
    const int t = lane & 15, h = lane >> 4;
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const Span codes = span(p.vc, rows[sub] * RB, there[sub] ? 16 * RB : 0);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int g = 0; g < NG; ++g)
          fetch<VB>(v.c[4 * sub + i][g], codes, 4 * h * RB + t * VB + i * RB + g * (G * BITS / 8));
      if constexpr (QUANT) load_scales(v.g, p.vs, p.vb, sub, rows[sub], there[sub], h);
    }
  }

  // scale or bias of the lane's token i (of 4) in group g
  static __device__ __forceinline__ float scale_at(const uint32_t *w, int i, int g) {
    const int e = i * NG + g;
    return half_at(w[e >> 1], e & 1);
  }

  // 8 codes of the keys as one operand: product s of the row's D/32
  static __device__ __forceinline__ u32x4v key_operand(const uint32_t *c, int s) {
    if constexpr (BITS == 16) {
      return u32x4v{c[4 * s], c[4 * s + 1], c[4 * s + 2], c[4 * s + 3]};
    } else if constexpr (BITS == 8) {
      const uint32_t a = c[2 * s], b = c[2 * s + 1];
      return u32x4v{__builtin_amdgcn_perm(0, a, 0x0C010C00u), __builtin_amdgcn_perm(0, a, 0x0C030C02u),
                    __builtin_amdgcn_perm(0, b, 0x0C010C00u), __builtin_amdgcn_perm(0, b, 0x0C030C02u)};
    } else {  // codes 0,4 | 1,5 | 2,6 | 3,7, the odd ones 16 times too large
      const uint32_t a = c[s], b = a >> 8;
      return u32x4v{a & 0x000F000Fu, a & 0x00F000F0u, b & 0x000F000Fu, b & 0x00F000F0u};
    }
  }

  // the operand of value n of group g: the lane's 8 tokens
  static __device__ __forceinline__ u32x4v value_operand(const Values &v, int g, int n) {
    u32x4v a;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t *x = v.c[2 * w][g], *y = v.c[2 * w + 1][g];
      if constexpr (BITS == 16) {
        a[w] = __builtin_amdgcn_perm(y[n >> 1], x[n >> 1], n & 1 ? 0x07060302u : 0x05040100u);
      } else if constexpr (BITS == 8) {
        const uint32_t k = n & 3;
        a[w] = __builtin_amdgcn_perm(y[n >> 2], x[n >> 2], 0x0C000C00u | k | (4 + k) << 16);
      } else {
        const uint32_t k = n >> 1;
        const uint32_t both = __builtin_amdgcn_perm(y[0], x[0], 0x0C000C00u | k | (4 + k) << 16);
        a[w] = both & (n & 1 ? 0x00F000F0u : 0x000F000Fu);
      }
    }
    return a;
  }

  // queries of rows slice*16*NT .. of (b, head): columns of this lane
  __device__ __forceinline__ void start(const Params &p, int b, int head, int slice, int len) {
    const int lane = lane_here(), h = lane >> 4;
    const int cols = p.L * p.group;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = (slice * NT + nt) * 16 + (lane & 15);
      const bool on = r < cols;
      const int rr = on ? r : 0, i = rr / p.group, j = rr - i * p.group;
      vis[nt] = on ? len - p.L + 1 + i : 0;
      const uint16_t *src = reinterpret_cast<const uint16_t *>(p.q) +
                            ((int64_t)b * p.L + i) * p.q_stride +
                            (int64_t)(head * p.group + j) * D;
      uint4 raw[KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        // where the keys' 8 values of this product lie along the row
        int d;
        if constexpr (QUANT) {
          const int c = (s % NKS) * 8;
          d = (s / NKS) * G + (c / CP) * (4 * CP) + h * CP + c % CP;
        } else {
          d = s * 32 + h * 8;
        }
        raw[s] = *reinterpret_cast<const uint4 *>(src + d);
        if (!on) raw[s] = make_uint4(0, 0, 0, 0);
      }
      if constexpr (QUANT) {
        float x[KS][8], top = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint32_t u[4] = {raw[s].x, raw[s].y, raw[s].z, raw[s].w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint16_t bits = (uint16_t)(u[e >> 1] >> (16 * (e & 1)));
            x[s][e] = p.x_dtype == X_F16 ? f16_to_f32(bits) : bf16_to_f32(bits);
            top = __builtin_fmaxf(top, __builtin_fabsf(x[s][e]));
          }
        }
        top = quarters_max(top);
        int e = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127;
        e = e < -100 ? -100 : (e > 100 ? 100 : e);
        const float down = __builtin_ldexpf(1.f, 8 - e);
        C[nt] = __builtin_ldexpf(p.scale * 1.44269504088896341f, 24 + e - 8);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float sum = 0.f;
#pragma unroll
          for (int k = 0; k < NKS; ++k)
#pragma unroll
            for (int i8 = 0; i8 < 8; ++i8) sum += x[g * NKS + k][i8];
          qsum[nt][g] = quarters_sum(sum) * down * 0x1p-24f;
        }
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if constexpr (BITS == 8) {
              q[nt][s][w] = pack_f16(x[s][2 * w] * down, x[s][2 * w + 1] * down);
            } else {
              const float f = w & 1 ? down * 0.0625f : down;
              q[nt][s][w] = pack_f16(x[s][w] * f, x[s][w + 4] * f);
            }
          }
      } else {
        C[nt] = p.scale * 1.44269504088896341f;
#pragma unroll
        for (int s = 0; s < KS; ++s) q[nt][s] = u32x4v{raw[s].x, raw[s].y, raw[s].z, raw[s].w};
      }
    }
    clear();
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = kNegInf;
      l[nt] = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        bacc[nt][g] = 0.f;
#pragma unroll
        for (int n = 0; n < VN; ++n) o[nt][g][n] = f32x4v{0.f, 0.f, 0.f, 0.f};
      }
    }
  }

  // scores of the tile's 32 tokens, in powers of two: t[nt][4*sub + i]
  __device__ __forceinline__ void scores(const Keys &k, float (&t)[NT][8]) const {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      f32x4v acc[NT][NG];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const u32x4v a = key_operand(k.c[sub], s);
        const int g = QUANT ? s / NKS : 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          acc[nt][g] = mfma<BF>(a, q[nt][s],
                                (QUANT ? s % NKS == 0 : s == 0) ? f32x4v{0.f, 0.f, 0.f, 0.f} : acc[nt][g]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x;
          if constexpr (QUANT) {
            x = 0.f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              x = __builtin_fmaf(scale_at(k.g.s[sub], i, g), acc[nt][g][i], x);
              x = __builtin_fmaf(scale_at(k.g.b[sub], i, g), qsum[nt][g], x);
            }
          } else {
            x = acc[nt][0][i];
          }
          t[nt][4 * sub + i] = x * C[nt];
        }
    }
  }

  // weights of the scores t against the new maximum; rescales o, l, bacc
  __device__ __forceinline__ void weigh(float (&t)[NT][8]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top = t[nt][0];
#pragma unroll
      for (int j = 1; j < 8; ++j) top = __builtin_fmaxf(top, t[nt][j]);
      top = __builtin_fmaxf(quarters_max(top), m[nt]);
      const float base = top == kNegInf ? 0.f : top;
      if (__ballot(top > m[nt])) {
        const float keep = exp2_fast(m[nt] - base);
        m[nt] = top;
        l[nt] *= keep;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          bacc[nt][g] *= keep;
#pragma unroll
          for (int n = 0; n < VN; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nt][g][n][i] *= keep;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        t[nt][j] = exp2_fast(t[nt][j] - (base - UP));
        l[nt] += t[nt][j];
      }
    }
  }

  // o += weights x values
  __device__ __forceinline__ void gather(const Values &v, const float (&p)[NT][8]) {
    u32x4v w[NT][NG], w2[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (QUANT) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          uint32_t words[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) words[j] = v.g.s[j >> 2][((j & 3) * NG + g) >> 1];
          if constexpr (NG == 1)
            w[nt][g] = scaled_weights<0, 1>(p[nt], words);
          else if (g & 1)
            w[nt][g] = scaled_weights<1, 1>(p[nt], words);
          else
            w[nt][g] = scaled_weights<0, 0>(p[nt], words);
          float add = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float s = scale_at(v.g.s[j >> 2], j & 3, g), b = scale_at(v.g.b[j >> 2], j & 3, g);
            add = __builtin_fmaf(p[nt][j], __builtin_fmaf(CENTRE, s, b), add);
            add = __builtin_fmaf(half_at(w[nt][g][j >> 1], j & 1), -CENTRE, add);
          }
          bacc[nt][g] += add;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          if constexpr (BF) {
            const uint32_t r = pack_bf16(p[nt][j], p[nt][j + 1]);
            w[nt][0][j >> 1] = r;
            w2[nt][j >> 1] = pack_bf16(p[nt][j] - __builtin_bit_cast(float, r << 16),
                                       p[nt][j + 1] - __builtin_bit_cast(float, r & 0xFFFF0000u));
          } else {
            w[nt][0][j >> 1] = pack_f16(p[nt][j], p[nt][j + 1]);
          }
        }
      }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int n = 0; n < VN; ++n) {
        const u32x4v a = value_operand(v, g, n);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          o[nt][g][n] = mfma<BF>(a, w[nt][g], o[nt][g][n]);
          if constexpr (BF) o[nt][g][n] = mfma<BF>(a, w2[nt], o[nt][g][n]);
        }
      }
  }

  // a tile that some column sees only in part, or with a page left out:
  // on[sub] = the 16 tokens' page is there
  __device__ __forceinline__ void edge_scores(float (&t)[NT][8], int token, const bool *on, int h) const {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = token + 16 * (j >> 2) + 4 * h + (j & 3);
        if (!on[j >> 2] || at >= vis[nt]) t[nt][j] = kNegInf;
      }
  }

  // The values of tokens a column does not see must not reach it, not even as
  // 0 * NaN.  Quantized values: the codes are finite, so this is a matter of
  // the lane's scales and biases: those of tokens past the lane's columns, and
  // any that are not finite, become 0; a NaN goes to the columns that see it.
  __device__ __forceinline__ void edge_values(Values &v, int token, const bool *on, int h) {
#pragma unroll
    for (int x = 0; x < 2 * SW; ++x) {
      const int sub = x / SW, w = x % SW;
      uint32_t keep = 0;
#pragma unroll
      for (int e = 2 * w; e < 2 * w + 2; ++e) {
        const int g = e % NG, at = token + 16 * sub + 4 * h + e / NG;
        const float zero = half_at(v.g.s[sub][w], e & 1) * 0.f + half_at(v.g.b[sub][w], e & 1) * 0.f;
        bool seen = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const bool here = on[sub] && at < vis[nt];
          seen |= here;
          bacc[nt][g] += here ? zero : 0.f;
        }
        if (seen && zero == 0.f) keep |= e & 1 ? 0xFFFF0000u : 0x0000FFFFu;
      }
      // (opaque, or the words of all tiles are taken apart into halves)
      asm volatile("" : "+v"(keep));
      v.g.s[sub][w] &= keep;
      v.g.b[sub][w] &= keep;
    }
  }

  // 16 bits: the values themselves may be infinite or NaN, and a lane's values
  // serve every column, so such a tile is taken once per query token, the
  // values past that token's sight and the other columns' weights zero
  __device__ __forceinline__ void edge_pass(Values &v, const float (&p)[NT][8], float (&w)[NT][8],
                                            int sees, int token, const bool *on, int h) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = token + 16 * (j >> 2) + 4 * h + (j & 3);
      const bool seen = on[j >> 2] && at < sees;
#pragma unroll
      for (int x = 0; x < VW; ++x) v.c[j][0][x] = seen ? v.c[j][0][x] : 0u;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) w[nt][j] = vis[nt] == sees ? p[nt][j] : 0.f;
    }
  }

  // the 32-token tiles of one wave in blocks [blk0, blk1) of a sequence
  __device__ __forceinline__ void run(const Params &p, int b, int head, int slice, int len,
                                      int blk0, int blk1) {
    const int lane = lane_here(), wave = uniform(threadIdx.x >> 6);
    const int least = len - p.L + 1 + (slice * NT * 16) / p.group;  // what every column sees
    for (int c0 = blk0; c0 < blk1; c0 += 32) {
      const int first = c0 * kBlock + wave * 32;
      const int most = blk1 - c0 < 32 ? blk1 - c0 : 32;
      // lane 2k + sub: the rows of tile k
      uint32_t row_lo = 0, row_hi = 0x80000000u;
      {
        const int64_t t = (int64_t)first + (lane >> 1) * kBlock + (lane & 1) * 16;
        if ((lane >> 1) < most && t < len) {
          const uint32_t s = (uint32_t)(t >> 4), pg = page_of(p, s);
          const int id = p.table[(int64_t)b * p.max_pages + pg];
          if (id >= 0 && id < p.num_pages) {
            const int64_t row = (((int64_t)id * p.kv_heads + head) * p.page_subs + (s - pg * p.page_subs)) * 16;
            row_lo = (uint32_t)row;
            row_hi = (uint32_t)(row >> 32);
          }
        }
      }
      // tiles past len are at the end only
      int tiles = (len - first + kBlock - 1) / kBlock;
      tiles = len <= first ? 0 : (tiles < most ? tiles : most);
      if (tiles == 0) continue;
      Keys k;
      Values v;
      int64_t rows[2];
      bool on[2], on_next[2];
      auto locate = [&](int tile, bool *there) {
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          const uint32_t lo = __builtin_amdgcn_readlane(row_lo, 2 * tile + sub);
          const uint32_t hi = __builtin_amdgcn_readlane(row_hi, 2 * tile + sub);
          there[sub] = !(hi >> 31);
          rows[sub] = (int64_t)(((uint64_t)(hi & 0x7FFFFFFFu) << 32) | lo);
        }
      };
      locate(0, on);
      load_keys(k, p, rows, on, lane);
      load_values(v, p, rows, on, lane);
      for (int tile = 0; tile < tiles; ++tile) {
        const int token = first + tile * kBlock;
        const bool last = tile + 1 == tiles;
        float t[NT][8];
        const bool edge = token + 32 > least || !on[0] || !on[1];
        scores(k, t);
        // the last tile fetches itself again: loads without a branch let the
        // waits count only what they need
        locate(last ? tile : tile + 1, on_next);
        // (into the registers just used: nothing moves across)
        __builtin_amdgcn_sched_barrier(0);
        load_keys(k, p, rows, on_next, lane);
        if (edge) edge_scores(t, token, on, lane >> 4);
        weigh(t);
        if constexpr (QUANT) {
          if (edge) edge_values(v, token, on, lane >> 4);
          gather(v, t);
        } else {
          const int passes = edge ? p.L : 1;
          for (int i = 0; i < passes; ++i) {
            float w[NT][8];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 8; ++j) w[nt][j] = t[nt][j];
            if (edge) {
              if (i) {
                locate(tile, on);
                load_values(v, p, rows, on, lane);
              }
              edge_pass(v, t, w, len - p.L + 1 + i, token, on, lane >> 4);
            }
            gather(v, w);
          }
          if (edge) locate(last ? tile : tile + 1, on_next);
        }
        __builtin_amdgcn_sched_barrier(0);
        load_values(v, p, rows, on_next, lane);
        on[0] = on_next[0];
        on[1] = on_next[1];
      }
    }
  }

  // (m, l, o) with the biases' part folded in and every lane holding its
  // column's whole sums
  __device__ __forceinline__ void fold(float (&r)[NR]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      l[nt] = quarters_sum(l[nt]);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float add = QUANT ? quarters_sum(bacc[nt][g]) : 0.f;
#pragma unroll
        for (int n = 0; n < VN; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            r[((nt * NG + g) * VN + n) * 4 + i] =
                QUANT ? __builtin_fmaf(o[nt][g][n][i], BITS == 4 && (n & 1) ? 0x1p20f : 0x1p24f, add)
                      : o[nt][g][n][i];
      }
    }
  }
};

// m, l and r of the four waves -> wave 0
template <int NT, int NR>
__device__ __forceinline__ void join_waves(float (&m)[NT], float (&l)[NT], float (&r)[NR],
                                           float *ml, float *buf) {
  const int lane = lane_here(), wave = threadIdx.x >> 6;
  __syncthreads();  // the buffers' last readers are done
  if (lane < 16)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      ml[(wave * NT + nt) * 32 + lane] = m[nt];
      ml[(wave * NT + nt) * 32 + 16 + lane] = l[nt];
    }
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float top = kNegInf, total = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = __builtin_fmaxf(top, ml[(w * NT + nt) * 32 + (lane & 15)]);
    const float base = top == kNegInf ? 0.f : top;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      total += ml[(w * NT + nt) * 32 + 16 + (lane & 15)] *
               exp2_fast(ml[(w * NT + nt) * 32 + (lane & 15)] - base);
    const float keep = exp2_fast(m[nt] - base);
#pragma unroll
    for (int i = 0; i < NR / NT; ++i) r[nt * (NR / NT) + i] *= keep;
    m[nt] = top;
    l[nt] = total;
  }
  if (wave >= 2)
#pragma unroll
    for (int i = 0; i < NR; ++i) buf[((wave - 2) * NR + i) * 64 + lane] = r[i];
  __syncthreads();
  if (wave < 2)
#pragma unroll
    for (int i = 0; i < NR; ++i) r[i] += buf[(wave * NR + i) * 64 + lane];
  __syncthreads();
  if (wave == 1)
#pragma unroll
    for (int i = 0; i < NR; ++i) buf[i * 64 + lane] = r[i];
  __syncthreads();
  if (wave == 0)
#pragma unroll
    for (int i = 0; i < NR; ++i) r[i] += buf[i * 64 + lane];
}

// One piece in the workspace: the results of 16 NT columns, D floats each, then
// the columns' m and l.  Pieces are read by other workgroups than wrote them,
// on other XCDs with L2s of their own, in the same launch: stores and loads go
// past the L2s (sc1, the cache policy of device scope), and a workgroup counts
// as arrived when its stores are done.  (Ordinary stores with a device-wide
// fence write back and drop whole L2s: 118 against 37 us for 16 sequences of
// up to 4096 tokens, 8 bits.)
constexpr int kDeviceScope = 16;
template <int D, int NT>
constexpr int piece_floats() { return NT * (16 * D + 32); }

__device__ __forceinline__ void put_piece(Span to, int at, f32x4v v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4v, v), to, at * 4, 0, kDeviceScope);
}
__device__ __forceinline__ f32x4v get_piece4(Span from, int at) {
  return __builtin_bit_cast(f32x4v, __builtin_amdgcn_raw_buffer_load_b128(from, at * 4, 0, kDeviceScope));
}
__device__ __forceinline__ float get_piece(Span from, int at) {
  const uint32_t u = __builtin_amdgcn_raw_buffer_load_b32(from, at * 4, 0, kDeviceScope);
  return __builtin_bit_cast(float, u);
}

// Joins a unit's pieces w0 .. w1 (the first is that workgroup's second) and
// writes the rows: m and l of each column over 16 strands of pieces, then
// every four values of a column over one strand per wave.  The order of all
// sums is the pieces' own.
template <int D, int NT>
__device__ __forceinline__ void join_pieces(const Params &p, int b, int head, int slice, int64_t w0,
                                            int n, float *ml, float *buf) {
  constexpr int PF = piece_floats<D, NT>(), ML = NT * 16 * D;
  const int lane = lane_here(), wave = uniform(threadIdx.x >> 6);
  const int cols = p.L * p.group - slice * NT * 16;
  const Span first = span(p.parts, (2 * w0 + 1) * (PF * 4), PF * 4);
  // piece i > 0 is at (2 i - 1) PF floats past the first
  const float *rest = p.parts + (2 * w0 + 1) * (int64_t)PF;
  auto piece = [&](int i) {
    return i ? span(rest, (2 * (int64_t)i - 1) * (PF * 4), PF * 4) : first;
  };
  {
    const int strand = threadIdx.x >> 4, c = threadIdx.x & 15;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float m = kNegInf, l = 0.f;
#pragma unroll 4
      for (int i0 = 0; i0 < n; i0 += 16) {
        const int i = i0 + strand;
        if (i < n) {
          // strands of a wave read different pieces: plain addresses
          const float *src = rest + (i ? (2 * (int64_t)i - 1) * PF : 0) + ML + nt * 32 + c;
          const float pm = __hip_atomic_load(src, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          const float pl = __hip_atomic_load(src + 16, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          const float top = __builtin_fmaxf(m, pm), base = top == kNegInf ? 0.f : top;
          l = l * exp2_fast(m - base) + pl * exp2_fast(pm - base);
          m = top;
        }
      }
      buf[(strand * NT + nt) * 32 + c] = m;
      buf[(strand * NT + nt) * 32 + 16 + c] = l;
    }
    __syncthreads();
    if (threadIdx.x < 16 * NT) {
      const int nt = threadIdx.x >> 4;
      float m = kNegInf, l = 0.f;
      for (int w = 0; w < 16; ++w) m = __builtin_fmaxf(m, buf[(w * NT + nt) * 32 + c]);
      const float base = m == kNegInf ? 0.f : m;
      for (int w = 0; w < 16; ++w)
        l += buf[(w * NT + nt) * 32 + 16 + c] * exp2_fast(buf[(w * NT + nt) * 32 + c] - base);
      ml[nt * 32 + c] = base;
      ml[nt * 32 + 16 + c] = l == 0.f ? 0.f : 1.f / l;
    }
    __syncthreads();
  }
  const int used = cols < 16 * NT ? cols : 16 * NT;
  constexpr int Q = D / 4;
  for (int i0 = 0; i0 < used * Q; i0 += 64) {
    const int item = i0 + lane, c = item / Q;  // past the columns in use: read, not written
    const float base = ml[(c >> 4) * 32 + (c & 15)];
    f32x4v acc = {0.f, 0.f, 0.f, 0.f};
    for (int i = wave; i < n; i += 32) {
      f32x4v v[8];
      float m[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const Span src = piece(i + 4 * x < n ? i + 4 * x : i);
        v[x] = get_piece4(src, item * 4);
        m[x] = get_piece(src, ML + (c >> 4) * 32 + (c & 15));
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float w = i + 4 * x < n ? exp2_fast(m[x] - base) : 0.f;
        if (i + 4 * x < n) acc += v[x] * w;
      }
    }
    *reinterpret_cast<f32x4v *>(buf + (wave * 64 + lane) * 4) = acc;
    __syncthreads();
    if (wave == ((i0 >> 6) & 3) && c < used) {
      const float inv = ml[(c >> 4) * 32 + 16 + (c & 15)];
      f32x4v y = *reinterpret_cast<f32x4v *>(buf + lane * 4);
      for (int w = 1; w < 4; ++w) y += *reinterpret_cast<f32x4v *>(buf + (w * 64 + lane) * 4);
      y *= inv;
      const int r = slice * NT * 16 + c, i = r / p.group, j = r - i * p.group;
      uint2 *out = reinterpret_cast<uint2 *>(
          reinterpret_cast<uint16_t *>(p.out) +
          (((int64_t)b * p.L + i) * p.kv_heads * p.group + head * p.group + j) * D + (item % Q) * 4);
      *out = p.x_dtype == X_F16 ? make_uint2(pack_f16(y[0], y[1]), pack_f16(y[2], y[3]))
                                : make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
    }
    __syncthreads();
  }
}

template <int BITS, bool BF, int D, int G, int NT, int WGS>
__global__ __launch_bounds__(256, WGS) void attn_kernel(Params p) {
  using W = Wave<BITS, BF, D, G, NT>;
  constexpr int NR = W::NR, NG = W::NG, VN = W::VN;
  __shared__ float buf[2 * NR * 64];
  __shared__ float ml[4 * NT * 32];
  __shared__ uint32_t sums[4];
  __shared__ int found[2];
  __shared__ uint32_t flag;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

  // sequences without tokens: zero rows
  const int64_t row_halves = (int64_t)p.L * p.kv_heads * p.group * D;
  for (int64_t b = blockIdx.x; b < p.B; b += gridDim.x)
    if (clamped_length(p, (int)b) == 0)
      for (int64_t i = threadIdx.x; i < row_halves / 8; i += 256)
        reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(p.out) + b * row_halves)[i] =
            make_uint4(0, 0, 0, 0);

  // blocks of all sequences, and this workgroup's part of the line
  const int per = (p.B + 255) / 256;
  const int b_lo = threadIdx.x * per < p.B ? threadIdx.x * per : p.B;
  const int b_hi = b_lo + per < p.B ? b_lo + per : p.B;
  uint32_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += (uint32_t)(clamped_length(p, b) + kBlock - 1) / kBlock;
  uint32_t upto = mine;  // inclusive sum over the threads
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t x = __shfl_up(upto, d);
    if (lane >= d) upto += x;
  }
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  uint32_t all = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < wave) upto += sums[w];
    all += sums[w];
  }
  const int64_t units = (int64_t)p.kv_heads * p.slices;  // per sequence
  const int64_t total = all * units;
  const int64_t grid = total < (int64_t)gridDim.x ? total : (int64_t)gridDim.x;
  if (blockIdx.x >= grid) return;
  int64_t pos = blockIdx.x * total / grid;
  const int64_t end = (blockIdx.x + 1) * total / grid;
  if ((int64_t)(upto - mine) * units <= pos && pos < (int64_t)upto * units) {
    uint32_t before = upto - mine;
    int b = b_lo;
    for (;; ++b) {
      const uint32_t n = (uint32_t)(clamped_length(p, b) + kBlock - 1) / kBlock;
      if (pos < (int64_t)(before + n) * units) break;
      before += n;
    }
    found[0] = b;
    found[1] = (int)before;
  }
  __syncthreads();
  int b = uniform(found[0]);
  uint32_t before = (uint32_t)uniform(found[1]);

  W st;
  while (pos < end) {
    int len = uniform(clamped_length(p, b));
    int blocks = (int)((uint32_t)(len + kBlock - 1) / kBlock);
    while (pos >= (int64_t)(before + blocks) * units) {
      before += blocks;
      ++b;
      len = uniform(clamped_length(p, b));
      blocks = (int)((uint32_t)(len + kBlock - 1) / kBlock);
    }
    const int64_t in_seq = pos - (int64_t)before * units;
    const int unit = uniform((int)(in_seq / blocks));
    const int blk0 = (int)(in_seq - (int64_t)unit * blocks);
    const int head = uniform(unit / p.slices), slice = unit - head * p.slices;
    const int64_t left = end - pos;
    const int blk1 = left < blocks - blk0 ? blk0 + (int)left : blocks;
    const int64_t unit_pos = pos - blk0;
    pos += blk1 - blk0;

    st.start(p, b, head, slice, len);
    st.run(p, b, head, slice, len, blk0, blk1);
    float r[NR];
    st.fold(r);
    join_waves<NT, NR>(st.m, st.l, r, ml, buf);

    if (blk0 != 0 || blk1 != blocks) {
      // a piece: to the workspace, and join if it is the unit's last to arrive
      const int lane = lane_here();
      constexpr int PF = piece_floats<D, NT>();
      const int64_t w0 = ((unit_pos + 1) * grid - 1) / total;
      const int n = uniform((int)(((unit_pos + blocks) * grid - 1) / total - w0) + 1);
      if (wave == 0) {
        const Span to = span(p.parts, (2 * (int64_t)blockIdx.x + (blk0 == 0)) * (PF * 4), PF * 4);
        const int c = lane & 15, h = lane >> 4;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int e = 0; e < 4 * VN; e += 4) {
              f32x4v y;
#pragma unroll
              for (int x = 0; x < 4; ++x)
                y[x] = r[((nt * NG + g) * VN + (e + x) % VN) * 4 + (e + x) / VN];
              put_piece(to, (nt * 16 + c) * D + g * G + 4 * h * VN + e, y);
            }
          if (h < 2) {
            const float x = h ? st.l[nt] : st.m[nt];
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), to,
                                                  (NT * 16 * D + nt * 32 + lane) * 4, 0, kDeviceScope);
          }
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        if (lane == 0)
          flag = __hip_atomic_fetch_add(p.arrived + w0, 1u, __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(n - 1);
      }
      __syncthreads();
      const bool last = uniform((int)flag) != 0;
      __syncthreads();
      if (last) {
        asm volatile("" ::: "memory");
        if (threadIdx.x == 0)
          __hip_atomic_store(p.arrived + w0, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        join_pieces<D, NT>(p, b, head, slice, w0, n, ml, buf);
      }
      continue;
    }
    if (wave == 0) {
      // a lane's results of a group are G/4 neighbouring values: 4 rows of VN
      const int lane = lane_here(), cols = p.L * p.group, h = lane >> 4;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int c = (slice * NT + nt) * 16 + (lane & 15);
        if (c >= cols) continue;
        const int i = c / p.group, j = c - i * p.group;
        uint16_t *out = reinterpret_cast<uint16_t *>(p.out) +
                        (((int64_t)b * p.L + i) * p.kv_heads * p.group + head * p.group + j) * D;
        const float inv = st.l[nt] == 0.f ? 0.f : 1.f / st.l[nt];
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int e = 0; e < 4 * VN; e += 8) {
            float y[8];
#pragma unroll
            for (int x = 0; x < 8; ++x)
              y[x] = r[((nt * NG + g) * VN + (e + x) % VN) * 4 + (e + x) / VN] * inv;
            const int64_t at = g * G + 4 * h * VN + e;
            if (p.x_dtype == X_F16)
              store8<X_F16>(out, at, y);
            else
              store8<X_BF16>(out, at, y);
          }
      }
    }
  }
}

// query rows per slice: two tiles of 16 where there are more than 16
int tiles_for(int64_t cols) { return cols > 16 ? 2 : 1; }

// workgroups per CU the kernel is built for: what its registers allow (a
// lane's scales and biases grow with the groups of a row)
constexpr int wgs_per_cu(int D, int NG, int NT) {
  return D * NT <= 128 && NG <= 2 ? 3 : (D * NT <= 128 || (D * NT <= 256 && NG <= 2) ? 2 : 1);
}

int grid_for(int D, int ng, int nt) {
  const int n = device_cus() * wgs_per_cu(D, ng, nt);
  return n < kMaxGrid ? n : kMaxGrid;
}

}  // namespace

int64_t attn_workspace_bytes(int64_t, int L, int q_heads, int kv_heads, int head_dim) {
  const int nt = tiles_for((int64_t)L * (q_heads / kv_heads));
  const int64_t piece = (int64_t)nt * head_dim * 16 + nt * 32;
  return kMaxGrid * 4 + 2 * (int64_t)grid_for(head_dim, 1, nt) * piece * 4;
}

hipError_t launch_paged_attention(const AttnArgs &a, const KvCache &c, hipStream_t s) {
  Params p;
  p.q = a.q;
  p.q_stride = a.q_stride;
  p.kc = c.k_codes;
  p.ks = c.k_scales;
  p.kb = c.k_biases;
  p.vc = c.v_codes;
  p.vs = c.v_scales;
  p.vb = c.v_biases;
  p.table = a.page_table;
  p.lengths = a.lengths;
  p.out = a.out;
  p.arrived = reinterpret_cast<uint32_t *>(a.workspace);
  p.parts = reinterpret_cast<float *>(a.workspace) + kMaxGrid;
  p.max_pages = a.max_pages;
  p.num_pages = c.num_pages;
  p.page_subs = (uint32_t)c.page_size / 16;
  p.page_magic = p.page_subs > 1 ? (uint32_t)(0x100000000ull / p.page_subs) + 1 : 0;
  p.kv_heads = c.kv_heads;
  p.group = a.q_heads / c.kv_heads;
  p.L = a.L;
  p.B = a.B;
  p.x_dtype = a.x_dtype;
  p.scale = a.scale;
  const int64_t cols = (int64_t)a.L * p.group;
  const int nt = tiles_for(cols);
  p.slices = (int)((cols + 16 * nt - 1) / (16 * nt));
  // no more workgroups than blocks the table can hold
  const int64_t blocks = (a.max_pages * c.page_size + kBlock - 1) / kBlock;
  int64_t grid = grid_for(c.head_dim, c.bits == 16 ? 1 : c.head_dim / c.group_size, nt);
  if (blocks * a.B < grid && blocks * a.B * c.kv_heads * p.slices < grid)
    grid = blocks * a.B * c.kv_heads * p.slices;
#define AQ_K(B, F, D, G)                                                                      \
  do {                                                                                        \
    if (nt == 1)                                                                              \
      hipLaunchKernelGGL((attn_kernel<B, F, D, G, 1, wgs_per_cu(D, D / G, 1)>), dim3((unsigned)grid), \
                         dim3(256), 0, s, p);                                                 \
    else                                                                                      \
      hipLaunchKernelGGL((attn_kernel<B, F, D, G, 2, wgs_per_cu(D, D / G, 2)>), dim3((unsigned)grid), \
                         dim3(256), 0, s, p);                                                 \
    return hipGetLastError();                                                                 \
  } while (0)
#define AQ_G(B, D)                                     \
  if (c.head_dim == D) {                               \
    if (c.group_size == 32) AQ_K(B, false, D, 32);     \
    if (c.group_size == 64) AQ_K(B, false, D, 64);     \
    if constexpr (D >= 128) AQ_K(B, false, D, 128);    \
  }
#define AQ_H(D)                                        \
  if (c.head_dim == D) {                               \
    if (c.dtype == X_BF16) AQ_K(16, true, D, D);       \
    AQ_K(16, false, D, D);                             \
  }
  if (c.bits == 4) { AQ_G(4, 64) AQ_G(4, 128) AQ_G(4, 256) }
  if (c.bits == 8) { AQ_G(8, 64) AQ_G(8, 128) AQ_G(8, 256) }
  if (c.bits == 16) { AQ_H(64) AQ_H(128) AQ_H(256) }
#undef AQ_H
#undef AQ_G
#undef AQ_K
  return hipErrorInvalidValue;
}

}  // namespace aq
