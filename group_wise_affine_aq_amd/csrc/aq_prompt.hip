// aq_prompt.hip -- attention of whole prompts over 16-bit rows of keys and
// values (gfx950).
//
//   out = sum_t p_t v_t,  p = softmax_t(score(q . k_t))
//
// in one pass over the keys with the running maximum and sum of the softmax.
//
// The query rows of one key head and sequence -- its tokens times the heads of
// the group, token by token -- are cut into tiles of 32 NW; a workgroup of NW
// waves takes one, 32 rows a wave, and walks over the keys that any of them
// sees, KT at a time.  Keys and values of a tile go through LDS once and serve
// all waves; while they are worked on, the next tile's are on their way.
//
// NW is 4, or 2 where a sequence has 64 rows or fewer.  With heads of up to 128
// two workgroups share a CU, and one's products run beside the other's softmax
// without any order between them.  8192 tokens of 32 heads on 8 of 128, bf16:
// 536 us (1026 TFLOP/s), capped 604; 4 x 4096 of heads of 64: 380 us and 463;
// heads of 256, which leave room for one wave a SIMD: 1171 and 1302 us.
// Compared at earlier steps, on one card each: workgroups of 8 waves in two
// groups half a tile apart 577 us capped and 509 not, against 592 and 528, but
// 83 against 72 us for 4 x 1024 tokens, 479 against 447 us for 4 x 4096 of heads
// of 64 and 117 against 107 us with a window of 512; heads of 256 with 32 keys a
// tile, whose sums are one chain of products, 1336 us against 1165 with 64;
// products of the tile before, put between the softmax's steps in one wave, 647
// and (heads of 256) 1199 us, more than they hid.
//
// Bound: the softmax's vector instructions and the products, hardly beside each
// other.  A score takes 10 vector instructions capped, 6.5 not (8192 tokens of
// heads of 128): 277 and 179 us of them at 2.4 GHz, and 222 us of products at the matrix
// cores' peak.
//
// Matrix layout (v_mfma_f32_32x32x16).  S^T = K q^T: a lane has one row of
// queries (lane % 32) and, with h = lane / 32, the tokens 8 i + 4 h .. + 3 of
// each 32.  So a row's maximum and sum stay in two lanes, and the 16 tokens of
// one k-step of the second product, O^T = V^T p^T, are taken in the order in
// which the lanes hold them: weights are rounded and packed where they are.  V
// enters as columns by transposing reads of LDS (4 tokens x 16 values each).
// 16-byte pieces of a row lie in LDS at their number xor the row's, keys and
// values in different ways, so that neither read meets a bank twice (heads of 64,
// whose rows are half as long, do: two conflict cycles for each product).
//
// A weight is rounded to the inputs' type once: half the products that two parts
// would take.  Errors of the measured cases' results against binary64 are 2.3e-4
// of their norm in fp16 and 2.1e-3 in bf16, 1.1 to 1.3 times the result's own
// rounding (2.0e-4, 1.6e-3), which two parts reach at 787 us against 602 for
// 8192 tokens capped and 96 against 80 for packed prompts.  The sums of weights
// are of the unrounded ones.
//
// Weights are 2^(t - m): m is set so that the largest weight is 2^(up - 4) and
// moves when one would pass 2^up, so that it seldom does; then everything summed
// is rescaled.  fp16: up = 15, the range below serves the small weights (down
// to 2^-35 of the largest, at least).  bf16 has binary32's range for weights and
// values, and a sum of weights of 1 times values near its end would pass it
// where the result does not: up = -12, so that 4096 tokens of the largest
// weights and of the type's largest value, 2^128, still have a finite sum (with
// up = 15 one token of 2^117 had none), and small values lose nothing down to
// 2^-110.
//
// Values that are not finite: 0 * inf is NaN, and a row that does not see a
// token must not see its value, nor lose an infinity to a weight that is
// rounded to 0.  Such a value leaves no finite result in its column of any row
// of the wave, so a workgroup that ends with one that is not finite starts
// again, with care: values are looked at on their way to LDS, those that are not
// finite become 0 there, and the waves add them, from memory, to the rows that
// see their token, one token of such a tile after the other.
#include "aq_device.hpp"
#include "aq_internal.hpp"

namespace aq {
namespace {

typedef _Float16 f16x8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef float f32x16v __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2v __attribute__((ext_vector_type(2)));
typedef short s16x4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4v lds_s16x4;
typedef __attribute__((address_space(3))) u32x4v lds_u32x4;
typedef __attribute__((address_space(3))) char lds_char;
typedef __amdgpu_buffer_rsrc_t Span;

constexpr float kNegInf = -__builtin_inff();
constexpr float kLog2e = 1.44269504088896341f;
template <bool BF> constexpr float kUp = BF ? -12.f : 15.f;  // weights are 2^kUp at most
constexpr int kMaxParts = 64;

struct Params {
  PromptArgs a;
  float C;         // |scale| log2 e
  uint32_t flip;   // sign of the scale, for pairs of queries
  // caps: cap2 (in powers of two; 0: none) and its inverse; where |s| <= small (smaller) the cap of a
  // score s is s times a polynomial of five (three) terms in s^2
  float cap2, inv_cap2, small, cap[5], smaller, cap3[3];
  int window, group;
  int tiles;       // of query rows, at most, of all sequences
  int parts;       // of every tile's keys
  float *piece;    // parts > 1: per tile, head and part: rows of D results, then m and l
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float as_float(uint32_t u) { return __builtin_bit_cast(float, u); }

// the value of lane ^ 32
__device__ __forceinline__ float other_half(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t x = r[0], y = r[1];
  return as_float(threadIdx.x & 32 ? x : y);
}

template <bool BF>
__device__ __forceinline__ f32x16v mfma(u32x4v a, u32x4v b, f32x16v c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8v, a), __builtin_bit_cast(bf16x8v, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8v, a), __builtin_bit_cast(f16x8v, b), c, 0, 0, 0);
}
template <bool BF>
__device__ __forceinline__ uint32_t pack(float a, float b) {
  if constexpr (BF)
    return __builtin_bit_cast(uint32_t, bf16x2v{(__bf16)a, (__bf16)b});
  else
    return __builtin_bit_cast(uint32_t, half2v{(_Float16)a, (_Float16)b});
}

// rows of one sequence: first and number, of queries and of keys
struct Sequence { int q0, n, k0, len; };
__device__ __forceinline__ Sequence sequence(const PromptArgs &a, int b) {
  auto clamp = [](int x, int lo, int64_t hi) { return x < lo ? lo : (x > hi ? (int)hi : x); };
  Sequence s;
  s.q0 = clamp(a.q_starts[b], 0, a.Tq);
  s.n = clamp(a.q_starts[b + 1], s.q0, a.Tq) - s.q0;
  s.k0 = clamp(a.k_starts[b], 0, a.Tk);
  s.len = clamp(a.k_starts[b + 1], s.k0, a.Tk) - s.k0;
  return s;
}

// The tile `at` of all sequences' tiles of R rows -> its sequence, and its number there,
// the last tiles, which see the most keys, first.  False past the last.
template <int R>
__device__ __forceinline__ bool find_tile(const PromptArgs &a, int group, int at, int &b, int &tile) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int mine = b0 + lane < a.B ? (sequence(a, b0 + lane).n * group + R - 1) / R : 0;
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int x = __shfl_up(upto, d);
      upto += lane >= d ? x : 0;
    }
    const uint64_t past = __ballot(at < before + upto);
    if (past) {
      const int l = __builtin_ctzll(past);
      b = uniform(b0 + l);
      const int own = __builtin_amdgcn_readlane(mine, l);
      tile = uniform(own - 1 - (at - before - (__builtin_amdgcn_readlane(upto, l) - own)));
      return true;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// a piece: results of R rows, then their m, then their l
template <int D>
constexpr int piece_floats(int R) { return R * (D + 2); }

template <bool BF, int D, int NW>
struct Shape {
  static constexpr int R = 32 * NW, THREADS = 64 * NW;
  static constexpr int KT = D > 128 && NW == 2 ? 32 : 64;  // keys of a tile
  static constexpr int X = KT / 32, KK = KT / 16;
  static constexpr int CH = D / 8;            // 16-byte pieces of a row
  static constexpr int RB = D * 2;            // bytes of a row
  static constexpr int EACH = KT * CH / THREADS;  // pieces a thread brings of each
  static constexpr int KS = D / 16, DB = D / 32;
  static constexpr int TILE = KT * RB;        // bytes of keys, or values
  static constexpr int LDS = 4 * TILE;
  static __device__ __forceinline__ int key_piece(int row, int c) { return row * RB + (c ^ key_swap(row)) * 16; }
  static __device__ __forceinline__ int value_swap(int row) { return CH < 16 ? row << 1 & 4 : row << 2 & 12; }
  static __device__ __forceinline__ int key_swap(int row) { return row & (CH < 16 ? CH - 1 : 15); }
  static __device__ __forceinline__ int value_piece(int row, int c) { return row * RB + (c ^ value_swap(row)) * 16; }
};

// the larger magnitude of each half, and whether one is infinite or NaN
__device__ __forceinline__ uint32_t larger_pair(uint32_t most, u32x4v w) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    most = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2v, most),
                                                                  __builtin_bit_cast(u16x2v, w[i] & 0x7FFF7FFFu)));
  return most;
}
template <bool BF>
__device__ __forceinline__ bool odd_value(uint32_t most) {
  constexpr uint32_t kTop = BF ? 0x7F80u : 0x7C00u;
  return (most & 0xFFFFu) >= kTop || (most >> 16) >= kTop;
}
// the values that are not finite, or the others, 0 in the places of the rest
template <bool BF>
__device__ __forceinline__ uint32_t odd_pair(uint32_t w) {
  constexpr uint32_t kTop = BF ? 0x7F80u : 0x7C00u;
  return ((w & kTop) == kTop ? w & 0xFFFFu : 0u) | ((w >> 16 & kTop) == kTop ? w & 0xFFFF0000u : 0u);
}
template <bool BF>
__device__ __forceinline__ float half_of(uint32_t w, int i) {
  return BF ? bf16_to_f32((uint16_t)(w >> (16 * i))) : f16_to_f32((uint16_t)(w >> (16 * i)));
}

template <int N> struct Count { static constexpr int value = N; };

// the largest of a lane's scores, or of their magnitudes
template <int X>
__device__ __forceinline__ float largest(const f32x16v (&s)[X], bool magnitude) {
  float top = magnitude ? __builtin_fabsf(s[0][0]) : s[0][0];
#pragma unroll
  for (int x = 0; x < X; ++x)
#pragma unroll
    for (int j = 0; j < 16; ++j) top = __builtin_fmaxf(top, magnitude ? __builtin_fabsf(s[x][j]) : s[x][j]);
  return top;
}
// a score below p.small, capped, is the score times this polynomial in its square
__device__ __forceinline__ float cap_factor(const Params &p, float s) {
  const float u = s * s;
  float f = __builtin_fmaf(u, p.cap[4], p.cap[3]);
  f = __builtin_fmaf(u, f, p.cap[2]);
  f = __builtin_fmaf(u, f, p.cap[1]);
  return __builtin_fmaf(u, f, p.cap[0]);
}
__device__ __forceinline__ float small_cap(const Params &p, float s) { return s * cap_factor(p, s); }

template <bool BF, int D, int NW>
__global__ __launch_bounds__(64 * NW, D > 128 || NW == 2 ? 1 : 2) void prompt_kernel(Params p) {
  using S = Shape<BF, D, NW>;
  constexpr int KT = S::KT, X = S::X, KK = S::KK, KS = S::KS, DB = S::DB, EACH = S::EACH;
  __shared__ __align__(16) char lds[S::LDS];
  __shared__ int range[NW][2], odd_tile[2][NW];
  const PromptArgs &a = p.a;
  const int head = blockIdx.x % (unsigned)a.kv_heads;
  const int unit = blockIdx.x / (unsigned)a.kv_heads;
  int b, tile;
  if (!find_tile<S::R>(a, p.group, unit, b, tile)) return;
  Sequence seq = sequence(a, b);
  seq.q0 = uniform(seq.q0), seq.n = uniform(seq.n), seq.k0 = uniform(seq.k0), seq.len = uniform(seq.len);

  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), h = lane >> 5;
  const int rows = seq.n * p.group, row = tile * S::R + wave * 32 + (lane & 31);
  const bool active = row < rows;
  const int token = (active ? row : 0) / p.group, qh = head * p.group + ((active ? row : 0) - token * p.group);
  const int pos = seq.len - seq.n + token;
  // what the row sees: lo <= t < hi
  int lo = 0, hi = 0;
  {
    const int first = a.scores.first ? a.scores.first[seq.q0 + token] : 0;
    const int prefix = a.scores.prefix ? a.scores.prefix[b] : 0;
    const int since = pos - p.window + 1;
    lo = first > since ? first : since;
    lo = lo < 0 ? 0 : lo;
    hi = pos + 1 > prefix ? pos + 1 : prefix;
    hi = hi < seq.len ? hi : seq.len;
    if (!active || hi < lo) hi = lo = 0;
  }
  const bool sees = hi > lo;
  // over the wave: the first and last key of any row, and the keys that all rows see
  int least = sees ? lo : 0x7FFFFFFF, most = hi, from = active ? lo : 0, upto = active ? hi : 0x7FFFFFFF;
  if (active && !sees) from = 0x7FFFFFFF;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_xor(least, d), y = __shfl_xor(most, d), z = __shfl_xor(from, d), w = __shfl_xor(upto, d);
    least = x < least ? x : least, most = y > most ? y : most;
    from = z > from ? z : from, upto = w < upto ? w : upto;
  }
  least = uniform(least), most = uniform(most), from = uniform(from), upto = uniform(upto);
  if (lane == 0) range[wave][0] = least, range[wave][1] = most;
  __syncthreads();
  int begin = 0x7FFFFFFF, end = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    begin = range[w][0] < begin ? range[w][0] : begin;
    end = range[w][1] > end ? range[w][1] : end;
  }
  // tiles of keys, of which this workgroup has a part
  int t0 = uniform(begin < end ? begin / KT : 0), t1 = uniform(begin < end ? (end + KT - 1) / KT : 0);
  if (p.parts > 1) {
    const int64_t all = t1 - t0;
    const int first = t0;
    t0 = first + (int)(all * blockIdx.y / p.parts);
    t1 = first + (int)(all * (blockIdx.y + 1) / p.parts);
  }

  // queries: the lane's row as the second operand, 8 values of each 16
  u32x4v q[KS];
  {
    const uint16_t *src = a.q + (int64_t)(seq.q0 + token) * a.q_stride + (int64_t)qh * D + 8 * h;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      q[s] = *reinterpret_cast<const u32x4v *>(src + 16 * s);
#pragma unroll
      for (int i = 0; i < 4; ++i) q[s][i] ^= p.flip;
    }
  }
  const float slope = a.scores.slopes ? a.scores.slopes[qh] * kLog2e : 0.f;

  // the rows of a tile of keys or values (counted from t0); those past the sequence, and all of a tile
  // past the last, read as zeros, without a memory access
  const int k_step = (int)a.k_stride * 2, v_step = (int)a.v_stride * 2;  // bytes of a token
  const int64_t row0 = (int64_t)seq.k0 + (int64_t)t0 * KT;
  auto scalar = [](const void *x) {
    const uint64_t u = reinterpret_cast<uint64_t>(x);
    return (uint64_t)(uint32_t)uniform((int)(u >> 32)) << 32 | (uint32_t)uniform((int)(uint32_t)u);
  };
  const uint64_t k0 = scalar(a.k + row0 * a.k_stride + (int64_t)head * D);
  const uint64_t v0 = scalar(a.v + row0 * a.v_stride + (int64_t)head * D);
  const int keys_left = (t1 * KT < seq.len ? t1 * KT : seq.len) - t0 * KT;
  auto rows_of = [&](uint64_t base, int step, int tile) {
    const uint64_t at = base + (uint64_t)(uint32_t)tile * (uint32_t)(step * KT);
    const int left = keys_left - tile * KT, there = left < KT ? left : KT;
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(at), 0,
                                             there > 0 ? (there - 1) * step + S::RB : 0, 0x00020000);
  };
  // Keys of tile `due` and values of the one before it (tiles counted from t0) go straight to
  // LDS, a kilobyte a load, the lanes' pieces in the order in which LDS has them.  The compiler
  // does not know of these loads: arrived() waits for them.
  int due = 0;
  lds_char *const mem = (lds_char *)lds;
  int from_k[EACH], from_v[EACH];
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int at = (wave * EACH + e) * 64 + lane, r = at / S::CH, c = at % S::CH;
    from_k[e] = r * k_step + (c ^ S::key_swap(r)) * 16;
    from_v[e] = r * v_step + (c ^ S::value_swap(r)) * 16;
  }
  auto fetch = [&](const int *from, uint64_t first, int step, int tile, int to) {
    const Span span = rows_of(first, step, tile);
    const uint32_t base = (uint32_t)(uintptr_t)mem + to + wave * (EACH * 1024);
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      uint32_t kept;  // (m0, which the compiler may have a use for)
      asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
                   "buffer_load_dwordx4 %2, %3, 0 offen lds\n\ts_mov_b32 m0, %0"
                   : "=&s"(kept) : "s"(base + e * 1024), "v"(from[e]), "s"(span) : "memory");
    }
  };
  auto arrived = [] { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); };
  bool careful = false;  // values are looked at on their way
  auto bring = [&] {
    fetch(from_k, k0, k_step, due, (due & 1) * S::TILE);
    if (due > 0) {
      const int half = (due - 1) & 1, to = (2 + half) * S::TILE;
      if (!careful) {
        fetch(from_v, v0, v_step, due - 1, to);
      } else {
        const Span span = rows_of(v0, v_step, due - 1);
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
          u32x4v x = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(span, from_v[e], 0, 0));
          top = larger_pair(top, x);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] ^= odd_pair<BF>(x[j]);
          *(lds_u32x4 *)(mem + to + ((wave * EACH + e) * 64 + lane) * 16) = x;
        }
        odd_tile[half][wave] = __ballot(odd_value<BF>(top)) != 0;
      }
    }
    ++due;
  };
  auto barrier = [] {
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
  };

  // Where the lane's operands begin, this tile's half of LDS included: the xor
  // reaches the low four bits of a piece's number, so pieces 16 apart, and rows 8
  // apart, are at fixed distances.
  constexpr int NK = KS < 8 ? KS : 8, NV = DB < 4 ? DB : 4;
  const int vr = 4 * h + ((lane & 15) >> 2), vc = (lane >> 4 & 1) * 16 + (lane & 3) * 4;
  int at_k[NK], at_v[NV];
  f32x16v o[DB];
  float m, l;

  // The first product of tile t, and the second one of the tile before, whose weights are w
  f32x16v s[X];
  u32x4v w[KK];
  bool have = false;  // (w: a tile that no row of the wave sees has none)
  auto value_operand = [&](int i, int k) {  // 4 tokens x 16 values a group of 16 lanes, twice
    const lds_char *from = mem + at_v[i % NV] + (16 * k * S::RB + i / NV * 256);
    const s16x4v x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)from);
    const s16x4v y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(from + 8 * S::RB));
    const u32x2v u = __builtin_bit_cast(u32x2v, x), v = __builtin_bit_cast(u32x2v, y);
    return u32x4v{u[0], u[1], v[0], v[1]};
  };
  // Operands are fetched kAhead products ahead of theirs, and stay kHold products longer: a read into
  // registers that a product under way still takes its operand from waits for that product (reads
  // right behind the product that frees their registers, as the compiler would have them: 66 cycles a
  // product instead of 34).
  auto multiply = [&](auto first, auto last) {
    constexpr int NKEYS = X * KS, FIRST = decltype(first)::value, N = decltype(last)::value - FIRST;
    constexpr int kAhead = 6, kHold = 2;
    if constexpr (FIRST == 0)
#pragma unroll
      for (int x = 0; x < X; ++x)
#pragma unroll
        for (int j = 0; j < 16; ++j) s[x][j] = 0.f;
    u32x4v f[N];
#pragma unroll
    for (int n = 0; n < N + kAhead; ++n) {
      if (n < N) {
        const int i = FIRST + n, j = i - NKEYS;
        f[n] = i < NKEYS ? *(const lds_u32x4 *)(mem + at_k[i / X % NK] + (32 * (i % X) * S::RB + i / X / NK * 256))
                         : value_operand(j % DB, j / DB);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (n >= kAhead) {
        const int d = n - kAhead, i = FIRST + d, j = i - NKEYS;
        if (i < NKEYS)
          s[i % X] = mfma<BF>(f[d], q[i / X], s[i % X]);
        else
          o[j % DB] = mfma<BF>(f[d], w[j / DB], o[j % DB]);
        if (d >= kHold) asm volatile("" ::"v"(f[d - kHold]));
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  constexpr Count<X * KS> keys_end;
  constexpr Count<X * KS + DB * KK> both_end;
  auto gather_odd = [&](int t) {
    if (!careful) return;
    int odd = 0;
#pragma unroll
    for (int x = 0; x < NW; ++x) odd |= odd_tile[(t - t0) & 1][x];
    if (uniform(odd)) {
      const int key0 = t * KT;
      const Span span = rows_of(v0, v_step, t - t0);
#pragma unroll 1
      for (int x = 0; x < KT; ++x) {
        const bool in = (uint32_t)(key0 + x - lo) < (uint32_t)(hi - lo);
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const u32x2v v = __builtin_bit_cast(u32x2v, __builtin_amdgcn_raw_buffer_load_b64(
                span, x * v_step + (32 * i + 2 * j + 4 * h) * 2, 0, 0));
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float z = half_of<BF>(odd_pair<BF>(v[y >> 1]), y & 1);
              o[i][j + y] += in ? z : 0.f;
            }
          }
      }
    }
  };

  for (;;) {
#pragma unroll
  for (int i = 0; i < DB; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
  m = kNegInf, l = 0.f;
  have = false;
#pragma unroll
  for (int k = 0; k < KK; ++k) w[k] = u32x4v{0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < EACH; ++e)  // (the values that the first weights of 0 meet)
    *(lds_u32x4 *)(mem + 3 * S::TILE + ((wave * EACH + e) * 64 + lane) * 16) = u32x4v{0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < NK; ++k) at_k[k] = S::key_piece(lane & 31, 2 * k + h);
#pragma unroll
  for (int i = 0; i < NV; ++i) at_v[i] = 3 * S::TILE + S::value_piece(vr, (32 * i + vc) >> 3) + (vc & 7) * 2;
  due = 0;
  // Behind a barrier every wave asks for its share of the keys of the next tile but one and the values
  // of the next, whose place was last read ahead of it.
  bring();
  arrived();
  barrier();
  bring();
  for (int t = t0; t < t1; ++t) {
    const int key0 = t * KT;
    const bool need = key0 < most && key0 + KT > least;
    if (need || have) {
      // Both products without a branch between them: a wave's first tile finds weights of 0 and
      // finite values, the one behind its last makes scores that nobody takes.
      multiply(Count<0>(), both_end);
    }
    if (have) gather_odd(t - 1);

#pragma unroll
    for (int k = 0; k < NK; ++k) at_k[k] ^= S::TILE;
#pragma unroll
    for (int i = 0; i < NV; ++i) at_v[i] ^= S::TILE;
    if (need) {
      // Scores in powers of two are t = s C, or its cap.  Three ways there, by what the wave has
      // (each of s, C and the cap's polynomial fused with the subtraction of m where it can be):
      // plain scores, capped ones that are small beside the cap, and all others.
      const bool edge = key0 < from || key0 + KT > upto;
      const bool simple = !edge && !a.scores.slopes;
      float top;
      int way = 0;
      if (simple && p.cap2 == 0.f) {
        // (a score past 2^23 has no room for what its product with C is rounded by)
        top = largest(s, false);
        if (__ballot(!(__builtin_fabsf(top * p.C) < 0x1p23f)) == 0) way = 1;
      } else if (simple) {
        top = largest(s, true);
        if (__ballot(!(top <= p.small)) == 0) way = __ballot(!(top <= p.smaller)) == 0 ? 3 : 2;
      }
      // (an if without an else, in which the scores change where they are: else they are copied for it,
      // in all ways)
      if (way) top = way == 1 ? top * p.C : small_cap(p, top);
      if (!way) {
        if (p.cap2 != 0.f) {
#pragma unroll
          for (int x = 0; x < X; ++x)
#pragma unroll
            for (int j = 0; j < 16; ++j) s[x][j] = capped_score(s[x][j] * p.C, p.cap2, p.inv_cap2);
        } else {
#pragma unroll
          for (int x = 0; x < X; ++x)
#pragma unroll
            for (int j = 0; j < 16; ++j) s[x][j] *= p.C;
        }
        if (a.scores.slopes) {
          const float away = (float)(pos - key0 - 4 * h);
#pragma unroll
          for (int x = 0; x < X; ++x)
#pragma unroll
            for (int j = 0; j < 16; ++j)
              s[x][j] = __builtin_fmaf(-slope, __builtin_fabsf(away - (float)(32 * x + 8 * (j >> 2) + (j & 3))), s[x][j]);
        }
        if (edge) {
          const int rel = key0 + 4 * h - lo;
          const uint32_t span = (uint32_t)(hi - lo);
#pragma unroll
          for (int x = 0; x < X; ++x)
#pragma unroll
            for (int j = 0; j < 16; ++j)
              s[x][j] = (uint32_t)(rel + 32 * x + 8 * (j >> 2) + (j & 3)) < span ? s[x][j] : kNegInf;
        }
        top = largest(s, false);
      }
      // (the lane's own half of the row, or what no score of it is above: enough to know that m stays)
      if (__ballot(top - m > kUp<BF>)) {
        if (way > 1) top = small_cap(p, largest(s, false));
        top = __builtin_fmaxf(top, other_half(top));
        const bool over = top - m > kUp<BF>;
        // (scores past 2^23 have no room for kUp: their weights are 1 at most, and m does not fall after
        // those that do)
        const float to = over ? (__builtin_fabsf(top) < 0x1p23f ? top - (kUp<BF> - 4.f) : __builtin_fmaxf(top, m)) : m;
        // (not 0: an infinite sum stays what it is)
        const float keep = __builtin_fmaxf(exp2_fast(m - (to == kNegInf ? 0.f : to)), 0x1p-126f);
        m = to;
        l *= keep;
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) o[i][j] *= keep;
      }
      const float base = m == kNegInf ? 0.f : m;
      // eight scores at a time, one step of all of them after the other: a result is not there for the
      // next instruction, and left to itself the compiler would take it in the next but one
      auto weigh = [&](auto... steps) {
#pragma unroll
        for (int x = 0; x < X; ++x)
#pragma unroll
          for (int j0 = 0; j0 < 16; j0 += 8) {
            float u[8], f[8];
            auto all = [&](auto step) {
#pragma unroll
              for (int j = 0; j < 8; ++j) step(s[x][j0 + j], u[j], f[j]);
              __builtin_amdgcn_sched_barrier(0);
            };
            (all(steps), ...);
            all([](float, float &, float &e) { e = exp2_fast(e); });
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              w[2 * x + (j0 >> 3)][j >> 1] = pack<BF>(f[j], f[j + 1]);
              u[j] = f[j] + f[j + 1];
            }
            l += (u[0] + u[2]) + (u[4] + u[6]);
          }
      };
      auto square = [](float y, float &u, float &) { u = y * y; };
      auto less_base = [&](float y, float &, float &f) { f = __builtin_fmaf(y, f, -base); };
      if (way == 1)
        weigh([&](float y, float &, float &f) { f = __builtin_fmaf(y, p.C, -base); });
      else if (way == 2)
        weigh(square, [&](float, float &u, float &f) { f = __builtin_fmaf(u, p.cap[4], p.cap[3]); },
              [&](float, float &u, float &f) { f = __builtin_fmaf(u, f, p.cap[2]); },
              [&](float, float &u, float &f) { f = __builtin_fmaf(u, f, p.cap[1]); },
              [&](float, float &u, float &f) { f = __builtin_fmaf(u, f, p.cap[0]); }, less_base);
      else if (way == 3)
        weigh(square, [&](float, float &u, float &f) { f = __builtin_fmaf(u, p.cap3[2], p.cap3[1]); },
              [&](float, float &u, float &f) { f = __builtin_fmaf(u, f, p.cap3[0]); }, less_base);
      else
        weigh([&](float y, float &, float &f) { f = y - base; });

    }
    have = need;
    arrived();
    barrier();
    bring();
  }
  if (have) {
    multiply(keys_end, both_end);
    gather_odd(t1 - 1);
  }
  arrived();

  // An infinity or NaN among the values has reached all rows of the waves that multiplied it, by a
  // weight of 0 too: then once more, with care.
  if (careful) break;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < DB; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) sum = __builtin_fmaf(o[i][j], 0.f, sum);
  const bool odd = __ballot(sum != 0.f) != 0;
  odd_tile[0][wave] = odd;
  barrier();
  int any = 0;
#pragma unroll
  for (int x = 0; x < NW; ++x) any |= odd_tile[0][x];
  if (!uniform(any)) break;
  barrier();
  careful = true;
  }

  l += other_half(l);
  if (p.parts > 1) {
    float *piece = p.piece + (((int64_t)unit * a.kv_heads + head) * p.parts + blockIdx.y) * piece_floats<D>(S::R);
    const int r = wave * 32 + (lane & 31);
    if (!active) return;
    piece[S::R * D + r] = m;
    piece[S::R * (D + 1) + r] = l;
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<float4 *>(piece + r * D + 32 * i + 2 * j + 4 * h) =
            make_float4(o[i][j], o[i][j + 1], o[i][j + 2], o[i][j + 3]);
    return;
  }
  if (!active) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t *out = a.out + ((int64_t)(seq.q0 + token) * a.q_heads + qh) * D;
#pragma unroll
  for (int i = 0; i < DB; ++i)
#pragma unroll
    for (int j = 0; j < 16; j += 4)
      *reinterpret_cast<uint2 *>(out + 32 * i + 2 * j + 4 * h) =
          make_uint2(pack<BF>(o[i][j] * inv, o[i][j + 1] * inv), pack<BF>(o[i][j + 2] * inv, o[i][j + 3] * inv));
  if (a.scores.lse && h == 0)
    a.scores.lse[(int64_t)(seq.q0 + token) * a.q_heads + qh] = log_scaled(m, l);
}

// Joins the parts of a tile's keys: four values of a row a thread, the parts in order
template <bool BF, int D, int R>
__global__ __launch_bounds__(256) void prompt_join_kernel(Params p) {
  const PromptArgs &a = p.a;
  const int head = blockIdx.x % (unsigned)a.kv_heads, unit = blockIdx.x / (unsigned)a.kv_heads;
  int b, tile;
  if (!find_tile<R>(a, p.group, unit, b, tile)) return;
  const Sequence seq = sequence(a, b);
  const int item = blockIdx.y * 256 + threadIdx.x, r = item / (D / 4), d = item % (D / 4) * 4;
  const int row = tile * R + r;
  if (r >= R || row >= seq.n * p.group) return;
  const float *piece = p.piece + ((int64_t)unit * a.kv_heads + head) * p.parts * piece_floats<D>(R);
  float m = kNegInf, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < p.parts; i0 += 8) {
    float4 v[8];
    float pm[8], pl[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float *src = piece + (int64_t)(i0 + x < p.parts ? i0 + x : i0) * piece_floats<D>(R);
      v[x] = *reinterpret_cast<const float4 *>(src + r * D + d);
      pm[x] = src[R * D + r];
      pl[x] = src[R * (D + 1) + r];
    }
#pragma unroll
    for (int x = 0; x < 8; ++x)
      if (i0 + x < p.parts) {
        const float top = __builtin_fmaxf(m, pm[x]), base = top == kNegInf ? 0.f : top;
        const float f = __builtin_fmaxf(exp2_fast(m - base), 0x1p-126f), g = __builtin_fmaxf(exp2_fast(pm[x] - base), 0x1p-126f);
        m = top;
        l = l * f + pl[x] * g;
        acc.x = acc.x * f + v[x].x * g, acc.y = acc.y * f + v[x].y * g;
        acc.z = acc.z * f + v[x].z * g, acc.w = acc.w * f + v[x].w * g;
      }
  }
  const int token = row / p.group, qh = head * p.group + row - token * p.group;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = (int64_t)(seq.q0 + token) * a.q_heads + qh;
  *reinterpret_cast<uint2 *>(a.out + at * D + d) =
      make_uint2(pack<BF>(acc.x * inv, acc.y * inv), pack<BF>(acc.z * inv, acc.w * inv));
  if (a.scores.lse && d == 0)
    a.scores.lse[at] = log_scaled(m, l);
}

// How a call is cut: waves of a workgroup, tiles of rows at most, and parts of every tile's keys
struct Cut { int waves, tiles, parts; };
Cut cut_for(int64_t Tq, int64_t Tk, int64_t B, int q_heads, int kv_heads, int D) {
  const int group = q_heads / kv_heads;
  Cut c;
  c.waves = Tq * group <= 64 * B ? 2 : 4;
  const int R = 32 * c.waves;
  c.tiles = (int)(Tq * group / R + B);
  // parts of at least 512 keys, as long as the chip is not full and pieces fit 64 MiB
  const int64_t wgs = (int64_t)c.tiles * kv_heads, room = ((int64_t)64 << 20) / ((int64_t)R * (D + 2) * 4);
  int64_t parts = (int64_t)device_cus() * (c.waves == 2 ? 4 : 1) / wgs;
  const int64_t keys = (Tk + B - 1) / B / 512;
  if (parts > keys) parts = keys;
  if (parts > room / wgs) parts = room / wgs;
  if (parts > kMaxParts) parts = kMaxParts;
  c.parts = parts < 2 ? 1 : (int)parts;
  return c;
}

// tanh y / y = sum c_i y^2i: five terms within 2^-23 for |y| <= 0.6, three for |y| <= 0.2 (fits of
// the least largest relative error).  So the cap of a small score costs five operations or three and no
// exponential or reciprocal, which take twice as long each: the softmax is the longer half of a tile
// (8192 tokens, cap 50: 754 us with them, 718 without, at that step).
void set_cap(Params &p) {
  constexpr double c3[3] = {0.999999894791025, -0.33328590894235166, 0.1301540743838377};
  p.inv_cap2 = 0.f, p.small = p.smaller = -1.f;
  for (float &x : p.cap) x = 0.f;
  for (float &x : p.cap3) x = 0.f;
  if (p.cap2 == 0.f) return;
  p.inv_cap2 = 1.f / p.cap2;
  const double y = (double)p.C / p.cap2, small = 0.6 / y;
  // (powers of scores are within binary32, and what is small has room for its rounding)
  if (!(small > 1e-3 && small < 1e9 && small * p.C < 0x1p22)) return;
  double f = p.C;
  for (int i = 0; i < 5; ++i, f *= y * y) {
    p.cap[i] = (float)(kTanhTerms[i] * f);
    if (i < 3) p.cap3[i] = (float)(c3[i] * f);
  }
  // (the terms hold powers of y up to y^8: where one is no normal number of binary32 it has lost bits,
  // or all of them, that scores near the cap would need.  With heads of 128 and the usual scale caps of
  // up to 2000 have normal terms)
  for (float x : p.cap)
    if (!(__builtin_fabsf(x) >= 0x1p-126f)) return;
  for (float x : p.cap3)
    if (!(__builtin_fabsf(x) >= 0x1p-126f)) return;
  p.small = (float)small;
  p.smaller = (float)(0.2 / y);
}

template <bool BF, int D, int NW>
hipError_t launch(const Params &p, hipStream_t s) {
  using S = Shape<BF, D, NW>;
  const unsigned wgs = (unsigned)p.tiles * (unsigned)p.a.kv_heads;
  hipLaunchKernelGGL((prompt_kernel<BF, D, NW>), dim3(wgs, p.parts), dim3(S::THREADS), 0, s, p);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || p.parts == 1) return err;
  hipLaunchKernelGGL((prompt_join_kernel<BF, D, S::R>), dim3(wgs, S::R * D / 4 / 256), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

int64_t prompt_workspace_bytes(int64_t Tq, int64_t Tk, int64_t B, int q_heads, int kv_heads, int D) {
  const Cut c = cut_for(Tq, Tk, B, q_heads, kv_heads, D);
  return c.parts == 1 ? 16 : (int64_t)c.tiles * kv_heads * c.parts * 32 * c.waves * (D + 2) * 4;
}

hipError_t launch_prompt_attention(const PromptArgs &a, hipStream_t s) {
  Params p;
  p.a = a;
  p.C = __builtin_fabsf(a.scale) * kLog2e;
  p.flip = a.scale < 0.f ? 0x80008000u : 0u;
  p.cap2 = a.scores.softcap * kLog2e;
  set_cap(p);
  p.window = a.scores.window > 0 && a.scores.window < (1 << 25) ? a.scores.window : 1 << 25;
  p.group = a.q_heads / a.kv_heads;
  const Cut c = cut_for(a.Tq, a.Tk, a.B, a.q_heads, a.kv_heads, a.head_dim);
  p.tiles = c.tiles;
  p.parts = c.parts;
  p.piece = reinterpret_cast<float *>(a.workspace);
#define AQ_W(B, D)                                                     \
  if (a.head_dim == D)                                                 \
    return c.waves == 2 ? launch<B, D, 2>(p, s) : launch<B, D, 4>(p, s);
#define AQ_D(B) AQ_W(B, 64) AQ_W(B, 128) AQ_W(B, 256)
  if (a.x_dtype == X_BF16) { AQ_D(true) } else { AQ_D(false) }
#undef AQ_D
#undef AQ_W
  return hipErrorInvalidValue;
}

}  // namespace aq
