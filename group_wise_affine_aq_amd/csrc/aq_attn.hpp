// aq_attn.hpp -- attention of each sequence's newest tokens over the paged,
// quantized key-value cache (gfx950): the kernels, which aq_attn.hip builds for
// plain scores and aq_attn_masked.hip for capped, biased and masked ones.
//
//   out = sum_t p_t v_t,  p = softmax_t(scale * q . k_t),  t <= len - L + i
//
// in one pass over the tokens with the running maximum m and sum l of the
// softmax: a tile of tokens with largest score m' > m rescales what was summed
// by exp(m - m') and adds exp(s - m').  The codes are never expanded into
// memory; with k = s code + b in each group g of G values of a row
//
//   q . k_t = sum_g s_tg (sum_{d in g} q_d code_td) + b_tg (sum_{d in g} q_d)
//   sum_t p_t v_td = sum_t (p_t s_tg) code_td + p_t b_tg,
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
//    one byte permute (8 bits) or a shift and a mask (4 bits, 16 times too
//    large) per pair.  2^24 or 2^20 goes into factors that are there anyway.
//    The sums of the matrix cores lose what lies some 24 bits below the
//    exponent an operand is written with, 2^-14 for all of these: codes of 4
//    bits in the lowest bits lost 2^-18 of their sums, two to four times the
//    rounding of an fp16 result that averages 60000 to 120000 tokens.
//  * bf16 queries become fp16, scaled by a power of two per row so that the
//    largest lies in [256, 512): exact down to 2^-22 of it.  fp16 queries are
//    taken as they are.
//  * A weight p s goes into the second product in two fp16 parts, rounded and
//    rest (two bf16 parts where the pages hold bf16), two products a tile.  (In
//    one part it would be off by 2^-12 at the mean, as much as an fp16 result's
//    own rounding: 1.1 to 1.7 times the error.)  Weights are as large as fp16
//    allows beside the scales of their tile: the exponent m that they are taken
//    from is not the largest score but up to 30 less, so that the largest weight
//    times the largest scale lies between 2^11 and 2^16, and down to 2^-35 of
//    that everything counts; o, l and the biases' sums have the same factor.
//    (With the factor that any scale allows, 2^6 at 8 bits, weights below 2^-25
//    were lost at scales of 0.02: of thousands of tokens beside one that takes
//    all but 2^-12 of the softmax, what they add to the result.)
//  * bits = 16: the pages' values are the operands.
//
// Work division.  The tokens of all units -- a unit is one sequence, one key
// head and one slice of at most 32 (heads of 256: 16) of its query rows -- form one line of
// 32-token tiles that the workgroups cut evenly, so a batch of ragged lengths
// and one long sequence load the chip alike and the launch does not depend on
// the lengths, which stay on the device.  The four waves of a workgroup take
// every fourth tile of its part; their (m, l, o) are joined through LDS.  A
// part that does not cover its unit is a piece in the workspace; the pieces
// are joined by the workgroup that finishes last among them or, where they may
// be many, by a second launch, in the pieces' order either way, so results do
// not depend on timing.
//
// Bound: HBM, the codes, scales and biases read once.  At 8 bits a tile of 32
// tokens x 128 values (groups of 64, one tile of query rows) is 8.7 KB and
// costs a wave about 245 vector and 24 matrix instructions (4 bits: 4.6 KB,
// 320); eight waves a CU could take 35 bytes a clock at that rate where HBM
// gives a CU about 9.  64 sequences of up to 16384 tokens (1.01 GB) take 185
// to 190 us, 5.4 TB/s; a large copy reaches 5.2, a large read 6.3.  Below about 100 MB
// what surrounds the stream shows: lengths, page ids and first codes are three
// loads that wait for each other (5 us to the first score), and joining pieces
// is three more (5 us): 16 sequences of up to 4096 tokens (71 MB) 19.0 us.
// (Figures in pairs, here and below, compare two variants at the step at which
// one was taken, not this code with one.)
#pragma once

#include "aq_device.hpp"
#include "aq_internal.hpp"

namespace aq {
namespace {

typedef _Float16 f16x8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2v __attribute__((ext_vector_type(2)));

constexpr int kTile = 32;         // tokens a wave takes at a time
constexpr int NW = 4;             // waves of a workgroup
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
  float *parts;  // two pieces per place of the work line
  int inside;    // pieces are joined by the workgroup that finishes a unit's last, else by
                 // attn_join_kernel
  uint32_t *arrived;  // inside: per place, pieces there of the unit that starts in its last piece;
                      // zero between calls
  uint2 *cuts;   // else: per unit, its pieces, 0 if it was not cut, and the first one's place
  int64_t max_pages, num_pages;
  uint32_t page_subs, page_magic;  // page_size / 16 and floor(2^32 / that) + 1
  int kv_heads, group, L, B, slices, x_dtype;
  uint32_t chunk;  // tokens of the work line's chunks, at least
  float scale;
  // MORE: scores s become cap2 tanh(s inv_cap2) (in powers of two; cap2 0: as
  // they are), less slopes[query head] times the distance to their token; a row
  // sees the last `window` tokens up to its own, from first[b] on; lse gets the
  // logarithm of each row's sum of weights.  Null pointers: none.
  float cap2, inv_cap2;
  int window;
  const float *slopes;
  const int32_t *first;
  float *lse;
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

// MORE: the first token that a row which sees the tokens before `vis` sees, and
// the tile that a sequence's oldest new token begins with (the last tile where
// it begins past the end: every sequence with tokens has a tile, which writes
// its rows)
__device__ __forceinline__ int first_seen(const Params &p, int first, int vis) {
  const int from = vis - p.window;
  return from > first ? from : first;
}
__device__ __forceinline__ int first_of(const Params &p, int b) {
  const int f = p.first ? p.first[b] : 0;
  return f < 0 ? 0 : f;
}
template <bool MORE>
__device__ __forceinline__ int first_tile(const Params &p, int b, int len) {
  if constexpr (!MORE) return 0;
  const int from = first_seen(p, first_of(p, b), len - p.L + 1);
  return (from < len ? from : (len > 0 ? len - 1 : 0)) / kTile;
}

// One piece in the workspace: the results of 16 NT columns, D floats each, then
// the columns' m and l.  Where a unit's pieces are joined inside the launch
// they are read by other workgroups than wrote them, on other XCDs with L2s of
// their own: stores and loads go past the L2s (sc1, the cache policy of device
// scope), and a workgroup counts as arrived when its stores are done.
// (Ordinary stores with a device-wide fence write back and drop whole L2s: 118
// against 37 us for 16 sequences of up to 4096 tokens, 8 bits, at that step.)
constexpr int kDeviceScope = 16;
constexpr int kMaxGrid = 1024;  // of counters, and of records of units, in the workspace
constexpr int piece_floats(int D, int NT) { return NT * (16 * D + 32); }

__device__ __forceinline__ void put_piece(Span to, int at, f32x4v v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4v, v), to, at * 4, 0, kDeviceScope);
}
__device__ __forceinline__ void put_piece1(Span to, int at, float v) {
  __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), to, at * 4, 0, kDeviceScope);
}
__device__ __forceinline__ f32x4v get_piece(Span from, int at) {
  return __builtin_bit_cast(f32x4v, __builtin_amdgcn_raw_buffer_load_b128(from, at * 4, 0, kDeviceScope));
}
__device__ __forceinline__ float get_piece1(Span from, int at) {
  const uint32_t u = __builtin_amdgcn_raw_buffer_load_b32(from, at * 4, 0, kDeviceScope);
  return __builtin_bit_cast(float, u);
}

// ---- the work line ------------------------------------------------------------------
// All tiles of all units in one line, sequences first, cut evenly.  A workgroup
// whose part begins in one unit and ends in another waits twice for first loads
// (about 5 us), so the line is counted in chunks that do not cross units, as
// many as there are workgroups at most, as long as they need not be more than
// 20 tiles larger than an even cut in single tiles.  (Cut evenly against in
// chunks: 26.9 and 21.9 us for 16 sequences of up to 4096 tokens, 8 bits; 50.1
// and 44.9 with 40 rows a key head; 59.1 and 53.6 at 16 bits; 195 and 196 for
// 64 sequences, whose parts are long.  4, 10 and 20 tiles measured the same.)

template <bool MORE>
struct Line {
  uint32_t rows;      // units per sequence
  uint32_t chunk;     // tokens
  // places, each a workgroup's: place w has share chunks, one more if w < longer
  uint32_t grid, share, longer;
  int per;            // sequences per lane
  uint32_t mine, upto;  // chunks (of one unit) of this lane's sequences, and up to them
  bool idle;          // this lane has a sequence without tokens

  // of a sequence, from its first tile on
  __device__ __forceinline__ uint32_t chunks(const Params &p, int b, uint32_t len) const {
    if constexpr (MORE) len -= first_tile<MORE>(p, b, (int)len) * kTile;
    return (len + chunk - 1) / chunk;
  }

  int len;            // its first sequence's length

  __device__ __forceinline__ uint32_t count(const Params &p, int lane) {
    const int lo = lane * per < p.B ? lane * per : p.B, hi = lo + per < p.B ? lo + per : p.B;
    mine = lo < hi ? chunks(p, lo, len) : 0;
    for (int b = lo + 1; b < hi; ++b) mine += chunks(p, b, clamped_length(p, b));
    upto = lanes_prefix(mine);
    return (uint32_t)uniform(__builtin_amdgcn_readlane(upto, 63)) * rows;
  }

  // `most`: workgroups there are
  __device__ __forceinline__ Line(const Params &p, uint32_t most, int lane) {
    rows = p.kv_heads * p.slices;
    per = (p.B + 63) / 64;
    const int lo = lane * per < p.B ? lane * per : p.B, hi = lo + per < p.B ? lo + per : p.B;
    len = lo < hi ? clamped_length(p, lo) : 1;
    idle = len == 0;
    for (int b = lo + 1; b < hi; ++b) idle |= clamped_length(p, b) == 0;
    chunk = p.chunk;
    uint32_t total = count(p, lane);
    if (chunk == kTile && rows * p.B <= most && total) {  // (no chunks of no tokens)
      const uint32_t even = (total + NW * most - 1) / (NW * most) * NW;
#pragma unroll 1
      for (uint32_t more = 0; more <= 20 && chunk == kTile; more += NW) {
        chunk = (even + more) * kTile;
        const uint32_t n = count(p, lane);
        if (n <= most)
          total = n;
        else
          chunk = kTile;
      }
      if (chunk == kTile) total = count(p, lane);
    }
    grid = total < most ? total : most;
    share = grid ? total / grid : 0;
    longer = total - share * grid;
  }

  __device__ __forceinline__ uint32_t begin(uint32_t w) const {
    return w * share + (w < longer ? w : longer);
  }
  // the place that has chunk `at`
  __device__ __forceinline__ uint32_t owner(uint32_t at) const {
    if (share == 1 && longer == 0) return at;
    const uint32_t first = longer * (share + 1);
    return at < first ? at / (share + 1) : longer + (at - first) / share;
  }
};

// N words moved as one, whatever they are otherwise accessed as
template <int N>
struct __attribute__((may_alias, aligned(N >= 4 ? 16 : 4 * N))) words { uint32_t w[N]; };
typedef uint16_t __attribute__((may_alias)) u16_any;

// ---- one wave's state over a segment of tokens -------------------------------------
// BITS 4, 8 or 16; BF: operands are bf16 (bits = 16 with a bf16 cache); G is
// head_dim for 16 bits.
template <int BITS, bool BF, int D, int G, int NT, bool MORE>
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
  static constexpr float UNIT = BITS == 4 ? 0x1p20f : 0x1p24f;  // 1 / what a code of 1 enters as

  struct Keys { uint32_t c[2][KW]; };
  struct Values { uint32_t c[8][NG][VW]; };
  // Scales and biases of a tile are fetched once: lane 16 a + t has array a
  // (K scales, K biases, V scales, V biases), token t of each 16.  Through a
  // strip of LDS of the wave's own every lane then gets those of its four
  // tokens.  (Every lane fetching its own: 32 registers for the time that
  // loads are under way instead of 2, and twice the codes' bytes through the
  // load path.)
  static constexpr int TB = NG * 2;            // bytes per token and array
  static constexpr int RW = TB < 4 ? 1 : TB / 4;
  struct Raw { uint32_t w[2][RW]; };
  struct Scales { uint32_t s[2][SW], b[2][SW]; };

  u32x4v q[NT][KS];
  float qsum[NT][NG], C[NT];
  int vis[NT];      // tokens the column sees (MORE: from `from` on)
  int from[MORE ? NT : 1];
  float slope[MORE ? NT : 1];
  // sums of 2^(t - m) over the scores t, alone and times biases and values
  float m[NT], l[NT], bacc[NT][NG];
  f32x4v o[NT][NG][VN];

  // The 16 tokens at rows[sub]; there[sub]: whether their page is (if not, zero
  // codes and the first row's scales, which edge tiles do not use)
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
    }
  }

  // the lane's array, from its token on; without bias arrays every bias is +0
  // (something is fetched all the same)
  static __device__ __forceinline__ const char *scales_of(const Params &p, int lane, bool &none) {
    const int a = lane >> 4;
    const void *s = a & 2 ? p.vs : p.ks, *b = a & 2 ? p.vb : p.kb;
    none = (a & 1) && !b;
    return reinterpret_cast<const char *>((a & 1) && b ? b : s) + (lane & 15) * TB;
  }
  static __device__ __forceinline__ void load_scales(Raw &r, const char *from, const int64_t *rows) {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const char *at = from + rows[sub] * TB;
      if constexpr (TB == 2) {
        r.w[sub][0] = *reinterpret_cast<const uint16_t *>(at);
      } else {
        const words<RW> x = *reinterpret_cast<const words<RW> *>(at);
#pragma unroll
        for (int i = 0; i < RW; ++i) r.w[sub][i] = x.w[i];
      }
    }
  }
  static __device__ __forceinline__ void share_scales(const Raw &r, char *strip, int lane, bool none) {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      char *at = strip + (sub * 64 + lane) * TB;
      if constexpr (TB == 2) {
        *reinterpret_cast<u16_any *>(at) = none ? 0 : (uint16_t)r.w[sub][0];
      } else {
        words<RW> x;
#pragma unroll
        for (int i = 0; i < RW; ++i) x.w[i] = none ? 0u : r.w[sub][i];
        *reinterpret_cast<words<RW> *>(at) = x;
      }
    }
  }
  // How large, in powers of two, a weight may be: times the tile's largest
  // scale of values it stays within fp16 (a scale of exponent field e is below
  // 2^(e - 14); infinities and NaN count as the next field).  Scales of tokens
  // that nobody sees do not count.  16 bits: the weight alone.  bf16 has
  // binary32's range for values too: weights stay so small that 4096 of the
  // largest, times the type's largest value, have a finite sum (at up to 2^4,
  // 2500 tokens of 2^121 had none).
  // Tokens since .. len - 1 are those that somebody sees.
  static __device__ __forceinline__ float room(const Raw &r, bool edge, int token, const bool *on,
                                               int since, int len, int lane) {
    if constexpr (!QUANT) return BF ? -12.f : 15.f;
    u16x2v most = {0, 0};
#pragma unroll
    for (int sub = 0; sub < 2; ++sub)
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        uint32_t w = r.w[sub][i] & 0x7FFF7FFFu;
        if (edge) w = on[sub] && (uint32_t)(token + 16 * sub - since + (lane & 15)) < (uint32_t)(len - since) ? w : 0u;
        most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2v, w));
      }
    int top = most[0] > most[1] ? most[0] : most[1];
    auto larger = [](int a, int b) { return a > b ? a : b; };
    top = larger(top, __builtin_amdgcn_update_dpp(0, top, 0x128, 0xF, 0xF, false));  // row_ror:8
    top = larger(top, __builtin_amdgcn_update_dpp(0, top, 0x124, 0xF, 0xF, false));
    top = larger(top, __builtin_amdgcn_update_dpp(0, top, 0x122, 0xF, 0xF, false));
    top = larger(top, __builtin_amdgcn_update_dpp(0, top, 0x121, 0xF, 0xF, false));
    return (float)(30 - (__builtin_amdgcn_readlane(top, 32) >> 10));  // (the lanes of V's scales)
  }

  // arrays a and a + 1 for the lane's four tokens of each 16
  static __device__ __forceinline__ void take_scales(Scales &g, const char *strip, int a, int lane) {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const char *at = strip + ((sub * 4 + a) * 16 + 4 * (lane >> 4)) * TB;
      const words<SW> s = *reinterpret_cast<const words<SW> *>(at);
      const words<SW> b = *reinterpret_cast<const words<SW> *>(at + 16 * TB);
#pragma unroll
      for (int i = 0; i < SW; ++i) g.s[sub][i] = s.w[i], g.b[sub][i] = b.w[i];
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
    } else {  // codes 0,4 | 1,5 | 2,6 | 3,7, 16 times too large
      const uint32_t a = c[s];
      return u32x4v{a << 4 & 0x00F000F0u, a & 0x00F000F0u, a >> 4 & 0x00F000F0u, a >> 8 & 0x00F000F0u};
    }
  }

  // the operand of value n of group g: the lane's 8 tokens
  static __device__ __forceinline__ u32x4v value_operand(const Values &v, int g, int n, uint32_t halves) {
    u32x4v a;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t *x = v.c[2 * w][g], *y = v.c[2 * w + 1][g];
      if constexpr (BITS == 16) {
        a[w] = __builtin_amdgcn_perm(y[n >> 1], x[n >> 1], halves + (n & 1) * 0x02020202u);
      } else if constexpr (BITS == 8) {
        const uint32_t k = n & 3;
        a[w] = __builtin_amdgcn_perm(y[n >> 2], x[n >> 2], 0x0C000C00u | k | (4 + k) << 16);
      } else {
        const uint32_t k = n >> 1;
        const uint32_t both = __builtin_amdgcn_perm(y[0], x[0], 0x0C000C00u | k | (4 + k) << 16);
        a[w] = (n & 1 ? both : both << 4) & 0x00F000F0u;
      }
    }
    return a;
  }

  // queries of rows slice*16*NT .. of (b, head), the columns of this lane:
  // fetched first, made into operands when the keys are on their way
  struct Queries { uint4 raw[NT][KS]; };
  __device__ __forceinline__ void load_queries(Queries &qs, const Params &p, int b, int head,
                                               int slice, int len, int lane) {
    const int h = lane >> 4, cols = p.L * p.group;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = (slice * NT + nt) * 16 + (lane & 15);
      const bool on = r < cols;
      const int rr = on ? r : 0, i = rr / p.group, j = rr - i * p.group;
      vis[nt] = on ? len - p.L + 1 + i : 0;
      if constexpr (MORE) {
        from[nt] = first_seen(p, first_of(p, b), vis[nt]);
        slope[nt] = p.slopes ? p.slopes[head * p.group + j] * 1.44269504088896341f : 0.f;
      }
      const uint16_t *src = reinterpret_cast<const uint16_t *>(p.q) +
                            ((int64_t)b * p.L + i) * p.q_stride +
                            (int64_t)(head * p.group + j) * D;
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
        qs.raw[nt][s] = *reinterpret_cast<const uint4 *>(src + d);
      }
    }
  }
  // (columns past the last hold the first row's queries: never written out)
  __device__ __forceinline__ void start(const Queries &qs, const Params &p) {
    const float log2s = p.scale * 1.44269504088896341f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (!QUANT) {
        C[nt] = log2s;
#pragma unroll
        for (int s = 0; s < KS; ++s)
          q[nt][s] = u32x4v{qs.raw[nt][s].x, qs.raw[nt][s].y, qs.raw[nt][s].z, qs.raw[nt][s].w};
        continue;
      }
      if (p.x_dtype == X_F16) {
        C[nt] = log2s * UNIT;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint32_t u[4] = {qs.raw[nt][s].x, qs.raw[nt][s].y, qs.raw[nt][s].z, qs.raw[nt][s].w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if constexpr (BITS == 8) {
              q[nt][s][w] = u[w];
            } else {  // queries w and w + 4
              q[nt][s][w] = __builtin_amdgcn_perm(u[2 + (w >> 1)], u[w >> 1],
                                                  w & 1 ? 0x07060302u : 0x05040100u);
            }
          }
        }
      } else {
        float x[KS][8], top = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint32_t u[4] = {qs.raw[nt][s].x, qs.raw[nt][s].y, qs.raw[nt][s].z, qs.raw[nt][s].w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[s][e] = __builtin_bit_cast(float, e & 1 ? u[e >> 1] & 0xFFFF0000u : u[e >> 1] << 16);
            top = __builtin_fmaxf(top, __builtin_fabsf(x[s][e]));
          }
        }
        top = quarters_max(top);
        int e = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127;
        e = e < -100 ? -100 : (e > 127 ? 127 : e);
        const float down = __builtin_ldexpf(1.f, 8 - e);
        // (a factor past binary32's range may be any smaller one: scores that
        // differ at all are then more than 2^20 apart either way)
        C[nt] = __builtin_amdgcn_fmed3f(__builtin_ldexpf(log2s * UNIT, e - 8), -0x1p127f, 0x1p127f);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if constexpr (BITS == 8) {
              q[nt][s][w] = pack_f16(x[s][2 * w] * down, x[s][2 * w + 1] * down);
            } else {
              q[nt][s][w] = pack_f16(x[s][w] * down, x[s][w + 4] * down);
            }
          }
      }
      // a group's sum, in the units of the scores of codes: a product with ones
      // (not with codes of 1, whose exponent is written as 2^-14: at 8 bits the
      // matrix cores lost all of the sum below 2^-14 of the largest query, and
      // the biases of keys, by which it is multiplied, may be large)
      constexpr uint32_t kOnes = 0x3C003C00u;
      const u32x4v ones = {kOnes, kOnes, kOnes, kOnes};
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        f32x4v sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NKS; ++k) sum = mfma<BF>(ones, q[nt][g * NKS + k], sum);
        qsum[nt][g] = sum[0] * (1.f / UNIT);
      }
    }
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
  __device__ __forceinline__ void scores(const Params &p, const Keys &k, const Scales &ks,
                                         float (&t)[NT][8], int token, int h) const {
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
              x = __builtin_fmaf(scale_at(ks.s[sub], i, g), acc[nt][g][i], x);
              x = __builtin_fmaf(scale_at(ks.b[sub], i, g), qsum[nt][g], x);
            }
          } else {
            x = acc[nt][0][i];
          }
          t[nt][4 * sub + i] = x * C[nt];
        }
    }
    if constexpr (MORE) {
      if (p.cap2 != 0.f)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 8; ++j) t[nt][j] = capped_score(t[nt][j], p.cap2, p.inv_cap2);
      if (p.slopes)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int away = vis[nt] - 1 - (token + 16 * (j >> 2) + 4 * h + (j & 3));
            t[nt][j] = __builtin_fmaf(-slope[nt], (float)away, t[nt][j]);
          }
    }
  }

  // The weights 2^(t - m) of the scores t, at most 2^up each: where one would be
  // larger, m moves up to 4 short of that, so that it seldom moves again, and
  // what was summed is rescaled.  (Scores past 2^23 have no room for up: their
  // weights are 1 at most, and m does not fall after those that do.)
  __device__ __forceinline__ void weigh(float (&t)[NT][8], float up) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top = t[nt][0];
#pragma unroll
      for (int j = 1; j < 8; ++j) top = __builtin_fmaxf(top, t[nt][j]);
      top = quarters_max(top);
      const bool over = top - m[nt] > up;
      if (__ballot(over)) {
        const float to = over ? (__builtin_fabsf(top) < 0x1p23f ? top - (up - 4.f) : __builtin_fmaxf(top, m[nt])) : m[nt];
        const float keep = exp2_fast(m[nt] - (to == kNegInf ? 0.f : to));
        m[nt] = to;
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
      const float base = m[nt] == kNegInf ? 0.f : m[nt];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        t[nt][j] = exp2_fast(t[nt][j] - base);
        l[nt] += t[nt][j];
      }
    }
  }

  // o += weights x values, the weights in two parts.  At 16 bits the first is
  // rounded down and the second is the least positive number at least, so that
  // an infinite value stays what it is (0 * inf or inf - inf would be NaN; a
  // weight not seen adds the least number times a value of 0).  SOME: only in the columns
  // that see `sees` tokens, from the halves of the values that `keep` has
  template <bool SOME = false>
  __device__ __forceinline__ void gather(const Values &v, const Scales &vs, const float (&p)[NT][8],
                                         int sees = 0, u32x4v keep = {}) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      // (opaque, or the operands of all passes are made, and kept, ahead of them)
      uint32_t halves = 0x05040100u;
      if constexpr (SOME) asm volatile("" : "+s"(halves));
      u32x4v w[NT], w2[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (QUANT) {
          uint32_t scale[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) scale[j] = vs.s[j >> 2][((j & 3) * NG + g) >> 1];
          if constexpr (NG == 1)
            w[nt] = scaled_weights<0, 1>(p[nt], scale);
          else if (g & 1)
            w[nt] = scaled_weights<1, 1>(p[nt], scale);
          else
            w[nt] = scaled_weights<0, 0>(p[nt], scale);
          float rest[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            rest[j] = __builtin_fmaf(p[nt][j], scale_at(vs.s[j >> 2], j & 3, g),
                                     -half_at(w[nt][j >> 1], j & 1));
            bacc[nt][g] = __builtin_fmaf(p[nt][j], scale_at(vs.b[j >> 2], j & 3, g), bacc[nt][g]);
          }
#pragma unroll
          for (int j = 0; j < 8; j += 2) w2[nt][j >> 1] = pack_f16(rest[j], rest[j + 1]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const float a = p[nt][j], b = p[nt][j + 1];
            if constexpr (BF) {
              const uint32_t ua = __builtin_bit_cast(uint32_t, a), ub = __builtin_bit_cast(uint32_t, b);
              w[nt][j >> 1] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
              const float ra = a - __builtin_bit_cast(float, ua & 0xFFFF0000u);
              const float rb = b - __builtin_bit_cast(float, ub & 0xFFFF0000u);
              w2[nt][j >> 1] = pack_bf16(__builtin_fmaxf(ra, 0x1p-126f), __builtin_fmaxf(rb, 0x1p-126f));
            } else {
              const uint32_t r = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
              w[nt][j >> 1] = r;
              w2[nt][j >> 1] = pack_f16(__builtin_fmaxf(a - half_at(r, 0), 0x1p-24f),
                                        __builtin_fmaxf(b - half_at(r, 1), 0x1p-24f));
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < VN; ++n) {
        u32x4v a = value_operand(v, g, n, halves);
        if constexpr (SOME) a &= keep;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (SOME) {
            f32x4v y = {0.f, 0.f, 0.f, 0.f};
            y = mfma<BF>(a, w[nt], y);
            y = mfma<BF>(a, w2[nt], y);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nt][g][n][i] += vis[nt] == sees ? y[i] : 0.f;
          } else {
            o[nt][g][n] = mfma<BF>(a, w[nt], o[nt][g][n]);
            o[nt][g][n] = mfma<BF>(a, w2[nt], o[nt][g][n]);
          }
        }
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
        if (!on[j >> 2] || at >= vis[nt] || (MORE && at < from[nt])) t[nt][j] = kNegInf;
      }
  }

  // The values of tokens a column does not see must not reach it, not even as
  // 0 * NaN.  Quantized values: the codes are finite, so this is a matter of
  // the lane's scales and biases.  Those of tokens past its column become 0;
  // where a lane has two columns, those of tokens past both do, and any that
  // are not finite, whose NaN goes to the columns that see it.
  __device__ __forceinline__ void edge_values(Scales &vs, int token, const bool *on, int h) {
#pragma unroll
    for (int x = 0; x < 2 * SW; ++x) {
      const int sub = x / SW, w = x % SW;
      uint32_t keep = 0;
#pragma unroll
      for (int e = 2 * w; e < 2 * w + 2; ++e) {
        const int g = e % NG, at = token + 16 * sub + 4 * h + e / NG;
        const uint32_t half = e & 1 ? 0xFFFF0000u : 0x0000FFFFu;
        if constexpr (NT == 1) {
          if (on[sub] && at < vis[0] && (!MORE || at >= from[0])) keep |= half;
        } else {
          const float zero = half_at(vs.s[sub][w], e & 1) * 0.f + half_at(vs.b[sub][w], e & 1) * 0.f;
          bool seen = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const bool here = on[sub] && at < vis[nt] && (!MORE || at >= from[nt]);
            seen |= here;
            bacc[nt][g] += here ? zero : 0.f;
          }
          if (seen && zero == 0.f) keep |= half;
        }
      }
      // (opaque, or the words of all tiles are taken apart into halves)
      asm volatile("" : "+v"(keep));
      vs.s[sub][w] &= keep;
      vs.b[sub][w] &= keep;
    }
  }

  // 16 bits: the values themselves may be infinite or NaN, and a lane's values
  // serve every column, so such a tile is taken once per query token: the
  // values past that token's sight are zero, and what the products give the
  // other columns (0 * NaN among it) is dropped, not weighed with 0
  __device__ __forceinline__ void edge_gather(const Values &v, const Scales &vs, const float (&p)[NT][8],
                                              int since, int sees, int token, const bool *on, int h) {
    u32x4v keep;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int at = token + 16 * (w >> 1) + 4 * h + 2 * (w & 1);
      keep[w] = on[w >> 1] && at + 1 < sees ? 0xFFFFFFFFu : (on[w >> 1] && at < sees ? 0x0000FFFFu : 0u);
      if constexpr (MORE) keep[w] &= at >= since ? 0xFFFFFFFFu : (at + 1 >= since ? 0xFFFF0000u : 0u);
    }
    gather<true>(v, vs, p, sees, keep);
  }

  // tiles first, first + NW, ... below end of a sequence: one wave's part
  __device__ __forceinline__ void run(const Params &p, int b, int head, int slice, int len,
                                      int tile0, int end, char *strip) {
    const int lane = lane_here();
    const int least = len - p.L + 1 + (slice * NT * 16) / p.group;  // what every column sees
    // MORE: and from where on; since: what any does
    int first_b = 0, most = 0, since = 0;
    if constexpr (MORE) {
      const int newest = ((slice + 1) * NT * 16 - 1) / p.group;
      first_b = uniform(first_of(p, b));
      since = first_seen(p, first_b, least);
      since = since < len ? since : len;
      most = first_seen(p, first_b, len - p.L + 1 + (newest < p.L ? newest : p.L - 1));
    }
    Keys k;
    Values v;
    Raw raw;
    bool none;
    const char *from = scales_of(p, lane, none);
    uint32_t row_lo, row_hi;  // lane 2 i + sub: the rows of the round's tile i
    int64_t rows[2];
    bool on[2], on_next[2];
    int c0 = tile0, first, tiles;
    // up to 32 tiles' pages at once; lanes without one look up the first.  No
    // branch: where some lanes of a wave leave a branch, the compiler may place
    // copies of any live register ahead of the instruction that turns the other
    // lanes on again, and those lose it.  It did so here in a build of two tiles
    // of columns at heads of 256: lanes lost their thread's number and with it
    // the address of the rows they write.
    auto look_up = [&] {
      first = c0 * kTile;
      const int left = (end - c0 + NW - 1) / NW;
      tiles = left < 32 ? left : 32;
      const int64_t t = (int64_t)first + (lane >> 1) * (NW * kTile) + (lane & 1) * 16;
      const bool want = (lane >> 1) < tiles && t < len;
      const uint32_t s = (uint32_t)((want ? t : (int64_t)first) >> 4), pg = page_of(p, s);
      const int id = p.table[(int64_t)b * p.max_pages + pg];
      const bool there = want && id >= 0 && id < p.num_pages;
      const int64_t row = (((int64_t)id * p.kv_heads + head) * p.page_subs + (s - pg * p.page_subs)) * 16;
      row_lo = there ? (uint32_t)row : 0u;
      row_hi = there ? (uint32_t)(row >> 32) : 0x80000000u;
    };
    auto locate = [&](int tile, bool *there) {
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const uint32_t lo = __builtin_amdgcn_readlane(row_lo, 2 * tile + sub);
        const uint32_t hi = __builtin_amdgcn_readlane(row_hi, 2 * tile + sub);
        there[sub] = !(hi >> 31);
        rows[sub] = (int64_t)(((uint64_t)(hi & 0x7FFFFFFFu) << 32) | lo);
      }
    };
    {
      Queries qs;
      load_queries(qs, p, b, head, slice, len, lane);
      look_up();
      locate(0, on);
      if constexpr (QUANT) load_scales(raw, from, rows);
      load_keys(k, p, rows, on, lane);
      load_values(v, p, rows, on, lane);
      __builtin_amdgcn_sched_barrier(0);
      start(qs, p);
      clear();
    }
    for (;;) {
      for (int tile = 0; tile < tiles; ++tile) {
        const int token = first + tile * (NW * kTile);
        const bool last = tile + 1 == tiles;
        float t[NT][8];
        const bool edge = token + 32 > least || !on[0] || !on[1] || (MORE && token < most);
        Scales g;
        if constexpr (QUANT) {
          share_scales(raw, strip, lane, none);
          take_scales(g, strip, 0, lane);
        }
        const float up = room(raw, edge, token, on, since, len, lane);
        scores(p, k, g, t, token, lane >> 4);
        // after the last tile fetches of no bytes: loads without a branch let
        // the waits count only what they need
        locate(last ? tile : tile + 1, on_next);
        if (last) on_next[0] = on_next[1] = false;
        // (into the registers just used: nothing moves across)
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (QUANT) load_scales(raw, from, rows);
        load_keys(k, p, rows, on_next, lane);
        if (edge) edge_scores(t, token, on, lane >> 4);
        weigh(t, up);
        if constexpr (QUANT) {
          take_scales(g, strip, 2, lane);
          if (edge) edge_values(g, token, on, lane >> 4);
          gather(v, g, t);
        } else if (edge) {
          for (int i = 0; i < p.L; ++i) {
            const int sees = len - p.L + 1 + i;
            edge_gather(v, g, t, MORE ? first_seen(p, first_b, sees) : 0, sees, token, on, lane >> 4);
          }
        } else {
          gather(v, g, t);
        }
        __builtin_amdgcn_sched_barrier(0);
        load_values(v, p, rows, on_next, lane);
        on[0] = on_next[0];
        on[1] = on_next[1];
      }
      c0 += 32 * NW;
      if (c0 >= end) break;
      look_up();
      locate(0, on);
      if constexpr (QUANT) load_scales(raw, from, rows);
      load_keys(k, p, rows, on, lane);
      load_values(v, p, rows, on, lane);
    }
  }

  // (m, l, o) of the wave's tile nt of columns, the biases' part folded in, to
  // its place in LDS: rows of D results per column, then the columns' m and l.
  // All lanes write (a column's m and l four times), for the reason that the
  // pages' look-up has no branch.
  static constexpr int PF = piece_floats(D, NT);
  static constexpr int ROW = D + 4;  // columns on different banks
  static constexpr int SHARE = 16 * ROW;
  __device__ __forceinline__ void give(int nt, float *o_at, float *ml_at) {
    const int lane = lane_here(), c = lane & 15, h = lane >> 4;
    ml_at[c] = m[nt];
    ml_at[16 + c] = quarters_sum(l[nt]);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const float add = QUANT ? quarters_sum(bacc[nt][g]) : 0.f;
      float *at = o_at + c * ROW + g * G + 4 * h * VN;
#pragma unroll
      for (int e = 0; e < 4 * VN; e += 4) {  // value e: row e / VN of product e % VN
        f32x4v y;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int n = (e + x) % VN;
          const float r = o[nt][g][n][(e + x) / VN];
          y[x] = QUANT ? __builtin_fmaf(r, UNIT, add) : r;
        }
        *reinterpret_cast<f32x4v *>(at + e) = y;
      }
    }
  }
};

// four values of a row of the result
template <int D>
__device__ __forceinline__ void put_result(const Params &p, int b, int head, int r, int at, f32x4v y) {
  const int i = r / p.group, j = r - i * p.group;
  uint2 *out = reinterpret_cast<uint2 *>(
      reinterpret_cast<uint16_t *>(p.out) +
      (((int64_t)b * p.L + i) * p.kv_heads * p.group + head * p.group + j) * D + at);
  *out = p.x_dtype == X_F16 ? make_uint2(pack_f16(y[0], y[1]), pack_f16(y[2], y[3]))
                            : make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
}

// MORE: the logarithm of a row's sum of weights l 2^m
__device__ __forceinline__ void put_lse(const Params &p, int b, int head, int r, float m, float l) {
  if (!p.lse) return;
  const int i = r / p.group, j = r - i * p.group;
  p.lse[((int64_t)b * p.L + i) * p.kv_heads * p.group + head * p.group + j] =
      log_scaled(m, l);
}

// Running (m, l, acc) of one strand of pieces
struct Strand {
  float m = kNegInf, l = 0.f;
  f32x4v acc = {0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(float pm, float pl, f32x4v v) {
    const float top = __builtin_fmaxf(m, pm), base = top == kNegInf ? 0.f : top;
    const float f = exp2_fast(m - base), g = exp2_fast(pm - base);
    m = top;
    l = l * f + pl * g;
    acc = acc * f + v * g;
  }
  __device__ __forceinline__ f32x4v result() const { return acc * (l == 0.f ? 0.f : 1.f / l); }
};

// Joins, inside the launch, the n pieces of a unit from place w0's second on,
// and writes the rows.  Every four values are one thread's, or, where the
// workgroup has more threads, several threads' (strands) with every so many-th
// piece each, joined through LDS: the order of all sums is the pieces' own.  A
// thread has the loads of U pieces for V times four values under way at once.
template <int D, int NT, int U, int V, bool MORE>
__device__ __forceinline__ void join_pieces(const Params &p, int b, int head, int slice, int w0,
                                            int n, int used, int strands, float *buf) {
  constexpr int PF = piece_floats(D, NT), ML = NT * 16 * D, Q = D / 4;
  const int items = used * Q;
  const int strand = strands == 1 ? 0 : (int)threadIdx.x / items;
  const int step = strands == 1 ? 64 * NW : items;  // items at a time
  const Span from = span(p.parts, (2 * (int64_t)w0 + 1) * (PF * 4), 0x7FFFFFFF);
  for (int i0 = 0; i0 < items; i0 += V * step) {
    Strand st[V];
    int c[V], at[V];
    bool on[V];
#pragma unroll
    for (int y = 0; y < V; ++y) {
      const int item = i0 + y * step + (int)threadIdx.x - strand * items;
      on[y] = strand < strands && item < items;
      c[y] = on[y] ? item / Q : 0;
      at[y] = on[y] ? (item % Q) * 4 : 0;
    }
    // every thread's piece of a round is `strand` past a uniform one, piece
    // k > 0 (2 k - 1) pieces past the first
    for (int k0 = 0; k0 < n; k0 += U * strands) {
      f32x4v v[U][V];
      float pm[U][V], pl[U][V];
#pragma unroll
      for (int x = 0; x < U; ++x) {
        const int k = k0 + x * strands + strand, kk = k < n ? k : n - 1;
        const int off = kk ? (2 * kk - 1) * PF : 0;
#pragma unroll
        for (int y = 0; y < V; ++y) {
          v[x][y] = get_piece(from, off + c[y] * D + at[y]);
          pm[x][y] = get_piece1(from, off + ML + c[y]);
          pl[x][y] = get_piece1(from, off + ML + NT * 16 + c[y]);
        }
      }
#pragma unroll
      for (int x = 0; x < U; ++x)
        if (k0 + x * strands + strand < n)
#pragma unroll
          for (int y = 0; y < V; ++y) st[y].add(pm[x][y], pl[x][y], v[x][y]);
    }
    if (strands > 1) {  // (one item a thread then)
      if (on[0]) {
        float *to = buf + (int)threadIdx.x * 6;
        to[0] = st[0].m, to[1] = st[0].l;
#pragma unroll
        for (int x = 0; x < 4; ++x) to[2 + x] = st[0].acc[x];
      }
      __syncthreads();
      if (on[0] && strand == 0)
        for (int k = 1; k < strands; ++k) {
          const float *other = buf + (k * items + (int)threadIdx.x) * 6;
          st[0].add(other[0], other[1], f32x4v{other[2], other[3], other[4], other[5]});
        }
    }
#pragma unroll
    for (int y = 0; y < V; ++y)
      if (on[y] && strand == 0) {
        put_result<D>(p, b, head, slice * NT * 16 + c[y], at[y], st[y].result());
        if constexpr (MORE)
          if (at[y] == 0) put_lse(p, b, head, slice * NT * 16 + c[y], st[y].m, st[y].l);
      }
  }
}

template <int D, int NT, bool MORE>
__device__ __forceinline__ void join_inside(const Params &p, int b, int head, int slice, int w0,
                                            int n, int used, float *buf) {
  const int items = used * (D / 4);
  int strands = 64 * NW / items;
  strands = strands < 1 ? 1 : (strands > n ? n : strands);
  // 16 loads a thread in as few rounds as the pieces and items make, fewer
  // loads where they are few
  if (items > 128 * NW && n <= 4)
    join_pieces<D, NT, 4, 4, MORE>(p, b, head, slice, w0, n, used, strands, buf);
  else if (items > 64 * NW)
    join_pieces<D, NT, 8, 2, MORE>(p, b, head, slice, w0, n, used, strands, buf);
  else if (n <= 4 * strands)
    join_pieces<D, NT, 4, 1, MORE>(p, b, head, slice, w0, n, used, strands, buf);
  else
    join_pieces<D, NT, 16, 1, MORE>(p, b, head, slice, w0, n, used, strands, buf);
}

template <int BITS, bool BF, int D, int G, int NT, int WGS, bool MORE>
__global__ __launch_bounds__(64 * NW, WGS) void attn_kernel(Params p) {
  using W = Wave<BITS, BF, D, G, NT, MORE>;
  __shared__ f32x4v buf4[NW * W::SHARE / 4];
  __shared__ float ml[NW * 32];
  __shared__ uint32_t last;
  float *buf = reinterpret_cast<float *>(buf4);
  const int wave = uniform(threadIdx.x >> 6);

  const Line<MORE> line(p, gridDim.x, lane_here());
  // sequences without tokens: zero rows
  if (__ballot(line.idle)) {
    const int64_t row_halves = (int64_t)p.L * p.kv_heads * p.group * D;
    for (int64_t b = blockIdx.x; b < p.B; b += gridDim.x)
      if (clamped_length(p, (int)b) == 0)
        for (int64_t i = threadIdx.x; i < row_halves / 8; i += 64 * NW)
          reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(p.out) + b * row_halves)[i] =
              make_uint4(0, 0, 0, 0);
    if constexpr (MORE)
      if (p.lse)
        for (int64_t b = blockIdx.x; b < p.B; b += gridDim.x)
          if (clamped_length(p, (int)b) == 0)
            for (int i = threadIdx.x; i < p.L * p.kv_heads * p.group; i += 64 * NW)
              p.lse[b * (p.L * p.kv_heads * p.group) + i] = kNegInf;
    if (!p.inside)
      for (int64_t b = blockIdx.x; b < p.B; b += gridDim.x)
        if (clamped_length(p, (int)b) == 0)
          for (uint32_t u = threadIdx.x; u < line.rows; u += 64 * NW)
            p.cuts[b * line.rows + u] = make_uint2(0, 0);
  }
  // Workgroups go to the 8 XCDs in turn; near places of the line are taken by
  // one XCD.  The slices of a key head read the same tokens at about the same
  // time and lie near each other, so the second reader finds the codes in that
  // XCD's L2 (8 sequences of up to 8192 tokens with 40 rows a key head: 90 MB
  // fetched against 174, 37.3 us against 40.3; without slices 20.1 against 20.9
  // for 16 sequences of up to 4096, the others the same).
  const uint32_t eighth = (line.grid + 7) / 8;
  const uint32_t place = (blockIdx.x & 7) * eighth + (blockIdx.x >> 3);
  if (place >= line.grid || (blockIdx.x >> 3) >= eighth) return;
  uint32_t pos = line.begin(place);
  const uint32_t end = line.begin(place + 1);
  const int at = __builtin_ctzll(__ballot(pos < line.upto * line.rows));
  int b = at * line.per;
  uint32_t before = (uint32_t)__builtin_amdgcn_readlane(line.upto - line.mine, at);

  W st;
  int len = uniform(__builtin_amdgcn_readlane(line.len, at));
  while (pos < end) {
    uint32_t chunks = line.chunks(p, b, len);
    while (pos >= (before + chunks) * line.rows) {
      before += chunks;
      ++b;
      len = uniform(clamped_length(p, b));
      chunks = line.chunks(p, b, len);
    }
    const uint32_t in_seq = pos - before * line.rows;
    const int unit = uniform(in_seq / chunks);
    const uint32_t c0 = in_seq - unit * chunks;
    const int head = uniform(unit / p.slices), slice = unit - head * p.slices;
    const uint32_t c1 = end - pos < chunks - c0 ? c0 + (end - pos) : chunks;
    const uint32_t unit_begin = pos - c0;
    pos += c1 - c0;

    const int base = uniform(first_tile<MORE>(p, b, len));
    const int tiles = (len + kTile - 1) / kTile, tile0 = base + (int)(c0 * (line.chunk / kTile));
    int tile1 = base + (int)(c1 * (line.chunk / kTile));
    tile1 = tile1 < tiles ? tile1 : tiles;
    const int busy = tile1 - tile0 < NW ? tile1 - tile0 : NW;
    const int cols = p.L * p.group - slice * NT * 16, used = cols < NT * 16 ? cols : NT * 16;
    const bool whole = c0 == 0 && c1 == chunks;
    const Span to = span(p.parts, (2 * (int64_t)place + (c0 == 0)) * (W::PF * 4), W::PF * 4);
    __syncthreads();  // the last round's readers of LDS are done
    if (wave < busy)
      st.run(p, b, head, slice, len, tile0 + wave, tile1,
             reinterpret_cast<char *>(buf + wave * W::SHARE));
    // a tile of columns after the other: the waves' shares, then every four
    // values of the rows over them, to the output or, where this is only a
    // piece of the unit, to the workspace (a place's second piece there is
    // the piece that starts its unit)
    constexpr int Q = D / 4;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (wave < busy) st.give(nt, buf + wave * W::SHARE, ml + wave * 32);
      __syncthreads();
      const int live = used - nt * 16 < 16 ? used - nt * 16 : 16;
      for (int item = threadIdx.x; item < live * Q; item += 64 * NW) {
        const int c = item / Q, at = (item % Q) * 4;
        // (all reads at once, the idle waves' too, which count for nothing)
        float wm[NW], wl[NW], top = kNegInf, l = 0.f;
        f32x4v wo[NW], y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          wm[w] = ml[w * 32 + c];
          wl[w] = ml[w * 32 + 16 + c];
          wo[w] = *reinterpret_cast<const f32x4v *>(buf + w * W::SHARE + c * W::ROW + at);
        }
#pragma unroll
        for (int w = 0; w < NW; ++w) top = __builtin_fmaxf(top, w < busy ? wm[w] : kNegInf);
        const float base = top == kNegInf ? 0.f : top;
#pragma unroll
        for (int w = 0; w < NW; ++w)
          if (w < busy) {
            const float f = exp2_fast(wm[w] - base);
            l += wl[w] * f;
            y += wo[w] * f;
          }
        const int r = nt * 16 + c;
        if (whole) {
          put_result<D>(p, b, head, slice * NT * 16 + r, at, y * (l == 0.f ? 0.f : 1.f / l));
          if constexpr (MORE)
            if (at == 0) put_lse(p, b, head, slice * NT * 16 + r, top, l);
        } else {
          put_piece(to, r * D + at, y);
          if (at == 0) {
            put_piece1(to, NT * 16 * D + r, top);
            put_piece1(to, NT * 16 * D + NT * 16 + r, l);
          }
        }
      }
      if (nt + 1 < NT) __syncthreads();
    }
    if (!p.inside) {
      if (c0 == 0 && threadIdx.x == 0) {
        const uint32_t n = whole ? 0 : line.owner(unit_begin + chunks - 1) - place + 1;
        p.cuts[b * line.rows + unit] = make_uint2(n, place);
      }
      continue;
    }
    if (whole) continue;

    // count this piece in, and join them if it is the unit's last to arrive
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    const int w0 = uniform(line.owner(unit_begin));
    const int n = uniform(line.owner(unit_begin + chunks - 1)) - w0 + 1;
    if (threadIdx.x == 0) {
      last = __hip_atomic_fetch_add(p.arrived + w0, 1u, __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(n - 1);
      if (last) __hip_atomic_store(p.arrived + w0, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (uniform((int)last)) {
      asm volatile("" ::: "memory");
      join_inside<D, NT, MORE>(p, b, head, slice, w0, n, used, buf);
    }
  }
}

// Joins the pieces of units that were cut, in a launch of its own: a workgroup
// takes 64 times four values of one unit, each of its JW waves every JW-th
// piece, and adds the waves' parts in order.
template <int N> struct Count { static constexpr int value = N; };
template <int D, int JW, bool MORE>
__global__ __launch_bounds__(64 * JW) void attn_join_kernel(Params p, int nt) {
  __shared__ float part[JW][6][64];
  const uint2 cut = p.cuts[blockIdx.x];
  const int n = uniform(cut.x), w0 = uniform(cut.y);
  if (n == 0) return;
  const int rows = p.kv_heads * p.slices, b = blockIdx.x / rows, unit = blockIdx.x - b * rows;
  const int head = unit / p.slices, slice = unit - head * p.slices;
  const int lane = lane_here(), wave = uniform(threadIdx.x >> 6);
  constexpr int Q = D / 4;
  const int cols = p.L * p.group - slice * nt * 16, used = cols < nt * 16 ? cols : nt * 16;
  const int item = blockIdx.y * 64 + lane;
  const bool on = item < used * Q;
  const int c = on ? item / Q : 0, d = on ? (item % Q) * 4 : 0;
  const int PF = piece_floats(D, nt);
  const float *first = p.parts + (2 * (int64_t)w0 + 1) * PF;
  // a wave's pieces, U at once (no more loads than there are pieces)
  Strand st;
  auto add = [&](auto at_once) {
    constexpr int U = decltype(at_once)::value;
    for (int i = wave; i < n; i += U * JW) {
      f32x4v v[U];
      float pm[U], pl[U];
#pragma unroll
      for (int x = 0; x < U; ++x) {
        const int k = i + x * JW < n ? i + x * JW : i;
        const float *src = first + (k ? (2 * (int64_t)k - 1) * PF : 0);
        v[x] = *reinterpret_cast<const f32x4v *>(src + c * D + d);
        pm[x] = src[nt * 16 * D + c];
        pl[x] = src[nt * 16 * D + nt * 16 + c];
      }
#pragma unroll
      for (int x = 0; x < U; ++x)
        if (i + x * JW < n) st.add(pm[x], pl[x], v[x]);
    }
  };
  if (n <= JW)
    add(Count<1>());
  else if (n <= 2 * JW)
    add(Count<2>());
  else
    add(Count<8>());
  part[wave][0][lane] = st.m;
  part[wave][1][lane] = st.l;
#pragma unroll
  for (int x = 0; x < 4; ++x) part[wave][2 + x][lane] = st.acc[x];
  __syncthreads();
  if (wave != 0 || !on) return;
  // (waves without a piece left a maximum of -inf and zeros)
#pragma unroll
  for (int w = 1; w < JW; ++w)
    st.add(part[w][0][lane], part[w][1][lane],
           f32x4v{part[w][2][lane], part[w][3][lane], part[w][4][lane], part[w][5][lane]});
  put_result<D>(p, b, head, slice * nt * 16 + c, d, st.result());
  if constexpr (MORE)
    if (d == 0) put_lse(p, b, head, slice * nt * 16 + c, st.m, st.l);
}

// Query rows per key head go to a wave in one or two tiles of 16; more rows are
// further slices, each of which reads the cache again, mostly from a cache of
// the chip.  (40 rows, 8 bits, 8 sequences of up to 8192 tokens, at one step: 45
// us in two slices of two tiles; 47 in one of three, which takes the registers
// of the second workgroup on a CU; 59 as four waves with a tile of rows each on
// the same tokens, too few tokens are then under way.  The second slice's one
// tile of 8 rows computed as one, not two: no faster, 46.4 against 45.3.)
// Heads of 256 have one tile a wave: with two the state does not fit the 512
// registers that a wave can have (8 bits: 40 to 275 of them in scratch memory,
// with the groups of a row; 16 bits 587).
constexpr int most_tiles(int D) { return D > 128 ? 1 : 2; }
inline void tiles_for(int64_t cols, int D, int &nt, int &slices) {
  const int64_t tiles = (cols + 15) / 16;
  nt = tiles > 1 ? most_tiles(D) : 1;
  slices = (int)((tiles + nt - 1) / nt);
}

// Workgroups per CU the kernel is built for: what its registers allow (a lane's
// scales and biases grow with the groups of a row), heads of 64 but for 9 to 15
// registers in scratch memory.  Two where three could be
// built with fewer loads under way: 16 sequences of up to 4096 tokens, 8 bits,
// 23.9 against 26.4 us at one step; 16 bits 54 against 60.
// Heads of 64, quantized, three: 32 sequences of up to 8192 tokens, 4 bits 41.8
// against 53.7 us (8 sequences of up to 2048 14.1 against 11.5); not at 16 bits,
// 34.5 against 29.6.  Heads of 256 at 16 bits one: 23.4 against 36.4 us, registers
// do not spill.
constexpr int wgs_per_cu(int BITS, int D, int NG, int NT) {
  return D * NT <= 64 && BITS != 16 ? 3 : (D * NT <= 128 || (D * NT <= 256 && NG <= 2 && BITS != 16) ? 2 : 1);
}

// what every launch has (not slices, chunk and the workspace)
inline Params common_params(const AttnArgs &a, const KvCache &c) {
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
  p.cap2 = a.scores.softcap * 1.44269504088896341f;
  p.inv_cap2 = a.scores.softcap != 0.f ? 1.f / p.cap2 : 0.f;
  p.window = a.scores.window > 0 && a.scores.window < 0x7FFFFF00 ? a.scores.window : 0x7FFFFF00;  // (vis - window in 32 bits)
  p.slopes = a.scores.slopes;
  p.first = a.scores.first;
  p.lse = a.scores.lse;
  return p;
}

template <bool MORE>
hipError_t launch(const AttnArgs &a, const KvCache &c, hipStream_t s) {
  Params p = common_params(a, c);
  const int64_t cols = (int64_t)a.L * p.group;
  int nt;
  tiles_for(cols, c.head_dim, nt, p.slices);
  // The line's chunks are counted in 32 bits: where the table could hold more
  // tiles than that they are longer.  A table that holds no more than one tile
  // per wave leaves units whole.
  const int64_t cap = a.max_pages * c.page_size, per_tile = (int64_t)a.B * c.kv_heads * p.slices;
  int64_t chunk = cap <= NW * kTile ? NW * kTile : kTile;
  while ((cap + chunk - 1) / chunk * per_tile > 0x7FFFFFFF) chunk *= 2;
  p.chunk = (uint32_t)chunk;
  // no more workgroups than chunks the table can hold
  const int64_t most = (cap + chunk - 1) / chunk * per_tile;
  int64_t grid = (int64_t)device_cus() *
                 wgs_per_cu(c.bits, c.head_dim, c.bits == 16 ? 1 : c.head_dim / c.group_size, nt);
  if (grid > kMaxGrid) grid = kMaxGrid;
  grid = grid / 8 * 8;  // (the same number on every XCD)
  if (most < grid) grid = (most + 7) / 8 * 8;
  p.cuts = reinterpret_cast<uint2 *>(a.workspace);
  p.arrived = reinterpret_cast<uint32_t *>(p.cuts + kMaxGrid);
  p.parts = reinterpret_cast<float *>(p.arrived + kMaxGrid);
  // A unit's pieces, each `items` times four values, are joined by one
  // workgroup inside the launch, unless one sequence could have so many (a
  // piece is four tiles at least) that a launch over the whole chip is faster:
  // one sequence, one key head, 64 pieces of 1024 items 15.7 us against 46.5;
  // one of 131072 tokens, 8 key heads, 64 of 128 items 41 against 46.  Where
  // there are few, that launch only costs: 16 sequences, 4 pieces of 128 items
  // each on average 21.8 us against 20.7; 16 with 40 rows a key head, 2 of 1024
  // items 133 against 123 (which the rule, not knowing lengths, puts there).
  const int items = (int)(cols < 16 * nt ? cols : 16 * nt) * c.head_dim / 4;
  const int64_t pieces = (cap + NW * kTile - 1) / (NW * kTile);
  p.inside = per_tile > kMaxGrid || (pieces < grid ? pieces : grid) * items <= 16384;
  hipError_t err = hipErrorInvalidValue;
#define AQ_KT(B, F, D, G, T)                                                           \
  hipLaunchKernelGGL((attn_kernel<B, F, D, G, T, wgs_per_cu(B, D, D / G, T), MORE>),         \
                     dim3((unsigned)grid), dim3(64 * NW), 0, s, p)
#define AQ_K(B, F, D, G)                                                               \
  do {                                                                                 \
    if (nt == 1)                                                                       \
      AQ_KT(B, F, D, G, 1);                                                            \
    else                                                                               \
      AQ_KT(B, F, D, G, most_tiles(D));                                                \
    err = hipGetLastError();                                                           \
  } while (0)
#define AQ_G(B, D)                                     \
  if (c.head_dim == D) {                               \
    if (c.group_size == 32) AQ_K(B, false, D, 32);     \
    if (c.group_size == 64) AQ_K(B, false, D, 64);     \
    if constexpr (D >= 128) {                          \
      if (c.group_size == 128) AQ_K(B, false, D, 128); \
    }                                                  \
  }
#define AQ_H(D)                                        \
  if (c.head_dim == D) {                               \
    if (c.dtype == X_BF16) AQ_K(16, true, D, D);       \
    else AQ_K(16, false, D, D);                        \
  }
  if (c.bits == 4) { AQ_G(4, 64) AQ_G(4, 128) AQ_G(4, 256) }
  if (c.bits == 8) { AQ_G(8, 64) AQ_G(8, 128) AQ_G(8, 256) }
  if (c.bits == 16) { AQ_H(64) AQ_H(128) AQ_H(256) }
#undef AQ_H
#undef AQ_G
#undef AQ_K
#undef AQ_KT
  // (a chunk that holds the whole table: no unit is cut)
  if (err != hipSuccess || cap <= chunk || p.inside) return err;
  const dim3 join((unsigned)per_tile, (unsigned)((items + 63) / 64));
  // Eight waves, as long as the chip holds them all; else four: 128 units of
  // 1024 items 39.5 us a call against 41.2, 256 124.5 against 127.8; 8 of 128
  // items 42.6 against 41.9.
  const bool room = (int64_t)join.x * join.y * 8 <= (int64_t)device_cus() * 32;
#define AQ_J(D)                                                                          \
  do {                                                                                   \
    if (room)                                                                            \
      hipLaunchKernelGGL((attn_join_kernel<D, 8, MORE>), join, dim3(64 * 8), 0, s, p, nt);     \
    else                                                                                 \
      hipLaunchKernelGGL((attn_join_kernel<D, 4, MORE>), join, dim3(64 * 4), 0, s, p, nt);     \
  } while (0)
  if (c.head_dim == 64) AQ_J(64);
  else if (c.head_dim == 128) AQ_J(128);
  else AQ_J(256);
#undef AQ_J
  return hipGetLastError();
}

}  // namespace
}  // namespace aq
