// aq_weigh.hip -- what every cached token gathers of the attention of new
// tokens: the sum over all rows of exp(score - lse), added to what it gathered
// before (gfx950).
//
// Scores are those of the attention (aq_attn.hpp: the same operands, the same
// products), so a wave has the scores of 32 tokens as S^T = K q^T, a lane one
// column and four tokens of each 16.  The weights 2^(t - lse) of the lane's
// columns are summed in its registers, then over the 16 lanes of the columns,
// and added to the token's place in a strip of LDS of the wave's own.  Key heads
// go to the waves of a workgroup in turn (fewer heads than waves: the tiles do),
// the waves' strips are added in order, and one thread adds a token's sum to
// its weight: no atomics, the same bits every time.
//
// Tokens are cut evenly over the chip in chunks, as in the attention, by the
// lengths on the device.
//
// Bound: neither HBM nor vector instructions are full, the waves of a CU (two a
// SIMD) wait in turn.  131072 tokens of 8 key heads of 128 at 4 bits, 32 rows
// each: 30 us, 12 of bytes at 6.2 TB/s and 16 of vector instructions at 2.4 GHz;
// 16 sequences of up to 4096 tokens at 8 bits, 4 rows: 17 us, 6 of bytes and 4 of
// instructions, the rest first loads that wait for each other.
#include "aq_attn.hpp"

namespace aq {
namespace {

constexpr int WV = 8;       // waves of a workgroup
constexpr int kSpan = 512;  // tokens of a workgroup's strip

// Sums of 8 values over the 16 lanes of a row; a lane gets the sum number lane / 2 % 8.  Partners
// are lanes that differ in bit 3, then 2, then 1: each time a lane keeps half of what it has, by
// that bit, and takes its partner's of it.
__device__ __forceinline__ float columns_sum(const float (&s)[8], int lane) {
  const bool b3 = lane & 8, b2 = lane & 4, b1 = lane & 2;
  float x[4], y[2];
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = (b3 ? s[j + 4] : s[j]) + dpp_f<0x140>(b3 ? s[j] : s[j + 4]);  // row_mirror
#pragma unroll
  for (int j = 0; j < 2; ++j) y[j] = (b2 ? x[j + 2] : x[j]) + dpp_f<0x141>(b2 ? x[j] : x[j + 2]);  // row_half_mirror
  const float z = (b1 ? y[1] : y[0]) + dpp_f<0x4E>(b1 ? y[0] : y[1]);  // quad_perm [2,3,0,1]
  return z + dpp_f<0xB1>(z);                                            // quad_perm [1,0,3,2]
}

template <int BITS, bool BF, int D, int G, int NT>
__global__ __launch_bounds__(64 * WV, 2) void weigh_kernel(Params p, float *weights, int64_t stride) {
  typedef Wave<BITS, BF, D, G, NT, true> W;
  constexpr int STRIP = 128 * W::TB;
  __shared__ float strips[WV][kSpan];
  __shared__ __align__(16) char scales[WV][W::QUANT ? STRIP : 16];
  const int wave = uniform(threadIdx.x >> 6);
  const int heads_at_once = p.kv_heads >= 8 ? 8 : (p.kv_heads >= 4 ? 4 : (p.kv_heads >= 2 ? 2 : 1)), split = WV / heads_at_once;
  const int head0 = wave % heads_at_once, part = wave / heads_at_once;

  Params lp = p;  // the line's units: sequences
  lp.kv_heads = lp.slices = 1;
  const Line<true> line(lp, gridDim.x, lane_here());
  if (blockIdx.x >= line.grid) return;
  uint32_t pos = line.begin(blockIdx.x);
  const uint32_t end = line.begin(blockIdx.x + 1);
  const int at = __builtin_ctzll(__ballot(pos < line.upto));
  int b = at * line.per;
  uint32_t before = (uint32_t)__builtin_amdgcn_readlane(line.upto - line.mine, at);
  int len = uniform(__builtin_amdgcn_readlane(line.len, at));
  W st;
  while (pos < end) {
    uint32_t chunks = line.chunks(lp, b, len);
    while (pos >= before + chunks) {
      before += chunks;
      ++b;
      len = uniform(clamped_length(p, b));
      chunks = line.chunks(lp, b, len);
    }
    // chunks c0 .. of sequence b, a strip's worth of tiles at a time
    const uint32_t c0 = pos - before, n = end - pos < chunks - c0 ? end - pos : chunks - c0;
    pos += n;
    const int base = uniform(first_tile<true>(p, b, len)), per = (int)(line.chunk / kTile);
    const int tiles = (len + kTile - 1) / kTile;
    int last_tile = base + (int)(c0 + n) * per;
    last_tile = last_tile < tiles ? last_tile : tiles;
    for (int tile0 = base + (int)c0 * per; tile0 < last_tile; tile0 += kSpan / kTile) {
    const int tile1 = last_tile - tile0 < kSpan / kTile ? last_tile : tile0 + kSpan / kTile;

    const int lane = lane_here(), h = lane >> 4;
    __syncthreads();  // the last strips' readers are done
#pragma unroll
    for (int i = 0; i < kSpan; i += 64) strips[wave][i + lane] = 0.f;

    // pages of the wave's tiles: lane 2 i + sub
    const int mine = tile1 - tile0 - part, count = mine > 0 ? (mine + split - 1) / split : 0;
    const int first = (tile0 + part) * kTile, step = split * kTile;
    uint32_t row_lo, row_hi;
    {
      const int64_t t = (int64_t)first + (lane >> 1) * step + (lane & 1) * 16;
      const bool want = (lane >> 1) < count && t < len;
      const uint32_t s = (uint32_t)((want ? t : (int64_t)tile0 * kTile) >> 4), pg = page_of(p, s);
      const int id = p.table[(int64_t)b * p.max_pages + pg];
      const bool there = want && id >= 0 && id < p.num_pages;
      const int64_t row = ((int64_t)id * p.kv_heads * p.page_subs + (s - pg * p.page_subs)) * 16;
      row_lo = there ? (uint32_t)row : 0u;
      row_hi = there ? (uint32_t)(row >> 32) : 0x80000000u;
    }
    if (count)
      for (int head = head0; head < p.kv_heads; head += heads_at_once) {
        const int64_t head_rows = (int64_t)head * p.page_subs * 16;
        int64_t rows[2];
        bool on[2], on_next[2];
        auto locate = [&](int tile, bool *there) {
#pragma unroll
          for (int sub = 0; sub < 2; ++sub) {
            const uint32_t lo = __builtin_amdgcn_readlane(row_lo, 2 * tile + sub);
            const uint32_t hi = __builtin_amdgcn_readlane(row_hi, 2 * tile + sub);
            there[sub] = !(hi >> 31);
            rows[sub] = there[sub] ? (int64_t)(((uint64_t)hi << 32) | lo) + head_rows : 0;
          }
        };
        for (int slice = 0; slice < p.slices; ++slice) {
          typename W::Keys k;
          typename W::Raw raw;
          bool none;
          const char *from = W::scales_of(p, lane, none);
          float lse[NT];
          bool idle[NT], some_idle = false;
          {
            typename W::Queries qs;
            st.load_queries(qs, p, b, head, slice, len, lane);
            locate(0, on);
            if constexpr (W::QUANT) W::load_scales(raw, from, rows);
            W::load_keys(k, p, rows, on, lane);
            const int cols = p.L * p.group;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int r = (slice * NT + nt) * 16 + (lane & 15), rr = r < cols ? r : 0;
              const int i = rr / p.group, j = rr - i * p.group;
              const float x = p.lse[((int64_t)b * p.L + i) * p.kv_heads * p.group + head * p.group + j];
              // A row that saw nothing, and columns without a row (which have the first row's query), add
              // nothing, by a choice and not by a logarithm of inf: a NaN would not yield to that.
              idle[nt] = r >= cols || x == kNegInf;
              some_idle |= __ballot(idle[nt]) != 0;
              lse[nt] = x * 1.44269504088896341f;
            }
            st.start(qs, p);
          }
          const int newest = ((slice + 1) * NT * 16 - 1) / p.group;
          const int least = len - p.L + 1 + (slice * NT * 16) / p.group;
          const int most = first_seen(p, uniform(first_of(p, b)), len - p.L + 1 + (newest < p.L ? newest : p.L - 1));
          for (int tile = 0; tile < count; ++tile) {
            const int token = first + tile * step;
            const bool last = tile + 1 == count;
            float t[NT][8];
            const bool edge = token + 32 > least || !on[0] || !on[1] || token < most;
            typename W::Scales g;
            if constexpr (W::QUANT) {
              W::share_scales(raw, scales[wave], lane, none);
              W::take_scales(g, scales[wave], 0, lane);
            }
            st.scores(p, k, g, t, token, h);
            locate(last ? tile : tile + 1, on_next);
            if (last) on_next[0] = on_next[1] = false;
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (W::QUANT) W::load_scales(raw, from, rows);
            W::load_keys(k, p, rows, on_next, lane);
            if (edge) st.edge_scores(t, token, on, h);
            // (what a row does not see gets nothing of it, be its logarithm NaN; a score of -inf that it
            // does see has a weight of 0 too)
            float sum[8];
            auto gather = [&](auto weight) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                sum[j] = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) sum[j] += weight(nt, j);
              }
            };
            auto weight = [&](int nt, int j) { return exp2_fast(t[nt][j] - lse[nt]); };
            // (one tile of columns mostly has idle ones, and a branch costs it more than the choices: 16
            // sequences of up to 4096 tokens 17.9 us against 17.0; two tiles without idle ones 32.9 against
            // 33.9, 131072 tokens; both with a copy of the weights)
            if (NT == 1 || edge || some_idle)
              gather([&](int nt, int j) { return idle[nt] || t[nt][j] == kNegInf ? 0.f : weight(nt, j); });
            else
              gather(weight);
            float *to = &strips[wave][token - tile0 * kTile + 16 * (lane >> 3 & 1) + 4 * h + (lane >> 1 & 3)];
            *to += columns_sum(sum, lane);
            on[0] = on_next[0];
            on[1] = on_next[1];
          }
        }
      }
    __syncthreads();
    const int64_t most_tokens = stride < len ? stride : len;
    for (int i = threadIdx.x; i < (tile1 - tile0) * kTile; i += 64 * WV) {
      const int64_t t = (int64_t)tile0 * kTile + i;
      if (t < most_tokens) {
        float sum = 0.f;
        // (the strips of a token: of the waves whose part its tile is in)
        const int q = (i / kTile) % split;
        for (int x = 0; x < heads_at_once; ++x) sum += strips[q * heads_at_once + x][i];
        weights[b * stride + t] += sum;
      }
    }
    }
  }
}

}  // namespace

hipError_t launch_kv_weigh(const AttnArgs &a, const KvCache &c, float *weights, int64_t stride,
                           hipStream_t s) {
  Params p = common_params(a, c);
  // only keys: their scales and biases in the place of the values'
  p.vc = p.kc;
  p.vs = p.ks;
  p.vb = p.kb;
  const int64_t cols = (int64_t)a.L * p.group;
  int nt;
  tiles_for(cols, c.head_dim, nt, p.slices);
  const int64_t cap = a.max_pages * c.page_size;
  // (the line's chunks are counted in 32 bits: where the table could hold more tiles than that they are longer)
  int64_t chunk = 2 * kTile;
  while ((cap + chunk - 1) / chunk * a.B > 0x7FFFFFFF) chunk *= 2;
  p.chunk = (uint32_t)chunk;
  int64_t grid = device_cus();
  const int64_t most = (cap + chunk - 1) / chunk * a.B;
  if (most < grid) grid = most;
  hipError_t err = hipErrorInvalidValue;
#define AQ_KT(B, F, D, G, T)                                                                    \
  hipLaunchKernelGGL((weigh_kernel<B, F, D, G, T>), dim3((unsigned)grid), dim3(64 * WV), 0, s, p, \
                     weights, stride)
#define AQ_K(B, F, D, G)               \
  do {                                 \
    if (nt == 1)                       \
      AQ_KT(B, F, D, G, 1);            \
    else                               \
      AQ_KT(B, F, D, G, most_tiles(D)); \
    err = hipGetLastError();           \
  } while (0)
#define AQ_G(B, D)                                     \
  if (c.head_dim == D) {                               \
    if (c.group_size == 32) AQ_K(B, false, D, 32);     \
    if (c.group_size == 64) AQ_K(B, false, D, 64);     \
    if constexpr (D >= 128) {                          \
      if (c.group_size == 128) AQ_K(B, false, D, 128); \
    }                                                  \
  }
#define AQ_H(D)                                  \
  if (c.head_dim == D) {                         \
    if (c.dtype == X_BF16) AQ_K(16, true, D, D); \
    else AQ_K(16, false, D, D);                  \
  }
  if (c.bits == 4) { AQ_G(4, 64) AQ_G(4, 128) AQ_G(4, 256) }
  if (c.bits == 8) { AQ_G(8, 64) AQ_G(8, 128) AQ_G(8, 256) }
  if (c.bits == 16) { AQ_H(64) AQ_H(128) AQ_H(256) }
#undef AQ_H
#undef AQ_G
#undef AQ_K
#undef AQ_KT
  return err;
}

}  // namespace aq
