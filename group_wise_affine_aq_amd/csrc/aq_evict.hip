// aq_evict.hip -- the tokens of each cached sequence that gathered most of the
// attention, chosen and moved to other pages (gfx950).
//
// Choosing.  One workgroup per sequence finds the least key that is kept, the
// M-th largest of the candidates' weights, by radix: weights become 32-bit keys
// in their order, and four counts of 8 bits each narrow down the key, each count
// over the candidates that share the bits found so far.  Then every wave takes
// a run of neighbouring tokens: it counts the larger keys and the equal ones,
// the counts of the waves before it say where its own kept tokens go and how
// many equal ones are still to be taken, and a second pass writes positions
// and weights, 64 tokens at a time by their ballots.  All counts are whole
// numbers, so the result does not depend on their order.
//
// Moving is copying rows: a workgroup takes neighbouring kept tokens of one
// head, keys or values, whose new places are neighbours, 16 bytes a thread and
// several loads under way.  It is bound by HBM; the choice by the latency of
// its passes.
#include "aq_internal.hpp"

namespace aq {
namespace {

constexpr int kSelect = 1024;  // threads that choose
constexpr int kWaves = kSelect / 64;

// weights in their order, NaN below everything
__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t u = __builtin_bit_cast(uint32_t, w);
  if (w != w) return 0;
  if (w == 0.f) return 0x80000000u;  // -0 and +0 are equal
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int clamped(const EvictArgs &a, const KvCache &c, int b) {
  int64_t cap = a.max_pages * c.page_size;
  cap = cap < a.stride ? cap : a.stride;
  const int n = a.lengths[b];
  return n < 0 ? 0 : (n > cap ? (int)cap : n);
}

__device__ __forceinline__ uint32_t lanes_before(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

__global__ __launch_bounds__(kSelect) void select_kernel(EvictArgs a, KvCache c) {
  constexpr int U = 16;      // tokens of a lane whose weights are fetched at once
  constexpr int kCopies = 8; // of the counts: equal digits are counted one after the other
  __shared__ uint32_t bins[kCopies][256 + 4], count_gt[kWaves], count_eq[kWaves];
  __shared__ uint32_t found, left;
  const int b = blockIdx.x, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = clamped(a, c, b);
  const float *w = a.weights + (int64_t)b * a.stride;
  int32_t *kept = a.kept + (int64_t)b * a.keep;
  float *got = a.new_weights + (int64_t)b * a.keep;
  const int total = n < a.keep ? n : a.keep;
  for (int i = total + (int)threadIdx.x; i < a.keep; i += kSelect) kept[i] = -1, got[i] = 0.f;
  if (n <= a.keep) {
    for (int i = threadIdx.x; i < n; i += kSelect) kept[i] = i, got[i] = w[i];
    __syncthreads();  // (lengths may be new_lengths)
    if (threadIdx.x == 0) a.new_lengths[b] = n;
    return;
  }

  // candidates: sinks <= i < n - recent, of which `want` are kept
  const int lo = a.sinks, hi = n - a.recent;
  const uint32_t want = (uint32_t)(a.keep - a.sinks - a.recent);
  // a wave's run of neighbouring tokens, in whole ballots; the keys of a run that is no longer than a
  // round stay in registers, others are fetched again for every pass
  const int per = (n + kSelect - 1) / kSelect * 64;
  const int begin = wave * per < n ? wave * per : n, end = begin + per < n ? begin + per : n;
  uint32_t keys[U];
  auto fetch = [&](int i0) {
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 64 + lane;
      x[u] = w[i < end ? i : 0];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) keys[u] = key_of(x[u]);
  };
  const bool once = per <= U * 64;
  if (once) fetch(begin);

  uint32_t key = 0, mask = 0, rest = want;
  if (want) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < kCopies * 260; i += kSelect) (&bins[0][0])[i] = 0;
      __syncthreads();
      for (int i0 = begin; i0 < end; i0 += U * 64) {
        if (!once) fetch(i0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * 64 + lane;
          if (i < end && i >= lo && i < hi && (keys[u] & mask) == key)
            atomicAdd(&bins[lane & (kCopies - 1)][(keys[u] >> shift) & 255], 1u);
        }
      }
      __syncthreads();
      if (wave == 0) {
        // from the top: the digit in which the count passes `rest`; lane l has the digits
        // 255 - 4 l down to 252 - 4 l
        uint32_t own[4] = {0, 0, 0, 0}, sum = 0;
#pragma unroll
        for (int x = 0; x < kCopies; ++x) {
          const uint4 four = *reinterpret_cast<const uint4 *>(&bins[x][252 - 4 * lane]);
          own[0] += four.w, own[1] += four.z, own[2] += four.y, own[3] += four.x;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sum += own[j];
        uint32_t upto = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const uint32_t x = __shfl_up(upto, d);
          upto += lane >= d ? x : 0;
        }
        const uint64_t past = __ballot(upto >= rest);
        if (lane == __builtin_ctzll(past)) {
          uint32_t before = upto - sum;
          int j = 0;
#pragma unroll
          for (int x = 0; x < 3; ++x)
            if (j == x && before + own[x] < rest) before += own[x], ++j;
          found = 255 - 4 * lane - j;
          left = rest - before;
        }
      }
      __syncthreads();
      key |= found << shift;
      mask |= 255u << shift;
      rest = left;
      __syncthreads();
    }
  }
  // larger keys are kept, and the first `rest` equal ones (none of no candidates)
  auto look = [&](int i, uint32_t k, uint64_t &gt, uint64_t &eq) {
    const bool in = i < end, edge = i < lo || i >= hi;
    gt = __ballot(in && (edge || (want && k > key)));
    eq = __ballot(in && !edge && want && k == key);
  };
  uint32_t gts = 0, eqs = 0;
  for (int i0 = begin; i0 < end; i0 += U * 64) {
    if (!once) fetch(i0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint64_t gt, eq;
      look(i0 + u * 64 + lane, keys[u], gt, eq);
      gts += __builtin_popcountll(gt);
      eqs += __builtin_popcountll(eq);
    }
  }
  if (lane == 0) count_gt[wave] = gts, count_eq[wave] = eqs;
  __syncthreads();
  uint32_t at = 0, seen = 0;  // kept tokens and equal ones ahead of this run
  for (int x = 0; x < wave; ++x) at += count_gt[x], seen += count_eq[x];
  at += seen < rest ? seen : rest;
  for (int i0 = begin; i0 < end; i0 += U * 64) {
    if (!once) fetch(i0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 64 + lane;
      uint64_t gt, eq;
      look(i, keys[u], gt, eq);
      const uint32_t before = lanes_before(eq);
      const bool in = gt >> lane & 1 || (eq >> lane & 1 && seen + before < rest);
      const uint64_t all = __ballot(in);
      if (in) {
        const uint32_t to = at + lanes_before(all);
        kept[to] = i;
        got[to] = w[i];
      }
      at += __builtin_popcountll(all);
      seen += __builtin_popcountll(eq);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) a.new_lengths[b] = total;
}

// one row of `bytes` is moved in pieces of P bytes, 1 << shift of them
template <int P> struct Piece;
template <> struct Piece<16> { typedef uint4 type; };
template <> struct Piece<8> { typedef uint2 type; };
template <> struct Piece<4> { typedef uint32_t type; };
template <> struct Piece<2> { typedef uint16_t type; };

constexpr int kMoveTokens = 64;  // of a workgroup

// Rows of `tokens` kept tokens: from[i], to[i] their row numbers in LDS (-1: not there)
template <int P>
__device__ __forceinline__ void move_rows(void *array, const int64_t *from, const int64_t *to, int n, int shift) {
  typedef typename Piece<P>::type T;
  constexpr int U = 4;
  T *x = reinterpret_cast<T *>(array);
  const int items = n << shift, mask = (1 << shift) - 1;
  for (int i0 = threadIdx.x; i0 < items; i0 += U * 256) {
    T got[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 256 < items ? i0 + u * 256 : i0;
      const int64_t row = from[i >> shift];
      got[u] = x[((row < 0 ? 0 : row) << shift) + (i & mask)];
      if (row < 0) got[u] = T{};
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 256;
      if (i < items && to[i >> shift] >= 0) x[(to[i >> shift] << shift) + (i & mask)] = got[u];
    }
  }
}

__device__ __forceinline__ void move_array(void *array, int bytes, const int64_t *from, const int64_t *to, int n) {
  if (bytes >= 16)
    move_rows<16>(array, from, to, n, __builtin_ctz(bytes) - 4);
  else if (bytes == 8)
    move_rows<8>(array, from, to, n, 0);
  else if (bytes == 4)
    move_rows<4>(array, from, to, n, 0);
  else
    move_rows<2>(array, from, to, n, 0);
}

// blockIdx.x: sequence, run of kept tokens, head; blockIdx.y: keys or values
__global__ __launch_bounds__(256) void move_kernel(EvictArgs a, KvCache c, uint32_t runs) {
  __shared__ int64_t from[kMoveTokens], to[kMoveTokens];
  const uint32_t h = blockIdx.x % (uint32_t)c.kv_heads, rest = blockIdx.x / (uint32_t)c.kv_heads;
  const uint32_t b = rest / runs, first = rest % runs * kMoveTokens;
  if ((int)threadIdx.x < kMoveTokens) {
    const uint32_t i = first + threadIdx.x;
    const int old = i < (uint32_t)a.keep ? a.kept[(int64_t)b * a.keep + i] : -1;
    int64_t x = -1, y = -1;
    if (old >= 0) {
      const uint32_t size = (uint32_t)c.page_size;
      const uint32_t op = (uint32_t)old / size, np = i / size;
      const int src = a.table[b * a.max_pages + op], dst = a.new_table[b * a.new_max_pages + np];
      if (src >= 0 && src < c.num_pages) x = ((int64_t)src * c.kv_heads + h) * size + ((uint32_t)old - op * size);
      if (dst >= 0 && dst < c.num_pages) y = ((int64_t)dst * c.kv_heads + h) * size + (i - np * size);
    }
    from[threadIdx.x] = x, to[threadIdx.x] = y;
  }
  __syncthreads();
  const int n = a.keep - first < kMoveTokens ? a.keep - (int)first : kMoveTokens;
  const bool is_v = blockIdx.y != 0;
  move_array(is_v ? c.v_codes : c.k_codes, c.head_dim * c.bits / 8, from, to, n);
  if (c.bits == 16) return;
  const int bytes = c.head_dim / c.group_size * 2;
  move_array(is_v ? c.v_scales : c.k_scales, bytes, from, to, n);
  uint16_t *biases = is_v ? c.v_biases : c.k_biases;
  if (biases) move_array(biases, bytes, from, to, n);
}

}  // namespace

hipError_t launch_kv_evict(const EvictArgs &a, const KvCache &c, hipStream_t s) {
  hipLaunchKernelGGL(select_kernel, dim3(a.B), dim3(kSelect), 0, s, a, c);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const uint32_t runs = (uint32_t)((a.keep + kMoveTokens - 1) / kMoveTokens);
  hipLaunchKernelGGL(move_kernel, dim3((unsigned)a.B * runs * (unsigned)c.kv_heads, 2), dim3(256), 0, s, a, c, runs);
  return hipGetLastError();
}

}  // namespace aq
