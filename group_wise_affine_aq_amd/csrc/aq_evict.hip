// aq_evict.hip -- the tokens of each cached sequence that gathered most of the
// attention, chosen and moved to other pages (gfx950).
//
// Choosing.  One workgroup per sequence finds the least key that is kept by
// radix: weights become 32-bit keys in their order, those of the first and last
// tokens the largest there is, and four counts of 8 bits each narrow down the key, each count
// over the keys that share the bits found so far.  Then every wave takes
// a run of neighbouring tokens: it counts the larger keys and the equal ones,
// the counts of the waves before it say where its own kept tokens go and how
// many equal ones are still to be taken, and a second pass writes positions
// and weights, 64 tokens at a time by their ballots.  All counts are whole
// numbers, so the result does not depend on their order.
//
// Moving is copying rows: a workgroup takes neighbouring kept tokens of one
// head, keys or values, whose new places are neighbours, 16 bytes a thread and
// several loads under way.  It is bound by HBM (24 sequences of 2048 kept tokens,
// 8 heads of 128 at 8 bits: 219 MB in 42 us, 5.2 TB/s); the choice by the latency
// of its passes in one workgroup a sequence (24 of up to 8192 tokens 13 us, one of
// 131072 131 us: past 16384 tokens every pass reads the weights again).
#include "aq_device.hpp"
#include "aq_internal.hpp"

namespace aq {
namespace {

constexpr int kSelect = 1024;  // threads that choose
constexpr int kWaves = kSelect / 64;

// Weights in their order: NaN, below everything, is 1, and no weight is 0 or
// kAlways (the patterns of NaNs).
constexpr uint32_t kNever = 0, kAlways = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t u = __builtin_bit_cast(uint32_t, w + 0.f);  // (-0 and +0 are equal)
  const uint32_t key = u ^ (0x80000000u | (uint32_t)((int)u >> 31));
  return w == w ? key : 1u;
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
  __shared__ __align__(16) uint32_t bins[4][kCopies][256 + 4];  // of every digit
  __shared__ uint32_t count_gt[kWaves], count_eq[kWaves];
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

  // a wave's run of neighbouring tokens, in whole ballots; the keys of a run that is no longer than a
  // round stay in registers, others are made again for every pass.  The first and last tokens have the
  // largest key, places behind the run one below all, so that the `keep` largest are what is kept.
  const int lo = a.sinks, hi = n - a.recent;
  const int per = (n + kSelect - 1) / kSelect * 64;
  const int begin = wave * per < n ? wave * per : n, end = begin + per < n ? begin + per : n;
  float x[U];
  uint32_t k[U];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 64 + lane;
      x[u] = w[i < end ? i : 0];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 64 + lane;
      k[u] = i < lo || i >= hi ? kAlways : key_of(x[u]);
      k[u] = i < end ? k[u] : kNever;
    }
  };
  const bool once = per <= U * 64;
  if (once) fetch(begin);
  // (rounds of a run, and within one the ballots that it has)
  auto every = [&](auto visit) {
    for (int i0 = begin; i0 < end; i0 += U * 64) {
      if (!once) fetch(i0);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * 64 < end) visit(i0 + u * 64 + lane, k[u], x[u]);
    }
  };

  uint32_t key = 0, mask = 0, rest = (uint32_t)a.keep;
  for (int i = threadIdx.x; i < 4 * kCopies * 260; i += kSelect) (&bins[0][0][0])[i] = 0;
  __syncthreads();
#pragma unroll 1
  for (int digit = 0; digit < 4; ++digit) {
    const int shift = 24 - 8 * digit;
    uint32_t *mine = bins[digit][lane & (kCopies - 1)];
    every([&](int, uint32_t k, float) {
      if ((k & mask) == key) atomicAdd(mine + (k >> shift & 255), 1u);
    });
    __syncthreads();
    // every wave finds, from the top, the digit in which the count passes `rest`; lane l has the
    // digits 255 - 4 l down to 252 - 4 l
    uint32_t own[4] = {0, 0, 0, 0}, sum = 0;
#pragma unroll
    for (int copy = 0; copy < kCopies; ++copy) {
      const uint4 four = *reinterpret_cast<const uint4 *>(&bins[digit][copy][252 - 4 * lane]);
      own[0] += four.w, own[1] += four.z, own[2] += four.y, own[3] += four.x;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sum += own[j];
    const uint32_t upto = lanes_prefix(sum);
    const int l = __builtin_ctzll(__ballot(upto >= rest));
    uint32_t before = upto - sum, found = 255u - 4u * (uint32_t)lane;
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (before + own[j] < rest && found == 255u - 4u * (uint32_t)lane - j) before += own[j], --found;
    key |= (uint32_t)__builtin_amdgcn_readlane((int)found, l) << shift;
    mask |= 255u << shift;
    rest -= (uint32_t)__builtin_amdgcn_readlane((int)before, l);
  }
  // larger keys are kept, and the first `rest` equal ones
  uint32_t gts = 0, eqs = 0;
  every([&](int, uint32_t k, float) { gts += k > key, eqs += k == key; });
  gts = (uint32_t)__builtin_amdgcn_readlane((int)lanes_prefix(gts), 63);
  eqs = (uint32_t)__builtin_amdgcn_readlane((int)lanes_prefix(eqs), 63);
  if (lane == 0) count_gt[wave] = gts, count_eq[wave] = eqs;
  __syncthreads();
  uint32_t at = 0, seen = 0;  // kept tokens and equal ones ahead of this run
  for (int i = 0; i < wave; ++i) at += count_gt[i], seen += count_eq[i];
  at += seen < rest ? seen : rest;
  every([&](int i, uint32_t k, float w) {
    bool in = k > key;
    const uint64_t eq = __ballot(k == key);
    if (eq && seen < rest) {
      in = in || (k == key && seen + lanes_before(eq) < rest);
      seen += __builtin_popcountll(eq);
    }
    const uint64_t all = __ballot(in);
    if (in) {
      const uint32_t to = at + lanes_before(all);
      kept[to] = i;
      got[to] = w;
    }
    at += __builtin_popcountll(all);
  });
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
