// aq_attn.hip -- attention of each sequence's newest tokens over the paged
// cache, plain scores (gfx950); aq_attn.hpp has the kernels.
#include "aq_attn.hpp"

namespace aq {

int64_t attn_workspace_bytes(int64_t, int L, int q_heads, int kv_heads, int head_dim) {
  int nt, slices;
  tiles_for((int64_t)L * (q_heads / kv_heads), head_dim, nt, slices);
  const int wgs = device_cus() * wgs_per_cu(8, head_dim, 1, nt);
  return kMaxGrid * 12 + (int64_t)(wgs < kMaxGrid ? wgs : kMaxGrid) * 2 * piece_floats(head_dim, nt) * 4;
}

hipError_t launch_paged_attention(const AttnArgs &a, const KvCache &c, hipStream_t s) {
  return launch<false>(a, c, s);
}

}  // namespace aq
