// aq_attn_masked.hip -- attention of each sequence's newest tokens over the
// paged cache, scores capped, biased by distance and masked (gfx950);
// aq_attn.hpp has the kernels.
#include "aq_attn.hpp"

namespace aq {

hipError_t launch_paged_attention_masked(const AttnArgs &a, const KvCache &c, hipStream_t s) {
  return launch<true>(a, c, s);
}

}  // namespace aq
