// Attention over the 8-bit cache for few query rows (cache_attn.cuh), the rows a tree of drafted tokens: a row's word has
// bits for them all.
#include "cache_attn.cuh"

namespace exattn {

static_assert(kCacheStreamRows <= 32, "one word a row");

cudaError_t launch_cache_attn_tree(const CacheAttnArgs& a, cudaStream_t stream) {
  if (static_cast<long long>(a.group) * a.Nq > kCacheStreamRows) return launch_cache_tile_tree(a, stream);
  return a.c.d == 128 ? launch_d<128, true>(a, stream) : launch_d<64, true>(a, stream);
}

}  // namespace exattn
