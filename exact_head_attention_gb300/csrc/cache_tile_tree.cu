// Attention over the 8-bit cache for many query rows (cache_tile.cuh), the rows a tree of drafted tokens.
#include "cache_tile.cuh"

namespace exattn {

cudaError_t launch_cache_tile_tree(const CacheAttnArgs& a, cudaStream_t stream) {
  return a.c.d == 128 ? launch_d<128, true>(a, stream) : launch_d<64, true>(a, stream);
}

}  // namespace exattn
