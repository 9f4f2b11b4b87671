// Attention over the 8-bit cache for many query rows (cache_tile.cuh).
#include "cache_tile.cuh"

namespace exattn {

cudaError_t launch_cache_tile(const CacheAttnArgs& a, cudaStream_t stream) {
  return a.c.d == 128 ? launch_d<128, false>(a, stream) : launch_d<64, false>(a, stream);
}

}  // namespace exattn
