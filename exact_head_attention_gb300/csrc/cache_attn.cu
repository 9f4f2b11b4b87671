// Attention over the 8-bit cache for few query rows (cache_attn.cuh): the launch without a tree, and the sizes that go with it.
#include "cache_attn.cuh"

namespace exattn {

int cache_attn_box_tokens(int page, int d) { return page < 4096 / d ? page : 4096 / d; }

CacheAttnShape cache_attn_shape(long long rows, int d) {
  if (rows > kCacheStreamRows) return {rows > 128 ? 256 : 128, 128};
  return {static_cast<int>((rows + 7) / 8 * 8), 4096 / d};
}

size_t cache_attn_workspace(long long rows, int d, int sm_count) {
  const int workers = rows > kCacheStreamRows ? sm_count : sm_count * kWorkers;
  return (cache_ws_bytes(cache_attn_shape(rows, d).rows, d, workers) + 255) & ~static_cast<size_t>(255);
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t stream) {
  if (static_cast<long long>(a.group) * a.Nq > kCacheStreamRows) return launch_cache_tile(a, stream);
  return a.c.d == 128 ? launch_d<128, false>(a, stream) : launch_d<64, false>(a, stream);
}

}  // namespace exattn
