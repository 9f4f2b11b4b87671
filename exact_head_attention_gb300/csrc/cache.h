// Arguments and launchers of the 8-bit key/value cache's kernels, shared by cache_api.cu and their translation
// units.  Not part of the public header.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "kernels.h"

namespace exattn {

// Device error word, besides the kErr* of ptx.cuh: a page number outside the pool, or a length outside its page table.
constexpr uint32_t kErrPage = 9;

// The 8-bit key/value cache (attn_cache) as the kernels take it.
struct CacheView {
  uint8_t *k, *v;            // [num_pages][heads][page][d] codes
  float *k_scale, *v_scale;  // [num_pages][heads]
  const int* table;          // [B][width]
  int num_pages, heads, page_shift, d, width;
  int capacity;  // tokens a table row can name: width << page_shift, at most 2^31 - 1
  int format;    // attn_cache_format
};

struct CacheIoArgs {
  CacheView c;
  void *k, *v;  // 16-bit [B][heads][N][d], strides sk and sv
  RowStrides sk, sv;
  const int *start, *count;  // write: may be nullptr; read: count is lens
  int B, N;
  int parts;  // units a sequence and head: pages that N tokens can reach (write), groups of rows (read)
  int sm_count;
  bool bf16;
  uint32_t* err_word;
};

// Attention over the cache.  The query rows of a key/value head are its group's heads and the Nq tokens
// together: row r is token r / group and head r % group of the group, so that the causal limit grows
// with r.
struct CacheAttnArgs {
  CUtensorMap tm_k, tm_v;  // 2-D byte maps {128, lines} over the codes, box {128, lines of box_tokens tokens}
  CacheView c;
  const void* q;
  void* o;
  RowStrides sq, so;
  const int* lens;
  float* lse;     // [B][heads * group][Nq]
  uint8_t* ws;    // cache_sched.cuh
  unsigned long long tag;  // of this call's counts in ws: not zero, the low 16 bits are
  uint32_t* err_word;
  int B, Nq, group, mask, sm_count;
  bool bf16;
  float scale;
  uint64_t timeout_ns;
};

// Allows `kernel` its dynamic shared memory, once on each device (`done`: a bit for each of the first 64).
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launches a kernel with programmatic stream serialisation: it may start before the kernel ahead of it
// on the stream has finished, and waits for that itself (griddep_wait).
template <typename Args>
cudaError_t launch_dependent(void (*kernel)(const Args), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                             const Args& args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

cudaError_t launch_cache_write(CacheIoArgs& a, cudaStream_t stream);
cudaError_t launch_cache_read(CacheIoArgs& a, cudaStream_t stream);
cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t stream);
cudaError_t launch_cache_tile(const CacheAttnArgs& a, cudaStream_t stream);
// Up to this many query rows a key/value head attn_fwd_cache streams the codes through the warp-level products
// (cache_attn.cu), above it through the tensor-memory ones (cache_tile.cu).  The first keep Q and O in registers: with
// 32 rows those run out, with 24 the codes still set the pace.  Measured, warp-level against tensor-memory:
//   8 sequences of 32k tokens, 12 heads of 128   17 rows 158 : 242 us   24 rows 160 : 243 us   32 rows 272 : 243 us
//   the same, 24 heads of 64                     17 rows 197 : 221 us   24 rows 197 : 221 us   32 rows 277 : 221 us
//   4 sequences of 300 tokens, 4 heads of 128    20 rows 15.6 : 13.8 us                        32 rows 29.5 : 14.5 us
// (the lengths are not known where the choice is made; the warp-level form for 32 rows is gone since its measurement).
constexpr int kCacheStreamRows = 24;
// Tokens per box of the tensor maps launch_cache_attn wants; query rows and keys of its tiles for so many
// rows a key/value head; its workspace bytes.
int cache_attn_box_tokens(int page, int d);
constexpr int kCacheItemCost = 32;  // above every cache_item_cost plus a rounded-up tile
struct CacheAttnShape {
  int rows, keys;
};
CacheAttnShape cache_attn_shape(long long rows, int d);
size_t cache_attn_workspace(long long rows, int d, int sm_count);

}  // namespace exattn
