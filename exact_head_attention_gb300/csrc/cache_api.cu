// C-ABI entry points of the 8-bit key/value cache: argument checks, tensor maps and dispatch.
#include <atomic>
#include <cmath>
#include <cstring>
#include <random>

#include "api_internal.h"
#include "cache.h"

using namespace exattn;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A number that no earlier call and no old contents of a workspace are likely to hold: a counter from a random
// start, through the finaliser of the splitmix64 generator (Steele, Lea and Flood, 2014).
unsigned long long next_tag() {
  static std::atomic<unsigned long long> count{[] {
    std::random_device r;
    return (static_cast<unsigned long long>(r()) << 32) ^ r();
  }()};
  unsigned long long z = count.fetch_add(0x9e3779b97f4a7c15ull, std::memory_order_relaxed);
  z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
  z = (z ^ (z >> 27)) * 0x94d049bb133111ebull;
  z ^= z >> 31;
  z &= ~0xffffull;                  // the count's place
  return z ? z : 0x10000ull;  // zero is a count at rest
}

// The rules of attn_cache, and its view for the kernels.
attn_status check_cache(const attn_cache* c, CacheView* out) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !c->page_table) return ATTN_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->heads <= 0 || c->table_width <= 0) return ATTN_ERR_INVALID_ARG;
  if (c->format != ATTN_CACHE_E4M3 && c->format != ATTN_CACHE_INT8) return ATTN_ERR_INVALID_ARG;
  int shift;
  switch (c->page_size) {
    case 16: shift = 4; break;
    case 32: shift = 5; break;
    case 64: shift = 6; break;
    case 128: shift = 7; break;
    default: return ATTN_ERR_INVALID_ARG;
  }
  if (c->d != 64 && c->d != 128) return ATTN_ERR_UNSUPPORTED;
  // Lines of 128 bytes are numbered in an int by the tensor maps.
  const long long lines_a_page = static_cast<long long>(c->page_size) * c->d / 128;
  if (static_cast<long long>(c->num_pages) * c->heads > 0x7fffffffLL / lines_a_page) return ATTN_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(c->page_table, 4))
    return ATTN_ERR_MISALIGNED;
  out->k = static_cast<uint8_t*>(c->k);
  out->v = static_cast<uint8_t*>(c->v);
  out->k_scale = c->k_scale;
  out->v_scale = c->v_scale;
  out->table = c->page_table;
  out->num_pages = c->num_pages;
  out->heads = c->heads;
  out->page_shift = shift;
  out->d = c->d;
  out->width = c->table_width;
  const long long cap = static_cast<long long>(c->table_width) << shift;
  out->capacity = static_cast<int>(cap < 0x7fffffffLL ? cap : 0x7fffffffLL);
  out->format = c->format;
  return ATTN_OK;
}

attn_status io_args(const attn_cache* cache, const void* K, attn_strides ks, const void* V, attn_strides vs,
                    const int* start, const int* count, int B, int N, attn_dtype dtype, CacheIoArgs* a) {
  if (B <= 0 || N <= 0 || !K || !V) return ATTN_ERR_INVALID_ARG;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16) return ATTN_ERR_INVALID_ARG;
  attn_status st = check_cache(cache, &a->c);
  if (st != ATTN_OK) return st;
  if (!api_strides(ks, B, cache->heads, cache->d, &a->sk) || !api_strides(vs, B, cache->heads, cache->d, &a->sv))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(start, 4) || !aligned(count, 4)) return ATTN_ERR_MISALIGNED;
  // units of the launches, at the fewest rows (16) that one takes
  if (static_cast<long long>(B) * cache->heads > 0x3fffffffLL / (N / 16 + 2)) return ATTN_ERR_INVALID_ARG;
  a->k = const_cast<void*>(K);
  a->v = const_cast<void*>(V);
  a->start = start;
  a->count = count;
  a->B = B;
  a->N = N;
  a->bf16 = dtype == ATTN_BF16;
  return ATTN_OK;
}

// Sizes of attn_fwd_cache; the rows of all heads together, and the tiles of the longest sequences that the
// table allows, are counted in 32 bits.
attn_status check_attn(const attn_cache* cache, int B, int H, int Nq, CacheView* view) {
  if (B <= 0 || H <= 0 || Nq <= 0) return ATTN_ERR_INVALID_ARG;
  const attn_status st = check_cache(cache, view);
  if (st != ATTN_OK) return st;
  if (H % cache->heads != 0) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * H > 0x7fffffffLL / Nq) return ATTN_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(H / cache->heads) * Nq;
  const CacheAttnShape sh = cache_attn_shape(rows, cache->d);
  const long long items = static_cast<long long>(B) * cache->heads * ((rows + sh.rows - 1) / sh.rows);
  if (items > 0x7fffffffLL / (view->capacity / sh.keys + kCacheItemCost)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

}  // namespace

extern "C" attn_status attn_cache_write(const attn_cache* cache, const void* K, attn_strides k_strides, const void* V,
                                        attn_strides v_strides, const int* start, const int* count, int B, int N,
                                        attn_dtype dtype, void* stream) {
  CacheIoArgs a;
  attn_status st = io_args(cache, K, k_strides, V, v_strides, start, count, B, N, dtype, &a);
  if (st != ATTN_OK) return st;
  DeviceInfo dev;
  if ((st = api_device(&dev)) != ATTN_OK) return st;
  a.err_word = dev.err_word;
  a.sm_count = dev.sm_count;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return api_finish(launch_cache_write(a, s), s);
}

extern "C" attn_status attn_cache_read(const attn_cache* cache, const int* start, const int* lens, void* K,
                                       attn_strides k_strides, void* V, attn_strides v_strides, int B, int N,
                                       attn_dtype dtype, void* stream) {
  if (!lens) return ATTN_ERR_INVALID_ARG;
  CacheIoArgs a;
  attn_status st = io_args(cache, K, k_strides, V, v_strides, start, lens, B, N, dtype, &a);
  if (st != ATTN_OK) return st;
  DeviceInfo dev;
  if ((st = api_device(&dev)) != ATTN_OK) return st;
  a.err_word = dev.err_word;
  a.sm_count = dev.sm_count;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return api_finish(launch_cache_read(a, s), s);
}

extern "C" size_t attn_fwd_cache_workspace_size(const attn_cache* cache, int B, int H, int Nq) {
  CacheView view;
  if (check_attn(cache, B, H, Nq, &view) != ATTN_OK) return 0;
  const int sms = api_sm_count();
  if (sms <= 0) return 0;
  return cache_attn_workspace(static_cast<long long>(H / cache->heads) * Nq, cache->d, sms);
}

extern "C" attn_status attn_fwd_cache(const void* Q, attn_strides q_strides, const attn_cache* cache, const int* lens,
                                      void* O, attn_strides o_strides, float* LSE, int B, int H, int Nq, int causal,
                                      float scale, attn_dtype dtype, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  CacheAttnArgs a;
  std::memset(&a, 0, sizeof(a));
  attn_status st = check_attn(cache, B, H, Nq, &a.c);
  if (st != ATTN_OK) return st;
  if (!Q || !O || !LSE || !lens) return ATTN_ERR_INVALID_ARG;
  if (causal != ATTN_MASK_NONE && causal != ATTN_MASK_CAUSAL && causal != ATTN_MASK_CAUSAL_BOTTOM_RIGHT)
    return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16) return ATTN_ERR_INVALID_ARG;
  if (!api_strides(q_strides, B, H, cache->d, &a.sq) || !api_strides(o_strides, B, H, cache->d, &a.so))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(O, 16) || !aligned(LSE, 4) || !aligned(lens, 4)) return ATTN_ERR_MISALIGNED;
  if (!workspace) return ATTN_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return ATTN_ERR_MISALIGNED;
  DeviceInfo dev;
  if ((st = api_device(&dev)) != ATTN_OK) return st;
  const int group = H / cache->heads;
  if (workspace_bytes < cache_attn_workspace(static_cast<long long>(group) * Nq, cache->d, dev.sm_count))
    return ATTN_ERR_WORKSPACE;
  const uint64_t lines = static_cast<uint64_t>(cache->num_pages) * cache->heads * cache->page_size * cache->d / 128;
  const uint32_t box = static_cast<uint32_t>(cache_attn_box_tokens(cache->page_size, cache->d) * cache->d / 128);
  CUresult r;
  if (group * static_cast<long long>(Nq) <= kCacheStreamRows &&
      ((r = api_encode_lines(&a.tm_k, cache->k, lines, box)) != CUDA_SUCCESS ||
       (r = api_encode_lines(&a.tm_v, cache->v, lines, box)) != CUDA_SUCCESS))
    return api_driver_fail("cuTensorMapEncodeTiled", r);
  a.q = Q;
  a.o = O;
  a.lens = lens;
  a.lse = LSE;
  a.ws = static_cast<uint8_t*>(workspace);
  a.tag = next_tag();
  a.err_word = dev.err_word;
  a.B = B;
  a.Nq = Nq;
  a.group = group;
  a.mask = causal;
  a.sm_count = dev.sm_count;
  a.bf16 = dtype == ATTN_BF16;
  a.scale = scale;
  a.timeout_ns = api_wait_timeout_ns();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return api_finish(launch_cache_attn(a, s), s);
}
