// C-ABI entry points of the 8-bit key/value cache: argument checks, tensor maps and dispatch.
#include <cmath>
#include <cstring>

#include "api_internal.h"
#include "cache.h"

using namespace exattn;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

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

extern "C" attn_status attn_cache_append(const attn_cache* cache, const void* Q, attn_strides q_strides, void* Qr,
                                         attn_strides qr_strides, const void* K, attn_strides k_strides, const void* V,
                                         attn_strides v_strides, const int* start, const int* count, int B, int H, int N,
                                         const attn_rope* rope, attn_dtype dtype, void* stream) {
  CacheAppendArgs a;
  std::memset(&a, 0, sizeof(a));
  attn_status st = io_args(cache, K, k_strides, V, v_strides, start, count, B, N, dtype, &a.io);
  if (st != ATTN_OK) return st;
  if (H < 0 || H > 65535 || static_cast<long long>(B) * N > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  const bool normed = rope && ((H && rope->q_weight) || rope->k_weight);
  if ((st = api_rope(rope, B, N, cache->d, normed, &a.rope.r)) != ATTN_OK) return st;
  if (!a.rope.r.start) a.rope.r.start = start;
  if (H > 0) {
    RopeSide& q = a.rope.side[0];
    if (!Q || !Qr || !api_strides(q_strides, B, H, cache->d, &q.sx) || !api_strides(qr_strides, B, H, cache->d, &q.sy))
      return ATTN_ERR_INVALID_ARG;
    if (!aligned(Q, 16) || !aligned(Qr, 16)) return ATTN_ERR_MISALIGNED;
    q.x = Q;
    q.y = Qr;
    q.weight = rope->q_weight;
    q.heads = H;
  }
  DeviceInfo dev;
  if ((st = api_device(&dev)) != ATTN_OK) return st;
  a.io.err_word = dev.err_word;
  a.io.sm_count = a.rope.sm_count = dev.sm_count;
  a.rope.B = B;
  a.rope.N = N;
  a.rope.d = cache->d;
  a.rope.tokens = B * N;
  a.rope.bf16 = a.io.bf16;
  a.rope.weight_fp32 = rope->weight_fp32 != 0;
  a.k_weight = rope->k_weight;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return api_finish(launch_cache_append(a, s), s);
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

namespace {

// attn_fwd_cache, and with a tree attn_fwd_cache_tree.
attn_status fwd_cache(const void* Q, attn_strides q_strides, const attn_cache* cache, const int* lens, void* O,
                      attn_strides o_strides, float* LSE, int B, int H, int Nq, int causal, float scale, attn_dtype dtype,
                      void* workspace, size_t workspace_bytes, void* stream, const uint32_t* tree, long long tree_stride) {
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
  a.tag = api_next_tag();
  a.err_word = dev.err_word;
  a.B = B;
  a.Nq = Nq;
  a.group = group;
  a.mask = causal;
  a.sm_count = dev.sm_count;
  a.bf16 = dtype == ATTN_BF16;
  a.scale = scale;
  a.timeout_ns = api_wait_timeout_ns();
  a.tree = tree;
  a.tree_stride = tree_stride;
  a.tree_words = (Nq + 31) / 32;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return api_finish(tree ? launch_cache_attn_tree(a, s) : launch_cache_attn(a, s), s);
}

}  // namespace

extern "C" attn_status attn_fwd_cache(const void* Q, attn_strides q_strides, const attn_cache* cache, const int* lens,
                                      void* O, attn_strides o_strides, float* LSE, int B, int H, int Nq, int causal,
                                      float scale, attn_dtype dtype, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  return fwd_cache(Q, q_strides, cache, lens, O, o_strides, LSE, B, H, Nq, causal, scale, dtype, workspace, workspace_bytes,
                   stream, nullptr, 0);
}

extern "C" attn_status attn_fwd_cache_tree(const void* Q, attn_strides q_strides, const attn_cache* cache, const int* lens,
                                           const uint32_t* tree, long long tree_stride, void* O, attn_strides o_strides,
                                           float* LSE, int B, int H, int Nq, float scale, attn_dtype dtype, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  if (!tree || Nq > ATTN_TREE_MAX_TOKENS) return ATTN_ERR_INVALID_ARG;
  if (!aligned(tree, 4)) return ATTN_ERR_MISALIGNED;
  const long long words = (Nq + 31) / 32 * static_cast<long long>(Nq);
  if (B > 1 && tree_stride != 0 && (tree_stride < words || tree_stride > (1ll << 39))) return ATTN_ERR_INVALID_ARG;
  return fwd_cache(Q, q_strides, cache, lens, O, o_strides, LSE, B, H, Nq, ATTN_MASK_CAUSAL_BOTTOM_RIGHT, scale, dtype, workspace,
                   workspace_bytes, stream, tree, B > 1 ? tree_stride : 0);
}

extern "C" attn_status attn_draft_tree(const int* parents, uint32_t* mask, int* depth, int B, int N, void* stream) {
  if (!parents || !mask || !depth || B <= 0 || N <= 0 || N > ATTN_TREE_MAX_TOKENS) return ATTN_ERR_INVALID_ARG;
  if (!aligned(parents, 4) || !aligned(mask, 4) || !aligned(depth, 4)) return ATTN_ERR_MISALIGNED;
  DeviceInfo dev;
  const attn_status st = api_device(&dev);
  if (st != ATTN_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return api_finish(launch_draft_tree(DraftTreeArgs{parents, mask, depth, N, dev.err_word}, B, s), s);
}
