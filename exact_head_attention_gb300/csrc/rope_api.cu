// C-ABI entry points of the rotary positions: argument checks and dispatch.
#include <atomic>
#include <cmath>
#include <cstring>
#include <random>

#include "api_internal.h"
#include "rope.h"

using namespace exattn;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }


// Sizes and the tensors' common rules; side i has heads[i] heads.
attn_status check_sizes(int B, int N, int d, const int (&heads)[2], attn_dtype dtype) {
  if (B <= 0 || N <= 0 || heads[0] < 0 || heads[1] < 0 || heads[0] + static_cast<long long>(heads[1]) == 0)
    return ATTN_ERR_INVALID_ARG;
  if (heads[0] > 65535 || heads[1] > 65535 || static_cast<long long>(B) * N > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16) return ATTN_ERR_INVALID_ARG;
  return d == 64 || d == 128 ? ATTN_OK : ATTN_ERR_UNSUPPORTED;
}

attn_status check_tensor(const void* p, const attn_strides& st, int B, int heads, int d, RowStrides* out) {
  if (!p || !api_strides(st, B, heads, d, out)) return ATTN_ERR_INVALID_ARG;
  return aligned(p, 16) ? ATTN_OK : ATTN_ERR_MISALIGNED;
}

}  // namespace

// A counter from a random start, through the finaliser of the splitmix64 generator (Steele, Lea and Flood, 2014).
unsigned long long exattn::api_next_tag() {
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

attn_status exattn::api_rope(const attn_rope* rope, int B, int N, int d, bool normed, RopeView* out) {
  if (!rope) return ATTN_ERR_INVALID_ARG;
  if (rope->rotary_dim < 0 || rope->rotary_dim > d || rope->rotary_dim % 16 != 0) return ATTN_ERR_INVALID_ARG;
  if (rope->layout != ATTN_ROPE_HALF && rope->layout != ATTN_ROPE_INTERLEAVED) return ATTN_ERR_INVALID_ARG;
  if (rope->rotary_dim > 0 && (!rope->freq || !std::isfinite(rope->amplitude))) return ATTN_ERR_INVALID_ARG;
  if (rope->offsets && B > 1 && rope->offset_stride != 0 && rope->offset_stride < N) return ATTN_ERR_INVALID_ARG;
  if (rope->offsets && rope->offset_stride > (1ll << 39)) return ATTN_ERR_INVALID_ARG;
  if (normed && (!std::isfinite(rope->eps) || !(rope->eps > 0.f))) return ATTN_ERR_INVALID_ARG;
  if (!aligned(rope->freq, 8) || !aligned(rope->start, 4) || !aligned(rope->offsets, 4) || !aligned(rope->q_weight, 16) ||
      !aligned(rope->k_weight, 16))
    return ATTN_ERR_MISALIGNED;
  out->freq = rope->freq;
  out->start = rope->start;
  out->offsets = rope->offsets;
  out->offset_stride = B > 1 ? rope->offset_stride : 0;
  out->rot = rope->rotary_dim;
  out->interleaved = rope->layout == ATTN_ROPE_INTERLEAVED;
  out->amplitude = rope->amplitude;
  out->eps = rope->eps;
  out->back = false;
  return ATTN_OK;
}

extern "C" attn_status attn_rope_fwd(const void* Q, attn_strides q_strides, const void* K, attn_strides k_strides, void* Qr,
                                     attn_strides qr_strides, void* Kr, attn_strides kr_strides, int B, int H, int Hk, int N,
                                     int d, const attn_rope* rope, attn_dtype dtype, void* stream) {
  const int heads[2] = {H, Hk};
  attn_status st = check_sizes(B, N, d, heads, dtype);
  if (st != ATTN_OK) return st;
  RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  const bool normed = rope && ((H && rope->q_weight) || (Hk && rope->k_weight));
  if ((st = api_rope(rope, B, N, d, normed, &a.r)) != ATTN_OK) return st;
  const void *x[2] = {Q, K}, *w[2] = {rope->q_weight, rope->k_weight};
  void* y[2] = {Qr, Kr};
  const attn_strides *sx[2] = {&q_strides, &k_strides}, *sy[2] = {&qr_strides, &kr_strides};
  for (int i = 0; i < 2; ++i) {
    RopeSide& sd = a.side[i];
    if (heads[i] == 0) continue;
    if ((st = check_tensor(x[i], *sx[i], B, heads[i], d, &sd.sx)) != ATTN_OK ||
        (st = check_tensor(y[i], *sy[i], B, heads[i], d, &sd.sy)) != ATTN_OK)
      return st;
    sd.x = x[i];
    sd.y = y[i];
    sd.weight = w[i];
    sd.heads = heads[i];
  }
  DeviceInfo dev;
  if ((st = api_device(&dev)) != ATTN_OK) return st;
  a.B = B;
  a.N = N;
  a.d = d;
  a.tokens = B * N;
  a.bf16 = dtype == ATTN_BF16;
  a.weight_fp32 = rope->weight_fp32 != 0;
  a.sm_count = dev.sm_count;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return api_finish(launch_rope(a, s), s);
}

extern "C" size_t attn_rope_bwd_workspace_size(int d) {
  if (d != 64 && d != 128) return 0;
  const int sms = api_sm_count();
  return sms > 0 ? (rope_bwd_workspace(d, sms) + 255) & ~static_cast<size_t>(255) : 0;
}

extern "C" attn_status attn_rope_bwd(const void* dQr, attn_strides dqr_strides, const void* dKr, attn_strides dkr_strides,
                                     const void* Q, attn_strides q_strides, const void* K, attn_strides k_strides, void* dQ,
                                     attn_strides dq_strides, void* dK, attn_strides dk_strides, void* dq_weight,
                                     void* dk_weight, int B, int H, int Hk, int N, int d, const attn_rope* rope,
                                     attn_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const int heads[2] = {H, Hk};
  attn_status st = check_sizes(B, N, d, heads, dtype);
  if (st != ATTN_OK) return st;
  RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  const bool normed = rope && ((H && rope->q_weight) || (Hk && rope->k_weight));
  if ((st = api_rope(rope, B, N, d, normed, &a.r)) != ATTN_OK) return st;
  a.r.back = true;
  const void *x[2] = {dQr, dKr}, *in[2] = {Q, K}, *w[2] = {rope->q_weight, rope->k_weight};
  void *y[2] = {dQ, dK}, *dw[2] = {dq_weight, dk_weight};
  const attn_strides *sx[2] = {&dqr_strides, &dkr_strides}, *sin[2] = {&q_strides, &k_strides}, *sy[2] = {&dq_strides, &dk_strides};
  for (int i = 0; i < 2; ++i) {
    RopeSide& sd = a.side[i];
    if (heads[i] == 0) continue;
    if ((st = check_tensor(x[i], *sx[i], B, heads[i], d, &sd.sx)) != ATTN_OK ||
        (st = check_tensor(y[i], *sy[i], B, heads[i], d, &sd.sy)) != ATTN_OK)
      return st;
    sd.x = x[i];
    sd.y = y[i];
    sd.heads = heads[i];
    if (w[i] == nullptr) continue;
    if ((st = check_tensor(in[i], *sin[i], B, heads[i], d, &sd.sin)) != ATTN_OK) return st;
    if (!dw[i]) return ATTN_ERR_INVALID_ARG;
    if (!aligned(dw[i], 16)) return ATTN_ERR_MISALIGNED;
    sd.in = in[i];
    sd.weight = w[i];
    sd.dweight = dw[i];
  }
  if (normed && !workspace) return ATTN_ERR_WORKSPACE;
  if (normed && !aligned(workspace, 256)) return ATTN_ERR_MISALIGNED;
  DeviceInfo dev;
  if ((st = api_device(&dev)) != ATTN_OK) return st;
  if (normed && workspace_bytes < rope_bwd_workspace(d, dev.sm_count)) return ATTN_ERR_WORKSPACE;
  a.B = B;
  a.N = N;
  a.d = d;
  a.tokens = B * N;
  a.bf16 = dtype == ATTN_BF16;
  a.weight_fp32 = rope->weight_fp32 != 0;
  a.sm_count = dev.sm_count;
  if (normed) {
    a.count = static_cast<unsigned long long*>(workspace);
    a.sums = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kRopeSumsAt);
    a.tag = api_next_tag();
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return api_finish(launch_rope_bwd(a, s), s);
}
