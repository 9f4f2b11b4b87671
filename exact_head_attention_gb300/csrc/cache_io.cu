// Writing tokens into the 8-bit key/value cache, and reading them back.
//
// Both are copies with a little arithmetic, bound by memory: a write reads 2 bytes and writes 1 for each
// value, a read the reverse.  The write takes one page of one head at a time and keeps its new tokens
// in registers between the search for the largest value and the rounding, so the input is read once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace exattn {
namespace {

constexpr int kIoThreads = 256;

// Rounds 8 fp32 values to codes: nearest even, clamped to the largest code.
template <int FMT>
__device__ __forceinline__ uint2 to_codes(const float (&x)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (FMT == kE4M3) {
      asm("{\n\t.reg .b16 a, b;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
          "mov.b32 %0, {a, b};\n\t}"
          : "=r"(w[h])
          : "f"(x[4 * h]), "f"(x[4 * h + 1]), "f"(x[4 * h + 2]), "f"(x[4 * h + 3]));
    } else {
      w[h] = 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = max(-127, min(127, __float2int_rn(x[4 * h + e])));
        w[h] |= static_cast<uint32_t>(i & 255) << (8 * e);
      }
    }
  }
  return make_uint2(w[0], w[1]);
}

// 8 codes as fp32.
template <int FMT>
__device__ __forceinline__ void from_codes(uint2 c, float (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t lo, hi;
    codes_to_f16<FMT>(h ? c.y : c.x, lo, hi);
    x[4 * h] = unpack_lo<false>(lo);
    x[4 * h + 1] = unpack_hi<false>(lo);
    x[4 * h + 2] = unpack_lo<false>(hi);
    x[4 * h + 3] = unpack_hi<false>(hi);
  }
}

// One unit is one page of one head, keys or values (blockIdx.y), of which GT threads each hold NV vectors
// of 8 values: GT * NV * 8 = page * d.  With 64 values a thread (32 at the smallest page) the loads of
// a whole page are in flight at once and its values fit the registers.
template <int FMT, bool BF16, int GT, int NV>
__global__ void __launch_bounds__(kIoThreads) cache_write_kernel(const __grid_constant__ CacheIoArgs a, int span) {
  constexpr int UNITS = kIoThreads / GT;
  __shared__ uint32_t s_max[kIoThreads / 32];
  const CacheView& c = a.c;
  const bool is_v = blockIdx.y != 0;
  const int g = threadIdx.x / GT, tid = threadIdx.x % GT;
  const long long unit = static_cast<long long>(blockIdx.x) * UNITS + g;
  const long long heads_span = static_cast<long long>(c.heads) * span;
  const int b = static_cast<int>(unit / heads_span);
  const int rest = static_cast<int>(unit % heads_span);
  const int head = rest / span, pj = rest % span;

  int page = -1;
  int r0 = 0, r1 = 0, inside = 0;  // rows [r0, r1) of the page are new; rows [0, inside) hold earlier tokens
  long long row_of_r0 = 0;         // input row of page row r0
  if (b < a.B) {
    const int start = a.start ? __ldg(a.start + b) : 0;
    const int want = a.count ? __ldg(a.count + b) : a.N;
    const int count = max(0, min(want, a.N));
    const long long end = static_cast<long long>(start) + count;
    bool bad = want != count || start < 0 || (count > 0 && end > c.capacity);
    if (start >= 0 && count > 0) {
      const int psize = 1 << c.page_shift;
      const long long first = (static_cast<long long>(start >> c.page_shift) + pj) << c.page_shift;  // first token of this page
      const long long stop = min(end, static_cast<long long>(c.capacity));
      if (first < stop) {
        page = cache_page(c, b, static_cast<int>(first));
        bad = bad || page < 0;
        inside = static_cast<int>(max(0ll, start - first));
        r0 = inside;
        r1 = static_cast<int>(min(static_cast<long long>(psize), stop - first));
        row_of_r0 = first + r0 - start;
      }
    }
    if (bad && tid == 0) record_page_error(a.err_word);
  }
  const int vshift = c.d == 128 ? 4 : 3;  // log2 of the vectors a row
  const RowStrides& st = is_v ? a.sv : a.sk;
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? a.v : a.k) + b * st.b + head * st.h +
                        (row_of_r0 - r0) * st.n;
  const long long ph = static_cast<long long>(page) * c.heads + head;
  float* scale_at = (is_v ? c.v_scale : c.k_scale) + ph;
  uint8_t* codes = (is_v ? c.v : c.k) + ((ph << c.page_shift) * c.d);
  float old = 0.f;
  if (page >= 0 && inside > 0) old = *scale_at;

  uint4 x[NV];
  uint32_t mx = 0u;  // largest |value| as a 16-bit pattern, NaN and infinity above all others
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vec = i * GT + tid, row = vec >> vshift;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (page >= 0 && row >= r0 && row < r1)
      x[i] = __ldg(reinterpret_cast<const uint4*>(src + row * st.n + ((vec & ((1 << vshift) - 1)) << 3)));
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) mx = __vmaxu2(mx, w[e] & 0x7fff7fffu);
  }
  mx = max(mx & 0xffffu, mx >> 16);
  mx = __reduce_max_sync(0xffffffffu, mx);
  if constexpr (GT > 32) {
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < GT / 32; ++w) mx = max(mx, s_max[g * (GT / 32) + w]);
  } else {
    __syncwarp();  // the old scale has been read by every lane before one of them writes the new
  }
  if (page < 0) return;

  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
  const float amax = mx >= kInf ? __int_as_float(0x7fffffff) : unpack_lo<BF16>(mx);
  constexpr float kUnit = 1.0f / (FMT == kE4M3 ? 448.f : 127.f);
  float f = __fmul_rn(amax, kUnit);
  if (f < 1.17549435e-38f) f = 0.f;
  float s = f;
  bool grew = false;
  if (inside > 0) {
    if (old >= f || old != old) s = old;  // a NaN on either side stays
    grew = s > old;
  }
  const float inv = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;  // NaN scale: codes 0, every token reads as NaN
  if (tid == 0) *scale_at = s;
  const bool alive = s > 0.f;
  const float again = old * inv;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vec = i * GT + tid, row = vec >> vshift;
    if (row >= r1) continue;
    uint2* at = reinterpret_cast<uint2*>(codes) + vec;
    float y[8];
    if (row >= r0) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[2 * e] = alive ? unpack_lo<BF16>(w[e]) * inv : 0.f;
        y[2 * e + 1] = alive ? unpack_hi<BF16>(w[e]) * inv : 0.f;
      }
      *at = to_codes<FMT>(y);
    } else if (grew) {
      from_codes<FMT>(*at, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= again;
      *at = to_codes<FMT>(y);
    }
  }
}

// Each thread reads NR vectors of 8 codes and writes 8 values for each: both sides of a warp's access are
// whole lines (256 bytes read, 512 written).
constexpr int kReadVecs = 8;

template <int FMT, bool BF16, int D>
__global__ void __launch_bounds__(kIoThreads) cache_read_kernel(const __grid_constant__ CacheIoArgs a, int chunks) {
  constexpr int VR = D / 8;                              // vectors a row
  constexpr int ROWS = kIoThreads * kReadVecs / VR;      // rows a block
  const CacheView& c = a.c;
  const bool is_v = blockIdx.y != 0;
  const int chunk = blockIdx.x % chunks;
  const long long bh = blockIdx.x / chunks;
  const int b = static_cast<int>(bh / c.heads), head = static_cast<int>(bh % c.heads);
  int start = a.start ? __ldg(a.start + b) : 0;
  const int want = __ldg(a.count + b);
  const int len = cache_len(c, want);
  if ((start < 0 || len != want) && threadIdx.x == 0) record_page_error(a.err_word);
  start = max(start, 0);
  const int rows = max(0, min(a.N, len - start));  // rows of this sequence that hold a token
  const int n0 = chunk * ROWS;
  if (n0 >= rows) return;
  const RowStrides& st = is_v ? a.sv : a.sk;
  uint16_t* dst = static_cast<uint16_t*>(is_v ? a.v : a.k) + b * st.b + head * st.h;
  const uint8_t* codes = is_v ? c.v : c.k;
  const float* scales = is_v ? c.v_scale : c.k_scale;
  const int col = threadIdx.x % VR;
  uint2 w[kReadVecs];
  float s[kReadVecs];
#pragma unroll
  for (int i = 0; i < kReadVecs; ++i) {
    const int n = n0 + (i * kIoThreads + threadIdx.x) / VR;
    s[i] = 0.f;
    w[i] = make_uint2(0u, 0u);
    if (n < rows) {
      const int t = start + n;
      const int page = cache_page(c, b, t);
      if (page < 0) {
        record_page_error(a.err_word);
        s[i] = __int_as_float(0x7fffffff);
      } else {
        const long long ph = static_cast<long long>(page) * c.heads + head;
        s[i] = __ldg(scales + ph);
        w[i] = __ldcs(reinterpret_cast<const uint2*>(codes + ((ph << c.page_shift) + (t & ((1 << c.page_shift) - 1))) * D) + col);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kReadVecs; ++i) {
    const int n = n0 + (i * kIoThreads + threadIdx.x) / VR;
    if (n < rows) {
      float y[8];
      from_codes<FMT>(w[i], y);
      uint4 o;
      o.x = pack2<BF16>(y[0] * s[i], y[1] * s[i]);
      o.y = pack2<BF16>(y[2] * s[i], y[3] * s[i]);
      o.z = pack2<BF16>(y[4] * s[i], y[5] * s[i]);
      o.w = pack2<BF16>(y[6] * s[i], y[7] * s[i]);
      *reinterpret_cast<uint4*>(dst + n * st.n + col * 8) = o;
    }
  }
}

template <int FMT, bool BF16, int GT, int NV>
cudaError_t write_t(const CacheIoArgs& a, int span, cudaStream_t stream) {
  const long long units = static_cast<long long>(a.B) * a.c.heads * span;
  constexpr int UNITS = kIoThreads / GT;
  const long long blocks = (units + UNITS - 1) / UNITS;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cache_write_kernel<FMT, BF16, GT, NV><<<dim3(static_cast<unsigned>(blocks), 2), kIoThreads, 0, stream>>>(a, span);
  return cudaGetLastError();
}

template <int FMT, bool BF16>
cudaError_t write_f(const CacheIoArgs& a, cudaStream_t stream) {
  const int psize = 1 << a.c.page_shift;
  const int span = static_cast<int>((a.N + static_cast<long long>(psize) - 2) / psize) + 1;  // pages that N tokens can reach
  switch (psize * a.c.d) {
    case 1024: return write_t<FMT, BF16, 32, 4>(a, span, stream);
    case 2048: return write_t<FMT, BF16, 32, 8>(a, span, stream);
    case 4096: return write_t<FMT, BF16, 64, 8>(a, span, stream);
    case 8192: return write_t<FMT, BF16, 128, 8>(a, span, stream);
    default: return write_t<FMT, BF16, 256, 8>(a, span, stream);
  }
}

template <int FMT, bool BF16, int D>
cudaError_t read_t(const CacheIoArgs& a, cudaStream_t stream) {
  constexpr int ROWS = kIoThreads * kReadVecs / (D / 8);
  const int chunks = (a.N - 1) / ROWS + 1;
  const long long blocks = static_cast<long long>(a.B) * a.c.heads * chunks;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cache_read_kernel<FMT, BF16, D><<<dim3(static_cast<unsigned>(blocks), 2), kIoThreads, 0, stream>>>(a, chunks);
  return cudaGetLastError();
}

template <int FMT, bool BF16>
cudaError_t read_f(const CacheIoArgs& a, cudaStream_t stream) {
  return a.c.d == 128 ? read_t<FMT, BF16, 128>(a, stream) : read_t<FMT, BF16, 64>(a, stream);
}

}  // namespace

cudaError_t launch_cache_write(const CacheIoArgs& a, cudaStream_t stream) {
  if (a.c.format == kE4M3) return a.bf16 ? write_f<kE4M3, true>(a, stream) : write_f<kE4M3, false>(a, stream);
  return a.bf16 ? write_f<kInt8, true>(a, stream) : write_f<kInt8, false>(a, stream);
}

cudaError_t launch_cache_read(const CacheIoArgs& a, cudaStream_t stream) {
  if (a.c.format == kE4M3) return a.bf16 ? read_f<kE4M3, true>(a, stream) : read_f<kE4M3, false>(a, stream);
  return a.bf16 ? read_f<kInt8, true>(a, stream) : read_f<kInt8, false>(a, stream);
}

}  // namespace exattn
