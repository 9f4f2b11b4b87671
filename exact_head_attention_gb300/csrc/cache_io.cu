// Writing tokens into the 8-bit key/value cache, and reading them back.
//
// Both are copies with a little arithmetic, bound by memory: a write reads 2 bytes and writes 1 for each
// value, a read the reverse.  The write takes one page of one head at a time and keeps its new tokens
// in registers between the search for the largest value and the rounding, so the input is read once.
// Measured, of what the bytes take at the copy rate: 4 prompts of 8k tokens on 12 heads of 128 written in 47 us (94%)
// and 4 sequences of 32k read in 179 us (99%); 16 chunks of up to 1537 tokens on 16 heads of 64 written in 17.8 us
// (61%: half the units are empty, and start and drain take 5 us); 16 prefixes of up to 4097 tokens on 8 heads of 128
// read in 34 us (85%); one token of each of 64 sequences written in 4.1 us, which is four dependent loads and the
// launch.  A grid of resident blocks that stride over the units was slower in all of these (ragged read 49 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache8.cuh"
#include "cache.h"
#include "cache_io.cuh"
#include "ptx.cuh"

namespace exattn {
namespace {

// One unit is one page of one head, keys or values, of which GT threads each hold NV vectors of 8 values:
// GT * NV * 8 = page * d.  With 64 values a thread (32 at the smallest page) the loads of a whole page are in
// flight at once and its values fit the registers.
template <int FMT, bool BF16, int GT, int NV>
__global__ void __launch_bounds__(kIoThreads, 4) cache_write_kernel(const __grid_constant__ CacheIoArgs a) {
  constexpr int UNITS = kIoThreads / GT;
  __shared__ uint32_t s_max[kIoThreads / 32];
  const CacheView& c = a.c;
  const int g = threadIdx.x / GT, tid = threadIdx.x % GT;
  const unsigned units = static_cast<unsigned>(a.B) * c.heads * a.parts;  // below 2^31, of the keys and again of the values
  const int vshift = c.d == 128 ? 4 : 3;  // log2 of the vectors a row
  griddep_wait();
  griddep_launch_dependents();
  const bool is_v = blockIdx.y != 0;
  const unsigned unit = blockIdx.x * UNITS + g;
  const unsigned bh = unit / a.parts;
  const int pj = unit - bh * a.parts, b = bh / c.heads, head = bh - b * c.heads;

  CacheUnit un;
  if (unit < units) un.find(a, b, pj, tid == 0);
  if (un.page < 0) return;  // all threads of a unit together
  const int r0 = un.r0, r1 = un.r1, inside = un.inside;
  const RowStrides& st = is_v ? a.sv : a.sk;
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? a.v : a.k) + b * st.b + head * st.h +
                        (un.row_of_r0 - r0) * st.n;
  const long long ph = static_cast<long long>(un.page) * c.heads + head;
  float* scale_at = (is_v ? c.v_scale : c.k_scale) + ph;
  uint8_t* codes = (is_v ? c.v : c.k) + ((ph << c.page_shift) * c.d);
  float old = 0.f;
  if (inside > 0) old = *scale_at;

  uint4 x[NV];
  uint32_t mx = 0u;  // largest |value| as a 16-bit pattern, NaN and infinity above all others
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vec = i * GT + tid, row = vec >> vshift;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row >= r0 && row < r1)
      x[i] = *reinterpret_cast<const uint4*>(src + row * st.n + ((vec & ((1 << vshift) - 1)) << 3));
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) loaded(x[i]);
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
    named_bar_sync(g + 1, GT);
#pragma unroll
    for (int w = 0; w < GT / 32; ++w) mx = max(mx, s_max[g * (GT / 32) + w]);
  } else {
    __syncwarp();  // the old scale has been read by every lane before one of them writes the new
  }

  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
  const float amax = mx >= kInf ? __int_as_float(0x7fffffff) : unpack_lo<BF16>(mx);
  const CacheScale sc(FMT, amax, inside > 0, old);
  if (tid == 0) *scale_at = sc.s;
  const bool alive = sc.s > 0.f, grew = sc.grew;
  const float inv = sc.inv, again = old * inv;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vec = i * GT + tid, row = vec >> vshift;
    if (row >= r1) continue;
    uint2* to = reinterpret_cast<uint2*>(codes) + vec;
    float y[8];
    if (row >= r0) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[2 * e] = alive ? unpack_lo<BF16>(w[e]) * inv : 0.f;
        y[2 * e + 1] = alive ? unpack_hi<BF16>(w[e]) * inv : 0.f;
      }
      *to = to_codes<FMT>(y);
    } else if (grew) {
      from_codes<FMT>(*to, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= again;
      *to = to_codes<FMT>(y);
    }
  }
}

// One unit is ROWS rows of one sequence and head, keys or values: each thread reads NR vectors of 8 codes
// and writes 8 values for each.  Both sides of a warp's access are whole lines (256 bytes read, 512 written).
template <int FMT, bool BF16, int D, int NR>
__global__ void __launch_bounds__(kIoThreads, NR == 8 ? 4 : 8) cache_read_kernel(const __grid_constant__ CacheIoArgs a) {
  constexpr int VR = D / 8;                 // vectors a row
  constexpr int STEP = kIoThreads / VR;     // rows between a thread's vectors
  constexpr int ROWS = STEP * NR;
  const CacheView& c = a.c;
  const int col = threadIdx.x % VR, row = threadIdx.x / VR;
  griddep_wait();
  griddep_launch_dependents();
  const bool is_v = blockIdx.y != 0;
  const unsigned unit = blockIdx.x;
  const unsigned bh = unit / a.parts;
  const int b = bh / c.heads, head = bh - b * c.heads;
  const int want = a.count[b], from = a.start ? a.start[b] : 0;
  const int len = cache_len(c, want), start = max(from, 0);
  if ((from < 0 || len != want) && threadIdx.x == 0) record_page_error(a.err_word);
  const int first = (unit - bh * a.parts) * ROWS;
  const int rows = max(0, min(a.N, len - start));  // rows of this sequence that hold a token
  if (first >= rows) return;
  const int left = rows - first - row;  // rows from this thread's first on
  const long long n0 = static_cast<long long>(first) + row;
  const RowStrides& st = is_v ? a.sv : a.sk;
  uint16_t* dst = static_cast<uint16_t*>(is_v ? a.v : a.k) + b * st.b + head * st.h + n0 * st.n + col * 8;
  const uint8_t* codes = (is_v ? c.v : c.k) + col * 8;
  const float* scales = is_v ? c.v_scale : c.k_scale;
  const int* table = c.table + static_cast<long long>(b) * c.width;
  // All loads of a kind before what needs them: pages, then scales and codes.
  int page[NR];
  uint2 w[NR];
  float s[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    page[i] = -1;
    if (i * STEP < left) page[i] = table[(start + n0 + i * STEP) >> c.page_shift];
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int t = static_cast<int>(start + n0) + i * STEP;
    const bool good = cache_page_checked(c, page[i]) >= 0;
    const long long ph = static_cast<long long>(page[i]) * c.heads + head;
    s[i] = __int_as_float(0x7fffffff);
    w[i] = make_uint2(0u, 0u);
    if (good) {
      s[i] = scales[ph];
      w[i] = __ldcs(reinterpret_cast<const uint2*>(codes + ((ph << c.page_shift) + (t & ((1 << c.page_shift) - 1))) * D));
    }
    bad = bad || (!good && i * STEP < left);
  }
  if (bad) record_page_error(a.err_word);
#pragma unroll
  for (int i = 0; i < NR; ++i) loaded(w[i]);
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    if (i * STEP < left) {
      float y[8];
      from_codes<FMT>(w[i], y);
      uint4 o;
      o.x = pack2<BF16>(y[0] * s[i], y[1] * s[i]);
      o.y = pack2<BF16>(y[2] * s[i], y[3] * s[i]);
      o.z = pack2<BF16>(y[4] * s[i], y[5] * s[i]);
      o.w = pack2<BF16>(y[6] * s[i], y[7] * s[i]);
      *reinterpret_cast<uint4*>(dst + i * STEP * st.n) = o;
    }
  }
}

template <typename Kernel>
cudaError_t launch_io(Kernel kernel, const CacheIoArgs& a, long long groups, cudaStream_t stream) {
  if (groups > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_dependent(kernel, dim3(static_cast<unsigned>(groups), 2), dim3(kIoThreads), 0, stream, a);
}

template <int FMT, bool BF16, int GT, int NV>
cudaError_t write_t(const CacheIoArgs& a, cudaStream_t stream) {
  const long long units = static_cast<long long>(a.B) * a.c.heads * a.parts;
  return launch_io(cache_write_kernel<FMT, BF16, GT, NV>, a, (units + kIoThreads / GT - 1) / (kIoThreads / GT), stream);
}

template <int FMT, bool BF16>
cudaError_t write_f(CacheIoArgs& a, cudaStream_t stream) {
  const int psize = 1 << a.c.page_shift;
  a.parts = static_cast<int>((a.N + static_cast<long long>(psize) - 2) / psize) + 1;
  switch (psize * a.c.d) {
    case 1024: return write_t<FMT, BF16, 32, 4>(a, stream);
    case 2048: return write_t<FMT, BF16, 32, 8>(a, stream);
    case 4096: return write_t<FMT, BF16, 64, 8>(a, stream);
    case 8192: return write_t<FMT, BF16, 128, 8>(a, stream);
    default: return write_t<FMT, BF16, 256, 8>(a, stream);
  }
}

template <int FMT, bool BF16, int D, int NR>
cudaError_t read_n(CacheIoArgs& a, cudaStream_t stream) {
  constexpr int ROWS = kIoThreads * NR / (D / 8);
  a.parts = (a.N - 1) / ROWS + 1;
  return launch_io(cache_read_kernel<FMT, BF16, D, NR>, a, static_cast<long long>(a.B) * a.c.heads * a.parts, stream);
}
// Few rows are spread over more blocks (B = 1, 8 heads, 333 rows of 64: 1.9 us at 2 vectors a thread, 2.8 us at 8);
// above, 8 vectors keep enough loads in flight (B = 16, 8 heads, up to 4097 rows of 128: 34 us, 36 us at 4, 44 us at 2).
template <int FMT, bool BF16, int D>
cudaError_t read_t(CacheIoArgs& a, cudaStream_t stream) {
  const long long vecs = static_cast<long long>(a.B) * a.c.heads * a.N * (D / 8) * 2;
  return vecs <= static_cast<long long>(a.sm_count) * kIoThreads * 2 ? read_n<FMT, BF16, D, 2>(a, stream) : read_n<FMT, BF16, D, 8>(a, stream);
}

template <int FMT, bool BF16>
cudaError_t read_f(CacheIoArgs& a, cudaStream_t stream) {
  return a.c.d == 128 ? read_t<FMT, BF16, 128>(a, stream) : read_t<FMT, BF16, 64>(a, stream);
}

}  // namespace

cudaError_t launch_cache_write(CacheIoArgs& a, cudaStream_t stream) {
  if (a.c.format == kE4M3) return a.bf16 ? write_f<kE4M3, true>(a, stream) : write_f<kE4M3, false>(a, stream);
  return a.bf16 ? write_f<kInt8, true>(a, stream) : write_f<kInt8, false>(a, stream);
}

cudaError_t launch_cache_read(CacheIoArgs& a, cudaStream_t stream) {
  if (a.c.format == kE4M3) return a.bf16 ? read_f<kE4M3, true>(a, stream) : read_f<kE4M3, false>(a, stream);
  return a.bf16 ? read_f<kInt8, true>(a, stream) : read_f<kInt8, false>(a, stream);
}

}  // namespace exattn
