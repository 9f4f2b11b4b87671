// Writing tokens into the 8-bit key/value cache with the keys' norm and rotary positions on the way, and the queries of the
// same tokens in the same launch.
//
// Mathematics: the keys of rope.cu in fp32, unrounded, then the rule of the cache's write (cache_io.cuh): the largest value
// of a page's new tokens gives its scale, and with that the codes.  So no rotated key is rounded twice or goes through memory.
//
// Bound: memory, 2 bytes read and 1 written a value, 2 and 2 of the queries.  As in cache_io.cu a unit is one page of one
// head, keys or values, of which GT threads hold 64 values each (32 at the smallest page), here widened to fp32 in their
// registers from the load to the codes.  A thread has whole lanes of rows (rope.cuh), NV / 2 of them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache8.cuh"
#include "cache.h"
#include "cache_io.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace exattn {
namespace {

static_assert(kIoThreads == kRopeThreads, "one launch for both");

__device__ __forceinline__ uint2 to_codes_of(int format, const float (&y)[8]) {
  return format == kE4M3 ? to_codes<kE4M3>(y) : to_codes<kInt8>(y);
}

template <int D, bool BF16, int GT, int NV>
__global__ void __launch_bounds__(kIoThreads, 2) cache_append_kernel(const __grid_constant__ CacheAppendArgs a) {
  using Lane = RopeLane<D>;
  constexpr int UNITS = kIoThreads / GT, ROWS = NV / 2, STEP = GT / Lane::LANES;  // rows of a thread, and between them
  __shared__ RopeShared sh;
  __shared__ uint32_t s_max[kIoThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x >= 2u * a.blocks) {
    const unsigned qb = blockIdx.x - 2u * a.blocks, cb = qb / a.q_token_blocks;
    rope_rows<D, BF16>(a.rope, sh, qb - cb * a.q_token_blocks, cb);
    return;
  }
  const CacheView& c = a.io.c;
  const RopeView& rv = a.rope.r;
  const int g = threadIdx.x / GT, tid = threadIdx.x % GT;
  const bool is_v = blockIdx.x >= static_cast<unsigned>(a.blocks);
  const unsigned units = static_cast<unsigned>(a.io.B) * c.heads * a.io.parts;  // below 2^31
  const unsigned unit = (blockIdx.x - (is_v ? a.blocks : 0)) * UNITS + g;
  const unsigned bh = unit / a.io.parts;
  const int pj = unit - bh * a.io.parts, b = bh / c.heads, head = bh - b * c.heads;
  CacheUnit un;
  if (unit < units) un.find(a.io, b, pj, tid == 0);
  if (!is_v) {
    sh.table.fill(rv, threadIdx.x, kIoThreads);
    __syncthreads();
  }
  if (un.page < 0) return;  // all threads of a unit together
  const int r0 = un.r0, r1 = un.r1, inside = un.inside;
  const Lane l(rv, tid % Lane::LANES);
  const int row0 = tid / Lane::LANES;
  const RowStrides& st = is_v ? a.io.sv : a.io.sk;
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? a.io.v : a.io.k) + b * st.b + head * st.h + (un.row_of_r0 - r0) * st.n;
  const long long ph = static_cast<long long>(un.page) * c.heads + head;
  float* scale_at = (is_v ? c.v_scale : c.k_scale) + ph;
  uint8_t* codes = (is_v ? c.v : c.k) + ((ph << c.page_shift) * D);
  float old = 0.f;
  if (inside > 0) old = *scale_at;

  uint4 xa[ROWS], xb[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int row = row0 + i * STEP;
    xa[i] = xb[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row >= r0 && row < r1) {
      xa[i] = reinterpret_cast<const uint4*>(src + row * st.n)[l.ua];
      xb[i] = reinterpret_cast<const uint4*>(src + row * st.n)[l.ub];
    }
  }
  float x[ROWS][16];
  const void* weight = is_v ? nullptr : a.k_weight;
  const bool turns = !is_v && l.turns();
  if (!is_v && (weight || rv.rot > 0)) {
    long long p[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int row = row0 + i * STEP;
      p[i] = 0;
      if (row >= r0 && row < r1) p[i] = rope_position(rv, b, static_cast<int>(un.row_of_r0) + row - r0, rv.start);
    }
    float w[16];
    if (weight) l.template weights<BF16>(weight, a.rope.weight_fp32, w);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      Lane::template widen<BF16>(xa[i], xb[i], x[i]);
      if (weight) {
        const float r = Lane::inverse_rms(x[i], rv.eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[i][e] *= r * w[e];
      }
      const int row = row0 + i * STEP;
      if (turns && row >= r0 && row < r1) {
        float co[8], si[8];
        l.angles(sh.table, p[i], false, co, si);
        l.rotate(x[i], co, si);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) Lane::template widen<BF16>(xa[i], xb[i], x[i]);
  }

  uint32_t mx = 0u;  // largest |value|, NaN and infinity above all others
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
#pragma unroll
    for (int e = 0; e < 16; ++e) mx = max(mx, __float_as_uint(x[i][e]) & 0x7fffffffu);
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if constexpr (GT > 32) {
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = mx;
    named_bar_sync(g + 1, GT);
#pragma unroll
    for (int w = 0; w < GT / 32; ++w) mx = max(mx, s_max[g * (GT / 32) + w]);
  } else {
    __syncwarp();  // the old scale has been read by every lane before one of them writes the new
  }
  const CacheScale sc(c.format, mx >= 0x7f800000u ? __int_as_float(0x7fffffff) : __uint_as_float(mx), inside > 0, old);
  if (tid == 0) *scale_at = sc.s;
  const bool alive = sc.s > 0.f;
  const float again = old * sc.inv;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int row = row0 + i * STEP;
    if (row >= r1) continue;
    uint2* to = reinterpret_cast<uint2*>(codes) + row * (D / 8);
    float y[2][8];
    if (row >= r0) {
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e >> 3][e & 7] = alive ? x[i][e] * sc.inv : 0.f;
      to[l.ua] = to_codes_of(c.format, y[0]);
      to[l.ub] = to_codes_of(c.format, y[1]);
    } else if (sc.grew) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint2* at = to + (h ? l.ub : l.ua);
        if (c.format == kE4M3) from_codes<kE4M3>(*at, y[h]); else from_codes<kInt8>(*at, y[h]);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[h][e] *= again;
        *at = to_codes_of(c.format, y[h]);
      }
    }
  }
}

template <int D, bool BF16, int GT, int NV>
cudaError_t append_t(CacheAppendArgs& a, cudaStream_t stream) {
  const int psize = 1 << a.io.c.page_shift;
  a.io.parts = static_cast<int>((a.io.N + static_cast<long long>(psize) - 2) / psize) + 1;
  const long long units = static_cast<long long>(a.io.B) * a.io.c.heads * a.io.parts;
  a.blocks = static_cast<int>((units + kIoThreads / GT - 1) / (kIoThreads / GT));
  long long q_blocks = 0;
  a.q_token_blocks = 1;
  if (a.rope.side[0].heads > 0) {
    const RopeGrid grid = rope_plan(a.rope);
    a.q_token_blocks = static_cast<int>(grid.token_blocks);
    q_blocks = static_cast<long long>(grid.token_blocks) * grid.chunk_blocks;
  }
  const long long grid = 2LL * a.blocks + q_blocks;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_dependent(cache_append_kernel<D, BF16, GT, NV>, dim3(static_cast<unsigned>(grid)), dim3(kIoThreads), 0, stream, a);
}

template <bool BF16>
cudaError_t append_f(CacheAppendArgs& a, cudaStream_t stream) {
  const int psize = 1 << a.io.c.page_shift;
  if (a.io.c.d == 64) {
    switch (psize) {
      case 16: return append_t<64, BF16, 32, 4>(a, stream);
      case 32: return append_t<64, BF16, 32, 8>(a, stream);
      case 64: return append_t<64, BF16, 64, 8>(a, stream);
      default: return append_t<64, BF16, 128, 8>(a, stream);
    }
  }
  switch (psize) {
    case 16: return append_t<128, BF16, 32, 8>(a, stream);
    case 32: return append_t<128, BF16, 64, 8>(a, stream);
    case 64: return append_t<128, BF16, 128, 8>(a, stream);
    default: return append_t<128, BF16, 256, 8>(a, stream);
  }
}

}  // namespace

cudaError_t launch_cache_append(CacheAppendArgs& a, cudaStream_t stream) {
  return a.io.bf16 ? append_f<true>(a, stream) : append_f<false>(a, stream);
}

}  // namespace exattn
