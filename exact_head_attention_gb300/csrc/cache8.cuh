// The 8-bit key/value cache on the device: what a kernel is told about it, page look-up with its bounds
// checks, and the conversion of codes to fp16.
#pragma once

#include <cstdint>

#include "../../include/exattn.h"
#include "cache.h"
#include "ptx.cuh"

namespace exattn {

constexpr int kE4M3 = ATTN_CACHE_E4M3, kInt8 = ATTN_CACHE_INT8;

__device__ __forceinline__ void record_page_error(uint32_t* err_word) { atomicCAS(err_word, 0u, kErrPage); }

// A sequence's length within [0, capacity of its table].
__device__ __forceinline__ int cache_len(const CacheView& c, int len) {
  return max(0, min(len, c.capacity));
}

// The kernels that use these are launched before the one ahead of them has finished, which may write what they
// read: no load of theirs is a read-only one.

// The table's entry for token t (0 <= t < capacity) of sequence b, and that as a page: -1 for a number
// outside the pool.
__device__ __forceinline__ int cache_page_number(const CacheView& c, int b, int t) {
  return c.table[static_cast<long long>(b) * c.width + (t >> c.page_shift)];
}
__device__ __forceinline__ int cache_page_checked(const CacheView& c, int p) {
  return static_cast<unsigned>(p) < static_cast<unsigned>(c.num_pages) ? p : -1;
}
__device__ __forceinline__ int cache_page(const CacheView& c, int b, int t) {
  return cache_page_checked(c, cache_page_number(c, b, t));
}

// A page's scale of the values.  An infinite one counts as NaN: as a number it would set the reference that the
// rows' probabilities are scaled by, for rows that do not see the page as well.
__device__ __forceinline__ float cache_v_scale(const CacheView& c, long long page_head) {
  const float s = c.v_scale[page_head];
  return s == INFINITY ? __int_as_float(0x7fffffff) : s;
}

// The upper bits of the bytes of w that are an e4m3 NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t nan_codes(const uint4& w) {
  return nan_codes(w.x) | nan_codes(w.y) | nan_codes(w.z) | nan_codes(w.w);
}
// w with zeros in their place.
__device__ __forceinline__ uint32_t without_nan(uint32_t w) { return w & ~((nan_codes(w) >> 7) * 0xffu); }
__device__ __forceinline__ uint4 without_nan(const uint4& w) {
  return make_uint4(without_nan(w.x), without_nan(w.y), without_nan(w.z), without_nan(w.w));
}

// Four codes as two fp16 pairs: bytes 0, 1 and bytes 2, 3.  fp16 holds every code exactly: e4m3 has 4
// significant bits and exponents from -9, and an integer of 8 bits has 8.
template <int FMT>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == kE4M3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // c + 128 as the low byte of an fp16 whose high byte is 0x64 is 1024 + 128 + c; the subtraction is exact.
    const uint32_t u = w ^ 0x80808080u;
    asm("{\n\t.reg .b32 a, b;\n\t"
        "prmt.b32 a, %2, 0x64646464, 0x4140;\n\tprmt.b32 b, %2, 0x64646464, 0x4342;\n\t"
        "sub.rn.f16x2 %0, a, %3;\n\tsub.rn.f16x2 %1, b, %3;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(u), "r"(0x64806480u));
  }
}

}  // namespace exattn
