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

// A page's scale of the values.  An infinite one counts as NaN.
__device__ __forceinline__ float cache_v_scale(const CacheView& c, long long page_head) {
  const float s = c.v_scale[page_head];
  return s == INFINITY ? __int_as_float(0x7fffffff) : s;
}

// What the attention kernels scale their O by.  Each row keeps, besides m >= max s - 8, a number w over the keys that it
// sees, with w >= max(s + log2 vs) - kValueLag and no greater than that maximum, vs the value scale of a key's page.  Its
// probabilities go into the product as 2^(s - m + 3) vs 2^(m - w), below 2^15 in fp16 whatever the scales are, and the
// sum of the products counts 2^(w - 3).  So a large scale costs the others nothing where it has no weight for the row:
// behind the row's last key, or with small scores.  (A reference over the scales alone lost such rows: with a hidden page's
// scale 2^28 times the others', a row's O was 0.)
constexpr float kValueLag = 12.f;
// w is no less than m - kValueFloor, so that 2^(m - w) is finite.
constexpr float kValueFloor = 126.f;

// log2 of a value scale, -inf below 2^-126; it needs no more accuracy than w's bounds do.
__device__ __forceinline__ float cache_log2(float vs) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(vs));
  return y;
}
// 2^x, also below 2^-126.
__device__ __forceinline__ float ex2_whole(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// w for a row whose maximum of s + log2 vs is z and of s is m, and the factor 2^(m - w) of its value scales.
__device__ __forceinline__ float value_reference(float w, float z, float m) { return fmaxf(fmaxf(w, z), m - kValueFloor); }
__device__ __forceinline__ float value_factor(float m, float w) { return w == -INFINITY ? 0.f : ex2_whole(m - w); }
// vs times that factor.  Finite, or NaN where vs is: with next to no probability behind it, it may be beyond fp32.
__device__ __forceinline__ float value_weight(float vs, float factor) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(vs * factor), "f"(3.402823466e38f));
  return y;
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
