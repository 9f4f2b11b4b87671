// What the kernels that write into the 8-bit key/value cache share: rounding to codes, the place of a page's new tokens, and
// the scale's rule.
#pragma once

#include <cstdint>

#include "cache8.cuh"

namespace exattn {

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
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // 1.5 * 2^23 + x has the rounded x in its low bits (the conversion to an integer has a quarter of the rate)
        const float r = __fadd_rn(fminf(fmaxf(x[4 * h + e], -127.f), 127.f), 12582912.f);
        w[h] = e == 0 ? __float_as_uint(r) : __byte_perm(w[h], __float_as_uint(r), e == 1 ? 0x3240 : e == 2 ? 0x3410 : 0x4210);
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

// Keeps the compiler from moving arithmetic on a loaded word up to its load, where it would wait for each load
// before the next is sent (reading int8 codes took 1.5 times as long).
__device__ __forceinline__ void loaded(uint2& w) { asm volatile("" : "+r"(w.x), "+r"(w.y)); }
__device__ __forceinline__ void loaded(uint4& w) { asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w)); }

// One page of one sequence that new tokens reach: the pj-th such page.
struct CacheUnit {
  int page = -1;                   // -1: there is none
  int r0 = 0, r1 = 0, inside = 0;  // rows [r0, r1) of the page are new; rows [0, inside) hold earlier tokens
  long long row_of_r0 = 0;         // input row of page row r0
  int start = 0;

  // `reports`: one of the threads that call this.
  __device__ __forceinline__ void find(const CacheIoArgs& a, int b, int pj, bool reports) {
    const CacheView& c = a.c;
    start = a.start ? a.start[b] : 0;
    const int want = a.count ? a.count[b] : a.N;
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
    if (bad && reports) record_page_error(a.err_word);
  }
};

// A page's scale from its new tokens' largest |value| (NaN: one was no number or infinite) and, where it holds earlier ones,
// the old scale; and what the values are multiplied by.
struct CacheScale {
  float s, inv;
  bool grew;

  __device__ __forceinline__ CacheScale(int format, float amax, bool holds, float old) {
    float f = __fmul_rn(amax, format == kE4M3 ? 1.0f / 448.f : 1.0f / 127.f);
    if (f < 1.17549435e-38f) f = 0.f;
    s = f;
    grew = false;
    if (holds) {
      if (old >= f || old != old) s = old;  // a NaN on either side stays
      grew = s > old;
    }
    // A scale that the page came with may be so small that its reciprocal is infinite, and zeros would become NaN.
    // NaN scale: codes 0, every token reads as NaN.
    inv = s > 0.f ? fminf(__fdiv_rn(1.f, s), 3.402823466e38f) : 0.f;
  }
};

}  // namespace exattn
