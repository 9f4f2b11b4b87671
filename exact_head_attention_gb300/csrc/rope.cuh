// Rotary positions and norms of single heads on the device, for the kernels of rope.cu and of cache_append.cu.
//
// A row (one head of one token, d values) lies in d / 16 lanes of a warp, 16 values each: two units of 8 values (16 bytes of
// memory).  Which two is chosen so that both values of a pair are in one lane and the lanes of a row read whole 128-byte
// lines: units u and u + rot / 16 in the half layout (what is behind the rotated part follows two by two), u and u + d / 16
// in the interleaved one.
//
// Angles.  The angle p f of a far position p is large, and only its fraction of a turn counts.  That is taken exactly:
// f / 2 pi is held as a fraction of a turn in 64 bits, whose product with p wraps round by itself, and the upper 32 bits of
// it are the angle in units of 2^-32 turns: the quadrant in two bits, and the rest of it within an eighth of a turn of its
// middle, where short polynomials do.  So no position is too far, and no 64-bit floating-point product (a sixty-fourth of
// the rate here), no reduction and no table of positions is needed.  Error of an angle: 2 p 2^-64 turns of the frequency,
// whatever its size, 2^-32 of the cut, and half a step of fp32 at up to an eighth of a turn.
#pragma once

#include <cstdint>

#include "ptx.cuh"
#include "rope.h"

namespace exattn {

constexpr int kRopeThreads = 256;

// f / 2 pi in units of 2^-64 turns, modulo one turn, within two of them.  f = m 2^(e - 52) with an m of 53 bits, so that f 2^64 / 2 pi
// is (m 2^11) (2^66 / 2 pi) 2^-64 shifted by e - 1; 2^66 / 2 pi has 64 bits and a fraction.  Up to f = 4 the upper half of one
// product has all bits of the result.  Above, 2^66 / 2 pi shifted by e - 1 has whole turns in front, of which the product's
// lower 64 bits count, and the bits behind them come out of its fraction.  `good`: f is finite and below 2^63.
__device__ __forceinline__ uint64_t turns_of(double f, bool& good) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(f));
  const int e = static_cast<int>((bits >> 52) & 0x7ff);
  good = e < 1023 + 63;
  const uint64_t m = e == 0 ? 0ull : (bits & 0xfffffffffffffull) | 0x10000000000000ull;  // below 2^-1022: zero
  const int left = e - 1023 - 1;
  uint64_t u = 0ull;
  if (left <= 0) {
    if (left > -64) u = __umul64hi(m << 11, 0xa2f9836e4e44152aull) >> -left;  // 2^66 / 2 pi, to the nearest
  } else if (good) {  // left from 1 to 61
    constexpr uint64_t whole = 0xa2f9836e4e441529ull, fraction = 0xfc2757d1f534ddc0ull;
    u = (m << 11) * (whole >> (64 - left)) + __umul64hi(m << 11, (whole << left) | (fraction >> (64 - left)));
  }
  return bits >> 63 ? 0ull - u : u;
}

// Sine and cosine of the angle h 2^-32 turns.  v in [-1, 1] counts eighths of a turn from the quadrant's middle; the
// coefficients were fitted to sin(pi v / 4) / v and (cos(pi v / 4) - 1) / v^2 in v^2 for the least largest error (below 2e-9).
// With the roundings of fp32 both are within 1e-7.  Angle 0 gives exactly 0 and 1.
__device__ __forceinline__ void sin_cos_turns(uint32_t h, float& sine, float& cosine) {
  const uint32_t q = h + 0x20000000u;  // the quadrant in bits 30 and 31
  const float v = static_cast<float>(static_cast<int>(q & 0x3fffffffu) - 0x20000000) * 1.862645149230957e-09f;  // 2^-29
  const float z = v * v;
  float s = fmaf(-3.587726e-05f, z, 0.002489872f);
  s = fmaf(s, z, -0.08074537f);
  s = fmaf(s, z, 0.7853981f) * v;
  float c = fmaf(3.5313346e-06f, z, -0.000325942f);
  c = fmaf(c, z, 0.015854327f);
  c = fmaf(c, z, -0.30842513f);
  c = fmaf(c, z, 1.f);
  const bool swap = q & 0x40000000u;
  sine = __uint_as_float(__float_as_uint(swap ? c : s) ^ (q & 0x80000000u));
  cosine = __uint_as_float(__float_as_uint(swap ? s : c) ^ ((q + 0x40000000u) & 0x80000000u));
}

// The pairs' turns a position and their amplitudes (NaN where the frequency is not finite, or 2^63 or more), in shared memory.
struct RopeTable {
  alignas(16) uint64_t turns[64];
  alignas(16) float amplitude[64];

  __device__ __forceinline__ void fill(const RopeView& r, int thread, int threads) {
    for (int i = thread; i < r.rot >> 1; i += threads) {
      bool good;
      turns[i] = turns_of(r.freq[i], good);
      amplitude[i] = good ? r.amplitude : __int_as_float(0x7fffffff);
    }
  }
};

__device__ __forceinline__ long long rope_position(const RopeView& r, int b, int n, const int* start) {
  long long p = start ? start[b] : 0;
  return p + (r.offsets ? r.offsets[b * r.offset_stride + n] : n);
}

// A lane's place in a row: its units, and whether they turn.
template <int D>
struct RopeLane {
  static constexpr int LANES = D / 16;
  int ua, ub;
  bool ta, tb, interleaved;

  __device__ __forceinline__ RopeLane(const RopeView& r, int u) : interleaved(r.interleaved) {
    if (!interleaved) {
      const int pairs = r.rot >> 4;
      ta = tb = u < pairs;
      ua = ta ? u : 2 * u;
      ub = ta ? u + pairs : 2 * u + 1;
    } else {
      ua = u;
      ub = u + LANES;
      ta = 8 * ua < r.rot;
      tb = 8 * ub < r.rot;
    }
  }
  __device__ __forceinline__ bool turns() const { return ta || tb; }
  __device__ __forceinline__ bool turns(int i) const { return i < 4 ? ta : tb; }

  // Cosines and sines of the lane's eight pairs at position p, times the amplitude.  `back`: the transposed rotation.
  __device__ __forceinline__ void angles(const RopeTable& t, long long p, bool back, float (&c)[8], float (&s)[8]) const {
    const uint32_t sign = back ? 0x80000000u : 0u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int first = interleaved ? 4 * (h ? ub : ua) : 8 * ua + 4 * h;
      if (!turns(4 * h)) continue;
      const ulonglong2 t0 = *reinterpret_cast<const ulonglong2*>(t.turns + first),
                       t1 = *reinterpret_cast<const ulonglong2*>(t.turns + first + 2);
      const float4 am = *reinterpret_cast<const float4*>(t.amplitude + first);
      const uint64_t tu[4] = {t0.x, t0.y, t1.x, t1.y};
      const float a[4] = {am.x, am.y, am.z, am.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float si, co;
        sin_cos_turns(static_cast<uint32_t>((static_cast<uint64_t>(p) * tu[i]) >> 32), si, co);
        c[4 * h + i] = co * a[i];
        s[4 * h + i] = __uint_as_float(__float_as_uint(si) ^ sign) * a[i];
      }
    }
  }
  // Where the values of pair i lie among the lane's 16.
  __device__ __forceinline__ static constexpr int first(bool inter, int i) { return inter ? 2 * i : i; }
  __device__ __forceinline__ static constexpr int second(bool inter, int i) { return inter ? 2 * i + 1 : 8 + i; }

  template <bool INTER>
  __device__ __forceinline__ void rotate_as(float (&x)[16], const float (&c)[8], const float (&s)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (turns(i)) {
        float &xa = x[first(INTER, i)], &xb = x[second(INTER, i)];
        const float a = xa, b = xb;
        xa = a * c[i] - b * s[i];
        xb = a * s[i] + b * c[i];
      }
    }
  }
  __device__ __forceinline__ void rotate(float (&x)[16], const float (&c)[8], const float (&s)[8]) const {
    if (interleaved) rotate_as<true>(x, c, s); else rotate_as<false>(x, c, s);
  }
  // The weights of the lane's values, in fp32.
  template <bool BF16>
  __device__ __forceinline__ void weights(const void* w, bool fp32, float (&x)[16]) const {
    if (fp32) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float4 v = reinterpret_cast<const float4*>(w)[2 * (h < 2 ? ua : ub) + (h & 1)];
        x[4 * h] = v.x;
        x[4 * h + 1] = v.y;
        x[4 * h + 2] = v.z;
        x[4 * h + 3] = v.w;
      }
    } else {
      widen<BF16>(reinterpret_cast<const uint4*>(w)[ua], reinterpret_cast<const uint4*>(w)[ub], x);
    }
  }
  template <bool BF16>
  static __device__ __forceinline__ void widen(const uint4& a, const uint4& b, float (&x)[16]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = unpack_lo<BF16>(w[i]);
      x[2 * i + 1] = unpack_hi<BF16>(w[i]);
    }
  }
  template <bool BF16>
  __device__ __forceinline__ void store(uint16_t* row, const float (&x)[16]) const {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack2<BF16>(x[2 * i], x[2 * i + 1]);
    reinterpret_cast<uint4*>(row)[ua] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(row)[ub] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  // The sum over the lanes of a row; all lanes of the warp are here.
  static __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  // 1 / sqrt(mean x^2 + eps)
  static __device__ __forceinline__ float inverse_rms(const float (&x)[16], float eps) {
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i & 1] = fmaf(x[i], x[i], q[i & 1]);
    return rsqrtf(row_sum(q[0] + q[1]) * (1.f / D) + eps);
  }
};

// A norm's weights and a rotation as one product for each pair: (a, b) -> (a ac - b bs, a as + b bc), with the weights of a
// and b in the four factors; values that do not turn have their weights in ac and bc.
template <int D, bool BF16>
struct RopeFactors {
  float ac[8], bs[8], as[8], bc[8];

  template <bool INTER>
  __device__ __forceinline__ void fold(const RopeLane<D>& l, const float (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float wa = w[l.first(INTER, i)], wb = w[l.second(INTER, i)], c = l.turns(i) ? ac[i] : 1.f, s = bs[i];
      ac[i] = wa * c;
      bc[i] = wb * c;
      as[i] = wa * s;
      bs[i] = wb * s;
    }
  }
  // For position p; weight nullptr: none.
  __device__ __forceinline__ RopeFactors(const RopeLane<D>& l, const RopeTable& t, long long p, bool back, const void* weight, bool fp32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) bs[i] = 0.f;
    l.angles(t, p, back, ac, bs);
    float w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = 1.f;
    if (weight) l.template weights<BF16>(weight, fp32, w);
    if (l.interleaved) fold<true>(l, w); else fold<false>(l, w);
  }
  template <bool INTER>
  __device__ __forceinline__ void apply_as(const RopeLane<D>& l, float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float &xa = x[l.first(INTER, i)], &xb = x[l.second(INTER, i)];
      const float a = xa, b = xb;
      xa = a * ac[i];
      xb = b * bc[i];
      if (l.turns(i)) {  // else a NaN in one would reach the other
        xa = fmaf(-b, bs[i], xa);
        xb = fmaf(a, as[i], xb);
      }
    }
  }
  __device__ __forceinline__ void apply(const RopeLane<D>& l, float (&x)[16]) const {
    if (l.interleaved) apply_as<true>(l, x); else apply_as<false>(l, x);
  }
};

// 16 bytes into shared memory, past the registers; zeros where `there` is false.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

constexpr int kRopeDepth = 4;

struct RopeShared {
  RopeTable table;
  uint4 slots[kRopeDepth][2][kRopeThreads];  // a thread's two units of the rows under way
};

// Norm (where there are weights) and rotation of the block's tokens, a thread taking `span` heads of one after the other.
// Called by all threads of a block; chunks of `span` heads of the queries come first, then those of the keys.
// Loads are kRopeDepth - 1 rows ahead, by way of places of the thread's own in shared memory, so that they stay under way
// while it computes and cost no registers (12 heads of 128 each, 32768 tokens: 62.9 us; 67.0 with one row ahead, 63.4 with
// two; 68.7 with two rows at a time through registers).
template <int D, bool BF16>
__device__ __forceinline__ void rope_rows(const RopeArgs& a, RopeShared& sh, unsigned token_block, unsigned chunk_block) {
  using Lane = RopeLane<D>;
  constexpr int GROUPS = kRopeThreads / Lane::LANES, DEPTH = kRopeDepth;
  const int g = threadIdx.x / Lane::LANES;
  const long long t = (static_cast<long long>(token_block) << a.token_shift) + (g & ((1 << a.token_shift) - 1));
  int chunk = chunk_block * (GROUPS >> a.token_shift) + (g >> a.token_shift);
  const bool is_k = chunk >= a.q_chunks;
  const RopeSide& sd = a.side[is_k];
  if (is_k) chunk -= a.q_chunks;
  const int h0 = chunk * a.span;
  const int here = t < a.tokens ? min(a.span, sd.heads - h0) : 0;  // heads of the chunk, where above 0
  const int b = static_cast<int>(t) / a.N, n = static_cast<int>(t) - b * a.N;
  const Lane l(a.r, threadIdx.x % Lane::LANES);
  const uint16_t* src = static_cast<const uint16_t*>(sd.x) + b * sd.sx.b + h0 * sd.sx.h + n * sd.sx.n;
  uint16_t* dst = static_cast<uint16_t*>(sd.y) + b * sd.sy.b + h0 * sd.sy.h + n * sd.sy.n;
  int slot = 0, ahead = 0;
  auto issue = [&]() {
    if (ahead < a.span) {
      const bool there = ahead < here;
      const uint4* from = reinterpret_cast<const uint4*>(there ? src : sd.x);
      copy16(&sh.slots[slot][0][threadIdx.x], from + l.ua, there);
      copy16(&sh.slots[slot][1][threadIdx.x], from + l.ub, there);
    }
    copies_commit();
    slot = slot + 1 == DEPTH ? 0 : slot + 1;
    src += sd.sx.h;
    ++ahead;
  };
#pragma unroll 1
  for (int k = 0; k < DEPTH - 1; ++k) issue();
  const long long p = here > 0 ? rope_position(a.r, b, n, a.r.start) : 0;
  sh.table.fill(a.r, threadIdx.x, kRopeThreads);
  __syncthreads();
  const bool norm = sd.weight != nullptr;
  // queries and keys may share a warp: all its lanes take part in the sums
  const bool any_norm = a.side[0].weight != nullptr || a.side[1].weight != nullptr;
  const RopeFactors<D, BF16> f(l, sh.table, p, a.r.back, sd.weight, a.weight_fp32);
  int from = 0;
  const int rows = __reduce_max_sync(0xffffffffu, max(here, 0));  // of the warp
#pragma unroll 1
  for (int i = 0; i < rows; ++i) {
    issue();
    copies_wait<DEPTH - 1>();
    float x[16];
    Lane::template widen<BF16>(sh.slots[from][0][threadIdx.x], sh.slots[from][1][threadIdx.x], x);
    from = from + 1 == DEPTH ? 0 : from + 1;
    if (any_norm) {
      const float r = Lane::inverse_rms(x, a.r.eps);
      if (norm) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= r;  // first, so that no product of a weight is out of range before
      }
    }
    f.apply(l, x);
    if (i < here) l.template store<BF16>(dst, x);
    dst += sd.sy.h;
  }
  copies_wait<0>();
}

}  // namespace exattn
