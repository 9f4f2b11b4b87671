// Writing tokens into the 8-bit key/value cache with the keys' norm and rotary positions on the way, and the queries of the
// same tokens in the same launch.
//
// Mathematics: the keys of rope.cu in fp32, unrounded, then the rule of the cache's write (cache_io.cuh): the largest value
// of a page's new tokens gives its scale, and with that the codes.  So no rotated key is rounded twice or goes through memory.
//
// Bound: memory, 2 bytes read and 1 written a value, 2 and 2 of the queries; but with 15 operations a value the instructions
// are close behind, and most of what is below is about them.  As in cache_io.cu one page of one head, keys or values, is held
// by GT threads, here widened to fp32 in their registers from the load to the codes: 32 values each (64 at the largest page),
// so that three blocks fit an SM.  A thread has whole lanes of rows (rope.cuh).
//   * A block has several heads of a page one after the other, since the angles, 25 instructions a token and pair, are the same
//     for all of them: they are computed once, into shared memory.
//   * The next head's rows come by asynchronous copies while the current one's are worked on.
//   * A lane's values are kept as first and second values of pairs, so that both layouts are one arithmetic of fp32 pairs.
// Measured, 4 prompts of 8192 tokens, 12 heads of 128, without queries (302 MB, 44.6 us at the copy rate; the write without
// norm and rotation takes 47.5): each thread the angles of its own page and head 110 us; from shared memory, 64 values a
// thread, 109 (spilled registers); 32 values and copies ahead 64; fp32 pairs 58; all 12 heads in a block 56.  With as many
// queries 80 us (503 MB, 93 %).  One token of each of 64 sequences, 8 heads, with 32 query heads: 6.3 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache8.cuh"
#include "cache.h"
#include "cache_io.cuh"
#include "ptx.cuh"
#include "rope.cuh"

#include <atomic>

namespace exattn {
namespace {

static_assert(kIoThreads == kRopeThreads, "one launch for both");
constexpr int kAppendBlocks = 3;  // resident an SM where a thread has two rows
// Shared memory: a cosine and a sine for each pair of a thread's NV * 8 values, and those in 16 bits.
template <int NV>
constexpr int kMostShared = kIoThreads * NV * (8 * 4 + 16);
static_assert(sizeof(RopeShared) <= kMostShared<4>, "room for the queries' part");

__device__ __forceinline__ uint2 to_codes_of(int format, const float (&y)[8]) {
  return format == kE4M3 ? to_codes<kE4M3>(y) : to_codes<kInt8>(y);
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// A lane's values of a row as fp32 pairs of neighbouring pairs' first, and second, values: with them the arithmetic is the same
// in both layouts and takes two values an instruction.
template <bool INTER>
struct PairedRow {
  uint64_t p[4], q[4];

  __device__ __forceinline__ void set(const float (&x)[16]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      p[k] = INTER ? f2_pack(x[4 * k], x[4 * k + 2]) : f2_pack(x[2 * k], x[2 * k + 1]);
      q[k] = INTER ? f2_pack(x[4 * k + 1], x[4 * k + 3]) : f2_pack(x[8 + 2 * k], x[9 + 2 * k]);
    }
  }
  __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (INTER) {
        f2_unpack(p[k], x[4 * k], x[4 * k + 2]);
        f2_unpack(q[k], x[4 * k + 1], x[4 * k + 3]);
      } else {
        f2_unpack(p[k], x[2 * k], x[2 * k + 1]);
        f2_unpack(q[k], x[8 + 2 * k], x[9 + 2 * k]);
      }
    }
  }
  // Where number k of p, or q, stands among the lane's 16.
  static __device__ __forceinline__ int place(bool second, int k) { return INTER ? 2 * k + second : k + 8 * second; }
  __device__ __forceinline__ float squares() const {
    uint64_t s = f2_mul(p[0], p[0]), t = f2_mul(q[0], q[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) {
      s = f2_fma(p[k], p[k], s);
      t = f2_fma(q[k], q[k], t);
    }
    float a, b;
    f2_unpack(f2_add(s, t), a, b);
    return a + b;
  }
  __device__ __forceinline__ void times(float f) {
    const uint64_t f2 = f2_pack(f, f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      p[k] = f2_mul(p[k], f2);
      q[k] = f2_mul(q[k], f2);
    }
  }
  __device__ __forceinline__ void times(const ulonglong2 (&w)[4]) {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      p[k] = f2_mul(p[k], w[k / 2].x);
      p[k + 1] = f2_mul(p[k + 1], w[k / 2].y);
      q[k] = f2_mul(q[k], w[2 + k / 2].x);
      q[k + 1] = f2_mul(q[k + 1], w[2 + k / 2].y);
    }
  }
  // Pairs 4 h to 4 h + 3 turned.
  __device__ __forceinline__ void turn(int h, const ulonglong2& c, const ulonglong2& s) {
    const uint64_t cs[2] = {c.x, c.y}, sn[2] = {s.x, s.y};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint64_t &a = p[2 * h + k], &b = q[2 * h + k];
      const uint64_t as = f2_mul(a, sn[k]);
      a = f2_sub(f2_mul(a, cs[k]), f2_mul(b, sn[k]));
      b = f2_fma(b, cs[k], as);
    }
  }
  // The largest |value|, or NaN.
  __device__ __forceinline__ float largest() const {
    float x[16];
    get(x);
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 16; e += 2) m = max3_nan(m, fabsf(x[e]), fabsf(x[e + 1]));
    return m;
  }
};

template <int D, bool BF16, bool INTER, int GT, int NV>
__global__ void __launch_bounds__(kIoThreads, NV == 4 ? kAppendBlocks : 2) cache_append_kernel(const __grid_constant__ CacheAppendArgs a) {
  using Lane = RopeLane<D>;
  constexpr int UNITS = kIoThreads / GT, ROWS = NV / 2, STEP = GT / Lane::LANES;  // rows of a thread, and between them
  constexpr int PAGE = ROWS * STEP, SLOTS = D / 2;                                // pairs of a row, a cosine and a sine each
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ __align__(16) uint32_t s_max[2][kIoThreads / 32];
  __shared__ __align__(16) float weights[2][SLOTS];  // in the order of PairedRow, lane by lane
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x >= 2u * a.blocks) {
    const unsigned qb = blockIdx.x - 2u * a.blocks, cb = qb / a.q_token_blocks;
    rope_rows<D, BF16>(a.rope, *reinterpret_cast<RopeShared*>(smem_raw), qb - cb * a.q_token_blocks, cb);
    return;
  }
  const CacheView& c = a.io.c;
  const RopeView& rv = a.rope.r;
  const bool is_v = blockIdx.x >= static_cast<unsigned>(a.blocks);
  const unsigned block = blockIdx.x - (is_v ? a.blocks : 0), chunk = block / a.page_blocks;
  // unit g: page group g >> head_shift of the block, and its head of those side by side
  const int g = threadIdx.x / GT, tid = threadIdx.x % GT, u = tid % Lane::LANES, side = 1 << a.head_shift, pg = g >> a.head_shift;
  const int head0 = chunk * a.span + (g & (side - 1)), heads = min(c.heads, static_cast<int>(chunk + 1) * a.span);
  const unsigned item = (block - chunk * a.page_blocks) * (UNITS >> a.head_shift) + pg;  // of B * parts pages
  const int b = item / a.io.parts, pj = item - b * a.io.parts;
  CacheUnit un;
  if (b < a.io.B) un.find(a.io, b, pj, tid == 0);
  const int r0 = un.r0, r1 = un.page < 0 ? r0 : un.r1, inside = un.inside;
  const Lane l(rv, u);

  // A head's rows under way: a thread's two units of each of its rows.  Rows that are not new stay zero.
  uint4 (*const slots)[kIoThreads] = reinterpret_cast<uint4 (*)[kIoThreads]>(smem_raw + a.slots_at);
  const RowStrides& st = is_v ? a.io.sv : a.io.sk;
  const int row0 = tid / Lane::LANES;
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? a.io.v : a.io.k) + b * st.b + head0 * st.h + (un.row_of_r0 - r0 + row0) * st.n + 8 * l.ua;
  const int to_ub = 8 * (l.ub - l.ua);
  const long long next_head = side * st.h, next_row = STEP * st.n;
  bool there[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int row = row0 + i * STEP;
    there[i] = row >= r0 && row < r1;
    if (!there[i]) slots[2 * i][threadIdx.x] = slots[2 * i + 1][threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
  }
  auto load = [&](bool some) {
    if (some) {
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        if (there[i]) {
          copy16(&slots[2 * i][threadIdx.x], src + i * next_row);
          copy16(&slots[2 * i + 1][threadIdx.x], src + i * next_row + to_ub);
        }
      }
      src += next_head;
    }
    copies_commit();
  };
  load(head0 < heads);

  float* const cosines = reinterpret_cast<float*>(smem_raw) + pg * PAGE * SLOTS;
  float* const sines = cosines + (UNITS >> a.head_shift) * PAGE * SLOTS;
  const void* weight = is_v ? nullptr : a.k_weight;
  if (!is_v) {
    if (weight) {
      for (int i = threadIdx.x; i < D; i += kIoThreads) {
        const int lane = i / 16, k = i % 16, second = k >> 3;
        const Lane at(rv, lane);
        const int e = PairedRow<INTER>::place(second, k & 7), col = 8 * (e < 8 ? at.ua : at.ub) + (e & 7);
        weights[second][8 * lane + (k & 7)] = a.rope.weight_fp32 ? static_cast<const float*>(weight)[col]
                                                                 : unpack_lo<BF16>(static_cast<const uint16_t*>(weight)[col]);
      }
    }
    // Angles, in the order in which lanes read them: four of the first half of the lanes' pairs side by side, then four of
    // the second.
    if (rv.rot > 0 && r0 < r1) {
      const long long first = (rv.start ? rv.start[b] : 0) + (rv.offsets ? 0 : un.row_of_r0 - r0);
      const int* offsets = rv.offsets ? rv.offsets + b * rv.offset_stride + (un.row_of_r0 - r0) : nullptr;
      static_assert(GT >= SLOTS, "a thread for each of a row's pairs at least");
      const int at = threadIdx.x & ((GT << a.head_shift) - 1), step = (GT << a.head_shift) / SLOTS, slot = at & (SLOTS - 1);
      const int h = slot / (SLOTS / 2), lane = slot / 4 % Lane::LANES;
      const int pair = (INTER ? 4 * (lane + h * Lane::LANES) : 8 * lane + 4 * h) + (slot & 3);
      if (pair < rv.rot >> 1) {
        bool good;
        const uint64_t turns = turns_of(rv.freq[pair], good);
        const float amplitude = good ? rv.amplitude : __int_as_float(0x7fffffff);
        const int first_row = r0 + at / SLOTS;
        auto direct = [&](uint64_t angle, float& co, float& si) { sin_cos_turns(static_cast<uint32_t>(angle >> 32), si, co); };
        auto put = [&](int row, float co, float si) {
          cosines[row * SLOTS + slot] = co;
          sines[row * SLOTS + slot] = si;
        };
        if (offsets || r1 - r0 < 4 * step) {
          for (int row = first_row; row < r1; row += step) {
            float co, si;
            direct(static_cast<uint64_t>(first + (offsets ? offsets[row] : row)) * turns, co, si);
            put(row, co * amplitude, si * amplitude);
          }
        } else {
          // Rows in order: every fourth angle of a thread's is computed, and the three behind it are that turned by one, two
          // and three steps.
          const uint64_t ahead = step * turns;
          float ch[3], sh[3];
#pragma unroll
          for (int k = 0; k < 3; ++k) direct((k + 1) * ahead, ch[k], sh[k]);
          uint64_t angle = static_cast<uint64_t>(first + first_row) * turns;
#pragma unroll 1
          for (int row = first_row; row < r1; row += 4 * step, angle += 4 * ahead) {
            float co, si;
            direct(angle, co, si);
            co *= amplitude;
            si *= amplitude;
            put(row, co, si);
#pragma unroll
            for (int k = 0; k < 3; ++k)
              if (row + (k + 1) * step < r1) put(row + (k + 1) * step, co * ch[k] - si * sh[k], co * sh[k] + si * ch[k]);
          }
        }
      }
    }
    __syncthreads();
  }
  if (un.page < 0) {  // all threads of a unit together
    copies_wait<0>();
    return;
  }
  const float* const angle = cosines + row0 * SLOTS + 4 * u;
  const int to_sines = static_cast<int>(sines - cosines);
  const long long ph0 = static_cast<long long>(un.page) * c.heads + head0;
  float* scale_at = (is_v ? c.v_scale : c.k_scale) + ph0;
  uint8_t* codes = (is_v ? c.v : c.k) + ph0 * (PAGE * D) + row0 * D;
  int turn = 0;
#pragma unroll 1
  for (int head = head0; head < heads; head += side, turn ^= 1, scale_at += side, codes += side * (PAGE * D)) {
    float old = 0.f;
    if (inside > 0) old = *scale_at;
    copies_wait<0>();
    uint4 raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) raw[i] = slots[i][threadIdx.x];
#pragma unroll
    for (int i = 0; i < NV; ++i) loaded(raw[i]);  // the places are free once the values are here
    load(head + side < heads);
    PairedRow<INTER> x[ROWS];
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      float v[16];
      Lane::template widen<BF16>(raw[2 * i], raw[2 * i + 1], v);
      x[i].set(v);
    }
    if (weight) {
      const ulonglong2* w = reinterpret_cast<const ulonglong2*>(weights[0] + 8 * u);
      const ulonglong2 ws[4] = {w[0], w[1], w[SLOTS / 4], w[SLOTS / 4 + 1]};
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        x[i].times(rsqrtf(Lane::row_sum(x[i].squares()) * (1.f / D) + rv.eps));
        x[i].times(ws);
      }
    }
    if (!is_v) {
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        if (!there[i]) continue;  // no angles there
        const float* at = angle + i * STEP * SLOTS;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (h ? l.tb : l.ta)
            x[i].turn(h, *reinterpret_cast<const ulonglong2*>(at + h * (SLOTS / 2)), *reinterpret_cast<const ulonglong2*>(at + to_sines + h * (SLOTS / 2)));
      }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) most = max3_nan(most, most, x[i].largest());
    uint32_t mx = __reduce_max_sync(0xffffffffu, __float_as_uint(most) & 0x7fffffffu);  // a NaN or an infinity above all others
    if constexpr (GT > 32) {
      if ((threadIdx.x & 31) == 0) s_max[turn][threadIdx.x >> 5] = mx;
      named_bar_sync(g + 1, GT);
      if constexpr (GT == 64) {
        const uint2 m = *reinterpret_cast<const uint2*>(&s_max[turn][2 * g]);
        mx = max(m.x, m.y);
      } else {
        mx = 0u;
#pragma unroll
        for (int k = 0; k < GT / 128; ++k) {
          const uint4 m = *reinterpret_cast<const uint4*>(&s_max[turn][GT / 32 * g + 4 * k]);
          mx = max(mx, max(max(m.x, m.y), max(m.z, m.w)));
        }
      }
    } else {
      __syncwarp();  // the old scale has been read by every lane before one of them writes the new
    }
    const CacheScale sc(c.format, mx >= 0x7f800000u ? __int_as_float(0x7fffffff) : __uint_as_float(mx), inside > 0, old);
    if (tid == 0) *scale_at = sc.s;
    const bool alive = sc.s > 0.f;  // else all codes are zero
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      uint2* to = reinterpret_cast<uint2*>(codes + i * STEP * D);
      if (there[i]) {
        x[i].times(sc.inv);
        float v[16];
        x[i].get(v);
        uint2 ca = make_uint2(0u, 0u), cb = ca;
        if (alive) {
          const float va[8] = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]}, vb[8] = {v[8], v[9], v[10], v[11], v[12], v[13], v[14], v[15]};
          ca = to_codes_of(c.format, va);
          cb = to_codes_of(c.format, vb);
        }
        to[l.ua] = ca;
        to[l.ub] = cb;
      } else if (sc.grew && row0 + i * STEP < r0) {
        const float again = old * sc.inv;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint2* at = to + (h ? l.ub : l.ua);
          float y[8];
          if (c.format == kE4M3) from_codes<kE4M3>(*at, y); else from_codes<kInt8>(*at, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] *= again;
          *at = to_codes_of(c.format, y);
        }
      }
    }
  }
  copies_wait<0>();  // a copy must not land after the block has ended
}

template <int D, bool BF16, bool INTER, int GT, int NV>
cudaError_t append_t(CacheAppendArgs& a, cudaStream_t stream) {
  constexpr int UNITS = kIoThreads / GT, PAGE = GT * NV * 8 / D;
  a.io.parts = static_cast<int>((a.io.N + static_cast<long long>(PAGE) - 2) / PAGE) + 1;
  const long long pages = static_cast<long long>(a.io.B) * a.io.parts;
  // Heads side by side: as many as a block has room for; where there are fewer, several pages.
  a.head_shift = 0;
  while ((1 << a.head_shift) < UNITS && (1 << a.head_shift) < a.io.c.heads) ++a.head_shift;
  const int side = 1 << a.head_shift, groups = UNITS >> a.head_shift;
  a.page_blocks = static_cast<int>((pages + groups - 1) / groups);
  // Turns of `side` heads a block: the angles take about as long as two and a half of them.  A second wave of few blocks takes as
  // long as a full one; where there are more, blocks that are done make room for others.  Without queries, 12 heads of 128 and
  // 32768 tokens: 111 us with 1, 77 with 2, 68 with 3, 62 with 4, 58 with 6, 56 with 12; 8 heads, one token of each of 64
  // sequences: 7.7, 5.9, 6.6 (the first of one wave), 7.0 and 8.6 us.
  const long long slots = static_cast<long long>(NV == 4 ? kAppendBlocks : 2) * a.io.sm_count;
  long long best = 0, blocks = 0;
  for (int turns : {1, 2, 3, 4, 6, 8, 12}) {
    const int span = turns * side;
    if (turns > 1 && span - side >= a.io.c.heads) break;
    const long long n = a.page_blocks * static_cast<long long>((a.io.c.heads + span - 1) / span);
    const long long waves16 = 2 * n > 2 * slots ? 32 * n / slots : 2 * n > slots ? 32 : 16;
    const long long cost = waves16 * (2 * turns + 5);
    if (best == 0 || cost < best) {
      best = cost;
      blocks = n;
      a.span = span;
    }
  }
  a.blocks = static_cast<int>(blocks);
  long long q_blocks = 0;
  a.q_token_blocks = 1;
  size_t smem = a.rope.r.rot > 0 ? static_cast<size_t>(2) * groups * PAGE * (D / 2) * sizeof(float) : 0;
  a.slots_at = static_cast<int>(smem);
  smem += NV * kIoThreads * sizeof(uint4);
  if (a.rope.side[0].heads > 0) {
    const RopeGrid grid = rope_plan(a.rope);
    a.q_token_blocks = static_cast<int>(grid.token_blocks);
    q_blocks = static_cast<long long>(grid.token_blocks) * grid.chunk_blocks;
    if (smem < sizeof(RopeShared)) smem = sizeof(RopeShared);
  }
  const long long grid = 2 * blocks + q_blocks;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  static std::atomic<uint64_t> done{0};
  auto kern = cache_append_kernel<D, BF16, INTER, GT, NV>;
  const cudaError_t e = allow_smem(kern, kMostShared<NV>, done);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(kIoThreads), smem, stream, a);
}

template <bool BF16, bool INTER>
cudaError_t append_f(CacheAppendArgs& a, cudaStream_t stream) {
  const int psize = 1 << a.io.c.page_shift;
  if (a.io.c.d == 64) {
    switch (psize) {
      case 16: return append_t<64, BF16, INTER, 32, 4>(a, stream);
      case 32: return append_t<64, BF16, INTER, 64, 4>(a, stream);
      case 64: return append_t<64, BF16, INTER, 128, 4>(a, stream);
      default: return append_t<64, BF16, INTER, 256, 4>(a, stream);
    }
  }
  switch (psize) {
    case 16: return append_t<128, BF16, INTER, 64, 4>(a, stream);
    case 32: return append_t<128, BF16, INTER, 128, 4>(a, stream);
    case 64: return append_t<128, BF16, INTER, 256, 4>(a, stream);
    default: return append_t<128, BF16, INTER, 256, 8>(a, stream);
  }
}

}  // namespace

cudaError_t launch_cache_append(CacheAppendArgs& a, cudaStream_t stream) {
  if (a.rope.r.interleaved) return a.io.bf16 ? append_f<true, true>(a, stream) : append_f<false, true>(a, stream);
  return a.io.bf16 ? append_f<true, false>(a, stream) : append_f<false, false>(a, stream);
}

}  // namespace exattn
