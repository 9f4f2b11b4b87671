// Attention over the 8-bit cache for many query rows a key/value head (chunks of a prompt, drafted tokens
// under shared heads): the tensor-core form of cache_attn.cuh.
//
// Mathematics as there: codes as they are in fp16, the key scale on the scores, the value scale on the probabilities, over
// a reference w for each row (cache8.cuh).
//
// Probabilities go into the product as one fp16 number, for fp16 outputs too: where many keys count alike, their rounding
// moves O by about as much as O's own, so that such outputs are 1.0 to 1.35 times as far off as their rounding (a bf16 output's
// rounding covers it).  Two numbers, as the trees of cache_attn.cuh have, bring that to 1.00, but here the products and the
// softmax set the pace.  Trees, one number against two, 128 columns a head: 16 sequences of 4096 tokens, 8 heads, 96 rows
// 60.4 : 77.9 us, 256 rows 74.9 : 119.2 us; 40 of 2048, 4 heads, 64 rows 57.2 : 65.7 us.
//
// Bound.  4 d flops for each row and key: the tensor cores, which tcgen05 reaches with 128 x 128 tiles in
// tensor memory.  Its operands are fp16 in shared memory, so six warps turn each 128-token tile of codes, copied
// in by the copy engine, into the swizzled operand tiles; 256 query rows share that work.
//
// Two chains of (scores, softmax, product) alternate on the tensor cores, one softmax warpgroup each:
//   PAIR    more than 128 rows: an item has 256, chain t works on rows [128 t, 128 t + 128)
//   else    an item has 128 rows, and chain t works on every second key tile; the two results are joined in
//           the epilogue.  Both chains then have work at any number of rows.  Up to 64 rows lie in the query tile
//           twice, and each copy's softmax takes half of a tile's keys (64 queries over 16k tokens on 16 heads of 64:
//           55 us without, 51 us with it).
// The chains' steps (one 128-token tile of one chain) form one sequence, and step i has score buffer i mod NB,
// which its P overwrites: S[0] .. S[NB-1] | O[0] S[NB] O[1] S[NB+1] ...  At d = 64 tensor memory has room for three
// buffers, so that a chain's next scores are there when its softmax has finished a step; at d = 128 for two.
// Steps of 64 keys with two buffers a chain were tried for d = 128: a score product of 64 columns takes as long as one
// of 128 (72 cycles for each 16 positions), and the whole became 1.4 times slower.
//
// Measured on GB300: 512 queries at the end of 12289 cached tokens, 2 sequences, 8 heads of 128 with 4 query heads each,
// in 180 us, 1.12 PFLOP/s, 58 % of the measured cuBLAS rate; 64 queries over 16k tokens of 4 sequences, 16 heads of 64, in
// 53 us (2.5 TB/s of codes).  The tensor pipe is active for 45 % of the first (ncu).  The warp that issues the
// products, whose instructions come back into an instruction cache that the softmax fills, is busy all the time: 1750
// cycles for the two products of a step.  Dropped, with what 176 us (before NaN codes were looked for) became:
// no issuing warp, each chain's softmax warps issuing its products (180, and 67 for the other's 56); the issuing warp's
// ring positions a lane each instead of all in every lane (181); the softmax as a loop over 64 keys, a quarter of the
// code (197).
//
// Warp roles (512 threads, registers re-split per warpgroup):
//   warps 0-3, 4-7  softmax of chain 0 and 1 (thread = query row = TMEM lane); they also bring the query rows
//                   into their operand tile and write the results
//   warp  8         product issue (the warp together, one elected lane), TMEM owner
//   warp  9         producer: walks the block's pieces (cache_sched.cuh), looks pages up, copies codes
//   warps 10-12, 13-15  converters of the keys and of the values, about 43 tokens of each tile apiece
// Tensor memory: score buffer b (P over its first 64 columns) at 128 b, O_t behind the buffers.
// Every role walks the same pieces and counts steps on, so the barriers are never re-armed.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "cache8.cuh"
#include "cache_sched.cuh"
#include "cache.h"
#include "ptx.cuh"

namespace exattn {
namespace {

constexpr int kThreads = 512;
// Registers: 128 a thread at launch; the softmax warpgroups hold a row of 128 scores.
constexpr uint32_t kRegsSoftmax = 176, kRegsOther = 80;
static_assert(2 * kRegsSoftmax + 2 * kRegsOther == 4 * 128, "register split must match the launch");
constexpr int kTK = 128;
constexpr uint32_t kChunk = 128 * 128;  // 128 rows x 128 bytes
constexpr int kPieceRing = 3;
// Flags of tiles that an item's rows see in part: at most 3 at a piece's end (the rows of an item see the keys of at
// most 256 tokens less or more; under a tree 5, of kTreeMost tokens), and the converters are at most NS tiles further.
constexpr int kFlagRing = 8;
static_assert((kTreeMost + 126) / kTK + 1 <= 5, "tiles that a tree's tokens reach into");
constexpr float kShift = 3.f;  // as in cache_attn.cuh
constexpr int kMeta = 24;      // numbers a tile: ks[8], vs[8], log2 vs[8]

template <int D, bool PAIR, bool TREE>
struct Cfg {
  static constexpr int R = PAIR ? 256 : 128;
  static constexpr int MIN_TILES = PAIR ? 2 : 4;
  static constexpr uint32_t TILE = 128 * D * 2;                // an fp16 operand tile
  static constexpr uint32_t RAW = 128 * D;                     // a tile of codes
  static constexpr int NS = D == 128 ? 2 : 3;                  // K and V operand slots
  static constexpr int NR = D == 128 ? (PAIR ? 2 : 3) : 8;     // slots of codes, K and V in turn
  static constexpr int NB = D == 64 ? 3 : 2;                   // score buffers
  // Scales stay in use from a tile's copy to its softmax, over tiles of codes, operand tiles, and steps under way.
  static constexpr int MR = D == 128 ? 8 : 16;
  static_assert((NR + 1) / 2 + NS + NB + 1 <= MR, "scales of the tiles under way");
  static constexpr uint32_t TM_O = NB * 128;                   // O_t at TM_O + t TM_OT
  static constexpr uint32_t TM_OT = D;
  static_assert(5 + NS <= kFlagRing, "flags of the tiles under way");
  static_assert(TM_O + 2 * TM_OT <= 512, "tensor memory");
  using Walk = CacheWalk<R, kTK, 32, MIN_TILES, TREE>;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = OFF_Q + (PAIR ? 2 : 1) * TILE;
  static constexpr uint32_t OFF_V = OFF_K + NS * TILE;
  static constexpr uint32_t OFF_RAW = OFF_V + NS * TILE;
  static constexpr uint32_t OFF_META = OFF_RAW + NR * RAW;           // [MR][kMeta]
  static constexpr uint32_t OFF_STAT = OFF_META + MR * kMeta * 4;    // !PAIR: {m, l} [2][128], w [2][128]
  static constexpr uint32_t OFF_FLAG = OFF_STAT + (PAIR ? 0 : 2 * 128 * 12);  // [kFlagRing][128]: a token has a NaN value
  static constexpr uint32_t OFF_PIECE = OFF_FLAG + kFlagRing * 128;
  static constexpr uint32_t OFF_BAR = OFF_PIECE + kPieceRing * kPieceInts * 4;
  static constexpr int NBAR = 2 + 4 * NS + NR + 2 * ((NR + 1) / 2) + 6 + MR + 2 * kPieceRing + 4;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr uint32_t OFF_SCHED = OFF_MISC + 16;
  static constexpr uint32_t BYTES = OFF_SCHED + sizeof(typename Walk::Shared);
  static_assert(BYTES <= 232448, "shared memory of a block");
};

// 16 consecutive 32-bit columns of a warp's 32 lanes; the load waits for its values.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0u;
}

template <int NS, int NR, int MR>
struct Bars {
  uint32_t base;
  __device__ uint32_t at(int i) const { return base + 8 * i; }
  __device__ uint32_t q_full(int t) const { return at(t); }
  __device__ uint32_t k_full(int s) const { return at(2 + s); }
  __device__ uint32_t k_empty(int s) const { return at(2 + NS + s); }
  __device__ uint32_t v_full(int s) const { return at(2 + 2 * NS + s); }
  __device__ uint32_t v_empty(int s) const { return at(2 + 3 * NS + s); }
  // Keys and values take the slots of codes in turn, but the barriers of their arrival are apart: with an odd number of
  // slots a converter would else wait on one whose last phase was the other operand's.  It has not seen that end, and
  // where that copy is still under way it finds the barrier a phase behind and passes early.  Two for each operand do
  // for three slots: the second copy after one is issued only once that one has been read.
  static constexpr int FR = (NR + 1) / 2;
  __device__ uint32_t raw_full(int v, int tile) const { return at(2 + 4 * NS + v * FR + tile % FR); }
  static __device__ uint32_t raw_parity(int tile) { return (tile / FR) & 1; }
  __device__ uint32_t raw_empty(int s) const { return at(2 + 4 * NS + 2 * FR + s); }
  static constexpr int kB = 2 + 4 * NS + NR + 2 * FR;
  __device__ uint32_t s_full(int b) const { return at(kB + b); }
  __device__ uint32_t p_full(int b) const { return at(kB + 3 + b); }
  static constexpr int kC = kB + 6;
  __device__ uint32_t meta_full(int s) const { return at(kC + s); }
  __device__ uint32_t piece_full(int s) const { return at(kC + MR + s); }
  __device__ uint32_t piece_empty(int s) const { return at(kC + MR + kPieceRing + s); }
  __device__ uint32_t join() const { return at(kC + MR + 2 * kPieceRing); }
  __device__ uint32_t mma_done() const { return at(kC + 1 + MR + 2 * kPieceRing); }
  __device__ uint32_t stored(int t) const { return at(kC + 2 + MR + 2 * kPieceRing + t); }
};

// One key tile of the online softmax for this thread's query row.  Scores of the 16-token group g count
// fac * ks[g]; P goes out in fp16 times vs[g] 2^(m - w) (sc: ks[8], vs[8], log2 vs[8]; vf: 2^(m - w)).  Columns at or past
// `lim` are hidden (MASKED), or those without their bit in `seen` (TREE).  All 128 scores are read for the maxima; the upper 64 are read again for P, which saves the
// registers that they would hold meanwhile.  P's packed columns overwrite scores of the lower 64 only.
// wait_pv() runs (warp-uniformly) before O is rescaled: the chain's last product may still be under way.
// HALF: the row is here twice, and this thread has 64 of its 128 scores: from column 64 `half` on, `sc` and `lim` likewise.
// The other half of its P is zero.
template <int D, bool MASKED, bool HALF, bool TREE, typename WaitPv>
__device__ __forceinline__ void softmax_scaled(uint32_t tS, int half, uint32_t tO, const float* sc, int lim,
                                               const uint32_t (&seen)[TREE ? 4 : 1], float fac, bool first, float& m, float& l, float& w, float& vf, WaitPv&& wait_pv) {
  auto hidden = [&](int col) {
    if constexpr (TREE) return (seen[col >> 5] & (1u << (col & 31))) == 0u;
    else return col >= lim;
  };
  constexpr int CHUNKS = HALF ? 2 : 4, GROUPS = 2 * CHUNKS;
  const uint32_t tX = HALF ? tS + half * 64 : tS, tP = HALF ? tS + half * 32 : tS;
  uint32_t sr[CHUNKS][32];
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) tmem_ld32(tX + c * 32, sr[c]);
  float f[GROUPS], vs[GROUPS];
#pragma unroll
  for (int g = 0; g < GROUPS; g += 4) {
    const float4 k = *reinterpret_cast<const float4*>(sc + g), v = *reinterpret_cast<const float4*>(sc + 8 + g);
    f[g] = fac * k.x;
    f[g + 1] = fac * k.y;
    f[g + 2] = fac * k.z;
    f[g + 3] = fac * k.w;
    vs[g] = v.x;
    vs[g + 1] = v.y;
    vs[g + 2] = v.z;
    vs[g + 3] = v.w;
  }
  tmem_wait_ld();
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) reg_fence32(sr[c]);
  float m_new = -INFINITY, w_new = -INFINITY;
  float4 lv;
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    if (g % 4 == 0) lv = *reinterpret_cast<const float4*>(sc + 16 + g);
    float a = -INFINITY, b = -INFINITY;  // a NaN is passed over: it is met below
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = __uint_as_float(sr[g >> 1][(g & 1) * 16 + i + e]);
        if constexpr (MASKED) v[e] = hidden(g * 16 + i + e) ? -INFINITY : v[e];
      }
      a = max3(a, v[0], v[1]);
      b = max3(b, v[2], v[3]);
    }
    const float x = fmaxf(a, b) * f[g];
    m_new = fmaxf(m_new, x);
    w_new = fmaxf(w_new, x + (g % 4 == 0 ? lv.x : g % 4 == 1 ? lv.y : g % 4 == 2 ? lv.z : lv.w));
  }
  const bool need = first || m_new > m + 8.0f;
  if (__any_sync(0xffffffffu, need || w_new > w + kValueLag)) {
    const float to = need ? m_new : m, wt = value_reference(w, w_new, to);
    const float al = need && !first ? ex2_approx(m - to) : 1.0f;
    const float ov = wt == -INFINITY ? 1.0f : ex2_approx(w - wt);
    if (!first) {
      wait_pv();
#pragma unroll 1
      for (int c = 0; c < D / 16; ++c) {
        uint32_t o[16];
        tmem_ld16(tO + c * 16, o);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * ov);
        tmem_st16(tO + c * 16, o);
      }
      tmem_wait_st();
    }
    l *= al;
    m = to;
    w = wt;
    vf = value_factor(to, wt);
  }
  const float ms = m == -INFINITY ? 0.f : m - kShift;
  const uint64_t nm2 = f2_pack(-ms, -ms);
  uint64_t acc[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) acc[i] = f2_pack(0.f, 0.f);
  auto chunk = [&](int c, const uint32_t (&x)[32]) __attribute__((always_inline)) {
    uint32_t pk[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float r = value_weight(vs[2 * c + h], vf);
      const uint64_t f2 = f2_pack(f[2 * c + h], f[2 * c + h]), r2 = f2_pack(r, r);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = h * 8 + k, col = c * 32 + 2 * i;  // scores col and col + 1
        const uint64_t z = f2_fma(f2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), f2, nm2);
        float z0, z1;
        f2_unpack(z, z0, z1);
        float p0 = ex2_approx(z0), p1 = ex2_approx(z1);
        if constexpr (MASKED) {  // whatever the scale
          p0 = hidden(col) ? 0.f : p0;
          p1 = hidden(col + 1) ? 0.f : p1;
        }
        acc[k & 1] = f2_add(acc[k & 1], f2_pack(p0, p1));
        float y0, y1;
        f2_unpack(f2_mul(f2_pack(p0, p1), r2), y0, y1);
        if constexpr (MASKED) {
          y0 = hidden(col) ? 0.f : y0;
          y1 = hidden(col + 1) ? 0.f : y1;
        }
        pk[i] = pack2<false>(y0, y1);
      }
    }
    tmem_st16(tP + c * 16, pk);
  };
  chunk(0, sr[0]);
  if constexpr (HALF) {
    chunk(1, sr[1]);
    uint32_t none[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) none[i] = 0u;
    const uint32_t tZ = tS + (1 - half) * 32;
    tmem_st16(tZ, none);
    tmem_st16(tZ + 16, none);
  } else {
    uint32_t x2[32], x3[32];
    tmem_ld32(tS + 64, x2);
    chunk(1, sr[1]);
    tmem_wait_ld();
    reg_fence32(x2);
    tmem_ld32(tS + 96, x3);
    chunk(2, x2);
    tmem_wait_ld();
    reg_fence32(x3);
    chunk(3, x3);
  }
  float s0, s1;
  f2_unpack(f2_add(acc[0], acc[1]), s0, s1);
  l += s0 + s1;
}

// A warp's 32 query rows in fp16 into an operand tile (rows tile_row ..), 16-byte units [u0, u1) of each, times
// a power of two where they are bf16.  Returns, for row `lane`, the factor that undoes it.  Lanes stand side by
// side over a row's units, so that the loads are whole lines; row_at(r) is where row r lies, nullptr a row that
// is not there, which becomes zero.
template <int D, bool BF16, typename RowAt>
__device__ __forceinline__ float stage_query_rows(RowAt&& row_at, uint32_t tile, int tile_row, int u0, int u1) {
  constexpr int UNITS = D / 8, ROWS = 32 / UNITS;  // units a row, rows a step
  const int lane = threadIdx.x & 31, u = lane % UNITS;
  float back = 1.f;
  constexpr int BATCH = 8;  // steps whose rows are loaded together, so that their latencies overlap
#pragma unroll 1
  for (int kb = 0; kb < 32; kb += BATCH * ROWS) {
    uint4 xs[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const uint16_t* src = row_at(kb + i * ROWS + lane / UNITS);
      xs[i] = src != nullptr ? reinterpret_cast<const uint4*>(src)[u] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int k = kb + i * ROWS, r = k + lane / UNITS;
      uint4 x = xs[i];
      if constexpr (BF16) {
        uint32_t mx = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
        mx = max(mx & 0xffffu, mx >> 16);
#pragma unroll
        for (int o = 1; o < UNITS; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        // As in cache_attn.cuh: the largest value comes to lie in [2^14, 2^15).
        const int e = static_cast<int>(mx >> 7) - 127;
        const int p = mx != 0u && e < 128 ? min(14 - e, 113) : 0;
        const float mul = __int_as_float((127 + p) << 23);
        x.x = pack2<false>(unpack_lo<true>(x.x) * mul, unpack_hi<true>(x.x) * mul);
        x.y = pack2<false>(unpack_lo<true>(x.y) * mul, unpack_hi<true>(x.y) * mul);
        x.z = pack2<false>(unpack_lo<true>(x.z) * mul, unpack_hi<true>(x.z) * mul);
        x.w = pack2<false>(unpack_lo<true>(x.w) * mul, unpack_hi<true>(x.w) * mul);
        const int q = __shfl_sync(0xffffffffu, p, (lane % ROWS) * UNITS);  // of row k + lane % ROWS
        if (lane / ROWS == k / ROWS) back = __int_as_float((127 - q) << 23);
      }
      if (u >= u0 && u < u1) st_shared_v4(tile + (u >> 3) * kChunk + sw128_offset(tile_row + r, u & 7), x.x, x.y, x.z, x.w);
    }
  }
  return back;
}

// A converter warp's third of a tile's 128 tokens, in two steps: the codes into registers, which frees their slot
// for the next copy (that takes longer than the conversion), then from there to the operand tile; tokens at or past
// `valid` become zero.  A warp takes 16-code units such that neither its reads nor its two writes meet a bank twice in
// 8 lanes.
template <int D>
struct Third {
  static constexpr int ROWS = D == 128 ? 4 : 8;  // token rows a step
  static constexpr int STEPS = 128 / ROWS, MOST = (STEPS + 2) / 3, LEAST = STEPS - 2 * MOST;  // in all, and of a third
  int q, row0, chunk, steps;
  uint4 c[MOST];

  __device__ Third(int third, int lane) {
    q = lane & 3;
    const int s0 = third * MOST;
    steps = min(MOST, STEPS - s0);
    if constexpr (D == 128) {
      const int p = (lane >> 2) & 1;
      row0 = s0 * ROWS + p + 2 * (lane >> 4);
      chunk = p ^ ((lane >> 3) & 1);
    } else {
      row0 = s0 * ROWS + (lane >> 2);
      chunk = 0;
    }
  }
  __device__ __forceinline__ void load(const uint8_t* raw) {
    const uint8_t* src = raw + row0 * D + chunk * 64 + q * 16;
#pragma unroll
    for (int i = 0; i < MOST; ++i)
      if (i < LEAST || i < steps) c[i] = *reinterpret_cast<const uint4*>(src + i * ROWS * D);
  }
  // NaN codes become zero where they lie, before load(); bit i: the unit of step i had one.  (In registers, between
  // load() and store(), this took the registers that both need: 3 % of the whole.)
  __device__ __forceinline__ uint32_t drop_nan(uint8_t* raw) const {
    uint32_t bad = 0u;
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      uint4* at = reinterpret_cast<uint4*>(raw + (row0 + i * ROWS) * D + chunk * 64 + q * 16);
      if (nan_codes(*at) != 0u) {
        *at = without_nan(*at);
        bad |= 1u << i;
      }
    }
    fence_proxy_async_smem();  // the next copy comes after these writes
    return bad;
  }
  // Flags of the tokens that had one.
  __device__ __forceinline__ void mark(uint8_t* flags, uint32_t bad) const {
#pragma unroll 1
    for (int i = 0; i < steps; ++i)
      if (q == 0 && chunk == 0) flags[row0 + i * ROWS] = 0;
    __syncwarp();
#pragma unroll 1
    for (; bad != 0u; bad &= bad - 1u) flags[row0 + (__ffs(bad) - 1) * ROWS] = 1;
  }
  template <int FMT>
  __device__ __forceinline__ void store(uint32_t tile, int valid) const {
    const uint32_t dst = tile + chunk * kChunk;
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      if (i >= LEAST && i >= steps) break;
      const int row = row0 + i * ROWS;
      uint32_t o[8];
      codes_to_f16<FMT>(c[i].x, o[0], o[1]);
      codes_to_f16<FMT>(c[i].y, o[2], o[3]);
      codes_to_f16<FMT>(c[i].z, o[4], o[5]);
      codes_to_f16<FMT>(c[i].w, o[6], o[7]);
      if (row >= valid) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0u;
      }
      st_shared_v4(dst + sw128_offset(row, 2 * q), o[0], o[1], o[2], o[3]);
      st_shared_v4(dst + sw128_offset(row, 2 * q + 1), o[4], o[5], o[6], o[7]);
    }
  }
};

template <int D, int FMT, bool BF16, bool PAIR, bool TREE>
__global__ void __launch_bounds__(kThreads, 1) cache_tile_kernel(const __grid_constant__ CacheAttnArgs a) {
  using C = Cfg<D, PAIR, TREE>;
  constexpr int NS = C::NS, NR = C::NR, MR = C::MR;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sbase = smem_u32(smem_raw);
  if (!smem_base_aligned(sbase, a.err_word)) return;
  const Bars<NS, NR, MR> bars{sbase + C::OFF_BAR};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + C::OFF_MISC);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem_raw + C::OFF_MISC + 4);
  const WaitCtx wc{abort_flag, a.err_word, a.timeout_ns};
  CachePiece* pieces = reinterpret_cast<CachePiece*>(smem_raw + C::OFF_PIECE);
  volatile uint32_t* merge_flag = reinterpret_cast<volatile uint32_t*>(smem_raw + C::OFF_MISC + 8);  // [2]
  float* meta = reinterpret_cast<float*>(smem_raw + C::OFF_META);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    for (int t = 0; t < 2; ++t) {
      mbar_init(bars.q_full(t), 4);
      mbar_init(bars.stored(t), 4);
    }
    for (int b = 0; b < C::NB; ++b) {
      mbar_init(bars.s_full(b), 1);
      mbar_init(bars.p_full(b), 4);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(bars.k_full(s), 3);
      mbar_init(bars.k_empty(s), 1);
      mbar_init(bars.v_full(s), 3);
      mbar_init(bars.v_empty(s), 1);
    }
    for (int s = 0; s < NR; ++s) mbar_init(bars.raw_empty(s), 3);
    for (int i = 0; i < 2 * bars.FR; ++i) mbar_init(bars.raw_full(i & 1, i >> 1), 1);
    for (int s = 0; s < MR; ++s) mbar_init(bars.meta_full(s), 1);
    for (int s = 0; s < kPieceRing; ++s) {
      mbar_init(bars.piece_full(s), 1);
      mbar_init(bars.piece_empty(s), 15);  // 8 softmax warps, 6 converters, the MMA issuer
    }
    mbar_init(bars.join(), 8);
    mbar_init(bars.mma_done(), 1);
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // A dependent launch: what is ahead on the stream has written its results before anything is read.
  griddep_wait();
  griddep_launch_dependents();
  const int rows = a.group * a.Nq;

  // The i-th piece, where it lies in shared memory (until this warp's arrival at piece_empty); nullptr at the
  // end, or after a failed wait.
  auto next_piece = [&](int i) -> const CachePiece* {
    if (!mbar_wait_warp(bars.piece_full(i % kPieceRing), (i / kPieceRing) & 1, wc)) return nullptr;
    const CachePiece* p = pieces + i % kPieceRing;
    return p->b >= 0 ? p : nullptr;
  };
  // The least number of keys that a row of a piece's item sees.  In tiles that some row sees in part only, a NaN among
  // the values would reach rows that do not see it through their zero probabilities.  There the converters turn
  // e4m3 NaN into zero and mark the token, and the softmax makes the sums of the rows that see it NaN.
  auto least_limit = [&](const CachePiece& p) {
    return TREE ? max(0, p.len - a.Nq) : cache_row_limit(a.mask, p.len, a.Nq, p.rt * C::R / a.group);
  };
  // Whether both chains have steps in a piece, and the steps of chain t.
  auto both_chains = [&](const CachePiece& p) { return PAIR ? rows - p.rt * C::R > 128 : p.end - p.begin > 1; };
  auto chain_steps = [&](const CachePiece& p, int t) {
    const int n = p.end - p.begin;
    if (PAIR) return t == 0 || both_chains(p) ? n : 0;
    return t == 0 ? (n + 1) / 2 : n / 2;
  };

  if (warp >= 8) {
    regs_decrease<kRegsOther>();
    if (warp == 9) {
      // ------------------------------------------------------------ producer
      // In rounds of four tiles: lane 8 q + g looks after 16-token group g of the round's tile q.  Page numbers,
      // scales and copies of a tile hang on one another, so rounds run through three stages, one behind the other.
      typename C::Walk walk(a, *reinterpret_cast<typename C::Walk::Shared*>(smem_raw + C::OFF_SCHED), lane, 0, blockIdx.x,
                            gridDim.x, blockIdx.x);
      const int psh = a.c.page_shift, box = min(1 << psh, kTK);
      const int group = lane & 7;
      const bool leads = ((16 * group) & (box - 1)) == 0;
      struct Round {
        int tiles, key, page, head;  // tiles: 0 for none (the same for all lanes)
        float ks, vs;
      };
      CachePiece p{};
      int tile = 0, announced = 0, issued = 0, raws = 0, left = 3;
      bool have = false, ok = true;
      Round r0, r1, r2;
      r1.tiles = r2.tiles = 0;
      auto copy = [&](const uint8_t* codes, const Round& r, int q) -> bool {
        const int s = raws % NR;
        const uint32_t full = bars.raw_full(raws & 1, raws >> 1);
        if (!mbar_wait_warp(bars.raw_empty(s), ((raws / NR) & 1) ^ 1, wc)) return false;
        const bool mine = lane >> 3 == q && leads && r.page >= 0;
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) mbar_arrive_expect_tx(full, n * box * D);
        __syncwarp();
        if (mine) {
          const long long row = ((static_cast<long long>(r.page) * a.c.heads + r.head) << psh) + (r.key & ((1 << psh) - 1));
          bulk_load(sbase + C::OFF_RAW + s * C::RAW + group * 16 * D, codes + row * D, box * D, full);
        }
        ++raws;
        return true;
      };
      while (left > 0 && ok) {
        r0 = r1;
        r1 = r2;
#pragma unroll 1
        for (int q = 0; q < r0.tiles; ++q) {
          if (!(ok = copy(a.c.k, r0, q))) break;
          const int ms = issued++ % MR;
          if (lane >> 3 == q) {
            meta[ms * kMeta + group] = r0.ks;
            meta[ms * kMeta + 8 + group] = r0.vs;
            meta[ms * kMeta + 16 + group] = cache_log2(r0.vs);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bars.meta_full(ms));
          if (!(ok = copy(a.c.v, r0, q))) break;
        }
        if (!ok) break;
        r2.tiles = 0;
        tile += 4;
        if (left == 3 && (!have || tile >= p.end)) {
          have = walk.next(p);
          if (!have) left = 2;
          tile = p.begin;
          const int i = announced % kPieceRing;
          ok = mbar_wait_warp(bars.piece_empty(i), ((announced / kPieceRing) & 1) ^ 1, wc);
          if (!ok) break;
          ++announced;
          if (lane == 0) {
            pieces[i] = p;
            if (!have) pieces[i].b = -1;
            mbar_arrive(bars.piece_full(i));
          }
        } else if (left < 3) {
          --left;
        }
        if (have && left == 3) {
          r2.tiles = min(4, p.end - tile);
          r2.head = p.head;
          r2.key = tile * kTK + 16 * lane;
          const bool there = lane >> 3 < r2.tiles && r2.key < p.len;
          r2.page = there ? cache_page_number(a.c, p.b, r2.key) : 0x7fffffff;
          r2.ks = there ? 0.f : 1.f;
        }
        if (r1.tiles > 0) {
          const bool there = r1.ks == 0.f;
          r1.page = cache_page_checked(a.c, r1.page);
          r1.ks = r1.vs = there ? __int_as_float(0x7fffffff) : 0.f;
          if (r1.page >= 0) {
            const long long h = static_cast<long long>(r1.page) * a.c.heads + r1.head;
            r1.ks = a.c.k_scale[h];
            r1.vs = cache_v_scale(a.c, h);
          } else if (there) {
            record_page_error(a.err_word);
          }
        }
      }
      cache_empty_items<D, C::R, kTK, C::MIN_TILES>(a, blockIdx.x, gridDim.x);
      // Every copy issued must land before the block exits, also where the other roles gave up.
      if (lane == 0)
        for (int n = max(0, raws - NR); n < raws; ++n) mbar_drain(bars.raw_full(n & 1, n >> 1), bars.raw_parity(n >> 1), a.timeout_ns);
    } else if (warp == 8) {
      // ------------------------------------------------------------ MMA issuer
      // The warp stays together and one elected lane issues: what the issue takes is then the same for all
      // lanes as the compiler sees it (hence the shuffles), and needs no moves to uniform registers for each
      // product.  The chains share their code: what this warp runs between its turns has to come back into an
      // instruction cache that the softmax fills.
      constexpr uint32_t idS = idesc_f16(128, 128, false, false, false);
      constexpr uint32_t idPV = idesc_f16(128, D, false, false, true);
      constexpr uint32_t kTileLo = C::TILE >> 4;
      const uint32_t ubase = __shfl_sync(0xffffffffu, sbase, 0), utmem = __shfl_sync(0xffffffffu, tmem, 0);
      const Bars<NS, NR, MR> ub{ubase + C::OFF_BAR};
      const uint32_t q_lo = sdesc_lo(ubase + C::OFF_Q, 16), k_lo = sdesc_lo(ubase + C::OFF_K, 16),
                     v_lo = sdesc_lo(ubase + C::OFF_V, kChunk);
      constexpr int NB = C::NB;
      int ks = 0, vs = 0, sb = 0, pb = 0;                       // next slots of K and V, next buffers of S and P ...
      uint32_t kph = 0, vph = 0, pph = 0, qph = 0;         // ... and the parities of the next waits
      bool ok = true;
      const CachePiece* p;
      for (int pi = 0; ok && (p = next_piece(pi)) != nullptr; ++pi) {
        const int n = __shfl_sync(0xffffffffu, chain_steps(*p, 0) + chain_steps(*p, 1), 0);  // steps of the piece
        const bool both = __shfl_sync(0xffffffffu, both_chains(*p), 0);
        const bool shared = PAIR && both;  // a tile has two steps, one of each chain, else one
        // The query tiles: each chain's own, or halves of one from both warpgroups.  A warpgroup without rows
        // arrives too: it then has seen the last piece's products end, before any barrier moves on.
        ok = mbar_wait_warp(ub.q_full(lane & 1), qph, wc);
        qph ^= 1;
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < n + NB; ++i) {
          // Turn i: O_t += P V of step j = i - NB, then the scores of step i.  Its three waits are one: a lane each.
          const int j = i - NB, tv = both ? j & 1 : 0, tk = both ? i & 1 : 0;
          const bool pv = j >= 0, sc = i < n;
          if (!pv && !sc) continue;  // a piece of fewer steps than buffers
          const bool first_v = pv && !(shared && tv), first_k = sc && !(shared && tk);  // the slot's first reader
          const bool last_v = !shared || tv, last_k = !shared || tk;                     // and its last
          uint32_t bar = pv ? ub.p_full(pb) : ub.k_full(ks), par = pv ? pph : kph;
          if (lane == 1 && first_v) {
            bar = ub.v_full(vs);
            par = vph;
          }
          if (lane == 2 && first_k) {
            bar = ub.k_full(ks);
            par = kph;
          }
          if (!(ok = mbar_wait_warp(bar, par, wc))) break;
          tc_fence_after();
          const uint32_t o = utmem + C::TM_O + tv * C::TM_OT, pa = utmem + pb * 128, vb = v_lo + vs * kTileLo;
          const uint32_t d = utmem + sb * 128, a_lo = q_lo + (PAIR ? tk * kTileLo : 0), b_lo = k_lo + ks * kTileLo;
          if (elect_one()) {
            if (pv) {
              mma_ts_lo_rt(o, pa, vb, idPV, both ? j >> 1 : j);
#pragma unroll
              for (int k = 1; k < kTK / 16; ++k) mma_ts_lo<true>(o, pa + k * 8, vb + k * (2048 >> 4), idPV);
              if (last_v) mma_commit(ub.v_empty(vs));
            }
            if (sc) {
              mma_ss_lo<false>(d, a_lo, b_lo, idS);
#pragma unroll
              for (int k = 1; k < D / 16; ++k) {
                const uint32_t off = ((k >> 2) * kChunk + (k & 3) * 32) >> 4;
                mma_ss_lo<true>(d, a_lo + off, b_lo + off, idS);
              }
              mma_commit(ub.s_full(sb));
              if (last_k) mma_commit(ub.k_empty(ks));
            }
          }
          if (pv) {
            if (last_v && ++vs == NS) {
              vs = 0;
              vph ^= 1;
            }
            if (++pb == NB) {
              pb = 0;
              pph ^= 1;
            }
          }
          if (sc) {
            if (last_k && ++ks == NS) {
              ks = 0;
              kph ^= 1;
            }
            if (++sb == NB) sb = 0;
          }
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bars.piece_empty(pi % kPieceRing));
      }
      // Every product issued above completes before TMEM can be released.
      __syncwarp();
      if (elect_one()) {
        mma_commit(bars.mma_done());
        mbar_drain(bars.mma_done(), 0, a.timeout_ns);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ converters
      const int v = warp >= 13, third = warp - (v ? 13 : 10);
      int kt = 0;
      bool ok = true;
      Third<D> part(third, lane);
      const CachePiece* p;
      for (int pi = 0; ok && (p = next_piece(pi)) != nullptr; ++pi) {
        const int len = p->len, end = p->end, lim_min = least_limit(*p);
        const int partly = FMT == kE4M3 && v && lim_min < len ? lim_min / kTK : end;  // the first tile that some row sees in part
        int t = p->begin;
        auto convert = [&](auto drop) __attribute__((always_inline)) -> bool {  // drop: NaN among the values
          constexpr bool kDrop = decltype(drop)::value;
          const int s = kt % NS, raws = 2 * kt + v, rs = raws % NR;
          if (!mbar_wait_warp(bars.raw_full(v, kt), bars.raw_parity(kt), wc)) return false;
          uint32_t bad = 0u;
          if constexpr (kDrop) bad = part.drop_nan(smem_raw + C::OFF_RAW + rs * C::RAW);
          part.load(smem_raw + C::OFF_RAW + rs * C::RAW);
          __syncwarp();
          if (lane == 0) mbar_arrive(bars.raw_empty(rs));
          if (!mbar_wait_warp(v ? bars.v_empty(s) : bars.k_empty(s), ((kt / NS) & 1) ^ 1, wc)) return false;
          // Hidden keys' scores are set aside by the softmax; their values must be finite.
          if constexpr (kDrop) part.mark(smem_raw + C::OFF_FLAG + kt % kFlagRing * 128, bad);
          part.template store<FMT>(sbase + (v ? C::OFF_V : C::OFF_K) + s * C::TILE, len - t * kTK);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(v ? bars.v_full(s) : bars.k_full(s));
          return true;
        };
        for (; ok && t < min(partly, end); ++t, ++kt) ok = convert(std::false_type{});
        if constexpr (FMT == kE4M3)
          for (; ok && t < end; ++t, ++kt) ok = convert(std::true_type{});
        if (ok && lane == 0) mbar_arrive(bars.piece_empty(pi % kPieceRing));
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    regs_increase<kRegsSoftmax>();
    const int t = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the operand tile = TMEM lane
    const uint32_t lane_bits = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_bits /* buffer 0 */, tO = tmem + C::TM_O + t * C::TM_OT + lane_bits;
    const CacheWs ws = cache_ws(a.ws, C::R, D, a.sm_count);
    float2* stat = reinterpret_cast<float2*>(smem_raw + C::OFF_STAT);
    float* stat_ref = reinterpret_cast<float*>(smem_raw + C::OFF_STAT + 2 * 128 * 8);
    constexpr int NB = C::NB;
    int kt = 0;
    uint32_t seq = 0;                        // steps of both chains in earlier pieces
    uint32_t jc = 0, dc = 0;                 // waits of join and stored
    bool ok = true;
    const bool twice = !PAIR && rows <= 64;  // lanes 64 + r have row r as well, and the second half of each tile's keys
    const int half = twice ? quarter >> 1 : 0;
    const int ri = PAIR ? t * 128 + r : twice ? r & 63 : r;  // row of the item
    // Both softmax warpgroups meet (!PAIR), or one.  Bounded waits: after a failed one elsewhere these give up too.
    auto join = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.join());
      return mbar_wait_warp(bars.join(), jc++ & 1, wc);
    };
    auto stored = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.stored(t));
      return mbar_wait_warp(bars.stored(t), dc++ & 1, wc);
    };
    // What the key-tile loop does not need is read from the piece in shared memory again after it.
    struct Row {
      bool there;
      int tok, hq;
    };
    auto row_of = [&](const CachePiece& p) -> Row {
      const int row = p.rt * C::R + ri, rc = min(row, rows - 1), tok = rc / a.group;
      return {row < rows, tok, p.head * a.group + rc - tok * a.group};
    };
    auto out_row = [&](const CachePiece& p, const Row& w) {
      return static_cast<uint16_t*>(a.o) + p.b * a.so.b + w.hq * a.so.h + w.tok * a.so.n;
    };
    auto out_lse = [&](const CachePiece& p, const Row& w) {
      return a.lse + (static_cast<long long>(p.b) * a.c.heads * a.group + w.hq) * a.Nq + w.tok;
    };
    const CachePiece* pp;
    for (int pi = 0; ok && (pp = next_piece(pi)) != nullptr; ++pi) {
      const CachePiece& p = *pp;
      const int n = chain_steps(p, t);
      const bool both = both_chains(p);
      if (!PAIR || n > 0) {
        const int row_first = p.rt * C::R + ri - lane;  // of this warp
        const bool idle = row_first >= rows;            // a warp of rows that are not there
        float m = -INFINITY, l = 0.f, ref = -INFINITY, vf = 0.f;
        {
          // The previous piece's score products have completed: this warpgroup has seen them all end,
          // the other (!PAIR) has before the join that ended the epilogue.
          const Row w = row_of(p);
          auto row_at = [&](int k) -> const uint16_t* {
            const int row = row_first + k, tok = row / a.group;
            if (row >= rows) return nullptr;
            return static_cast<const uint16_t*>(a.q) + p.b * a.sq.b +
                   (static_cast<long long>(p.head) * a.group + row - tok * a.group) * a.sq.h + tok * a.sq.n;
          };
          const float back = stage_query_rows<D, BF16>(row_at, sbase + C::OFF_Q + (PAIR ? t * C::TILE : 0), quarter * 32,
                                                       PAIR ? 0 : t * (D / 16), PAIR ? D / 8 : (t + 1) * (D / 16));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars.q_full(t));
          const float fac = a.scale * 1.4426950408889634f * back;
          const int key_first = p.begin * kTK;
          const int lim_row = cache_row_limit(a.mask, p.len, a.Nq, w.tok) - key_first;
          const int lim_min = least_limit(p) - key_first;
          for (int j = 0; j < n; ++j) {
            const int i = PAIR ? j : 2 * j + t, nt = kt + i;  // key tile
            const uint32_t g = seq + (both ? 2 * j + t : j), b = g % NB;
            if (!(ok = mbar_wait_warp(bars.s_full(b), (g / NB) & 1, wc))) break;
            if (!(ok = mbar_wait_warp(bars.meta_full(nt % MR), (nt / MR) & 1, wc))) break;
            tc_fence_after();
            if (!idle) {
              const float* scales = meta + (nt % MR) * kMeta;
              // The chain's last product.  With two buffers that the chains share, these scores were issued after it.
              // With three, or with two and the steps of one chain only, it may still be under way: its end (and that
              // of the other chain's on the same values) frees the tile's slot.
              auto wait_pv = [&] {
                if (NB > 2 || (PAIR && !both)) {
                  const int nv = nt - (PAIR ? 1 : 2);
                  if (!mbar_wait_warp(bars.v_empty(nv % NS), (nv / NS) & 1, wc)) ok = false;
                  tc_fence_after();
                }
              };
              const bool masked = (i + 1) * kTK > lim_min;
              const int lim = lim_row - i * kTK;
              uint32_t seen[TREE ? 4 : 1];
              if constexpr (TREE) {
                if (masked) {
                  const int s0 = key_first + i * kTK + 64 * half - (p.len - a.Nq);
#pragma unroll
                  for (int c = 0; c < 4; ++c) seen[c] = tree_bits(tree_row(a, p.b, w.tok), a.tree_words, w.tok, s0 + 32 * c);
                }
              }
              if (!PAIR && twice) {
                if (masked)
                  softmax_scaled<D, true, true, TREE>(tS + b * 128, half, tO, scales + 4 * half, lim - 64 * half, seen, fac, j == 0, m, l, ref, vf, wait_pv);
                else
                  softmax_scaled<D, false, true, TREE>(tS + b * 128, half, tO, scales + 4 * half, kTK, seen, fac, j == 0, m, l, ref, vf, wait_pv);
              } else if (masked) {
                softmax_scaled<D, true, false, TREE>(tS + b * 128, 0, tO, scales, lim, seen, fac, j == 0, m, l, ref, vf, wait_pv);
              } else {
                softmax_scaled<D, false, false, TREE>(tS + b * 128, 0, tO, scales, kTK, seen, fac, j == 0, m, l, ref, vf, wait_pv);
              }
              tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.p_full(b));
            if (!ok) break;
          }
        }
        // Every product of the piece has completed once its last value tile is free.  (!PAIR: the chain that had no part
        // in that tile may find the barrier a phase behind and pass early; it goes on only once both have met below.)
        if (ok) {
          const int nv = kt + p.end - p.begin - 1;
          ok = mbar_wait_warp(bars.v_empty(nv % NS), (nv / NS) & 1, wc);
        }
        if (PAIR && !both && ok) ok = join();  // lets the other warpgroup go on, see below

        // ------------------------------------------------------------ epilogue
        float w0 = 0.f, w1 = 0.f, lse2;  // factors of O_0 and O_1 (PAIR: of O_t)
        bool use1 = false;
        if constexpr (PAIR) {
          w0 = l == 0.f ? 0.f : ex2_whole(ref - m) / l;
          lse2 = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) - kShift + __log2f(l);
        } else {
          stat[t * 128 + r] = make_float2(m, l);
          stat_ref[t * 128 + r] = ref;
          tc_fence_before();
          if (!(ok = ok && join())) break;
          use1 = both;
          // The row's statistics: of both chains, and of both halves of the keys.
          float2 x = stat[r], y = stat[128 + r], x2 = make_float2(-INFINITY, 0.f), y2 = x2;
          if (twice) {
            x2 = stat[r ^ 64];
            y2 = stat[128 + (r ^ 64)];
          }
          const float mx = fmaxf(fmaxf(x.x, y.x), fmaxf(x2.x, y2.x)), ms = mx == -INFINITY ? 0.f : mx;
          auto share = [&](float2 v) { return v.y == 0.f ? 0.f : ex2_approx(v.x - ms); };
          auto part_sum = [&](float2 v) { return v.y == 0.f ? 0.f : share(v) * v.y; };
          const float sum = part_sum(x) + part_sum(y) + (part_sum(x2) + part_sum(y2));
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          auto weight = [&](float2 v, int at) { return v.y == 0.f ? 0.f : ex2_whole(stat_ref[at] - ms) * inv; };
          w0 = weight(x, r);
          w1 = use1 ? weight(y, 128 + r) : 0.f;
          lse2 = sum == 0.f ? -INFINITY : ms - kShift + __log2f(sum);
        }
        if (!ok) break;
        tc_fence_after();
        // Rows that see a token with a NaN among its values.  Flags are written before their tile's products are issued,
        // and those have completed.  (Looked at tile by tile in the loop, 4 % of the whole.)
        if (FMT == kE4M3 && !idle) {
          const int lim_min = least_limit(p), tok = row_of(p).tok, lim_row = cache_row_limit(a.mask, p.len, a.Nq, tok);
          if (lim_min < p.len) {
#pragma unroll 1
            for (int tile = max(p.begin, lim_min / kTK); tile < p.end; ++tile) {
              const uint8_t* flags = smem_raw + C::OFF_FLAG + ((kt + tile - p.begin) % kFlagRing) * 128;
              uint32_t found = 0u;
#pragma unroll 1
              for (int c = 0; c < 128; c += 16) {
                const uint4 x = *reinterpret_cast<const uint4*>(flags + c);
                found |= x.x | x.y | x.z | x.w;
              }
              if (found == 0u) continue;
#pragma unroll 1
              for (int c = 0; c < min(lim_row - tile * kTK, 128); ++c)
                if (flags[c] && (!TREE || (tree_bits(tree_row(a, p.b, tok), a.tree_words, tok, tile * kTK + c - (p.len - a.Nq)) & 1u)))
                  w0 = w1 = lse2 = __int_as_float(0x7fffffff);
            }
          }
        }
        constexpr int COLS = PAIR ? D : D / 2;  // this thread's columns of its row
        const int c0 = PAIR ? 0 : t * COLS;
        const Row w = row_of(p);
        const int slot = p.slot;
        // A partial result lies column by column, four at a time, so that the lanes (rows) stand side by side.
        auto part_of = [&](int slot) {
          return reinterpret_cast<float4*>(ws.o) + (static_cast<size_t>(slot) * (D / 4) + c0 / 4) * C::R + ri;
        };
        const uint32_t at0 = PAIR ? tO : tmem + C::TM_O + lane_bits;
        // Two halves meet in the query tile, which is free: column by column, the rows side by side.
        float* const meet = reinterpret_cast<float*>(smem_raw + C::OFF_Q) + c0 * 64 + ri;
        if (!PAIR && twice) {
          if (half && !idle) {
#pragma unroll 1
            for (int c = 0; c < COLS; c += 16) {
              uint32_t x[16], y[16];
              tmem_ld16(at0 + c0 + c, x);
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = 0u;
              if (use1) tmem_ld16(at0 + C::TM_OT + c0 + c, y);
#pragma unroll
              for (int e = 0; e < 16; ++e) meet[(c + e) * 64] = fmaf(__uint_as_float(y[e]), w1, __uint_as_float(x[e]) * w0);
            }
          }
          if (!(ok = stored())) break;
        }
        const bool writes = !idle && half == 0;
        if (writes) {
          uint16_t* dst = out_row(p, w) + c0;
          float4* part = part_of(max(slot, 0));
#pragma unroll 1
          for (int c = 0; c < COLS; c += 16) {
            uint32_t x[16];
            tmem_ld16(at0 + c0 + c, x);
            if (!PAIR && use1) {
              uint32_t y[16];
              tmem_ld16(at0 + C::TM_OT + c0 + c, y);
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(fmaf(__uint_as_float(y[e]), w1, __uint_as_float(x[e]) * w0));
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * w0);
            }
            if (!PAIR && twice) {
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) + meet[(c + e) * 64]);
            }
            if (slot >= 0) {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                part[(c + e) / 4 * C::R] = make_float4(__uint_as_float(x[e]), __uint_as_float(x[e + 1]), __uint_as_float(x[e + 2]),
                                                       __uint_as_float(x[e + 3]));
            } else if (w.there) {
#pragma unroll
              for (int e = 0; e < 16; e += 8)
                *reinterpret_cast<uint4*>(dst + c + e) =
                    make_uint4(pack2<BF16>(__uint_as_float(x[e]), __uint_as_float(x[e + 1])),
                               pack2<BF16>(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])),
                               pack2<BF16>(__uint_as_float(x[e + 4]), __uint_as_float(x[e + 5])),
                               pack2<BF16>(__uint_as_float(x[e + 6]), __uint_as_float(x[e + 7])));
            }
          }
          if (slot >= 0)
            ws.l[(static_cast<size_t>(slot) * 2 + t) * C::R + ri] = lse2;
          else if (w.there && (PAIR || t == 0))
            *out_lse(p, w) = lse2 * 0.6931471805599453f;
        }
        tc_fence_before();

        // ------------------------------------------------------------ merge, where this piece completes its item
        // Each warpgroup for itself: it has its own rows (PAIR) or columns.  (What runs once a piece is kept short: its
        // instructions come from far each time.)
        if (slot >= 0) {
          if (!(ok = stored())) break;
          if (quarter == 0) {
            const bool all = cache_piece_done(ws, p, t, a.tag);
            if (lane == 0) merge_flag[t] = all;
          }
          if (!(ok = stored())) break;
          if (merge_flag[t] && writes) {
            // L = log2 sum 2^(L_s), O = sum 2^(L_s - L) O_s over the row's pieces in key order.
            const int np = p.pieces;
            auto lse_at = [&](int s) { return __ldcg(ws.l + (static_cast<size_t>(s) * 2 + t) * C::R + ri); };
            float mx = -INFINITY, sum = 0.f;
#pragma unroll 1
            for (int i = 0; i < np; ++i) {
              const float L = lse_at(p.slot_of(i)), to = fmaxf(mx, L), mt = to == -INFINITY ? 0.f : to;
              sum = fmaf(sum, mx == -INFINITY ? 0.f : ex2_approx(mx - mt), ex2_approx(L - mt));  // a NaN counts
              mx = to;
            }
            const float ms = mx == -INFINITY ? 0.f : mx, inv = sum == 0.f ? 0.f : 1.f / sum;
            uint16_t* dst = out_row(p, w) + c0;
            constexpr int CH = COLS < 64 ? COLS : 64;  // columns whose loads are under way together
#pragma unroll 1
            for (int c = 0; c < COLS; c += CH) {
              float4 acc[CH / 4];
#pragma unroll
              for (int e = 0; e < CH / 4; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
              for (int i = 0; i < np; ++i) {
                const int s = p.slot_of(i);
                const float4* src = part_of(s) + c / 4 * C::R;
                float4 x[CH / 4];
#pragma unroll
                for (int e = 0; e < CH / 4; ++e) x[e] = __ldcg(src + e * C::R);
                const float wi = ex2_approx(lse_at(s) - ms) * inv;
#pragma unroll
                for (int e = 0; e < CH / 4; ++e) {
                  acc[e].x = fmaf(wi, x[e].x, acc[e].x);
                  acc[e].y = fmaf(wi, x[e].y, acc[e].y);
                  acc[e].z = fmaf(wi, x[e].z, acc[e].z);
                  acc[e].w = fmaf(wi, x[e].w, acc[e].w);
                }
              }
              if (w.there) {
#pragma unroll
                for (int e = 0; e < CH / 4; e += 2)
                  *reinterpret_cast<uint4*>(dst + c + 4 * e) =
                      make_uint4(pack2<BF16>(acc[e].x, acc[e].y), pack2<BF16>(acc[e].z, acc[e].w),
                                 pack2<BF16>(acc[e + 1].x, acc[e + 1].y), pack2<BF16>(acc[e + 1].z, acc[e + 1].w));
              }
            }
            if (w.there && (PAIR || t == 0))
              *out_lse(p, w) = sum == 0.f ? -INFINITY : (ms + __log2f(sum)) * 0.6931471805599453f;
          }
        }
        // O_t, the statistics and the query tile are free once both warpgroups are here.
        if (!PAIR && !(ok = join())) break;
      } else {
        // No rows here in this piece (PAIR).  Its steps use the barriers that this warpgroup waits on next, so that it
        // must not wait for its own steps of a later piece before they have ended.
        if (lane == 0) mbar_arrive(bars.q_full(t));
        ok = join();
      }
      kt += p.end - p.begin;
      seq += chain_steps(p, 0) + chain_steps(p, 1);
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(bars.piece_empty(pi % kPieceRing));
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int FMT, bool BF16, bool PAIR, bool TREE>
cudaError_t launch_t(const CacheAttnArgs& a, cudaStream_t stream) {
  using C = Cfg<D, PAIR, TREE>;
  auto kern = cache_tile_kernel<D, FMT, BF16, PAIR, TREE>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kern, C::BYTES, done);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(a.sm_count), dim3(kThreads), C::BYTES, stream, a);
}

template <int D, int FMT, bool BF16, bool TREE>
cudaError_t launch_p(const CacheAttnArgs& a, cudaStream_t stream) {
  return static_cast<long long>(a.group) * a.Nq > 128 ? launch_t<D, FMT, BF16, true, TREE>(a, stream)
                                                     : launch_t<D, FMT, BF16, false, TREE>(a, stream);
}

template <int D, bool TREE>
cudaError_t launch_d(const CacheAttnArgs& a, cudaStream_t stream) {
  if (a.c.format == kE4M3) return a.bf16 ? launch_p<D, kE4M3, true, TREE>(a, stream) : launch_p<D, kE4M3, false, TREE>(a, stream);
  return a.bf16 ? launch_p<D, kInt8, true, TREE>(a, stream) : launch_p<D, kInt8, false, TREE>(a, stream);
}

}  // namespace
}  // namespace exattn
