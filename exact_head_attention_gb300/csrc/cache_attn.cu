// Attention over the 8-bit cache for few query rows (decoding): O = softmax(scale Q K^T) V with K and V in
// 8-bit codes and one scale for each page and head.
//
// Mathematics.  With codes k, v and the scales ks, vs of their page, a score is s = c (q . k) ks with
// c = scale * log2(e), and the online softmax keeps m >= max s - 8, l = sum 2^(s - m) and
// O = sum 2^(s - m) (vs / vref) v with vref the largest vs met so far, so that the probabilities times
// vs / vref stay below 2^15 in fp16 whatever the scales are.  The codes enter the products as they are
// (fp16 holds them exactly).  Pieces of the key axis are merged by their log-sum-exp.
//
// Bound.  With one to some tens of query rows a key/value head the time is that of reading the codes: 2 d
// bytes a token and head against 4 d rows flops.  A block (one an SM) therefore keeps up to 128 KB of
// copies in flight: warp 8 walks the block's share of the work (cache_sched.cuh), looks the pages up and
// has the copy engine fill a ring of 32-token tiles for each of the eight computing warps.  Each of these
// owns every eighth tile of a piece and its own (m, l, O), and meets the others only at the end of a
// piece, where the eight results are joined in shared memory.
//
// Products.  The tensor cores are far from busy here, so the rows go through the warp-level
// m16n8k16 product: the rows are its M (16, padded), and both the code-to-fp16 conversion and the operand
// layout happen in registers:
//   S = Q K^T: a lane reads 16-byte pieces of its key's row; which 4 d-positions form a k-step is the same
//     for Q and K, so any order serves, and no transposition is needed.
//   O = P V: the accumulator layout of S is the operand layout of P; a lane reads 16-byte (d = 128) or
//     8-byte (d = 64) pieces of the four key rows its B operand wants and pairs their bytes.
// Two 64-byte rows share a 128-byte line at d = 64; tiles are stored with the 128-byte swizzle, and the order of
// keys inside a tile (key_row) is chosen for either d so that no read of 8 lanes meets a bank twice.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache8.cuh"
#include "cache_sched.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace exattn {
namespace {

constexpr int kWarps = 8;                       // computing warps
constexpr int kThreads = 32 * (kWarps + 4);     // and a warpgroup of which one warp is the producer
// Registers: 168 a thread at launch (65,536 over 384 threads); the third warpgroup gives most of its share to
// the first two, which hold O and the codes in flight: 2 x 216 + 72 = 3 x 168.
constexpr int kComputeRegs = 216, kProducerRegs = 72;
constexpr int kTileKeys = 32;
constexpr int kPieceRing = 4;                   // pieces announced ahead
constexpr float kShift = 7.f;                   // P is held times 2^7: fewer of the small ones become subnormal

template <int D, int MT>
struct Cfg {
  static constexpr int R = 16 * MT;                           // query rows an item
  static constexpr int TILE = kTileKeys * D;                  // bytes of codes, K or V
  static constexpr int STAGES = D == 128 ? 2 : 4;             // of K and V together, a warp
  static constexpr int RING = kWarps * STAGES * 2 * TILE;     // 128 KB
  static constexpr int JOIN = kWarps * 16 * D * 4;            // one 16-row tile of O from every warp
  static constexpr int QBYTES = MT > 1 ? MT * (D / 16) * 32 * 16 : 0;
  static constexpr int OFF_JOIN = RING;
  static constexpr int OFF_Q = OFF_JOIN + JOIN;
  static constexpr int OFF_META = OFF_Q + QBYTES;             // [warp][stage] {ks0, ks1, vs0, vs1}
  static constexpr int OFF_STAT = OFF_META + kWarps * STAGES * 16;  // m[warp][R], l[warp][R], vref[warp]
  static constexpr int OFF_PIECE = OFF_STAT + (2 * kWarps * R + kWarps) * 4;
  static constexpr int OFF_BAR = (OFF_PIECE + kPieceRing * 32 + 7) & ~7;
  static constexpr int OFF_MISC = OFF_BAR + 8 * (2 * kWarps * STAGES + 2 * kPieceRing + 1);
  static constexpr int OFF_SCHED = (OFF_MISC + 16 + 7) & ~7;
  static constexpr int BYTES = OFF_SCHED + static_cast<int>(sizeof(typename CacheWalk<R, kTileKeys, kThreads, kWarps>::Shared));
  static_assert(BYTES <= 232448, "shared memory of a block");
};

// Row of the 32-token tile that stands at column n of 8-key block nb of the score product.
template <int D>
__device__ __forceinline__ constexpr int key_row(int nb, int n) {
  return D == 128 ? nb * 8 + n : 4 * (n >> 1) + (n & 1) + 2 * (nb & 1) + 16 * (nb >> 1);
}

// Shared-memory address of byte `col` of token row r in a tile.
template <int D>
__device__ __forceinline__ uint32_t tile_at(uint32_t base, int r, int col) {
  if constexpr (D == 128) return base + r * 128 + ((((col >> 4) ^ r) & 7) << 4) + (col & 15);
  const int line = r >> 1;
  return base + line * 128 + (((((r & 1) * 4 + (col >> 4)) ^ line) & 7) << 4) + (col & 15);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void tma_load_lines(uint32_t dst, const CUtensorMap* map, int line, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(line), "r"(bar)
      : "memory");
}

__device__ __forceinline__ float qnan() { return __int_as_float(0x7fffffff); }

// One query row in fp16 for a lane: 4-value groups of its d positions, times the power of two `mul`.
template <bool BF16>
__device__ __forceinline__ uint2 q_to_f16(uint2 w, float mul) {
  if constexpr (!BF16) return w;
  return make_uint2(pack2<false>(unpack_lo<true>(w.x) * mul, unpack_hi<true>(w.x) * mul),
                    pack2<false>(unpack_lo<true>(w.y) * mul, unpack_hi<true>(w.y) * mul));
}

template <int D, int FMT, bool BF16, int MT>
__global__ void __launch_bounds__(kThreads, 1) cache_attn_kernel(const __grid_constant__ CacheAttnArgs a) {
  using C = Cfg<D, MT>;
  using Walk = CacheWalk<C::R, kTileKeys, kThreads, kWarps>;
  constexpr int NST = C::STAGES, KS = D / 16, NB = D / 8;  // k-steps of S; 8-column blocks of O
  griddep_launch_dependents();  // the merge may start; it waits for this kernel before it reads
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sbase = smem_u32(smem_raw);
  if (!smem_base_aligned(sbase, a.err_word)) return;
  const uint32_t bars = sbase + C::OFF_BAR;
  auto full = [&](int w, int s) { return bars + 8 * (w * NST + s); };
  auto empty = [&](int w, int s) { return bars + 8 * (kWarps * NST + w * NST + s); };
  auto piece_full = [&](int i) { return bars + 8 * (2 * kWarps * NST + i); };
  auto piece_empty = [&](int i) { return bars + 8 * (2 * kWarps * NST + kPieceRing + i); };
  const uint32_t join_bar = bars + 8 * (2 * kWarps * NST + 2 * kPieceRing);
  float4* meta = reinterpret_cast<float4*>(smem_raw + C::OFF_META);
  int* pieces = reinterpret_cast<int*>(smem_raw + C::OFF_PIECE);  // [kPieceRing][8]
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem_raw + C::OFF_MISC);
  const WaitCtx wc{abort_flag, a.err_word, a.timeout_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    for (int i = 0; i < kWarps * NST; ++i) {
      mbar_init(bars + 8 * i, 1);
      mbar_init(bars + 8 * (kWarps * NST + i), 1);
    }
    for (int i = 0; i < kPieceRing; ++i) {
      mbar_init(piece_full(i), 1);
      mbar_init(piece_empty(i), kWarps);
    }
    mbar_init(join_bar, kWarps);
    fence_mbar_init();
    prefetch_tmap(&a.tm_k);
    prefetch_tmap(&a.tm_v);
  }
  // Ends with a barrier of the block, after which the mbarriers above are set up too.
  Walk walk(a, *reinterpret_cast<typename Walk::Shared*>(smem_raw + C::OFF_SCHED), blockIdx.x, gridDim.x);

  if (warp >= kWarps) {
    regs_decrease<kProducerRegs>();
    if (warp > kWarps) return;
    // ------------------------------------------------------------ producer: lane w feeds computing warp w
    const int psh = a.c.page_shift;
    const uint32_t ring = sbase + lane * (NST * 2 * C::TILE);
    int issued = 0;
    bool ok = true;
    CachePiece p;
    for (int i = 0; ; ++i) {
      const bool more = ok && walk.next(p);
      ok = mbar_wait_warp(piece_empty(i % kPieceRing), ((i / kPieceRing) & 1) ^ 1, wc) && ok;
      if (lane == 0) {
        int* d = pieces + (i % kPieceRing) * 8;
        d[0] = more && ok ? p.b : -1;
        d[1] = p.head;
        d[2] = p.rt;
        d[3] = p.len;
        d[4] = p.begin;
        d[5] = p.end;
        d[6] = p.slot;
        mbar_arrive(piece_full(i % kPieceRing));
      }
      if (!more || !ok) break;
      for (int base = p.begin; base < p.end; base += kWarps) {
        const int t = base + lane;
        if (lane < kWarps && t < p.end && ok) {
          const int s = issued % NST;
          const int key = t * kTileKeys;
          // The pages of the tile's two halves (the same one where a page holds 32 tokens or more).
          const int pg0 = cache_page(a.c, p.b, key);
          const bool two = psh == 4;
          const bool second = two && key + 16 < p.len;
          const int pg1 = second ? cache_page(a.c, p.b, key + 16) : pg0;
          const long long h0 = static_cast<long long>(pg0) * a.c.heads + p.head;
          const long long h1 = static_cast<long long>(pg1) * a.c.heads + p.head;
          float4 sc;
          sc.x = pg0 >= 0 ? __ldg(a.c.k_scale + h0) : qnan();
          sc.z = pg0 >= 0 ? __ldg(a.c.v_scale + h0) : qnan();
          sc.y = sc.x;
          sc.w = sc.z;
          if (two) {
            sc.y = pg1 >= 0 ? __ldg(a.c.k_scale + h1) : qnan();
            sc.w = pg1 >= 0 ? __ldg(a.c.v_scale + h1) : qnan();
          }
          if (pg0 < 0 || pg1 < 0) record_page_error(a.err_word);
          if (mbar_wait(empty(lane, s), ((issued / NST) & 1) ^ 1, wc)) {
            const uint32_t bk = ring + s * 2 * C::TILE, bv = bk + C::TILE, bar = full(lane, s);
            uint32_t bytes = 0;
            constexpr int kLineShift = D == 128 ? 0 : 1;  // tokens a 128-byte line
            if (pg0 >= 0) {
              const int line = static_cast<int>(((h0 << psh) + (key & ((1 << psh) - 1))) >> kLineShift);
              tma_load_lines(bk, &a.tm_k, line, bar);
              tma_load_lines(bv, &a.tm_v, line, bar);
              bytes += two ? C::TILE : 2 * C::TILE;
            }
            if (second && pg1 >= 0) {
              const int line = static_cast<int>((h1 << psh) >> kLineShift);
              tma_load_lines(bk + C::TILE / 2, &a.tm_k, line, bar);
              tma_load_lines(bv + C::TILE / 2, &a.tm_v, line, bar);
              bytes += C::TILE;
            }
            meta[lane * NST + s] = sc;
            mbar_arrive_expect_tx(bar, bytes);
            ++issued;
          } else {
            ok = false;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
    }
    // Every copy issued must land before the block exits, also where the computing warps gave up.
    if (lane < kWarps)
      for (int n = max(0, issued - NST); n < issued; ++n) mbar_drain(full(lane, n % NST), (n / NST) & 1, a.timeout_ns);
    return;
  }

  // -------------------------------------------------------------- computing warps
  regs_increase<kComputeRegs>();
  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t ring = sbase + warp * (NST * 2 * C::TILE);
  float* st_m = reinterpret_cast<float*>(smem_raw + C::OFF_STAT);
  float* st_l = st_m + kWarps * C::R;
  float* st_v = st_l + kWarps * C::R;
  float4* join = reinterpret_cast<float4*>(smem_raw + C::OFF_JOIN);
  const CacheWs ws = cache_ws(a.ws, a.B, C::R, D, a.sm_count);
  const int rows = a.group * a.Nq;
  int used = 0;
  bool ok = true;
  // Barrier of the computing warps.  After a failed wait a warp leaves, so this one gives up too (a
  // hardware barrier would wait for it for ever).
  uint32_t joins = 0;
  auto sync_warps = [&]() -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(join_bar);
    return mbar_wait_warp(join_bar, joins++ & 1, wc);
  };

  for (int pi = 0; ; ++pi) {
    ok = mbar_wait_warp(piece_full(pi % kPieceRing), (pi / kPieceRing) & 1, wc) && ok;
    if (!ok) break;
    const int* d = pieces + (pi % kPieceRing) * 8;
    const int b = d[0], head = d[1], rt = d[2], len = d[3], begin = d[4], end = d[5], slot = d[6];
    if (b < 0) break;
    const int row0 = rt * C::R;

    // Query rows: lane (g, t4) holds d positions [t4 D/4, (t4 + 1) D/4) of rows g and g + 8 of each 16.
    uint32_t qf[MT == 1 ? KS : 1][4];
    float fac[MT][2];  // c over the power of two in Q
    int lim[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint4 raw[2][D / 32];
      float mul[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = min(row0 + mt * 16 + h * 8 + g, rows - 1);
        const int tok = r / a.group, hg = r - tok * a.group;
        lim[mt][h] = cache_row_limit(a.mask, len, a.Nq, tok);
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(a.q) + b * a.sq.b +
            (static_cast<long long>(head) * a.group + hg) * a.sq.h + tok * a.sq.n + t4 * (D / 4));
        uint32_t mx = 0u;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          raw[h][i] = __ldg(src + i);
          if constexpr (BF16) {
            mx = __vmaxu2(mx, raw[h][i].x & 0x7fff7fffu);
            mx = __vmaxu2(mx, raw[h][i].y & 0x7fff7fffu);
            mx = __vmaxu2(mx, raw[h][i].z & 0x7fff7fffu);
            mx = __vmaxu2(mx, raw[h][i].w & 0x7fff7fffu);
          }
        }
        mul[h] = 1.f;
        float back = 1.f;
        if constexpr (BF16) {
          mx = max(mx & 0xffffu, mx >> 16);
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          // Exponent e of the largest value: times 2^(14 - e) it lies in [2^14, 2^15), and the row keeps 38
          // binades.  The factor is held to [2^-113, 2^113]; rows of zeros, NaN or infinity stay as they are.
          const int e = static_cast<int>(mx >> 7) - 127;
          if (mx != 0u && e < 128) {
            const int k = min(14 - e, 113);
            mul[h] = __int_as_float((127 + k) << 23);
            back = __int_as_float((127 - k) << 23);
          }
        }
        fac[mt][h] = a.scale * 1.4426950408889634f * back;
      }
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const uint32_t* r0 = reinterpret_cast<const uint32_t*>(&raw[0][0]) + 2 * j;
        const uint32_t* r1 = reinterpret_cast<const uint32_t*>(&raw[1][0]) + 2 * j;
        const uint2 x = q_to_f16<BF16>(make_uint2(r0[0], r0[1]), mul[0]);
        const uint2 y = q_to_f16<BF16>(make_uint2(r1[0], r1[1]), mul[1]);
        if constexpr (MT == 1) {
          qf[j][0] = x.x;
          qf[j][1] = y.x;
          qf[j][2] = x.y;
          qf[j][3] = y.y;
        } else if (warp == 0) {  // every warp holds the same: one writes them
          st_shared_v4(sbase + C::OFF_Q + ((mt * KS + j) * 32 + lane) * 16, x.x, y.x, x.y, y.y);
        }
      }
    }
    if constexpr (MT > 1) ok = sync_warps();
    const int tok0 = row0 / a.group;
    const int lim_min = cache_row_limit(a.mask, len, a.Nq, tok0);  // of the tile's first row

    float o[MT][NB][4];
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][j][e] = 0.f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
    }
    float vref = 0.f;

    for (int t = begin + warp; t < end; t += kWarps, ++used) {
      const int s = used % NST;
      if (ok) ok = mbar_wait_warp(full(warp, s), (used / NST) & 1, wc);
      if (!ok) break;
      const uint32_t bk = ring + s * 2 * C::TILE, bv = bk + C::TILE;
      const float4 sc = meta[warp * NST + s];
      const int key0 = t * kTileKeys;

      // S = Q K^T over the codes
      float sv[MT][4][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) sv[mt][nb][e] = 0.f;
#pragma unroll
      for (int c16 = 0; c16 < D / 64; ++c16) {  // 16 of the lane's d positions at a time
        uint4 kw[4];
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) kw[nb] = lds128(tile_at<D>(bk, key_row<D>(nb, g), t4 * (D / 4) + c16 * 16));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int j = c16 * 4 + w;
          uint32_t qa[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if constexpr (MT == 1) {
#pragma unroll
              for (int e = 0; e < 4; ++e) qa[mt][e] = qf[j][e];
            } else {
              const uint4 x = lds128(sbase + C::OFF_Q + ((mt * KS + j) * 32 + lane) * 16);
              qa[mt][0] = x.x;
              qa[mt][1] = x.y;
              qa[mt][2] = x.z;
              qa[mt][3] = x.w;
            }
          }
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) {
            const uint32_t word = w == 0 ? kw[nb].x : w == 1 ? kw[nb].y : w == 2 ? kw[nb].z : kw[nb].w;
            uint32_t b0, b1;
            codes_to_f16<FMT>(word, b0, b1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma16816(sv[mt][nb], qa[mt], b0, b1);
          }
        }
      }

      // Online softmax.  kf: score of a unit product, for each 16-key half of the tile.
      const bool masked = key0 + kTileKeys > lim_min;
      const float vnew = fmaxf(vref, fmaxf(sc.z, sc.w));  // a NaN scale is passed over here and met below
      bool grow = vnew > vref;
      float mnew[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float f0 = fac[mt][h] * sc.x, f1 = fac[mt][h] * sc.y;
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) {
            const float f = nb < 2 ? f0 : f1;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& x = sv[mt][nb][2 * h + e];
              x *= f;
              if (masked && key0 + key_row<D>(nb, 2 * t4 + e) >= lim[mt][h]) x = -INFINITY;
            }
          }
          float mx = sv[mt][0][2 * h];
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) mx = fmaxf(mx, fmaxf(sv[mt][nb][2 * h], sv[mt][nb][2 * h + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          mnew[mt][h] = mx;
          grow = grow || mx > m[mt][h] + 8.f;
        }
      if (__any_sync(0xffffffffu, grow)) {
        const float vr = vnew > 0.f ? vref / vnew : 1.f;
        vref = vnew;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float to = fmaxf(m[mt][h], mnew[mt][h]);
            const float al = to == -INFINITY ? 1.f : ex2_approx(m[mt][h] - to);
            m[mt][h] = to;
            l[mt][h] *= al;
            const float ov = al * vr;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              o[mt][j][2 * h] *= ov;
              o[mt][j][2 * h + 1] *= ov;
            }
          }
      }
      const float vinv = vref > 0.f ? 1.f / vref : 0.f;
      const float r0 = sc.z * vinv, r1 = sc.w * vinv;
      uint32_t pf[MT][2][4];  // operand of each 16-key half
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float ms = m[mt][h] == -INFINITY ? 0.f : m[mt][h] - kShift;
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) {
            const float r = nb < 2 ? r0 : r1;
            const float x0 = sv[mt][nb][2 * h], x1 = sv[mt][nb][2 * h + 1];
            const float p0 = ex2_approx(x0 - ms), p1 = ex2_approx(x1 - ms);
            l[mt][h] += p0 + p1;
            float y0 = p0 * r, y1 = p1 * r;
            if (masked) {  // a hidden key must not bring in a NaN scale
              y0 = x0 == -INFINITY ? 0.f : y0;
              y1 = x1 == -INFINITY ? 0.f : y1;
            }
            pf[mt][nb >> 1][(nb & 1) * 2 + h] = pack2<false>(y0, y1);
          }
        }

      // O += P V over the codes
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        constexpr int WORDS = D / 32;  // words of a lane's piece of a key row: NB values
        uint32_t vw[4][WORDS];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = key_row<D>(2 * half + (i >> 1), 2 * t4 + (i & 1));
          if constexpr (D == 128) {
            const uint4 x = lds128(tile_at<D>(bv, r, g * 16));
            vw[i][0] = x.x;
            vw[i][1] = x.y;
            vw[i][2] = x.z;
            vw[i][3] = x.w;
          } else {
            const uint2 x = lds64(tile_at<D>(bv, r, g * 8));
            vw[i][0] = x.x;
            vw[i][1] = x.y;
          }
          // Codes past the sequence's end may be anything, a NaN among them.
          if (key0 + kTileKeys > len && key0 + r >= len) {
#pragma unroll
            for (int w = 0; w < WORDS; ++w) vw[i][w] = 0u;
          }
        }
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
          uint32_t b0[4], b1[4];  // of d positions 4 w .. 4 w + 3 of the lane's piece
          codes_to_f16<FMT>(__byte_perm(vw[0][w], vw[1][w], 0x5140), b0[0], b0[1]);
          codes_to_f16<FMT>(__byte_perm(vw[0][w], vw[1][w], 0x7362), b0[2], b0[3]);
          codes_to_f16<FMT>(__byte_perm(vw[2][w], vw[3][w], 0x5140), b1[0], b1[1]);
          codes_to_f16<FMT>(__byte_perm(vw[2][w], vw[3][w], 0x7362), b1[2], b1[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma16816(o[mt][4 * w + e], pf[mt][half], b0[e], b1[e]);
        }
      }
      __syncwarp();  // every lane has read the tile
      if (lane == 0) mbar_arrive(empty(warp, s));
    }

    // ------------------------------------------------------------ join the warps' results
    const int nrows = min(C::R, rows - row0);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = l[mt][h];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (t4 == 0) {
          st_m[warp * C::R + mt * 16 + h * 8 + g] = m[mt][h];
          st_l[warp * C::R + mt * 16 + h * 8 + g] = x;
        }
      }
    if (lane == 0) {
      st_v[warp] = vref;
      mbar_arrive(piece_empty(pi % kPieceRing));
    }
    constexpr int Q4 = D / 4;       // float4s a row
    constexpr int LQ = D / 16;      // float4s of a lane's row part (dims t4 D/4 ..)
    auto place = [&](int r, int q) {  // bank-conflict-free order of a row's float4s
      const int k = D == 128 ? ((q >> 3) | ((r & 1) << 2)) : ((q >> 3) | ((r & 1) << 1));
      return r * Q4 + (q ^ k);
    };
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt * 16 >= nrows) break;  // the same for all warps
      if (begin + warp < end) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (mt * 16 + h * 8 + g < nrows) {
            float4* dst = join + warp * (16 * Q4);
#pragma unroll
            for (int q = 0; q < LQ; ++q) {
              // d position t4 D/4 + 4 q + e is column 2 t4 + (q >= LQ/2) of block 4 (q % (LQ/2)) + e
              const int col = q >= LQ / 2 ? 1 : 0, j = 4 * (q % (LQ / 2));
              dst[place(h * 8 + g, t4 * LQ + q)] = make_float4(o[mt][j][2 * h + col], o[mt][j + 1][2 * h + col],
                                                               o[mt][j + 2][2 * h + col], o[mt][j + 3][2 * h + col]);
            }
          }
        }
      }
      if (!(ok = ok && sync_warps())) break;
      const int nr = min(16, nrows - mt * 16);
      for (int i = threadIdx.x; i < nr * Q4; i += 32 * kWarps) {
        const int r = i / Q4, q = i % Q4, ri = mt * 16 + r;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, st_m[w * C::R + ri]);
        const float ms = mx == -INFINITY ? 0.f : mx;
        float lsum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float lw = st_l[w * C::R + ri];
          if (lw != 0.f) {
            const float e = ex2_approx(st_m[w * C::R + ri] - ms), ev = e * st_v[w];
            const float4 x = join[w * (16 * Q4) + place(r, q)];
            lsum = fmaf(e, lw, lsum);
            acc.x = fmaf(ev, x.x, acc.x);
            acc.y = fmaf(ev, x.y, acc.y);
            acc.z = fmaf(ev, x.z, acc.z);
            acc.w = fmaf(ev, x.w, acc.w);
          }
        }
        const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
        acc.x *= inv;
        acc.y *= inv;
        acc.z *= inv;
        acc.w *= inv;
        const float lse2 = lsum == 0.f ? -INFINITY : ms - kShift + __log2f(lsum);
        if (slot < 0) {
          const int rr = row0 + ri, tok = rr / a.group, hq = head * a.group + rr - tok * a.group;
          uint16_t* dst = static_cast<uint16_t*>(a.o) + b * a.so.b + hq * a.so.h + tok * a.so.n + q * 4;
          *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF16>(acc.x, acc.y), pack2<BF16>(acc.z, acc.w));
          if (q == 0)
            a.lse[(static_cast<long long>(b) * a.c.heads * a.group + hq) * a.Nq + tok] = lse2 * 0.6931471805599453f;
        } else {
          reinterpret_cast<float4*>(ws.o)[(static_cast<size_t>(slot) * C::R + ri) * Q4 + q] = acc;
          if (q == 0) ws.l[static_cast<size_t>(slot) * C::R + ri] = lse2;
        }
      }
      if (!(ok = sync_warps())) break;
    }
    if (!ok) break;
  }
}

// Merge of the pieces of divided items, one warp a query row, and the rows that see no token:
// L = log2 sum 2^(L_s), O = sum 2^(L_s - L) O_s over the row's pieces in key order.
template <int D, bool BF16, int R, int TK>
__global__ void __launch_bounds__(256) cache_merge_kernel(const __grid_constant__ CacheAttnArgs a) {
  griddep_wait();
  constexpr int V = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheItems<R, TK> items(a);
  const long long rid = static_cast<long long>(blockIdx.x) * 8 + warp;
  if (rid >= static_cast<long long>(a.B) * a.c.heads * items.rows) return;
  const int r = static_cast<int>(rid % items.rows);
  const long long bh = rid / items.rows;
  const int head = static_cast<int>(bh % a.c.heads), b = static_cast<int>(bh / a.c.heads);
  const int rt = r / R;
  const CacheWs ws = cache_ws(a.ws, a.B, R, D, a.sm_count);
  const int len = items.seq_len(a, b);
  const int nt = items.tiles(a, len, rt);
  const int C = ws.head->per_piece;
  long long first = 0;
  int pieces = 0;
  if (nt > 0) {
    first = ws.first[b];
    if (head > 0) first += head * items.head_units(a, len, 0);
    for (int i = 0; i < rt; ++i) first += items.tiles(a, len, i);
    pieces = ws.head->pieces ? (nt + C - 1) / C : static_cast<int>((first + nt - 1) / C - first / C) + 1;
    if (pieces == 1) return;  // written by the block that had all of it
  }
  const bool by_piece = ws.head->pieces != 0;
  auto row_of = [&](int i) {  // workspace row of piece i
    const long long start = by_piece ? first + static_cast<long long>(i) * C : (i == 0 ? first : (first / C + i) * C);
    return static_cast<size_t>(2 * (start / C) + (i != 0)) * R + (r - rt * R);
  };
  float mx = -INFINITY;
  for (int i = lane; i < pieces; i += 32) mx = fmaxf(mx, ws.l[row_of(i)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float ms = mx == -INFINITY ? 0.f : mx;
  float acc[V], sum = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  for (int i = 0; i < pieces; ++i) {
    const size_t at = row_of(i);
    const float w = ex2_approx(ws.l[at] - ms);
    if (w != 0.f) {  // a NaN counts
      const float* op = ws.o + at * D + lane * V;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = fmaf(w, op[e], acc[e]);
      sum += w;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int tok = r / a.group, hq = head * a.group + r - tok * a.group;
  uint16_t* dst = static_cast<uint16_t*>(a.o) + b * a.so.b + hq * a.so.h + tok * a.so.n + lane * V;
  if constexpr (V == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF16>(acc[0] * inv, acc[1] * inv), pack2<BF16>(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack2<BF16>(acc[0] * inv, acc[1] * inv);
  if (lane == 0)
    a.lse[(static_cast<long long>(b) * a.c.heads * a.group + hq) * a.Nq + tok] =
        sum == 0.f ? -INFINITY : (ms + __log2f(sum)) * 0.6931471805599453f;
}

template <int D, bool BF16, int R, int TK>
cudaError_t launch_merge(const CacheAttnArgs& a, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.B) * a.c.heads * a.group * a.Nq;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + 7) / 8));
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_merge_kernel<D, BF16, R, TK>, a);
}

template <int D, int FMT, bool BF16, int MT>
cudaError_t launch_t(const CacheAttnArgs& a, cudaStream_t stream) {
  using C = Cfg<D, MT>;
  auto kern = cache_attn_kernel<D, FMT, BF16, MT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
  if (e != cudaSuccess) return e;
  kern<<<a.sm_count, kThreads, C::BYTES, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_merge<D, BF16, C::R, kTileKeys>(a, stream);
}

template <int D, int FMT, bool BF16>
cudaError_t launch_m(const CacheAttnArgs& a, cudaStream_t stream) {
  return static_cast<long long>(a.group) * a.Nq <= 16 ? launch_t<D, FMT, BF16, 1>(a, stream) : launch_t<D, FMT, BF16, 2>(a, stream);
}

template <int D>
cudaError_t launch_d(const CacheAttnArgs& a, cudaStream_t stream) {
  if (a.c.format == kE4M3) return a.bf16 ? launch_m<D, kE4M3, true>(a, stream) : launch_m<D, kE4M3, false>(a, stream);
  return a.bf16 ? launch_m<D, kInt8, true>(a, stream) : launch_m<D, kInt8, false>(a, stream);
}

}  // namespace

int cache_attn_box_tokens(int page) { return page < kTileKeys ? page : kTileKeys; }

size_t cache_attn_workspace(int B, int rows, int d, int sm_count) {
  const int R = rows <= 16 ? 16 : 32;
  return cache_align256(cache_ws_first_bytes(B) + cache_slots(sm_count) * R * (static_cast<size_t>(d) + 1) * sizeof(float));
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t stream) {
  return a.c.d == 128 ? launch_d<128>(a, stream) : launch_d<64>(a, stream);
}

}  // namespace exattn
