// Attention over the 8-bit cache for few query rows (decoding): O = softmax(scale Q K^T) V with K and V in
// 8-bit codes and one scale for each page and head.
//
// Mathematics.  With codes k, v and the scales ks, vs of their page, a score is s = c (q . k) ks with
// c = scale * log2(e), and the online softmax keeps m >= max s - 8, l = sum 2^(s - m) and
// O = sum 2^(s - w) vs v with w >= max(s + log2 vs) - 12 (cache8.cuh), so that what stands before v stays below 2^15 in
// fp16 whatever the scales are.  The codes enter the products as they are (fp16 holds them exactly).  Pieces of the key
// axis are merged by their log-sum-exp.
//   A row's w is m + kappa.  As long as all value scales that a warp meets lie within [vref, 16 vref], vref half the
// least of its first tile or less, kappa is log2 vref for every row, which satisfies w's bounds without a look at the
// scores.  From the first tile on where one does not, the warp keeps a kappa for each row in shared memory and looks for
// the maxima of s + log2 vs, a path of its own.  (One path, with a kappa in registers for each row, took 27.3 us for five
// tokens on 32 ragged sequences, which take 26.3; a reference over the scales alone, whatever the rows see of them, 25.8.
// With every 7th page's scale 100 times the others' these five tokens take 36 us, one token over 32k the same 125.)
//
// Bound.  With one to some tens of query rows a key/value head the time is that of reading the codes: 2 d
// bytes a token and head against 4 d rows flops.  A block (one an SM) therefore keeps 128 to 192 KB of copies
// under way.  It holds two workers, each with its own share of the work (cache_sched.cuh): two producer warps walk
// it, look the pages up and have the copy engine fill, for each of the worker's four computing warps, a ring of two or
// three tiles of 4 KB of keys and 4 KB of values.  A computing warp owns every fourth tile of a piece and its own
// (m, l, O), and meets the others only at the end of a piece, where their results are joined in shared memory.
//
// Measured on GB300: 12 heads of 128, one token over 32k cached tokens of 8 sequences (805 MB of codes) in 124 us,
// 96 % of the measured copy rate; 64 sequences of 1 to 8191 tokens, 8 heads of 128 with 8 query heads each, pages of 16,
// in 102 us (79 %; the uneven end of the blocks' shares, and a copy for each 16 tokens).  From 162 us for the first:
// four producer warps instead of one, 142 (one took 190 cycles for each 4 KB box, and they arrive every 175); 32-bit
// arithmetic and one pass in the division of the work, 130; the query rows copied ahead with each piece, 128; two
// workers, 124.  A call over one short sequence takes 6.5 us, 20 rows instead of 8 add 3 us and a division of the keys
// 6 us: code that runs once a piece comes from far, and is kept short.
//
// Products.  The tensor cores are far from busy here, so the work goes through the warp-level m16n8k16
// product with keys (for the scores) and d positions (for O) as its M and query rows as its N, eight at a
// time: a head without a group wastes the least that way.  Conversion to fp16 and operand layout both
// happen in registers:
//   S^T = K Q^T: a lane reads 16-byte pieces of its keys' rows; which d positions form a k-step is the same for
//     Q and K, so any order serves, and no transposition is needed.
//   O^T = V^T P^T: a lane reads 16-byte (d = 128) or 8-byte (d = 64) pieces of the four key rows that its
//     operand wants and pairs their bytes; P^T is S^T's accumulator with its 8 x 8 blocks transposed
//     between the lanes (movmatrix).
// Two 64-byte rows share a 128-byte line at d = 64; tiles are stored with the 128-byte swizzle, and the order of
// keys inside a tile (key_row) is chosen for either d so that no read of 8 lanes meets a bank twice.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache8.cuh"
#include "cache_sched.cuh"
#include "cache.h"
#include "ptx.cuh"

namespace exattn {
namespace {

// P is held times 2^kShift, so that fewer of the small ones become subnormal in fp16.  With the value scales it stays below
// 2^15: s - m may be 8, and vs / vref 2^4.
constexpr float kShift = 3.f;

constexpr int kWorkers = 2;                     // of a block: each with its own share of the work
constexpr int kGroup = 4;                       // computing warps of a worker
constexpr int W = kWorkers * kGroup;
constexpr int kThreads = 32 * (W + 4);          // and a warpgroup of producers, two warps a worker
// Registers: 168 a thread at launch (65,536 over 384 threads); the producers give a part of their share to the
// computing warps, which hold O, Q and the codes in flight: 2 x 208 + 88 = 3 x 168.
constexpr int kComputeRegs = 208, kProducerRegs = 88;
static_assert(2 * kComputeRegs + kProducerRegs == 3 * 168, "register split must match the launch");
constexpr int kMinTiles = 2 * kGroup;           // the smallest piece: two tiles a warp

// NT: query rows in eights.
template <int D, int NT>
struct Cfg {
  static constexpr int R = 8 * NT;                            // query rows an item
  static constexpr int TK = 4096 / D;                         // tokens a tile: 32 or 64
  static constexpr int NH = TK / 16;                          // 16-token groups of it, each in one page
  static constexpr int TILE = TK * D;                         // bytes of codes, K or V
  static constexpr int STAGES = NT == 1 ? 3 : 2;              // of K and V together, a warp
  static constexpr int RING = W * STAGES * 2 * TILE;          // 192 or 128 KB
  // Rows joined at a time, a power of two: all of them where shared memory has the room.
  static constexpr int JR = D == 64 ? (NT == 3 ? 32 : R) : NT == 1 ? 4 : NT == 2 ? R : 8;
  static constexpr int JOIN = kGroup * JR * D * 4;            // a worker
  static constexpr bool Q_IN_SMEM = NT > 2;                   // registers hold Q up to 16 rows
  static constexpr int QBYTES = Q_IN_SMEM ? NT * (D / 16) * 32 * 8 : 0;
  static constexpr int RINGQ = 2;                             // pieces announced ahead
  static constexpr int QROWS = R * D * 2;                     // the rows of one piece as they lie in memory
  static constexpr int STAT = 3 * kGroup * R * 4;        // m, l, kappa [R][warp]
  using Walk = CacheWalk<R, TK, 64, kMinTiles>;
  // a worker's part of shared memory
  static constexpr int W_JOIN = 0;
  static constexpr int W_QROWS = W_JOIN + JOIN;
  static constexpr int W_Q = W_QROWS + RINGQ * QROWS;
  static constexpr int W_STAT = W_Q + QBYTES;
  static constexpr int W_PIECE = W_STAT + STAT;
  static constexpr int W_SCHED = W_PIECE + RINGQ * kPieceInts * 4;
  static constexpr int WORKER = (W_SCHED + static_cast<int>(sizeof(typename Walk::Shared)) + 15) & ~15;
  static constexpr int OFF_WORKER = RING;
  static constexpr int OFF_META = OFF_WORKER + kWorkers * WORKER;  // [warp][stage][group] {ks, vs}
  static constexpr int OFF_BAR = OFF_META + W * STAGES * NH * 8;
  static constexpr int OFF_MISC = OFF_BAR + 8 * (2 * W * STAGES + kWorkers * (2 * RINGQ + 1));
  static constexpr int BYTES = OFF_MISC + 16;
  static_assert(BYTES <= 232448, "shared memory of a block");
};

// Row of the tile that stands at place n of its 8-key block nb in the products.
template <int D>
__device__ __forceinline__ constexpr int key_row(int nb, int n) {
  return D == 128 ? nb * 8 + n : 4 * (n >> 1) + (n & 1) + 2 * (nb & 1) + 16 * (nb >> 1);
}

// Offset of byte `col` of token row r in a tile.
template <int D>
__device__ __forceinline__ int tile_at(int r, int col) {
  if constexpr (D == 128) return r * 128 + ((((col >> 4) ^ r) & 7) << 4) + (col & 15);
  const int line = r >> 1;
  return line * 128 + (((((r & 1) * 4 + (col >> 4)) ^ line) & 7) << 4) + (col & 15);
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 block of 16-bit values held by the warp (lane 4 i + j: row i, columns 2 j and 2 j + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void tma_load_lines(uint32_t dst, const CUtensorMap* map, int line, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(line), "r"(bar)
      : "memory");
}

// log2 of a power of two.
__device__ __forceinline__ float exponent_of(float x) { return static_cast<float>((__float_as_int(x) >> 23) - 127); }

__device__ __forceinline__ float qnan() { return __int_as_float(0x7fffffff); }

template <int D, int FMT, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, 1) cache_attn_kernel(const __grid_constant__ CacheAttnArgs a) {
  using C = Cfg<D, NT>;
  constexpr int NST = C::STAGES, NH = C::NH, RQ = C::RINGQ;
  constexpr int KS = D / 16, MT = D / 16;  // k-steps of S^T; 16-row tiles of O^T
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sbase = smem_u32(smem_raw);
  if (!smem_base_aligned(sbase, a.err_word)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = warp < W ? warp / kGroup : (warp - W) / 2;
  uint8_t* wmem = smem_raw + C::OFF_WORKER + worker * C::WORKER;
  const uint32_t bars = sbase + C::OFF_BAR, wbars = bars + 8 * (2 * W * NST + worker * (2 * RQ + 1));
  auto full = [&](int w, int s) { return bars + 8 * (w * NST + s); };
  auto empty = [&](int w, int s) { return bars + 8 * (W * NST + w * NST + s); };
  auto piece_full = [&](int i) { return wbars + 8 * i; };
  auto piece_empty = [&](int i) { return wbars + 8 * (RQ + i); };
  const uint32_t join_bar = wbars + 8 * (2 * RQ);
  float2* meta = reinterpret_cast<float2*>(smem_raw + C::OFF_META);
  CachePiece* pieces = reinterpret_cast<CachePiece*>(wmem + C::W_PIECE);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem_raw + C::OFF_MISC);
  volatile uint32_t* merge_flag = reinterpret_cast<volatile uint32_t*>(smem_raw + C::OFF_MISC + 4 + 4 * worker);
  const WaitCtx wc{abort_flag, a.err_word, a.timeout_ns};

  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    for (int i = 0; i < W * NST; ++i) {
      mbar_init(bars + 8 * i, NH);
      mbar_init(bars + 8 * (W * NST + i), 1);
    }
    for (int k = 0; k < kWorkers; ++k) {
      const uint32_t at = bars + 8 * (2 * W * NST + k * (2 * RQ + 1));
      for (int i = 0; i < RQ; ++i) {
        mbar_init(at + 8 * i, 1);
        mbar_init(at + 8 * (RQ + i), kGroup);
      }
      mbar_init(at + 8 * (2 * RQ), kGroup);
    }
    fence_mbar_init();
    prefetch_tmap(&a.tm_k);
    prefetch_tmap(&a.tm_v);
  }
  __syncthreads();
  // A dependent launch: what is ahead on the stream has written its results before anything is read.
  griddep_wait();
  griddep_launch_dependents();

  if (warp >= W) {
    regs_decrease<kProducerRegs>();
    // ------------------------------------------------------------ producers
    // Producer p of a worker feeds its computing warps 2 p and 2 p + 1, with one lane for each 16-token group of
    // their tiles.  (One warp that copied for a whole block took 190 cycles for each 4 KB box, more than the 175 in
    // which they arrive at the memory's rate.)
    // A warp works in rounds of one tile a computing warp.  A group's page number, then its scales and codes
    // hang on one another, so the rounds run through three stages, one behind the other: the pages of
    // one are loaded while the scales of the round before are, and the codes of the one before that copied.
    const int pw = (warp - W) & 1;
    typename C::Walk walk(a, *reinterpret_cast<typename C::Walk::Shared*>(wmem + C::W_SCHED), pw * 32 + lane, 1 + worker,
                          blockIdx.x * kWorkers + worker, gridDim.x * kWorkers);
    const int psh = a.c.page_shift;
    const bool feeds = lane < 2 * NH;
    const int gw = feeds ? 2 * pw + lane / NH : 0;  // the computing warp in its worker
    const int cw = worker * kGroup + gw;
    const int group = lane % NH;
    const int box = min(1 << psh, C::TK);              // tokens a copy
    const bool leads = ((16 * group) & (box - 1)) == 0;  // this lane's copy takes the groups behind it along
    const uint32_t ring = sbase + cw * (NST * 2 * C::TILE);
    constexpr int kNoTile = -2;  // as `page`: no tile here; -1: not a page, or behind the sequence's end
    struct Round {
      int key, page, head;
      float ks, vs;
    };
    CachePiece p{};
    int base = 0, announced = 0, issued = 0, left = 3;  // left: 3, then rounds until the last is through
    bool have = false, ok = true;
    Round r0, r1, r2;
    r1.page = r2.page = kNoTile;
    while (left > 0) {
      r0 = r1;
      r1 = r2;
      // Third stage: this round's copies, and the bytes that its barrier waits for.
      if (r0.page != kNoTile) {
        const int s = issued % NST;
        if (mbar_wait(empty(cw, s), ((issued / NST) & 1) ^ 1, wc)) {
          const uint32_t bar = full(cw, s);
          uint32_t bytes = 0;
          if (leads && r0.page >= 0) {
            const long long at = ((static_cast<long long>(r0.page) * a.c.heads + r0.head) << psh) + (r0.key & ((1 << psh) - 1));
            const int line = static_cast<int>(at >> (D == 128 ? 0 : 1));  // two tokens a 128-byte line at d = 64
            const uint32_t bk = ring + s * 2 * C::TILE + group * 16 * D;
            tma_load_lines(bk, &a.tm_k, line, bar);
            tma_load_lines(bk + C::TILE, &a.tm_v, line, bar);
            bytes = 2 * box * D;
          }
          meta[(cw * NST + s) * NH + group] = make_float2(r0.ks, r0.vs);
          mbar_arrive_expect_tx(bar, bytes);
          ++issued;
        } else {
          ok = false;
        }
      }
      // First stage: the next round, its piece announced where it is new, and its page numbers.
      r2.page = kNoTile;
      base += kGroup;
      if (left == 3 && (!have || base >= p.end)) {
        have = ok && walk.next(p);
        if (!have) left = 2;
        base = p.begin;
        if (pw == 0) {
          const int i = announced++ % RQ;
          ok = mbar_wait_warp(piece_empty(i), (((announced - 1) / RQ) & 1) ^ 1, wc) && ok;
          const int nrows = have && ok ? min(C::R, a.group * a.Nq - p.rt * C::R) : 0;
          if (lane == 0) {
            pieces[i] = p;
            if (!have) pieces[i].b = -1;
            mbar_arrive_expect_tx(piece_full(i), nrows * D * 2);
          }
          if (lane < nrows) {
            const int r = p.rt * C::R + lane, tok = r / a.group, hg = r - tok * a.group;
            bulk_load(smem_u32(wmem) + C::W_QROWS + i * C::QROWS + lane * D * 2,
                      static_cast<const uint16_t*>(a.q) + p.b * a.sq.b +
                          (static_cast<long long>(p.head) * a.group + hg) * a.sq.h + tok * a.sq.n,
                      D * 2, piece_full(i));
          }
        }
      } else if (left < 3) {
        --left;
      }
      if (have && feeds && base + gw < p.end) {
        r2.head = p.head;
        r2.key = (base + gw) * C::TK + 16 * group;
        r2.page = r2.key < p.len ? cache_page_number(a.c, p.b, r2.key) : 0x7fffffff;  // no entry there
        r2.ks = r2.key < p.len ? 0.f : 1.f;
      }
      // Second stage: the scales.
      if (r1.page != kNoTile) {
        const bool there = r1.ks == 0.f;
        r1.page = cache_page_checked(a.c, r1.page);
        r1.ks = there ? qnan() : 0.f;
        r1.vs = qnan();  // behind the sequence's end: not counted among the scales that the tile has
        if (r1.page >= 0) {
          const long long h = static_cast<long long>(r1.page) * a.c.heads + r1.head;
          r1.ks = a.c.k_scale[h];
          r1.vs = cache_v_scale(a.c, h);
        } else if (there) {
          record_page_error(a.err_word);
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
    }
    cache_empty_items<D, C::R, C::TK, kMinTiles>(a, blockIdx.x * 4 + warp - W, gridDim.x * 4);
    // Every copy issued must land before the block exits, also where the computing warps gave up.
    if (feeds)
      for (int n = max(0, issued - NST); n < issued; ++n) mbar_drain(full(cw, n % NST), (n / NST) & 1, a.timeout_ns);
    if (pw == 0)
      for (int n = max(0, announced - RQ); n < announced; ++n) mbar_drain(piece_full(n % RQ), (n / RQ) & 1, a.timeout_ns);
    return;
  }

  // -------------------------------------------------------------- computing warps
  regs_increase<kComputeRegs>();
  const int gw = warp % kGroup, tid = threadIdx.x % (32 * kGroup);  // in the worker
  const int g = lane >> 2, t4 = lane & 3;
  uint8_t* ring = smem_raw + warp * (NST * 2 * C::TILE);
  float* st_m = reinterpret_cast<float*>(wmem + C::W_STAT);
  float* st_l = st_m + kGroup * C::R;
  float* st_k = st_l + kGroup * C::R;
  float4* join = reinterpret_cast<float4*>(wmem + C::W_JOIN);
  uint2* qs = reinterpret_cast<uint2*>(wmem + C::W_Q);
  const CacheWs ws = cache_ws(a.ws, C::R, D, a.sm_count * kWorkers);
  const int rows = a.group * a.Nq;
  int used = 0;
  bool ok = true;
  // Barrier of the worker's computing warps.  After a failed wait a warp leaves, so this one gives up too (a
  // hardware barrier would wait for it for ever).
  uint32_t joins = 0;
  auto sync_warps = [&]() -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(join_bar);
    return mbar_wait_warp(join_bar, joins++ & 1, wc);
  };

  for (int pi = 0; ; ++pi) {
    ok = mbar_wait_warp(piece_full(pi % RQ), (pi / RQ) & 1, wc) && ok;
    if (!ok) break;
    const CachePiece piece = pieces[pi % RQ];
    const int b = piece.b, head = piece.head, rt = piece.rt, len = piece.len, begin = piece.begin, end = piece.end,
              slot = piece.slot;
    if (b < 0) break;
    const int row0 = rt * C::R;

    // Query rows: lane (g, t4) holds d positions [t4 D/4, (t4 + 1) D/4) of row g of each eight.
    uint2 qf[C::Q_IN_SMEM ? 1 : NT][KS];
    float fac[NT][2];  // c over the power of two in Q, of the rows 2 t4 and 2 t4 + 1
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + nt * 8 + g;
      const uint4* src = reinterpret_cast<const uint4*>(wmem + C::W_QROWS + (pi % RQ) * C::QROWS +
                                                        (nt * 8 + g) * D * 2 + t4 * (D / 2));
      uint4 raw[D / 32];
      uint32_t mx = 0u;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) raw[i] = r < rows ? src[i] : make_uint4(0u, 0u, 0u, 0u);
      float mul = 1.f, back = 1.f;
      if constexpr (BF16) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          mx = __vmaxu2(mx, raw[i].x & 0x7fff7fffu);
          mx = __vmaxu2(mx, raw[i].y & 0x7fff7fffu);
          mx = __vmaxu2(mx, raw[i].z & 0x7fff7fffu);
          mx = __vmaxu2(mx, raw[i].w & 0x7fff7fffu);
        }
        mx = max(mx & 0xffffu, mx >> 16);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // Exponent e of the largest value: times 2^(14 - e) it lies in [2^14, 2^15), and the row keeps 38
        // binades.  The factor is held to [2^-113, 2^113]; rows of zeros, NaN or infinity stay as they are.
        const int e = static_cast<int>(mx >> 7) - 127;
        if (mx != 0u && e < 128) {
          const int k = min(14 - e, 113);
          mul = __int_as_float((127 + k) << 23);
          back = __int_as_float((127 - k) << 23);
        }
      }
      const float f = a.scale * 1.4426950408889634f * back;
      const int lm = cache_row_limit(a.mask, len, a.Nq, min(r, rows - 1) / a.group);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        fac[nt][e] = __shfl_sync(0xffffffffu, f, (2 * t4 + e) * 4);
        lim[nt][e] = __shfl_sync(0xffffffffu, lm, (2 * t4 + e) * 4);
      }
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(raw) + 2 * j;
        uint2 x = make_uint2(w[0], w[1]);
        if constexpr (BF16)
          x = make_uint2(pack2<false>(unpack_lo<true>(w[0]) * mul, unpack_hi<true>(w[0]) * mul),
                         pack2<false>(unpack_lo<true>(w[1]) * mul, unpack_hi<true>(w[1]) * mul));
        if constexpr (!C::Q_IN_SMEM)
          qf[nt][j] = x;
        else if (gw == 0)  // every warp holds the same: one writes them
          qs[(nt * KS + j) * 32 + lane] = x;
      }
    }
    if constexpr (C::Q_IN_SMEM) ok = sync_warps();
    const int lim_min = cache_row_limit(a.mask, len, a.Nq, row0 / a.group);  // of the item's first row

    float o[NT][MT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
    float vref = 0.f, vinv = 0.f;  // powers of two, until `uneven`
    bool uneven = false;           // the rows' kappa are in st_k

    for (int t = begin + gw; t < end; t += kGroup, ++used) {
      const int s = used % NST;
      if (ok) ok = mbar_wait_warp(full(warp, s), (used / NST) & 1, wc);
      if (!ok) break;
      const uint8_t *bk = ring + s * 2 * C::TILE, *bv = bk + C::TILE;
      float2 sc[NH];
#pragma unroll
      for (int i = 0; i < NH; ++i) sc[i] = meta[(warp * NST + s) * NH + i];
      const int key0 = t * C::TK;

      // S^T = K Q^T over the codes.  sv[i][nt][2 h + e]: key place g of block 2 i + h, row 2 t4 + e.
      float sv[NH][NT][4];
#pragma unroll
      for (int i = 0; i < NH; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sv[i][nt][e] = 0.f;
#pragma unroll
      for (int c16 = 0; c16 < D / 64; ++c16) {  // 16 of the lane's d positions at a time
        uint4 kw[2 * NH];
#pragma unroll
        for (int nb = 0; nb < 2 * NH; ++nb)
          kw[nb] = *reinterpret_cast<const uint4*>(bk + tile_at<D>(key_row<D>(nb, g), t4 * (D / 4) + c16 * 16));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int j = c16 * 4 + w;
          uint2 qb[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (C::Q_IN_SMEM) qb[nt] = qs[(nt * KS + j) * 32 + lane]; else qb[nt] = qf[nt][j];
          }
#pragma unroll
          for (int i = 0; i < NH; ++i) {
            const uint4 &x = kw[2 * i], &y = kw[2 * i + 1];
            uint32_t a0, a1, a2, a3;
            codes_to_f16<FMT>(w == 0 ? x.x : w == 1 ? x.y : w == 2 ? x.z : x.w, a0, a2);
            codes_to_f16<FMT>(w == 0 ? y.x : w == 1 ? y.y : w == 2 ? y.z : y.w, a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(sv[i][nt], a0, a1, a2, a3, qb[nt].x, qb[nt].y);
          }
        }
      }

      // Online softmax; group i of the tile has one page and so one scale of each kind.  The maximum is looked for only
      // where a score passes the running one by more than 2^8: until then it may lag.
      const bool masked = key0 + C::TK > lim_min;
      float vmin = sc[0].y, vmax = sc[0].y;  // a NaN scale is passed over here and met below
#pragma unroll
      for (int i = 1; i < NH; ++i) {
        vmin = fminf(vmin, sc[i].y);
        vmax = fmaxf(vmax, sc[i].y);
      }
      if (t == begin + gw) {
        const int e = max((__float_as_int(vmin) & 0x7f800000) - 0x00800000, 0);
        vref = __int_as_float(e);
        vinv = __int_as_float(0x7f000000 - e);
      }
      uneven = uneven || !(vref > 0.f) || vmin < vref || vmax > 16.f * vref;
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < NH; ++i) {
            const float f = fac[nt][e] * sc[i].x;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float& x = sv[i][nt][2 * h + e];
              x *= f;
              if (masked && key0 + key_row<D>(2 * i + h, g) >= lim[nt][e]) x = -INFINITY;
              grow = grow || x > m[nt][e] + 8.f;
            }
          }
      uint32_t pb[NT][2 * NH];  // P^T operand of each 8-key block
      if (!uneven) {
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float to = m[nt][e];
#pragma unroll
              for (int i = 0; i < NH; ++i) to = fmaxf(to, fmaxf(sv[i][nt][e], sv[i][nt][2 + e]));
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, x));
              const float al = to == -INFINITY ? 1.f : ex2_approx(m[nt][e] - to);
              m[nt][e] = to;
              l[nt][e] *= al;
#pragma unroll
              for (int j = 0; j < MT; ++j) {
                o[nt][j][e] *= al;
                o[nt][j][2 + e] *= al;
              }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float ms0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0] - kShift;
          const float ms1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1] - kShift;
          uint64_t l2 = f2_pack(l[nt][0], l[nt][1]);
#pragma unroll
          for (int nb = 0; nb < 2 * NH; ++nb) {
            const float r = sc[nb >> 1].y * vinv;
            const float x0 = sv[nb >> 1][nt][2 * (nb & 1)], x1 = sv[nb >> 1][nt][2 * (nb & 1) + 1];
            const uint64_t p2 = f2_pack(ex2_approx(x0 - ms0), ex2_approx(x1 - ms1));
            l2 = f2_add(l2, p2);
            float y0, y1;
            f2_unpack(f2_mul(p2, f2_pack(r, r)), y0, y1);
            if (masked) {  // a hidden key must not bring in a NaN scale
              y0 = x0 == -INFINITY ? 0.f : y0;
              y1 = x1 == -INFINITY ? 0.f : y1;
            }
            pb[nt][nb] = transpose8(pack2<false>(y0, y1));
          }
          f2_unpack(l2, l[nt][0], l[nt][1]);
        }
      } else {
        // Scales far apart: each row for itself, the maxima looked for in every tile.
        const bool first = vref >= 0.f;  // of these tiles; kappa was log2 vref, of no meaning where no key has been seen
        const float even = exponent_of(vref);
        vref = -1.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float vf[2], ms[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float* const kappa = st_k + (nt * 8 + 2 * t4 + e) * kGroup + gw;
            const float was = m[nt][e], k0 = first ? even : *kappa;
            float to = was;
#pragma unroll
            for (int i = 0; i < NH; ++i) to = fmaxf(to, fmaxf(sv[i][nt][e], sv[i][nt][2 + e]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, x));
            // kappa = max(s + log2 vs) - m over all keys; never below the last one's, as w goes
            const bool seen = was > -INFINITY, some = to > -INFINITY;
            const float fall = seen ? was - to : 0.f;
            float k = seen ? k0 + fall : -kValueFloor;
#pragma unroll
            for (int i = 0; i < NH; ++i)
              k = fmaxf(k, fmaxf(sv[i][nt][e], sv[i][nt][2 + e]) - to + cache_log2(sc[i].y));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) k = fmaxf(k, __shfl_xor_sync(0xffffffffu, k, x));
            k = fmaxf(k, -kValueFloor);
            const float ov = seen ? ex2_approx(fall + k0 - k) : 1.f;
            l[nt][e] *= seen ? ex2_approx(fall) : 1.f;
            m[nt][e] = to;
            ms[e] = some ? to - kShift : 0.f;
            vf[e] = ex2_whole(-k);
            __syncwarp();
            if (g == 0) *kappa = k;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              o[nt][j][e] *= ov;
              o[nt][j][2 + e] *= ov;
            }
          }
#pragma unroll
          for (int nb = 0; nb < 2 * NH; ++nb) {
            const float x0 = sv[nb >> 1][nt][2 * (nb & 1)], x1 = sv[nb >> 1][nt][2 * (nb & 1) + 1];
            const float p0 = ex2_approx(x0 - ms[0]), p1 = ex2_approx(x1 - ms[1]);
            l[nt][0] += p0;
            l[nt][1] += p1;
            const float y0 = p0 * value_weight(sc[nb >> 1].y, vf[0]), y1 = p1 * value_weight(sc[nb >> 1].y, vf[1]);
            pb[nt][nb] = transpose8(pack2<false>(x0 == -INFINITY ? 0.f : y0, x1 == -INFINITY ? 0.f : y1));
          }
        }
        __syncwarp();
      }

      // A NaN among the values of a token that some row does not see would reach that row through its zero
      // probability: such codes become zero, and the sums of the rows that see the token NaN.
      if (FMT == kE4M3 && masked && lim_min < len) {
        uint32_t found = 0u;
#pragma unroll
        for (int i = 0; i < C::TILE / 512; ++i) found |= nan_codes(reinterpret_cast<const uint4*>(bv)[i * 32 + lane]);
        if (__any_sync(0xffffffffu, found != 0u)) {
#pragma unroll 1
          for (int r = 0; r < C::TK; r += 32) {
            bool bad = false;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint4* at = reinterpret_cast<uint4*>(ring + s * 2 * C::TILE + C::TILE + tile_at<D>(r + lane, c));
              bad = bad || nan_codes(*at) != 0u;
              *at = without_nan(*at);
            }
            const uint32_t tokens = __ballot_sync(0xffffffffu, bad);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int seen = lim[nt][e] - key0 - r;
                if (seen > 0 && (tokens & (seen >= 32 ? ~0u : (1u << seen) - 1u)) != 0u) l[nt][e] = __int_as_float(0x7fffffff);
              }
          }
          __syncwarp();
          fence_proxy_async_smem();  // the next copy into the slot comes after these writes
        }
      }

      // O^T += V^T P^T over the codes
#pragma unroll
      for (int half = 0; half < NH; ++half) {
        constexpr int WORDS = D / 32;  // words of a lane's piece of a key row
        uint32_t vw[4][WORDS];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = key_row<D>(2 * half + (i >> 1), 2 * t4 + (i & 1));
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(bv + tile_at<D>(r, g * 16));
            vw[i][0] = x.x;
            vw[i][1] = x.y;
            vw[i][2] = x.z;
            vw[i][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(bv + tile_at<D>(r, g * 8));
            vw[i][0] = x.x;
            vw[i][1] = x.y;
          }
        }
        if (key0 + C::TK > len) {  // codes past the sequence's end may be anything, a NaN among them
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key0 + key_row<D>(2 * half + (i >> 1), 2 * t4 + (i & 1)) >= len) {
#pragma unroll
              for (int w = 0; w < WORDS; ++w) vw[i][w] = 0u;
            }
        }
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
          uint32_t x[4], y[4];  // d positions 4 w .. 4 w + 3 of the lane's piece; first and second pair of keys
          codes_to_f16<FMT>(__byte_perm(vw[0][w], vw[1][w], 0x5140), x[0], x[1]);
          codes_to_f16<FMT>(__byte_perm(vw[0][w], vw[1][w], 0x7362), x[2], x[3]);
          codes_to_f16<FMT>(__byte_perm(vw[2][w], vw[3][w], 0x5140), y[0], y[1]);
          codes_to_f16<FMT>(__byte_perm(vw[2][w], vw[3][w], 0x7362), y[2], y[3]);
#pragma unroll
          for (int h = 0; h < 2; ++h)  // tile rows g and g + 8: d positions 2 j and 2 j + 1 of the piece
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816(o[nt][2 * w + h], x[2 * h], x[2 * h + 1], y[2 * h], y[2 * h + 1], pb[nt][2 * half], pb[nt][2 * half + 1]);
        }
      }
      __syncwarp();  // every lane has read the tile
      if (lane == 0) mbar_arrive(empty(warp, s));
    }

    // ------------------------------------------------------------ join the warps' results
    const int nrows = min(C::R, rows - row0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
        if (g == 0) {
          st_m[(nt * 8 + 2 * t4 + e) * kGroup + gw] = m[nt][e];
          st_l[(nt * 8 + 2 * t4 + e) * kGroup + gw] = x;
          if (!uneven) st_k[(nt * 8 + 2 * t4 + e) * kGroup + gw] = exponent_of(vref);
        }
      }
    if (lane == 0) mbar_arrive(piece_empty(pi % RQ));
    constexpr int Q4 = D / 4;   // float4s a row
    constexpr int LQ = D / 32;  // float4s of a lane's part of a row (d positions g D/8 ..)
    auto place = [&](int r, int q) {  // order of a row's float4s in which 8 lanes never meet a bank twice
      const int t = (r >> 1) & 3;
      return (r & (C::JR - 1)) * Q4 + (q ^ (D == 128 ? t : (t & 1) | ((t & 2) << 1)));
    };
    for (int base = 0; base < nrows; base += C::JR) {  // the same for all warps
      if (begin + gw < end) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = nt * 8 + 2 * t4 + e;
            if (r >= base && r < min(nrows, base + C::JR)) {
#pragma unroll
              for (int q = 0; q < LQ; ++q)
                join[gw * (C::JR * Q4) + place(r, g * LQ + q)] =
                    make_float4(o[nt][2 * q][e], o[nt][2 * q][2 + e], o[nt][2 * q + 1][e], o[nt][2 * q + 1][2 + e]);
            }
          }
      }
      if (!(ok = ok && sync_warps())) break;
      const int nr = min(C::JR, nrows - base);
      for (int i = tid; i < nr * Q4; i += 32 * kGroup) {
        const int ri = base + i / Q4, q = i % Q4;
        const float4 sm4 = *reinterpret_cast<const float4*>(st_m + ri * kGroup), sl4 = *reinterpret_cast<const float4*>(st_l + ri * kGroup),
                     sk4 = *reinterpret_cast<const float4*>(st_k + ri * kGroup);
        const float sm[kGroup] = {sm4.x, sm4.y, sm4.z, sm4.w}, sl[kGroup] = {sl4.x, sl4.y, sl4.z, sl4.w},
                    sk[kGroup] = {sk4.x, sk4.y, sk4.z, sk4.w};
        const float mx = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
        const float ms = mx == -INFINITY ? 0.f : mx;
        float lsum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kGroup; ++w) {
          if (sl[w] != 0.f) {
            const float e = ex2_approx(sm[w] - ms), ev = ex2_whole(sm[w] - ms + sk[w]);
            const float4 x = join[w * (C::JR * Q4) + place(ri, q)];
            lsum = fmaf(e, sl[w], lsum);
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
          if (q == 0) ws.l[static_cast<size_t>(slot) * 2 * C::R + ri] = lse2;
        }
      }
      if (!(ok = sync_warps())) break;
    }
    if (!ok) break;

    // ------------------------------------------------------------ merge, where this piece completes its item
    if (slot >= 0) {
      if (gw == 0) {
        const bool all = cache_piece_done(ws, piece, 0, a.tag);
        if (lane == 0) *merge_flag = all;
      }
      if (!(ok = sync_warps())) break;
      if (*merge_flag) {
        // L = log2 sum 2^(L_s), O = sum 2^(L_s - L) O_s over the row's pieces.  Where threads are left over, G of them
        // share a row's four columns, each with every G-th piece, and join in shared memory.
        const int n = piece.pieces, cells = nrows * Q4;
        const int G = max(1, min(n, 32 * kGroup / cells));
        float4* m_acc = join;
        float2* m_stat = reinterpret_cast<float2*>(join + 32 * kGroup);
        static_assert(C::JOIN >= 32 * kGroup * 24, "room for the shares");
        for (int i = tid; i < cells * G; i += 32 * kGroup) {
          const int cell = i % cells, g0 = i / cells, ri = cell / Q4, q = cell % Q4;
          float mx = -INFINITY, sum = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int k = g0; k < n; k += G) {
            const size_t at = static_cast<size_t>(piece.slot_of(k));
            const float L = __ldcg(ws.l + at * 2 * C::R + ri);
            const float4 x = __ldcg(reinterpret_cast<const float4*>(ws.o) + (at * C::R + ri) * Q4 + q);
            const float to = fmaxf(mx, L), mt = to == -INFINITY ? 0.f : to;
            const float e0 = mx == -INFINITY ? 0.f : ex2_approx(mx - mt), e1 = ex2_approx(L - mt);  // a NaN counts
            mx = to;
            sum = fmaf(sum, e0, e1);
            acc.x = fmaf(acc.x, e0, e1 * x.x);
            acc.y = fmaf(acc.y, e0, e1 * x.y);
            acc.z = fmaf(acc.z, e0, e1 * x.z);
            acc.w = fmaf(acc.w, e0, e1 * x.w);
          }
          auto finish = [&]() {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int rr = row0 + ri, tok = rr / a.group, hq = head * a.group + rr - tok * a.group;
            uint16_t* dst = static_cast<uint16_t*>(a.o) + b * a.so.b + hq * a.so.h + tok * a.so.n + q * 4;
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
            if (q == 0)
              a.lse[(static_cast<long long>(b) * a.c.heads * a.group + hq) * a.Nq + tok] =
                  sum == 0.f ? -INFINITY : ((mx == -INFINITY ? 0.f : mx) + __log2f(sum)) * 0.6931471805599453f;
          };
          if (G == 1) {
            finish();
          } else {  // cells * G threads at most: one turn of the loop
            m_acc[i] = acc;
            m_stat[i] = make_float2(mx, sum);
          }
        }
        if (G > 1) {
          if (!(ok = sync_warps())) break;
          for (int cell = tid; cell < cells; cell += 32 * kGroup) {
            const int ri = cell / Q4, q = cell % Q4;
            float mx = -INFINITY;
            for (int k = 0; k < G; ++k) mx = fmaxf(mx, m_stat[k * cells + cell].x);
            const float ms = mx == -INFINITY ? 0.f : mx;
            float sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < G; ++k) {
              const float2 st = m_stat[k * cells + cell];
              if (st.y == 0.f) continue;
              const float4 x = m_acc[k * cells + cell];
              const float e = ex2_approx(st.x - ms);
              sum = fmaf(e, st.y, sum);
              acc.x = fmaf(e, x.x, acc.x);
              acc.y = fmaf(e, x.y, acc.y);
              acc.z = fmaf(e, x.z, acc.z);
              acc.w = fmaf(e, x.w, acc.w);
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int rr = row0 + ri, tok = rr / a.group, hq = head * a.group + rr - tok * a.group;
            uint16_t* dst = static_cast<uint16_t*>(a.o) + b * a.so.b + hq * a.so.h + tok * a.so.n + q * 4;
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
            if (q == 0)
              a.lse[(static_cast<long long>(b) * a.c.heads * a.group + hq) * a.Nq + tok] =
                  sum == 0.f ? -INFINITY : (ms + __log2f(sum)) * 0.6931471805599453f;
          }
        }
        if (!(ok = sync_warps())) break;  // `join` is free again
      }
    }
  }
}

template <int D, int FMT, bool BF16, int NT>
cudaError_t launch_t(const CacheAttnArgs& a, cudaStream_t stream) {
  using C = Cfg<D, NT>;
  auto kern = cache_attn_kernel<D, FMT, BF16, NT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kern, C::BYTES, done);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(a.sm_count), dim3(kThreads), C::BYTES, stream, a);
}

template <int D, int FMT, bool BF16>
cudaError_t launch_m(const CacheAttnArgs& a, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.group) * a.Nq;
  if (rows <= 8) return launch_t<D, FMT, BF16, 1>(a, stream);
  if (rows <= 16) return launch_t<D, FMT, BF16, 2>(a, stream);
  static_assert(kCacheStreamRows == 24, "the variants of launch_m");
  return launch_t<D, FMT, BF16, 3>(a, stream);
}

template <int D>
cudaError_t launch_d(const CacheAttnArgs& a, cudaStream_t stream) {
  if (a.c.format == kE4M3) return a.bf16 ? launch_m<D, kE4M3, true>(a, stream) : launch_m<D, kE4M3, false>(a, stream);
  return a.bf16 ? launch_m<D, kInt8, true>(a, stream) : launch_m<D, kInt8, false>(a, stream);
}

}  // namespace

int cache_attn_box_tokens(int page, int d) { return page < 4096 / d ? page : 4096 / d; }

CacheAttnShape cache_attn_shape(long long rows, int d) {
  if (rows > kCacheStreamRows) return {rows > 128 ? 256 : 128, 128};
  return {static_cast<int>((rows + 7) / 8 * 8), 4096 / d};
}

size_t cache_attn_workspace(long long rows, int d, int sm_count) {
  const int workers = rows > kCacheStreamRows ? sm_count : sm_count * kWorkers;
  return (cache_ws_bytes(cache_attn_shape(rows, d).rows, d, workers) + 255) & ~static_cast<size_t>(255);
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t stream) {
  if (static_cast<long long>(a.group) * a.Nq > kCacheStreamRows) return launch_cache_tile(a, stream);
  return a.c.d == 128 ? launch_d<128>(a, stream) : launch_d<64>(a, stream);
}

}  // namespace exattn
