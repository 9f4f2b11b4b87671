// How the attention over the cache divides its work, computed on the device from the lengths there.
//
// An item is one tile of query rows of one key/value head of one sequence; its keys are cut into tiles of
// TK tokens.  All tiles of all items, in the order (sequence, head, row tile, key tile), are numbered
// 0 .. T - 1 (below 2^31: the host checks the largest T that the page table allows).  With
// C = ceil(T / P) for P blocks (or workers, several to a block),
//   * in general block c takes the tiles [c C, (c + 1) C), whichever items they belong to, so every block has the
//     same work however uneven the lengths are;
//   * where the items cut into pieces of C tiles make no more pieces than there are blocks, a block takes one of
//     those, so that short items are not cut for nothing.  C is kMinTiles, twice that where it cuts no item at all (a
//     merge takes longer than kMinTiles more tiles), or 2 or 4 times that where smaller ones are too many and blocks
//     would have as many tiles in the first form.  Measured when this was chosen, five tokens on 32 sequences, 4 heads of
//     64, 20 rows each: 1024 cached tokens 16.3 us, 2048 22.0 us (16.5 and 22.3 now); with kMinTiles alone 16.8 and 26.0.
// In the first form an item also counts kItemCost tiles that are not there, before its own: what it costs to
// begin and to end a piece.  Without them a block whose share were many short sequences took 1.6 times as
// long as the average block (64 sequences spread over 1 to 8191 tokens, 8 heads).
// A piece is a run of an item's tiles in one block.  Where an item has several, each leaves a partial
// result in slot 2 (start / C) + (start != item's first tile) of the workspace, `start` being the number
// of the piece's first tile (kItemCost past the item's first number): at most one piece in each block begins an item
// that it does not finish, and at most one continues an item, so no two pieces share a slot.  In the second form the
// pieces are numbered, and that takes the place of start / C.
#pragma once

#include <cstdint>
#include <type_traits>

#include "cache8.cuh"

namespace exattn {

// Merging.  The block whose piece completes an item merges all its pieces, in key order, so the result does
// not depend on which block that is.  Each piece, once stored, adds one to its item's count, in the first
// slot's word; the one that brings it to the number of pieces merges, and sets the word back to zero.  The
// workspace needs no preparation: a word counts from nothing unless its upper 48 bits are a tag drawn for the call,
// and a captured call, whose tag is the same at each replay, finds zeros.

// Workspace: counts, then the slots (R rows of D values in fp32, normalised by the piece's own sum, in an order
// that each kernel chooses) and their base-2 log-sum-exps.  Counts and log-sum-exps are kept twice, for the two warpgroups of cache_tile.cuh.
struct CacheWs {
  unsigned long long* count;  // [slots][2]
  float* o;                   // [slots][R * D]
  float* l;                   // [slots][2][R]
};

// Slots are numbered below 2 (T / C + 1) <= 2 (P + 1), T with the items' costs, or below 2 P.
inline __host__ __device__ size_t cache_slots(int sm_count) { return 2 * (static_cast<size_t>(sm_count) + 1); }

inline __host__ __device__ size_t cache_ws_bytes(int R, int D, int sm_count) {
  return cache_slots(sm_count) * (16 + static_cast<size_t>(R) * (D + 2) * sizeof(float));
}

inline __host__ __device__ CacheWs cache_ws(uint8_t* ws, int R, int D, int sm_count) {
  CacheWs w;
  w.count = reinterpret_cast<unsigned long long*>(ws);
  w.o = reinterpret_cast<float*>(ws + cache_slots(sm_count) * 16);
  w.l = w.o + cache_slots(sm_count) * R * D;
  return w;
}

// Beginning and ending a piece takes about as long as 768 of its tokens (256, 384 and 768 were tried).
constexpr __host__ __device__ int cache_item_cost(int TK) { return 768 / TK; }

// Number of keys that token i of Nq queries sees in a sequence of `len` tokens.
__device__ __forceinline__ int cache_row_limit(int mask, int len, int Nq, int i) {
  if (mask == ATTN_MASK_NONE) return len;
  if (mask == ATTN_MASK_CAUSAL) return min(len, i + 1);
  return max(0, len - Nq + i + 1);
}

// A tree's rows.  Token i of the Nq at a sequence's end sees what is before them, and of them those j <= i whose bit is set:
// a part of what it sees under the bottom-right mask, which divides the work.
constexpr int kTreeMost = ATTN_TREE_MAX_TOKENS;
__device__ __forceinline__ const uint32_t* tree_row(const CacheAttnArgs& a, int b, int i) {
  return a.tree + b * a.tree_stride + static_cast<long long>(i) * a.tree_words;
}
// The n lowest bits, n from below 0 to above 32.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : n > 0 ? (1u << n) - 1u : 0u; }
// The 32 tokens of the tree from s on (below 0: what is before it) that token i sees, `row` its words.
__device__ __forceinline__ uint32_t tree_bits(const uint32_t* row, int words, int i, int s) {
  if (s <= -32) return ~0u;
  if (s > i) return 0u;
  const int w = s >> 5;  // -1 to words - 1
  const uint32_t lo = w < 0 ? ~0u : row[w], hi = w + 1 < words ? row[w + 1] : 0u;
  return __funnelshift_r(lo, hi, s & 31) & low_bits(i - s + 1);
}

// R query rows an item, TK keys a tile.
template <int R, int TK, int kMinTiles>
struct CacheItems {
  static constexpr int kItemCost = cache_item_cost(TK);
  int rows, row_tiles;
  __device__ explicit CacheItems(const CacheAttnArgs& a) : rows(a.group * a.Nq), row_tiles((a.group * a.Nq + R - 1) / R) {}

  __device__ int tiles(const CacheAttnArgs& a, int len, int rt) const {
    // the item's last row sees the most; the last item ends with the last token
    const int tok = rt + 1 == row_tiles ? a.Nq - 1 : ((rt + 1) * R - 1) / a.group;
    return (cache_row_limit(a.mask, len, a.Nq, tok) + TK - 1) / TK;
  }
  __device__ static int cost(int tiles) { return tiles > 0 ? tiles + kItemCost : 0; }
  __device__ static int cut(int tiles, int shift) { return (tiles + (1 << shift) - 1) >> shift; }
  // Tiles of one head of a sequence with the items' costs, and its pieces of at most 2^shift tiles.
  __device__ void head_units(const CacheAttnArgs& a, int len, int shift, int& ntiles, int& npieces) const {
    ntiles = npieces = 0;
#pragma unroll 1
    for (int rt = 0; rt < row_tiles; ++rt) {
      const int t = tiles(a, len, rt);
      ntiles += cost(t);
      npieces += cut(t, shift);
    }
  }
  __device__ int seq_len(const CacheAttnArgs& a, int b) const { return cache_len(a.c, a.lens[b]); }
};

// A piece of an item for one worker, as the producer announces it.
struct CachePiece {
  int b, head, rt, len;  // b < 0: there are no more
  int begin, end;        // key tiles of the item
  int slot;              // -1: the whole item, else its place in the workspace
  int bucket, pieces;    // first / C of the item's first tile, or the number of its first piece; and its pieces

  __device__ int slot_of(int i) const { return 2 * (bucket + i) + (i != 0); }  // of the item's i-th piece
};
constexpr int kPieceInts = 12;  // room for one

// Called by a warp (all lanes) after the block's worker, or the warpgroup `part`, has stored its piece and met:
// counts the piece; true where every piece of the item has been, and the count is at rest again.  The other pieces'
// partial results are then visible to lane 0, and to other threads once they have met it at a barrier.
__device__ __forceinline__ bool cache_piece_done(const CacheWs& ws, const CachePiece& p, int part, unsigned long long tag) {
  bool all = false;
  if ((threadIdx.x & 31) == 0) {
    unsigned long long* at = ws.count + 2 * p.slot_of(0) + part;
    const unsigned long long n = static_cast<unsigned long long>(p.pieces);
    unsigned long long seen, old;
    // release: the partial result before the count; acquire: the others' partial results after it, for this lane
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(seen) : "l"(at) : "memory");
    for (;;) {
      if ((seen & ~0xffffull) == tag) {  // nobody puts it to rest before this piece is counted
        asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], %2;" : "=l"(old) : "l"(at), "l"(1ull) : "memory");
        all = (old & 0xffffull) + 1ull == n;
        if (all) asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(at), "l"(0ull) : "memory");
        break;
      }
      asm volatile("atom.acq_rel.gpu.global.cas.b64 %0, [%1], %2, %3;" : "=l"(old) : "l"(at), "l"(seen), "l"(tag | 1ull) : "memory");
      if (old == seen) break;  // the first of several
      seen = old;
    }
  }
  return __shfl_sync(0xffffffffu, all, 0);
}
// The division, and a block's walk over its pieces.  Built by NT threads of a block (numbered `tid`, whole
// warps that meet at hardware barrier `bar`), then walked by each of their warps, all lanes alike.
// A third form, for trees over many query rows (WHOLE): no item is divided, and so nothing is stored, counted and merged.  Where
// there are more items than blocks they go, longest sequences first, to the blocks in turn, there and back (block c has the
// c-th, the (2 P - 1 - c)-th, the (2 P + c)-th ...).  It is taken where the block with the most has no more than kWholeSlack
// tiles, items' costs counted, above what the other forms give each: dividing items costs about as much.  Measured, divided
// against whole, 8 heads of 128:
//   16 sequences of 4096 tokens, 96 rows  71.5 : 61.4 us;  of 2048, 256 rows  62.2 : 45.3 us;  of 4096, 256 rows  86.2 : 75.3 us
//   32 sequences spread over 1 to 4065 tokens, 256 rows  111.4 : 89.2 us
// and where the rule does not take it, 40 sequences of 2048 tokens, 4 heads, 64 rows (20 tiles above)  59.2 : 69.4 us, 8 of
// 2088, 4 heads, 256 rows (18 above)  38.5 : 47.2 us.
// Of no more than kWholeMost sequences: every block puts them in order by itself, in the square of their number.  64 against 256
// at most: 100 sequences of 2048 tokens, 4 heads, 64 rows 117.6 : 130.1 us; 250 of 512, 4 heads, 64 rows 129 : 208 us; 128 spread
// over 1 to 2063, 8 heads, 256 rows 273 : 256 us.
// (attn_fwd_cache keeps the first two forms, and with them the bits of its results.)
constexpr int kWholeMost = 64;   // sequences
constexpr int kWholeTurns = 8;   // items a block
constexpr int kWholeSlack = 15;  // tiles
template <int NT>
struct CacheWalkShared {  // first tile and first unit of each of the NT runs that the sequences are summed in
  int tiles[NT + 1], units[NT + 1], warp_sums[NT / 32][5];
};
struct CacheWholeShared : CacheWalkShared<32> {  // and the sequences by length
  uint8_t order[kWholeMost];
};
template <int R, int TK, int NT, int kMinTiles, bool WHOLE = false>
struct CacheWalk {
  using Shared = std::conditional_t<WHOLE, CacheWholeShared, CacheWalkShared<NT>>;
  const CacheAttnArgs& a;
  Shared& sh;
  CacheItems<R, TK, kMinTiles> items;
  int at, stop, step;  // first form: tile numbers; second: piece numbers
  int C, shift, per;   // C: 2^shift by pieces; per: sequences a run
  bool by_piece, placed = false;
  bool whole = false, sorted = false;  // third form
  int turn = 0, block, blocks, per_seq = 1;
  float per_seq_inverse = 1.f;
  // place of the next tile (first form)
  int b = 0, head = 0, rt = 0, len = 0, tile = 0, ntiles = 0, item_first = 0;

  // spread: this block's (or worker's) number where pieces are dealt out one each: the first ones then are on an SM each
  // (16 sequences of 448 tokens, 8 heads of 128, 16 rows: 13.4 us with neighbours on an SM, 11.2; in the first form, whose
  // blocks share items with their neighbours, 28.2 and 28.7 for 4032)
  __device__ CacheWalk(const CacheAttnArgs& args, Shared& s, int tid, int bar, int block_, int blocks_, int spread)
      : a(args), sh(s), items(args), block(block_), blocks(blocks_) {
    per = (a.B + NT - 1) / NT;
    const int b0 = static_cast<int>(min(static_cast<long long>(a.B), static_cast<long long>(tid) * per));
    const int b1 = min(a.B - b0, per) + b0;
    constexpr int kLog = kMinTiles == 2 ? 1 : kMinTiles == 4 ? 2 : 3;
    static_assert(1 << kLog == kMinTiles, "a power of two");
    int n[4] = {0, 0, 0, 0}, count = 0;  // tiles; pieces of 1, 2 and 4 kMinTiles; items
    int longest = 0;                     // WHOLE: the most tiles of an item, with its cost
    for (int i = b0; i < b1; ++i) {
      const int raw = a.lens[i], l = cache_len(a.c, raw);
      if (raw != l && block == 0) record_page_error(a.err_word);
#pragma unroll 1
      for (int r = 0; r < items.row_tiles; ++r) {
        const int t = items.tiles(a, l, r);
        n[0] += a.c.heads * items.cost(t);
#pragma unroll
        for (int k = 0; k < 3; ++k) n[1 + k] += a.c.heads * items.cut(t, kLog + k);
        count += t > 0 ? a.c.heads : 0;
        if constexpr (WHOLE) longest = max(longest, items.cost(t));
      }
    }
    // inclusive sums over the warp, then over the warps
    const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int u = __shfl_up_sync(0xffffffffu, n[k], o);
        if (lane >= o) n[k] += u;
      }
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 31) {
#pragma unroll
      for (int k = 0; k < 4; ++k) sh.warp_sums[warp][k] = n[k];
      sh.warp_sums[warp][4] = count;
    }
    sync(bar);
    int sum[5] = {0, 0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
#pragma unroll
      for (int k = 0; k < 5; ++k) {
        const int s = sh.warp_sums[w][k];
        if (k < 4 && w < warp) n[k] += s;
        sum[k] += s;
      }
    }
    const int total = sum[0], even = (total - 1) / blocks + 1;
    int k = -1;
    if (sum[2] == sum[4] && sum[2] <= blocks) k = 1;
    else if (sum[1] <= blocks) k = 0;
    else if (sum[2] <= blocks && 2 * kMinTiles <= even) k = 1;
    else if (sum[3] <= blocks && 4 * kMinTiles <= even) k = 2;
    by_piece = k >= 0;
    shift = kLog + max(k, 0);
    C = by_piece ? 1 << shift : even;
    const int pieces = k == 0 ? sum[1] : k == 1 ? sum[2] : sum[3];
    sh.tiles[tid + 1] = n[0];
    sh.units[tid + 1] = k < 0 ? n[0] : k == 0 ? n[1] : k == 1 ? n[2] : n[3];
    if (tid == 0) sh.tiles[0] = sh.units[0] = 0;
    sync(bar);
    if (by_piece) {
      at = spread;
      stop = pieces;
      step = blocks;
    } else {
      at = block * C;
      stop = total - at > C ? at + C : total;
      step = 0;
    }
    if constexpr (WHOLE) {
      static_assert(NT == 32 && kWholeMost <= 256, "one warp, and a byte a sequence");
      const long long n = static_cast<long long>(a.B) * a.c.heads * items.row_tiles;
      per_seq = a.c.heads * items.row_tiles;
      per_seq_inverse = 1.f / static_cast<float>(per_seq);
      if (n <= blocks) {  // an item a block: in any order
        whole = __reduce_max_sync(0xffffffffu, longest) <= C + kWholeSlack;
      } else if (a.B <= kWholeMost && n <= kWholeTurns * blocks) {
        sorted = true;
        // A sequence's place among all, the lengths by shuffles.  (Loops are kept as such: what runs once comes from far, and
        // unrolled this took 4 us of a call instead of 1.)
#pragma unroll 1
        for (int g = tid; g - tid < a.B; g += 32) {
          const int own = g < a.B ? items.seq_len(a, g) : -1;
          int rank = 0;
#pragma unroll 1
          for (int h = tid; h - tid < a.B; h += 32) {
            const int others = h < a.B ? items.seq_len(a, h) : -1;
#pragma unroll 1
            for (int j = 0; j < 32; ++j) {
              const int other = __shfl_sync(0xffffffffu, others, j);
              rank += other > own || (other == own && h - tid + j < g);
            }
          }
          if (g < a.B) sh.order[rank] = static_cast<uint8_t>(g);
        }
        __syncwarp();
        // A bound of all blocks' tiles.  The items of a turn get shorter with the block's number there and longer on the way
        // back (each counted as its sequence's longest), so that no block from c0 to c1 has more than the sum of c0's there and
        // c1's back.  (32 blocks by themselves missed the last, which alone have a second item where those are few more than
        // blocks: 39 sequences of 8192 tokens, 4 heads, 64 rows 189.6 us for 129.4; all blocks cost 1 us a call.)
        const int c0 = (blocks - 1) * tid / (NT - 1), c1 = (blocks - 1) * min(tid + 1, NT - 1) / (NT - 1);
        int worst = 0;
#pragma unroll 1
        for (int k = 0; k < kWholeTurns; ++k) {
          const int i = whole_item(k, k & 1 ? c1 : c0);
          if (i < n) worst += items.cost(whole_tiles(whole_rank(i), items.row_tiles - 1));
        }
        whole = __reduce_max_sync(0xffffffffu, worst) <= C + kWholeSlack;
      }
    }
  }
  // The third form's items: number k of block c, in the order of length, there and back; the place of item i's sequence (items
  // are few, and the quotient exact); and the tiles of one of a sequence's items (row tile `rt`).
  __device__ int whole_item(int k, int c) const { return k & 1 ? (k + 1) * blocks - 1 - c : k * blocks + c; }
  __device__ int whole_rank(int i) const { return static_cast<int>((static_cast<float>(i) + 0.5f) * per_seq_inverse); }
  __device__ int whole_tiles(int rank, int rt) const { return items.tiles(a, items.seq_len(a, whole_seq(rank)), rt); }
  __device__ int whole_seq(int rank) const { return sorted ? sh.order[rank] : rank; }
  __device__ bool next_whole(CachePiece& p) {
    int i, rank;
    do {
      i = whole_item(turn++, block);
      if (i >= a.B * per_seq) return false;
      rank = whole_rank(i);
      const int rest = i - rank * per_seq;
      p.head = items.row_tiles == 1 ? rest : rest / items.row_tiles;
      p.rt = rest - p.head * items.row_tiles;
      p.end = whole_tiles(rank, p.rt);
    } while (p.end == 0);
    p.b = whole_seq(rank);
    p.len = items.seq_len(a, p.b);
    p.begin = 0;
    p.slot = -1;
    p.bucket = 0;
    p.pieces = 1;
    return true;
  }

  __device__ static void sync(int bar) {
    if constexpr (NT > 32) named_bar_sync(bar, NT); else __syncwarp();
  }

  // Finds unit x: sets b, len, head, rt and item_first, and returns the unit's number inside its item.
  __device__ int locate(int x) {
    // the run: the last whose first unit is at most x
    int run = -1;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) run += __popc(__ballot_sync(0xffffffffu, sh.units[i * 32 + (threadIdx.x & 31)] <= x));
    x -= sh.units[run];
    item_first = sh.tiles[run];
    int ht, hp, hu;
    for (b = run * per;; ++b) {
      len = items.seq_len(a, b);
      items.head_units(a, len, shift, ht, hp);
      hu = by_piece ? hp : ht;
      if (x < hu * a.c.heads) break;
      x -= hu * a.c.heads;
      item_first += a.c.heads * ht;
    }
    head = x / hu;
    x -= head * hu;
    item_first += head * ht;
    for (rt = 0;; ++rt) {
      ntiles = items.tiles(a, len, rt);
      const int u = by_piece ? items.cut(ntiles, shift) : items.cost(ntiles);
      if (x < u) break;
      x -= u;
      item_first += items.cost(ntiles);
    }
    return x;
  }

  __device__ bool next(CachePiece& p) {
    if constexpr (WHOLE) {
      if (whole) return next_whole(p);
    }
    int first_piece = 0;  // the number of the item's first
    for (;;) {
      if (at >= stop) return false;
      int x;  // unit of the item at which the piece begins
      if (by_piece || !placed) {
        x = locate(at);
        placed = true;
      } else {  // the item after the last one, passing those without tiles
        item_first += items.cost(ntiles);
        x = 0;
        do {
          if (++rt == items.row_tiles) {
            rt = 0;
            if (++head == a.c.heads) {
              head = 0;
              ++b;
              len = items.seq_len(a, b);
            }
          }
          ntiles = items.tiles(a, len, rt);
        } while (ntiles == 0);
      }
      if (by_piece) {
        tile = x << shift;
        p.end = min(ntiles, tile + C);
        first_piece = at - x;
        at += step;
      } else {
        const int y = min(items.cost(ntiles), x + (stop - at));
        at += y - x;
        if (y <= items.kItemCost) continue;  // nothing but the item's cost
        tile = max(0, x - items.kItemCost);
        p.end = y - items.kItemCost;
      }
      break;
    }
    p.b = b;
    p.head = head;
    p.rt = rt;
    p.len = len;
    p.begin = tile;
    const int first = item_first + items.kItemCost;
    p.bucket = by_piece ? first_piece : first / C;
    p.pieces = by_piece ? items.cut(ntiles, shift) : (first + ntiles - 1) / C - p.bucket + 1;
    p.slot = p.pieces == 1 ? -1 : p.slot_of(by_piece ? tile / C : (first + tile) / C - p.bucket);
    return true;
  }
};

// O = 0 and LSE = -inf for the rows of items without a key tile (sequences without tokens, and queries before
// the first token), the items dealt out to all `warps` of the grid.
template <int D, int R, int TK, int kMinTiles>
__device__ void cache_empty_items(const CacheAttnArgs& a, int warp, int warps) {
  const CacheItems<R, TK, kMinTiles> items(a);
  const int lane = threadIdx.x & 31, n = a.B * a.c.heads * items.row_tiles;  // below 2^31: the host has counted tiles
  for (int i = warp; i < n; i += warps) {
    const int rt = i % items.row_tiles, bh = i / items.row_tiles, head = bh % a.c.heads, b = bh / a.c.heads;
    if (items.tiles(a, items.seq_len(a, b), rt) != 0) continue;
    for (int r = rt * R; r < min(items.rows, (rt + 1) * R); ++r) {
      const int tok = r / a.group, hq = head * a.group + r - tok * a.group;
      if (lane < D / 8)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + b * a.so.b + hq * a.so.h + tok * a.so.n + lane * 8) =
            make_uint4(0u, 0u, 0u, 0u);
      if (lane == 0) a.lse[(static_cast<long long>(b) * a.c.heads * a.group + hq) * a.Nq + tok] = -INFINITY;
    }
  }
}

}  // namespace exattn
