// How the attention over the cache divides its work, computed on the device from the lengths there.
//
// An item is one tile of query rows of one key/value head of one sequence; its keys are cut into tiles of
// TK tokens.  All tiles of all items, in the order (sequence, head, row tile, key tile), are numbered
// 0 .. T - 1.  With C = ceil(T / P) for P blocks,
//   * more than kMinTiles tiles a block: block c takes the tiles [c C, (c + 1) C), whichever items they
//     belong to, so every block has the same work however uneven the lengths are;
//   * fewer: C = kMinTiles, and a block takes whole pieces of at most C tiles that begin at an item's
//     start or C, 2 C, ... tiles behind it, so that short items are not cut for nothing.
// A piece is a run of an item's tiles in one block.  Where an item has several, each leaves a partial
// result in slot 2 (start / C) + (start != item's first tile) of the workspace, `start` being the number
// of the piece's first tile: at most one piece in each block begins an item that it does not finish, and
// at most one continues an item, so no two pieces share a slot.
#pragma once

#include <cstdint>

#include "cache8.cuh"

namespace exattn {

// Workspace: a header, the first tile number of every sequence, then the slots (fp32 rows of D values,
// normalised by the piece's own sum) and their base-2 log-sum-exps.
struct CacheSchedHeader {
  long long total;
  int per_piece;  // C
  int pieces;     // 1: the second form above
};

inline size_t cache_align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct CacheWs {
  CacheSchedHeader* head;
  long long* first;  // [B]
  float* o;          // [slots][R][D]
  float* l;          // [slots][R]
};

// Slots are numbered below 2 (T / C + 1) <= 2 (P + 1).
inline __host__ __device__ size_t cache_slots(int sm_count) { return 2 * (static_cast<size_t>(sm_count) + 1); }

inline __host__ __device__ size_t cache_ws_first_bytes(int B) { return (256 + 8 * static_cast<size_t>(B) + 255) & ~static_cast<size_t>(255); }

__host__ __device__ inline CacheWs cache_ws(uint8_t* ws, int B, int R, int D, int sm_count) {
  CacheWs w;
  w.head = reinterpret_cast<CacheSchedHeader*>(ws);
  w.first = reinterpret_cast<long long*>(ws + 256);
  w.o = reinterpret_cast<float*>(ws + cache_ws_first_bytes(B));
  w.l = w.o + cache_slots(sm_count) * R * D;
  return w;
}

// Number of keys that token i of Nq queries sees in a sequence of `len` tokens.
__device__ __forceinline__ int cache_row_limit(int mask, int len, int Nq, int i) {
  if (mask == ATTN_MASK_NONE) return len;
  if (mask == ATTN_MASK_CAUSAL) return min(len, i + 1);
  return max(0, len - Nq + i + 1);
}

// R query rows an item, TK keys a tile.
template <int R, int TK>
struct CacheItems {
  int rows, row_tiles;
  __device__ explicit CacheItems(const CacheAttnArgs& a) : rows(a.group * a.Nq), row_tiles((a.group * a.Nq + R - 1) / R) {}

  __device__ int tiles(const CacheAttnArgs& a, int len, int rt) const {
    const int last = min(rows, (rt + 1) * R) - 1;
    return (cache_row_limit(a.mask, len, a.Nq, last / a.group) + TK - 1) / TK;
  }
  // Units of one head of a sequence: its tiles, or with C > 0 its pieces of at most C tiles.
  __device__ long long head_units(const CacheAttnArgs& a, int len, int C) const {
    long long n = 0;
    for (int rt = 0; rt < row_tiles; ++rt) {
      const int t = tiles(a, len, rt);
      n += C > 0 ? (t + C - 1) / C : t;
    }
    return n;
  }
  __device__ int seq_len(const CacheAttnArgs& a, int b) const { return cache_len(a.c, __ldg(a.lens + b)); }
};

// Exclusive prefix sums over the block's threads of one value each; `out` has NT + 1 entries.
template <int NT>
__device__ void block_prefix(long long v, long long* out, long long* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  long long base = 0;
  for (int w = 0; w < warp; ++w) base += warp_sums[w];
  out[threadIdx.x + 1] = base + x;
  if (threadIdx.x == 0) out[0] = 0;
  __syncthreads();
}

// A piece of an item for one block.
struct CachePiece {
  int b, head, rt, len;
  int begin, end;     // key tiles of the item
  int slot;           // -1: the whole item, else its place in the workspace
};

// The division, and a block's walk over its pieces.  Built by all NT threads of a block; next() is then
// called by one warp, all lanes alike.
template <int R, int TK, int NT, int kMinTiles>
struct CacheWalk {
  struct Shared {
    long long tiles[NT + 1], units[NT + 1], warp_sums[NT / 32];
  };
  const CacheAttnArgs& a;
  Shared& sh;
  CacheItems<R, TK> items;
  long long total, at, stop;  // first form: tile numbers; second: piece numbers
  int C, per;                 // per: sequences a thread of the prefix sums
  bool by_piece;
  int step;
  // place of the next tile (first form)
  int b = 0, head = 0, rt = 0, len = 0, tile = 0, ntiles = 0;
  long long item_first = 0;
  bool placed = false;

  __device__ CacheWalk(const CacheAttnArgs& args, Shared& s, int block, int blocks)
      : a(args), sh(s), items(args) {
    per = (a.B + NT - 1) / NT;
    const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    long long n = 0;
    for (int i = b0; i < b1; ++i) n += a.c.heads * items.head_units(a, items.seq_len(a, i), 0);
    block_prefix<NT>(n, sh.tiles, sh.warp_sums);
    total = sh.tiles[NT];
    by_piece = total <= static_cast<long long>(blocks) * kMinTiles;
    C = by_piece ? kMinTiles : static_cast<int>((total + blocks - 1) / blocks);
    if (by_piece) {
      n = 0;
      for (int i = b0; i < b1; ++i) n += a.c.heads * items.head_units(a, items.seq_len(a, i), C);
      block_prefix<NT>(n, sh.units, sh.warp_sums);
      at = block;
      stop = sh.units[NT];
      step = blocks;
    } else {
      sh.units[threadIdx.x + 1] = sh.tiles[threadIdx.x + 1];
      if (threadIdx.x == 0) sh.units[0] = 0;
      at = static_cast<long long>(block) * C;
      stop = min(total, at + C);
      step = 0;
    }
    __syncthreads();
    if (block == 0) {  // for the merge
      const CacheWs ws = cache_ws(a.ws, a.B, R, a.c.d, a.sm_count);
      long long f = sh.tiles[threadIdx.x];
      for (int i = b0; i < b1; ++i) {
        ws.first[i] = f;
        const int raw = __ldg(a.lens + i), l = cache_len(a.c, raw);
        if (raw != l) record_page_error(a.err_word);
        f += a.c.heads * items.head_units(a, l, 0);
      }
      if (threadIdx.x == 0) *ws.head = CacheSchedHeader{total, C, by_piece ? 1 : 0};
    }
  }

  // Finds unit x: sets b, len, head, rt and item_first, and returns the unit's number inside its item.
  __device__ long long locate(long long x) {
    int lo = 0, hi = NT;  // units[lo] <= x < units[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sh.units[mid] <= x) lo = mid; else hi = mid;
    }
    x -= sh.units[lo];
    item_first = sh.tiles[lo];
    const int piece = by_piece ? C : 0;
    long long hu = 0;
    for (b = lo * per;; ++b) {
      len = items.seq_len(a, b);
      hu = items.head_units(a, len, piece);
      if (x < hu * a.c.heads) break;
      x -= hu * a.c.heads;
      item_first += a.c.heads * items.head_units(a, len, 0);
    }
    head = static_cast<int>(x / hu);
    x -= head * hu;
    item_first += head * items.head_units(a, len, 0);
    for (rt = 0;; ++rt) {
      ntiles = items.tiles(a, len, rt);
      const long long u = by_piece ? (ntiles + C - 1) / C : ntiles;
      if (x < u) break;
      x -= u;
      item_first += ntiles;
    }
    return x;
  }

  __device__ bool next(CachePiece& p) {
    if (at >= stop) return false;
    if (by_piece) {
      tile = static_cast<int>(locate(at)) * C;
      at += step;
    } else {
      if (!placed) {
        tile = static_cast<int>(locate(at));
        placed = true;
      } else {  // the item after the last one, passing those without tiles
        item_first += ntiles;
        tile = 0;
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
    }
    p.b = b;
    p.head = head;
    p.rt = rt;
    p.len = len;
    p.begin = tile;
    p.end = by_piece ? min(ntiles, tile + C)
                     : static_cast<int>(min(static_cast<long long>(ntiles), tile + (stop - at)));
    const long long start = item_first + tile;
    p.slot = (p.begin == 0 && p.end == ntiles) ? -1 : static_cast<int>(2 * (start / C) + (tile != 0));
    if (!by_piece) at += p.end - p.begin;
    return true;
  }
};

}  // namespace exattn
