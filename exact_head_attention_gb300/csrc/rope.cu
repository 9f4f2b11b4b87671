// Rotary positions with optional RMS norms per head, and their gradients.
//
// Mathematics.  A head x of a token at position p becomes y = x r w, r = 1 / sqrt(mean x^2 + eps), whose pairs (a, b) turn by
// the angle p f: (a cos - b sin, a sin + b cos).  Backwards, with g the gradient turned back,
//   dw = sum over tokens and heads of g x r,    dx = r (g w - x r mean(g w x r)),
// and r is computed again from x, which has to be read anyway.  All in fp32, rounded once; the sums of dw in a fixed order.
//
// Bound: memory.  Forward 2 bytes read and 2 written a value, the gradients 4 read (2 without weights) and 2 written.  What
// the angles take (about 25 instructions a pair and token) is shared by the heads that a thread has.
//
// Measured on GB300, 4 sequences of 8192 tokens, 12 query and 12 key heads of 128, bf16: with norms in 62.9 us, 95 % of the
// measured copy rate; the gradients in 96.5 us, 93 %.  One token, 24 heads: 2.3 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.h"  // launch_dependent
#include "rope.cuh"

namespace exattn {
namespace {

constexpr int kFwdBlocks = 3;  // resident an SM

template <int D, bool BF16>
__global__ void __launch_bounds__(kRopeThreads, kFwdBlocks) rope_kernel(const __grid_constant__ RopeArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ RopeShared sh;
  rope_rows<D, BF16>(a, sh, blockIdx.x, blockIdx.y);
}

constexpr int kBwdBlocks = 2;  // resident an SM

// A count of the blocks that are done.  It needs no preparation: every block first makes it the call's tag where its upper 48
// bits are another (cache_sched.cuh), which costs nothing beside the block's first loads, and the last to be counted puts it
// to rest.
__device__ __forceinline__ void count_open(unsigned long long* at, unsigned long long tag) {
  unsigned long long seen, old;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(seen) : "l"(at) : "memory");
  while ((seen & ~0xffffull) != tag) {
    asm volatile("atom.relaxed.gpu.global.cas.b64 %0, [%1], %2, %3;" : "=l"(old) : "l"(at), "l"(seen), "l"(tag) : "memory");
    if (old == seen) break;
    seen = old;
  }
}
// Adds one, by a thread whose block has met; true for the last of `n`: what the others' blocks wrote is then visible to it, and
// to its block after a barrier.
__device__ __forceinline__ bool count_close(unsigned long long* at, unsigned n) {
  unsigned long long old;
  asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], %2;" : "=l"(old) : "l"(at), "l"(1ull) : "memory");
  const bool all = (old & 0xffffull) + 1ull == n;
  if (all) asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(at), "l"(0ull) : "memory");
  return all;
}

// One thread takes `span` heads of a token after another (an item), the block's threads different tokens or chunks of heads.
// Its loads are a row ahead, by way of places of its own in shared memory, so that they stay under way while it computes
// (held in registers, two rows at a time, the whole took 111 us for 96; two and more rows ahead 97 to 111).
template <int D, bool BF16>
__global__ void __launch_bounds__(kRopeThreads, kBwdBlocks) rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
  using Lane = RopeLane<D>;
  constexpr int GROUPS = kRopeThreads / Lane::LANES;
  constexpr int DEPTH = 2;
  __shared__ uint4 slots[DEPTH][4][kRopeThreads];  // a thread's units of the gradient and of the input, of the rows under way
  __shared__ float sums[kRopeThreads / 32][D];
  __shared__ RopeTable table;
  griddep_wait();
  griddep_launch_dependents();
  const bool is_k = blockIdx.x >= static_cast<unsigned>(a.blocks[0]);
  const RopeSide& sd = a.side[is_k];
  const unsigned blocks = a.blocks[is_k];
  const int g = threadIdx.x / Lane::LANES, span = min(a.span, sd.heads);
  const int chunks_a_block = GROUPS >> a.token_shift, chunks = (sd.heads + span - 1) / span;
  const unsigned token_blocks = (static_cast<unsigned>(a.tokens) + (1u << a.token_shift) - 1) >> a.token_shift;
  const unsigned chunk_blocks = (chunks + chunks_a_block - 1) / chunks_a_block;
  const Lane l(a.r, threadIdx.x % Lane::LANES);

  // A place in the block's sequence of rows: row i of `here` of the item (tb, cb), of which a block has every `blocks`-th in
  // the order token blocks first.
  const unsigned step_cb = blocks / token_blocks, step_tb = blocks - step_cb * token_blocks;
  struct Cursor {
    unsigned tb, cb;
    int i, here, b, n, h0;
  };
  auto enter = [&](Cursor& c) {
    const unsigned t = (c.tb << a.token_shift) + (g & ((1 << a.token_shift) - 1));
    c.i = 0;
    c.h0 = (c.cb * chunks_a_block + (g >> a.token_shift)) * span;
    c.here = c.cb < chunk_blocks && t < static_cast<unsigned>(a.tokens) ? min(span, sd.heads - c.h0) : 0;
    c.b = t / static_cast<unsigned>(a.N);
    c.n = t - c.b * a.N;
  };
  auto next = [&](Cursor& c) {
    c.tb += step_tb;
    c.cb += step_cb;
    if (c.tb >= token_blocks) {
      c.tb -= token_blocks;
      ++c.cb;
    }
    enter(c);
  };
  auto row_of = [&](const void* x, const RowStrides& st, const Cursor& c) {
    return static_cast<const uint16_t*>(x) + c.b * st.b + c.h0 * st.h + c.n * st.n;
  };
  Cursor ahead, at;
  const unsigned first = blockIdx.x - (is_k ? a.blocks[0] : 0);
  ahead.cb = first / token_blocks;
  ahead.tb = first - ahead.cb * token_blocks;
  enter(ahead);
  at = ahead;
  const uint16_t *dy = row_of(sd.x, sd.sx, ahead), *in = row_of(sd.in, sd.sin, ahead);
  int slot = 0;
  auto issue = [&]() {
    const bool there = ahead.i < ahead.here;
    uint4 (&to)[4][kRopeThreads] = slots[slot];
    const uint4 *from_dy = reinterpret_cast<const uint4*>(there ? dy : sd.x), *from_in = reinterpret_cast<const uint4*>(there ? in : sd.in);
    copy16(&to[0][threadIdx.x], from_dy + l.ua, there);
    copy16(&to[1][threadIdx.x], from_dy + l.ub, there);
    copy16(&to[2][threadIdx.x], from_in + l.ua, there);
    copy16(&to[3][threadIdx.x], from_in + l.ub, there);
    copies_commit();
    slot = slot + 1 == DEPTH ? 0 : slot + 1;
    dy += sd.sx.h;
    in += sd.sin.h;
    if (++ahead.i == span) {
      next(ahead);
      dy = row_of(sd.x, sd.sx, ahead);
      in = row_of(sd.in, sd.sin, ahead);
    }
  };
  issue();
  if (threadIdx.x == 0 && a.tag != 0) count_open(a.count + is_k, a.tag);

  table.fill(a.r, threadIdx.x, kRopeThreads);
  __syncthreads();
  float w[16], dw[16];
  l.template weights<BF16>(sd.weight, a.weight_fp32, w);
#pragma unroll
  for (int e = 0; e < 16; ++e) dw[e] = 0.f;
  float c[8], s[8];
  int from = 0;
  uint16_t* dx = const_cast<uint16_t*>(row_of(sd.y, sd.sy, at));
#pragma unroll 1
  while (at.cb < chunk_blocks) {
    if (at.i == 0 && at.here > 0) l.angles(table, rope_position(a.r, at.b, at.n, a.r.start), true, c, s);
    issue();
    copies_wait<DEPTH - 1>();
    float gr[16], x[16];
    const uint4 (&in)[4][kRopeThreads] = slots[from];
    Lane::template widen<BF16>(in[0][threadIdx.x], in[1][threadIdx.x], gr);
    Lane::template widen<BF16>(in[2][threadIdx.x], in[3][threadIdx.x], x);
    from = from + 1 == DEPTH ? 0 : from + 1;
    const bool there = at.i < at.here;
    if (there) l.rotate(gr, c, s);
    const float r = Lane::inverse_rms(x, a.r.eps);
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      x[e] *= r;
      dw[e] = fmaf(gr[e], x[e], dw[e]);
      gr[e] *= w[e];
      dot = fmaf(gr[e], x[e], dot);
    }
    dot = Lane::row_sum(dot) * (1.f / D);
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = r * (gr[e] - x[e] * dot);
    if (there) l.template store<BF16>(dx, x);
    dx += sd.sy.h;
    if (++at.i == span) {
      next(at);
      dx = const_cast<uint16_t*>(row_of(sd.y, sd.sy, at));
    }
  }
  copies_wait<0>();  // a copy must not land after the block has ended
  // The block's sums: over the rows of a warp, then over the warps.
#pragma unroll
  for (int e = 0; e < 16; ++e) {
#pragma unroll
    for (int o = Lane::LANES; o < 32; o <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], o);
  }
  if ((threadIdx.x & 31) < Lane::LANES) {
#pragma unroll
    for (int e = 0; e < 16; ++e) sums[threadIdx.x >> 5][8 * (e < 8 ? l.ua : l.ub) + (e & 7)] = dw[e];
  }
  __syncthreads();
  float* const mine = a.sums + static_cast<size_t>(blockIdx.x) * D;
  for (int col = threadIdx.x; col < D; col += kRopeThreads) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kRopeThreads / 32; ++i) v += sums[i][col];
    mine[col] = v;
  }
  if (a.tag == 0) return;  // rope_dw_kernel adds them up
  // The side's last block to come here does.
  __shared__ bool last;
  __syncthreads();
  if (threadIdx.x == 0) last = count_close(a.count + is_k, blocks);
  __syncthreads();
  if (!last) return;
  constexpr int COLS = D / 4, PARTS = kRopeThreads / COLS;  // four columns a thread, every PARTS-th block
  const float4* parts = reinterpret_cast<const float4*>(a.sums + (is_k ? static_cast<size_t>(a.blocks[0]) * D : 0));
  const int col = threadIdx.x % COLS, part = threadIdx.x / COLS;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (unsigned i = part; i < blocks; i += PARTS) {
    const float4 x = __ldcg(parts + static_cast<size_t>(i) * COLS + col);
    v.x += x.x;
    v.y += x.y;
    v.z += x.z;
    v.w += x.w;
  }
  float4* const joint = reinterpret_cast<float4*>(slots);  // every copy into them has landed
  joint[part * COLS + col] = v;
  __syncthreads();
  if (threadIdx.x < COLS) {
#pragma unroll
    for (int i = 1; i < PARTS; ++i) {
      const float4 x = joint[i * COLS + col];
      v.x += x.x;
      v.y += x.y;
      v.z += x.z;
      v.w += x.w;
    }
    if (a.weight_fp32)
      reinterpret_cast<float4*>(sd.dweight)[col] = v;
    else
      reinterpret_cast<uint2*>(sd.dweight)[col] = make_uint2(pack2<BF16>(v.x, v.y), pack2<BF16>(v.z, v.w));
  }
}

// dw from the blocks' sums where those are many: 32 columns a block, each over 32 threads.
template <bool BF16>
__global__ void __launch_bounds__(1024) rope_dw_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float sums[32][33];
  griddep_wait();
  griddep_launch_dependents();
  const RopeSide& sd = a.side[blockIdx.y];
  const int first = blockIdx.y ? a.blocks[0] : 0, blocks = a.blocks[blockIdx.y];
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float v = 0.f;
  for (int i = part; i < blocks; i += 32) v += a.sums[static_cast<size_t>(first + i) * a.d + col];
  sums[part][lane] = v;
  __syncthreads();
  v = sums[lane][part];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0 && blocks > 0) {
    const int to = blockIdx.x * 32 + part;
    if (a.weight_fp32) static_cast<float*>(sd.dweight)[to] = v;
    else static_cast<uint16_t*>(sd.dweight)[to] = static_cast<uint16_t>(pack2<BF16>(v, 0.f));
  }
}

// log2 of the tokens that stand side by side in a block of `groups` rows: as many as there are, up to all of them.
int token_shift(int tokens, int groups) {
  int s = 0;
  while ((1 << s) < groups && (1 << s) < tokens) ++s;
  return s;
}

template <int D, bool BF16>
cudaError_t fwd_d(RopeArgs& a, cudaStream_t stream) {
  const RopeGrid g = rope_plan(a);
  return launch_dependent(rope_kernel<D, BF16>, dim3(g.token_blocks, g.chunk_blocks), dim3(kRopeThreads), 0, stream, a);
}

template <int D, bool BF16>
cudaError_t bwd_d(RopeArgs& a, cudaStream_t stream) {
  constexpr int GROUPS = kRopeThreads / RopeLane<D>::LANES;
  a.token_shift = token_shift(a.tokens, GROUPS);
  const long long token_blocks = (static_cast<long long>(a.tokens) + (1 << a.token_shift) - 1) >> a.token_shift;
  const int per = GROUPS >> a.token_shift;
  // the blocks that are resident at once, shared out by heads
  const long long heads = static_cast<long long>(a.side[0].heads) + a.side[1].heads;
  const long long resident = static_cast<long long>(kBwdBlocks) * a.sm_count;
  // Heads an item: beginning one costs about one and a half rows.  12 heads of 128 each, 32768 tokens: 155 us with 1, 115 with
  // 2, 102 with 4, 99 with 6, 97 with 12; 16 and 4 heads of 64, 666 tokens: 6.7, 5.8, 6.8, 7.6 and 11.3 us.
  long long best = 0;
  int span_best = 2;
  for (int s : {2, 4, 6, 12}) {
    long long rounds = 0;
    for (int i = 0; i < 2; ++i) {
      const long long share = resident * a.side[i].heads / heads, chunks = (a.side[i].heads + s - 1) / s;
      const long long items = token_blocks * ((chunks + per - 1) / per), r = (items + (share > 0 ? share - 1 : 0)) / (share > 0 ? share : 1);
      if (r > rounds) rounds = r;
    }
    const long long cost = rounds * (2 * s + 3);
    if (best == 0 || cost < best) {
      best = cost;
      span_best = s;
    }
  }
  a.span = span_best;
  for (int i = 0; i < 2; ++i) {
    const int span = a.span < a.side[i].heads ? a.span : a.side[i].heads;
    const long long chunks = span ? (a.side[i].heads + span - 1) / span : 0, items = token_blocks * ((chunks + per - 1) / per);
    long long share = resident * a.side[i].heads / heads;
    if (share < 1) share = 1;
    a.blocks[i] = static_cast<int>(items < share ? items : share);
  }
  // Few blocks' sums are added up by the last one, many by a launch of their own, more of whose loads are under way: 110 blocks
  // 6.8 us and 29 for the host's part, 5.9 and 32 with a second launch; 304 blocks 98.8 us, 96.6 with a second launch.
  const int blocks = a.blocks[0] + a.blocks[1];
  if (blocks > a.sm_count) a.tag = 0;
  const cudaError_t e = launch_dependent(rope_bwd_kernel<D, BF16>, dim3(blocks), dim3(kRopeThreads), 0, stream, a);
  if (e != cudaSuccess || a.tag != 0) return e;
  return launch_dependent(rope_dw_kernel<BF16>, dim3(D / 32, 2), dim3(1024), 0, stream, a);
}

}  // namespace

RopeGrid rope_plan(RopeArgs& a) {
  // Heads a thread.  What it does before the first takes about as long as four of them; all threads' work over the blocks that
  // are resident at once, and about half a thread's for the blocks that end last.  us with 1, 2, 3, 4, 6, 8 and 12:
  //   12 and 12 heads of 128, 32768 tokens   153  96  78  70  63  65  64
  //   14 and 2 heads of 64, 20072 tokens     30.0 19.8 17.5 16.3 15.5 14.8 14.5
  //   28 and 4 heads of 64, 4611 tokens      14.8 9.4 8.4 7.4 6.7 7.9 9.2
  //   16 and 16 heads of 128, 2048 tokens    15.2 10.7 9.5 8.8 7.5 8.6 10.7
  //   42 and 6 heads of 128, 114 tokens      3.3 2.9 3.2 3.4 3.8 4.3 5.2
  // It takes 12, 8, 6, 8 and 2 of them.
  const int hq = a.side[0].heads, hk = a.side[1].heads, most = hq > hk ? hq : hk, groups = kRopeThreads / (a.d / 16);
  a.token_shift = token_shift(a.tokens, groups);
  const int per = groups >> a.token_shift;  // chunks a block
  const long long token_blocks = (static_cast<long long>(a.tokens) + (1 << a.token_shift) - 1) >> a.token_shift;
  const long long slots = static_cast<long long>(kFwdBlocks) * a.sm_count;
  long long best = 0, chunk_blocks = 0;
  for (int s : {1, 2, 3, 4, 6, 8, 12}) {
    if (s > 1 && s > most) break;
    const long long chunks = (hq + s - 1) / s + (hk + s - 1) / s, cb = (chunks + per - 1) / per;
    const long long cost = 200 * token_blocks * (4 * chunks + hq + hk) / per / slots + 100 * (4 + s);
    if (best == 0 || cost < best) {
      best = cost;
      chunk_blocks = cb;
      a.span = s;
    }
  }
  a.q_chunks = (hq + a.span - 1) / a.span;
  // a side without heads has rows that no load reads, but whose addresses are formed
  for (int i = 0; i < 2; ++i)
    if (a.side[i].heads == 0) {
      a.side[i].x = a.side[1 - i].x;
      a.side[i].weight = nullptr;
    }
  return {static_cast<unsigned>(token_blocks), static_cast<unsigned>(chunk_blocks)};
}

cudaError_t launch_rope(RopeArgs& a, cudaStream_t stream) {
  if (a.d == 128) return a.bf16 ? fwd_d<128, true>(a, stream) : fwd_d<128, false>(a, stream);
  return a.bf16 ? fwd_d<64, true>(a, stream) : fwd_d<64, false>(a, stream);
}

// Two counts, and a row of sums for each block: no more than two an SM, and one more for either side.
size_t rope_bwd_workspace(int d, int sm_count) { return kRopeSumsAt + static_cast<size_t>(kBwdBlocks * sm_count + 2) * d * sizeof(float); }

cudaError_t launch_rope_bwd(RopeArgs& a, cudaStream_t stream) {
  // A side without weights needs no more than the rotation turned back.
  RopeArgs plain = a, normed = a;
  for (int i = 0; i < 2; ++i) {
    (a.side[i].weight ? plain : normed).side[i].heads = 0;
    plain.side[i].weight = nullptr;
  }
  if (plain.side[0].heads + plain.side[1].heads > 0) {
    const cudaError_t e = launch_rope(plain, stream);
    if (e != cudaSuccess) return e;
  }
  if (normed.side[0].heads + normed.side[1].heads == 0) return cudaSuccess;
  if (a.d == 128) return a.bf16 ? bwd_d<128, true>(normed, stream) : bwd_d<128, false>(normed, stream);
  return a.bf16 ? bwd_d<64, true>(normed, stream) : bwd_d<64, false>(normed, stream);
}

}  // namespace exattn
