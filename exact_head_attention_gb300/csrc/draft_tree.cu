// Masks and depths of trees of drafted tokens from their parents.
//
// A token sees itself and its ancestors.  By doubling: with row i holding the nearest 2^k of them (itself among them) and
// up[i] the 2^k-th, row i | row up[i] holds the nearest 2^(k+1), so that no chain is walked: at most 9 rounds for 512 tokens,
// as many as the deepest token's depth has binary digits.  A block for each tree, a thread for each token; rows lie word by
// word, so that a warp's own words never meet a bank twice.  All latency: trees of 24 tokens take as long as a launch.
#include "cache_sched.cuh"
#include "ptx.cuh"

namespace exattn {
namespace {

constexpr int kWords = kTreeMost / 32;

__global__ void __launch_bounds__(kTreeMost) draft_tree_kernel(const __grid_constant__ DraftTreeArgs a) {
  __shared__ uint32_t rows[kWords][kTreeMost];
  __shared__ int up[kTreeMost];
  griddep_wait();
  griddep_launch_dependents();
  const int i = threadIdx.x, words = (a.N + 31) >> 5;
  const long long first = static_cast<long long>(blockIdx.x) * a.N;
  int parent = -1;
  if (i < a.N) {
    parent = a.parents[first + i];
    if (parent < -1 || parent >= i) {
      parent = -1;
      atomicCAS(a.err_word, 0u, kErrTree);
    }
  }
  up[i] = parent;
  uint32_t mine[kWords];
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    mine[w] = w == i >> 5 ? 1u << (i & 31) : 0u;
    if (w < words) rows[w][i] = mine[w];
  }
  while (__syncthreads_or(parent >= 0)) {
    int next = -1;
    if (parent >= 0) {
      next = up[parent];
#pragma unroll
      for (int w = 0; w < kWords; ++w)
        if (w <= parent >> 5) mine[w] |= rows[w][parent];
    }
    __syncthreads();
    if (parent >= 0) {
      up[i] = parent = next;
#pragma unroll
      for (int w = 0; w < kWords; ++w)
        if (w < words) rows[w][i] = mine[w];
    }
  }
  if (i < a.N) {
    int n = -1;
#pragma unroll
    for (int w = 0; w < kWords; ++w) n += __popc(mine[w]);
    a.depth[first + i] = n;
  }
  // no thread is behind the last round's writes: the loop's barrier came after them
  for (int k = i; k < a.N * words; k += blockDim.x) {
    const int row = k / words;
    a.mask[first * words + k] = rows[k - row * words][row];
  }
}

}  // namespace

cudaError_t launch_draft_tree(const DraftTreeArgs& a, int B, cudaStream_t stream) {
  return launch_dependent(draft_tree_kernel, dim3(B), dim3((a.N + 31) / 32 * 32), 0, stream, a);
}

}  // namespace exattn
