// Arguments and launchers of the kernels for rotary positions and norms per head, shared by rope_api.cu, cache_api.cu
// and their translation units.  Not part of the public header.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"

namespace exattn {

// attn_rope as the kernels take it.
struct RopeView {
  const double* freq;  // [rot / 2]
  const int* start;    // [B], or nullptr
  const int* offsets;  // [B][N] at offset_stride, or nullptr
  long long offset_stride;
  int rot, interleaved;
  float amplitude, eps;
  bool back;  // the transposed rotation
};

// One tensor of heads: 16-bit views [B][heads][N][d], its weights of the norm (nullptr: none).
struct RopeSide {
  const void* x;   // forward: the input; backward: the gradient of the output
  const void* in;  // backward with weights: the forward's input
  void* y;
  const void* weight;
  void* dweight;
  RowStrides sx, sin, sy;
  int heads;
};

struct RopeArgs {
  RopeView r;
  RopeSide side[2];  // queries and keys
  int B, N, d;
  int tokens;       // B * N
  int token_shift;  // log2 of the tokens that a block takes side by side
  int span;         // forward: heads that a thread takes one after the other
  int q_chunks;     // forward: chunks of `span` heads of the queries
  bool bf16, weight_fp32;
  int sm_count;
  // backward
  unsigned long long* count;  // blocks that are done, of the queries and of the keys
  unsigned long long tag;     // of this call's counts, the low 16 bits zero; 0: there are none
  float* sums;                // a row of d for each block
  int blocks[2];              // of the queries and of the keys
};

// Chooses how the forward is divided over blocks of 256 threads: token_shift, span and q_chunks, and the blocks of tokens and
// of chunks.
struct RopeGrid {
  unsigned token_blocks, chunk_blocks;
};
RopeGrid rope_plan(RopeArgs& a);
cudaError_t launch_rope(RopeArgs& a, cudaStream_t stream);
cudaError_t launch_rope_bwd(RopeArgs& a, cudaStream_t stream);
constexpr size_t kRopeSumsAt = 256;  // of the workspace, behind the counts
size_t rope_bwd_workspace(int d, int sm_count);

}  // namespace exattn
