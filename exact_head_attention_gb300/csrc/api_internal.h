// What the C-ABI translation units share: per-device state, argument rules and error reporting, defined
// in api.cu.  Not part of the public header.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/exattn.h"
#include "kernels.h"
#include "rope.h"

namespace exattn {

struct DeviceInfo {
  uint32_t* err_word;  // device address of the error word
  int sm_count;
};

// State of the current device (first call on a device sets it up); ATTN_ERR_UNSUPPORTED off sm_103a.
attn_status api_device(DeviceInfo* out);
// SM count of the current device, or 0 where no device answers.
int api_sm_count();
uint64_t api_wait_timeout_ns();
// Status of a launch (and, in checked mode, of the kernels after a synchronisation).
attn_status api_finish(cudaError_t e, cudaStream_t stream);
attn_status api_driver_fail(const char* what, int code);
// attn_strides rules; extents of 1 get a stride that nothing uses.
bool api_strides(const attn_strides& in, int B, int H, int d, RowStrides* out);
// attn_rope rules, and its view for the kernels; `normed`: there are weights of a norm.
attn_status api_rope(const attn_rope* rope, int B, int N, int d, bool normed, RopeView* out);
// A number that no earlier call and no old contents of a workspace are likely to hold, its low 16 bits zero.
unsigned long long api_next_tag();
// 2-D byte map {128, lines} over contiguous 128-byte lines, box {128, box_lines}, 128-byte swizzle.
CUresult api_encode_lines(CUtensorMap* map, const void* base, uint64_t lines, uint32_t box_lines);

}  // namespace exattn
