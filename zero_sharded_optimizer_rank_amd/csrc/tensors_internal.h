// Internal interface between the host side of the tensor-list calls
// (zero_tensors.cpp) and their kernels (zero_tensors.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "zero_internal.h"
#include "zero_shard.h"

namespace zk {

// The norm cuts every tensor into chunks, one workgroup and one fp64 partial
// each.  A chunk is kTensorChunk << s elements, with the smallest s that keeps
// the list at kTensorPartials chunks (each tensor's last, short one aside): few
// enough for one workgroup per tensor to sum, many enough to fill the chip.
constexpr int64_t kTensorChunk = 16384;
constexpr int64_t kTensorPartials = 32768;

struct TensorLayout {
  int32_t shift;       // s above
  int64_t chunks;      // over all tensors; an empty tensor has one
  int64_t longest;     // most chunks of one tensor
};
TensorLayout tensor_layout(const zero_tensor_t* tensors, int32_t n);
size_t tensors_workspace_bytes(const zero_tensor_t* tensors, int32_t n);

// Launchers: arguments already validated.  Return hipSuccess or the error.
int launch_tensors_norm(const zero_tensor_t* tensors, int32_t n, double* tensor_sq,
                        void* workspace, const FinalizeArgs& fa, zero_step_result_t* res,
                        hipStream_t stream);
int launch_tensors_clip(const zero_tensor_t* tensors, int32_t n, float scale,
                        const zero_step_result_t* res, hipStream_t stream);
int launch_tensors_norm_clip(const zero_tensor_t* tensors, int32_t n, double* tensor_sq,
                             void* workspace, const FinalizeArgs& fa, float scale,
                             zero_step_result_t* res, hipStream_t stream);

}  // namespace zk
