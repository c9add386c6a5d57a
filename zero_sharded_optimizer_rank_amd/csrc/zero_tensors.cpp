// Host side of the tensor-list calls: argument checks and the chunk layout.
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "host_internal.h"
#include "tensors_internal.h"
#include "zero_shard.h"

using namespace zk::host;

namespace {

size_t elem_bytes(int32_t dtype) { return dtype == ZERO_F32 ? 4 : 2; }
bool known(int32_t dtype) { return dtype == ZERO_F32 || dtype == ZERO_F16 || dtype == ZERO_BF16; }

int check_list(const zero_tensor_t* t, int32_t n) {
  if (n < 0 || (n > 0 && !t)) return fail(ZERO_EINVAL, "bad tensor list");
  for (int32_t i = 0; i < n; ++i) {
    if (t[i].numel < 0 || t[i].numel > INT64_MAX / 8)
      return fail(ZERO_EINVAL, "tensor %d: numel %lld", i, (long long)t[i].numel);
    if (!known(t[i].src_dtype))
      return fail(ZERO_EINVAL, "tensor %d: unknown dtype %d", i, t[i].src_dtype);
    if (t[i].numel == 0) continue;
    if (!t[i].src) return fail(ZERO_EINVAL, "tensor %d: src is NULL", i);
    if (!aligned(t[i].src, elem_bytes(t[i].src_dtype)))
      return fail(ZERO_EALIGN, "tensor %d: src not aligned to its elements", i);
  }
  return ZERO_OK;
}

int check_result(const zero_step_result_t* dev_result) {
  if (!dev_result) return fail(ZERO_EINVAL, "dev_result is NULL");
  if (!aligned(dev_result, 8)) return fail(ZERO_EALIGN, "dev_result not 8-byte aligned");
  return ZERO_OK;
}

int check_norm(const zero_tensor_t* t, int32_t n, const zero_step_args_t* args, double* tensor_sq,
               void* workspace, size_t ws_bytes, zero_step_result_t* dev_result) {
  int rc = check_list(t, n);
  if (!rc) rc = check_norm_args(args);
  if (!rc) rc = check_result(dev_result);
  if (rc) return rc;
  if (args->other_q_lo || args->other_q_hi)
    return fail(ZERO_EINVAL, "other_q must be 0 (combine with other_sq)");
  if (!aligned(tensor_sq, 8)) return fail(ZERO_EALIGN, "tensor_sq not 8-byte aligned");
  if (!workspace) return fail(ZERO_EINVAL, "workspace is NULL");
  if (!aligned(workspace, 16)) return fail(ZERO_EALIGN, "workspace not 16-byte aligned");
  const size_t need = zk::tensors_workspace_bytes(t, n);
  if (ws_bytes < need) return fail(ZERO_ENOSPC, "workspace %zu bytes < %zu", ws_bytes, need);
  return ZERO_OK;
}

int check_clip(const zero_tensor_t* t, int32_t n, const zero_step_args_t* args, double out_scale,
               const zero_step_result_t* dev_result) {
  int rc = check_list(t, n);
  if (!rc) rc = check_norm_args(args);
  if (!rc) rc = check_result(dev_result);
  if (rc) return rc;
  const float s = (float)(out_scale / args->loss_scale);
  if (!(out_scale > 0.0) || !isfinite(out_scale) || !(s > 0.0f) || !isfinite(s))
    return fail(ZERO_EINVAL, "out_scale and out_scale / loss_scale must be finite and > 0");
  for (int32_t i = 0; i < n; ++i) {
    if (!known(t[i].dst_dtype))
      return fail(ZERO_EINVAL, "tensor %d: unknown dst dtype %d", i, t[i].dst_dtype);
    if (t[i].numel == 0) continue;
    if (!t[i].dst) return fail(ZERO_EINVAL, "tensor %d: dst is NULL", i);
    const size_t es = elem_bytes(t[i].src_dtype), ed = elem_bytes(t[i].dst_dtype);
    if (!aligned(t[i].dst, ed))
      return fail(ZERO_EALIGN, "tensor %d: dst not aligned to its elements", i);
    const bool in_place = t[i].src == t[i].dst && t[i].src_dtype == t[i].dst_dtype;
    if (!in_place && overlap(t[i].src, es * (size_t)t[i].numel, t[i].dst,
                             ed * (size_t)t[i].numel))
      return fail(ZERO_EINVAL, "tensor %d: dst overlaps src", i);
  }
  return ZERO_OK;
}

zk::FinalizeArgs norm_finalize_args(const zero_step_args_t* a) {
  const zero_plan_t one = {0, 1, 1, 0, 0};  // the gradients are sums already: N = 1
  return finalize_args(&one, a);
}

}  // namespace

namespace zk {

TensorLayout tensor_layout(const zero_tensor_t* t, int32_t n) {
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i)
    total = t[i].numel > INT64_MAX - total ? INT64_MAX : total + t[i].numel;
  TensorLayout l{0, 0, 0};
  while ((total >> l.shift) > kTensorChunk * kTensorPartials) ++l.shift;
  const int64_t chunk = kTensorChunk << l.shift;
  for (int32_t i = 0; i < n; ++i) {
    const int64_t c = t[i].numel ? (t[i].numel - 1) / chunk + 1 : 1;
    l.chunks += c;
    if (c > l.longest) l.longest = c;
  }
  return l;
}

// Ticket, one record and one fp64 sum per tensor, one partial per chunk.
size_t tensors_workspace_bytes(const zero_tensor_t* t, int32_t n) {
  return kTicketBytes + 32 * (size_t)n + kPartialBytes * (size_t)tensor_layout(t, n).chunks;
}

}  // namespace zk

extern "C" {

size_t zero_tensors_workspace_bytes(const zero_tensor_t* tensors, int32_t n_tensors) {
  if (n_tensors < 0 || (n_tensors > 0 && !tensors)) return 0;
  for (int32_t i = 0; i < n_tensors; ++i)
    if (tensors[i].numel < 0 || tensors[i].numel > INT64_MAX / 8) return 0;
  return zk::tensors_workspace_bytes(tensors, n_tensors);
}

int zero_tensors_norm(const zero_tensor_t* tensors, int32_t n_tensors,
                      const zero_step_args_t* args, double* tensor_sq, void* workspace,
                      size_t ws_bytes, zero_step_result_t* dev_result, hipStream_t stream) {
  g_err[0] = 0;
  const int rc = check_norm(tensors, n_tensors, args, tensor_sq, workspace, ws_bytes, dev_result);
  if (rc) return rc;
  return hip_status(zk::launch_tensors_norm(tensors, n_tensors, tensor_sq, workspace,
                                            norm_finalize_args(args), dev_result, stream),
                    "tensors_norm launch");
}

int zero_tensors_clip(const zero_tensor_t* tensors, int32_t n_tensors,
                      const zero_step_args_t* args, double out_scale,
                      const zero_step_result_t* dev_result, hipStream_t stream) {
  g_err[0] = 0;
  const int rc = check_clip(tensors, n_tensors, args, out_scale, dev_result);
  if (rc) return rc;
  return hip_status(zk::launch_tensors_clip(tensors, n_tensors,
                                            (float)(out_scale / args->loss_scale),
                                            dev_result, stream),
                    "tensors_clip launch");
}

int zero_tensors_norm_clip(const zero_tensor_t* tensors, int32_t n_tensors,
                           const zero_step_args_t* args, double out_scale, double* tensor_sq,
                           void* workspace, size_t ws_bytes, zero_step_result_t* dev_result,
                           hipStream_t stream) {
  g_err[0] = 0;
  int rc = check_norm(tensors, n_tensors, args, tensor_sq, workspace, ws_bytes, dev_result);
  if (!rc) rc = check_clip(tensors, n_tensors, args, out_scale, dev_result);
  if (rc) return rc;
  return hip_status(zk::launch_tensors_norm_clip(tensors, n_tensors, tensor_sq, workspace,
                                                 norm_finalize_args(args),
                                                 (float)(out_scale / args->loss_scale),
                                                 dev_result, stream),
                    "tensors_norm_clip launch");
}

}  // extern "C"
