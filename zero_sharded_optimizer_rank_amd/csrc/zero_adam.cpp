// Host side of the list update: argument checks, the table and the scalars.
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "adam_internal.h"
#include "host_internal.h"
#include "zero_shard.h"

using namespace zk::host;

namespace {

bool known(int32_t dtype) { return dtype == ZERO_F32 || dtype == ZERO_F16 || dtype == ZERO_BF16; }
size_t elem_bytes(int32_t dtype) { return dtype == ZERO_F32 ? 4 : 2; }
constexpr int64_t kMostElements = (int64_t)1 << 39;  // workgroups are counted in 32 bits

int check_tensor(const zero_adam_tensor_t& t, int32_t i) {
  if (t.numel < 0 || t.numel > kMostElements)
    return fail(ZERO_EINVAL, "tensor %d: numel %lld", i, (long long)t.numel);
  if (!known(t.grad_dtype))
    return fail(ZERO_EINVAL, "tensor %d: unknown gradient dtype %d", i, t.grad_dtype);
  if (t.moment_bits != 8 && t.moment_bits != 32)
    return fail(ZERO_EINVAL, "tensor %d: moments of %d bits (8 or 32)", i, t.moment_bits);
  if (t.param && !known(t.param_dtype))
    return fail(ZERO_EINVAL, "tensor %d: unknown parameter dtype %d", i, t.param_dtype);
  if (!isfinite(t.weight_decay))
    return fail(ZERO_EINVAL, "tensor %d: weight_decay is not finite", i);
  if (!(t.lr_scale >= 0.0) || !isfinite(t.lr_scale))
    return fail(ZERO_EINVAL, "tensor %d: lr_scale must be finite and >= 0", i);
  if (t.numel == 0) return ZERO_OK;
  if (!t.grad || !t.master || !t.m || !t.v)
    return fail(ZERO_EINVAL, "tensor %d: grad, master, m or v is NULL", i);
  if (!aligned(t.grad, elem_bytes(t.grad_dtype)) || !aligned(t.master, 4) || !aligned(t.m, 4) ||
      !aligned(t.v, 4) || (t.param && !aligned(t.param, elem_bytes(t.param_dtype))))
    return fail(ZERO_EALIGN, "tensor %d: gradient and parameter must be aligned to their "
                "elements, master, m and v to 4 bytes", i);
  const bool small = t.moment_bits == 8;
  if (small && (!t.m_exp || !t.v_exp))
    return fail(ZERO_EINVAL, "tensor %d: m_exp or v_exp is NULL", i);
  const size_t n = (size_t)t.numel, b = (n + ZERO_ADAM_BLOCK - 1) / ZERO_ADAM_BLOCK;
  struct Range { const void* p; size_t n; };
  const Range r[7] = {{t.grad, n * elem_bytes(t.grad_dtype)},
                      {t.master, 4 * n},
                      {t.m, small ? n : 4 * n},
                      {t.v, small ? n : 4 * n},
                      {t.param, t.param ? n * elem_bytes(t.param_dtype) : 0},
                      {t.m_exp, small ? b : 0},
                      {t.v_exp, small ? b : 0}};
  for (int x = 0; x < 7; ++x)
    for (int y = 0; y < x; ++y)
      if (r[x].n && r[y].n && overlap(r[x].p, r[x].n, r[y].p, r[y].n))
        return fail(ZERO_EINVAL, "tensor %d: its buffers overlap", i);
  return ZERO_OK;
}

int check_list(const zero_adam_list_t* l) {
  if (!l) return fail(ZERO_EINVAL, "list is NULL");
  if (!l->table || l->n_tensors < 0 || l->blocks32 < 0 || l->blocks32 > UINT32_MAX ||
      l->blocks8 < 0 || l->blocks8 > UINT32_MAX)
    return fail(ZERO_EINVAL, "list was not prepared");
  return ZERO_OK;
}

}  // namespace

extern "C" {

size_t zero_adam_table_bytes(int32_t n_tensors) {
  if (n_tensors < 0) return 0;
  return (sizeof(zk::AdamEntry) + 2 * sizeof(uint32_t)) * (size_t)(n_tensors > 0 ? n_tensors : 1);
}

int zero_tensors_adam_prepare(const zero_adam_tensor_t* tensors, int32_t n_tensors, void* table,
                              size_t table_bytes, zero_adam_list_t* list, hipStream_t stream) {
  g_err[0] = 0;
  if (n_tensors < 0 || (n_tensors > 0 && !tensors)) return fail(ZERO_EINVAL, "bad tensor list");
  if (!list) return fail(ZERO_EINVAL, "list is NULL");
  if (!table) return fail(ZERO_EINVAL, "table is NULL");
  if (!aligned(table, 8)) return fail(ZERO_EALIGN, "table not 8-byte aligned");
  int64_t total = 0, blocks[2] = {0, 0}, elements = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    const int rc = check_tensor(tensors[i], i);
    if (rc) return rc;
    total += tensors[i].numel;
    if (total > kMostElements) return fail(ZERO_EINVAL, "too many elements");
    const bool small = tensors[i].moment_bits == 8;
    blocks[small] += zk::adam_blocks(tensors[i].numel, small);
    elements += (tensors[i].numel + ZERO_ADAM_BLOCK - 1) / ZERO_ADAM_BLOCK * ZERO_ADAM_BLOCK;
  }
  if (blocks[0] > UINT32_MAX || blocks[1] > UINT32_MAX)
    return fail(ZERO_EINVAL, "too many elements");
  const size_t need = zero_adam_table_bytes(n_tensors);
  if (table_bytes < need) return fail(ZERO_ENOSPC, "table %zu bytes < %zu", table_bytes, need);
  const int e = zk::launch_adam_table(tensors, n_tensors, table, stream);
  if (e) return hip_status(e, "adam table launch");
  *list = zero_adam_list_t{table, blocks[0], blocks[1], elements, n_tensors, 0};
  return ZERO_OK;
}

int zero_tensors_adam(const zero_adam_list_t* list, const zero_step_args_t* args, uint32_t seed,
                      const zero_step_result_t* dev_result, hipStream_t stream) {
  g_err[0] = 0;
  int rc = check_list(list);
  if (!rc) rc = check_adam_args(args);
  if (rc) return rc;
  if (!aligned(dev_result, 8)) return fail(ZERO_EALIGN, "dev_result not 8-byte aligned");
  const float scale = (float)(1.0 / args->loss_scale);
  if (!(scale > 0.0f) || !isfinite(scale))
    return fail(ZERO_EINVAL, "1 / loss_scale must be finite and > 0 in fp32");
  const double c1 = 1.0 - pow(args->beta1, (double)args->step);
  const double c2 = 1.0 - pow(args->beta2, (double)args->step);
  zk::ListScalars s;
  s.b1 = (float)args->beta1;
  s.omb1 = (float)(1.0 - args->beta1);
  s.b2 = (float)args->beta2;
  s.omb2 = (float)(1.0 - args->beta2);
  s.eps = (float)args->eps;
  s.sqrt_bc2 = (float)sqrt(c2);
  s.inv_root = (float)(1.0 / sqrt(c2));
  s.inv_root_low = 0x1p-12f * s.inv_root;
  s.scale = scale;
  s.key = seed;
  s.step_size = args->lr / c1;
  s.lr = args->lr;
  return hip_status(zk::launch_tensors_adam(list, s, dev_result, stream), "tensors_adam launch");
}

int zero_tensors_adam_moments(const zero_adam_list_t* list, void* m, void* v, int32_t dtype,
                              hipStream_t stream) {
  g_err[0] = 0;
  const int rc = check_list(list);
  if (rc) return rc;
  if (dtype != ZERO_F32 && dtype != ZERO_BF16)
    return fail(ZERO_EINVAL, "dtype %d: fp32 or bf16", dtype);
  if (list->elements > 0 && (!m || !v)) return fail(ZERO_EINVAL, "m or v is NULL");
  if (!aligned(m, elem_bytes(dtype)) || !aligned(v, elem_bytes(dtype)))
    return fail(ZERO_EALIGN, "m and v must be aligned to their elements");
  const size_t n = elem_bytes(dtype) * (size_t)list->elements;
  if (n && overlap(m, n, v, n)) return fail(ZERO_EINVAL, "m overlaps v");
  return hip_status(zk::launch_adam_moments(list, m, v, dtype == ZERO_F32, stream),
                    "adam_moments launch");
}

}  // extern "C"
