// Internal interface between the host side of the list update (zero_adam.cpp)
// and its kernels (zero_adam.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "zero_internal.h"
#include "zero_shard.h"

namespace zk {

// Elements a workgroup updates.
constexpr int64_t kAdamChunk = 4096;
// Elements of one key of the dither; a chunk lies within one.
constexpr int kKeyShift = 12;
static_assert(((int64_t)1 << kKeyShift) % kAdamChunk == 0, "one key a workgroup");

// A tensor as the kernels read it, in the device table: entries [n], then the
// first workgroups [n] (32 bits each).
struct AdamEntry {
  const void* grad;
  float* master;
  void *m, *v;
  uint8_t *m_exp, *v_exp;
  void* param;
  int64_t numel, offset;
  double weight_decay, lr_scale;
  uint32_t kind;  // grad dtype | param dtype << 2 (3: none) | 8-bit moments << 4
  uint32_t reserved;
};

struct ListScalars {
  float b1, omb1, b2, omb2, eps, sqrt_bc2;
  float scale;       // 1 / loss_scale
  uint32_t key;      // the seed, mixed once
  double step_size;  // lr / (1 - b1^t); a tensor's factor follows
  double lr;
};

inline int64_t adam_blocks(int64_t numel) { return (numel + kAdamChunk - 1) / kAdamChunk; }

// Launchers: arguments already validated.  Return hipSuccess or the error.
int launch_adam_table(const zero_adam_tensor_t* tensors, int32_t n, void* table,
                      hipStream_t stream);
int launch_tensors_adam(const zero_adam_list_t* list, const ListScalars& sc,
                        const zero_step_result_t* res, hipStream_t stream);
int launch_adam_moments(const zero_adam_list_t* list, void* m, void* v, bool f32,
                        hipStream_t stream);

}  // namespace zk
