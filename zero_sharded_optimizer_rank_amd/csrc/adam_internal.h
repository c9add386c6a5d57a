// Internal interface between the host side of the list update (zero_adam.cpp)
// and its kernels (zero_adam.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "zero_internal.h"
#include "zero_shard.h"

namespace zk {

// Threads of a workgroup and 4-element quads of a thread, for moments in 32 and in
// 8 bits; bytes of LDS that the 32-bit kernel reserves and never touches, so that a
// CU holds 20 of its one-wave workgroups: the seven streams of more waves get in
// each other's way.  Llama-3 block (218 M elements, bf16 gradients): 32 bits, one wave
// with one quad, 32 / 20 / 16 / 13 / 12 a CU 1025 / 975 / 971 / 1048 / 1086 us, GPT-2
// (1.56 G) 7.20 / 6.90 / 6.95 / 7.45 / 7.70 ms; two or four quads a thread 1000 and 1092
// us, four waves with one 1050.  8 bits, limited by the vector units as much as by
// memory: one wave with one quad 618 us, with two or four 598; four waves with one, two,
// four quads 617, 598, 605; fewer a CU, no faster.
constexpr int kAdamThreads32 = 64, kAdamQuads32 = 1, kAdamLds32 = 8192;
constexpr int kAdamThreads8 = 256, kAdamQuads8 = 2;
// Elements of a launch: long grids run slower the longer they are (GPT-2, in launches
// of 2^26 / 2^27 / 2^28 / in one: 32 bits 6.90 / 6.87 / 6.94 / 7.14 ms; 8 bits, 2^25 / 2^27
// / 2^28 / one: 4.78 / 4.76 / 4.82 / 5.01).
constexpr int64_t kAdamLaunch = (int64_t)1 << 27;
// Elements a workgroup updates.
constexpr int64_t kAdamChunk32 = 4 * kAdamThreads32 * kAdamQuads32;
constexpr int64_t kAdamChunk8 = 4 * kAdamThreads8 * kAdamQuads8;
// Elements of one key of the dither; a chunk lies within one.
constexpr int kKeyShift = 12;
static_assert(((int64_t)1 << kKeyShift) % kAdamChunk8 == 0, "one key a workgroup");

// A tensor as the kernels read it, in the device table: entries [n], then the
// first workgroups [n] of the kernel for 32-bit moments, and those of the one for
// 8-bit moments (32 bits each; a tensor of the other kind has none).
struct AdamEntry {
  const void* grad;
  float* master;
  void *m, *v;
  uint8_t *m_exp, *v_exp;
  void* param;
  int64_t numel, offset;
  double weight_decay, lr_scale;
  uint32_t kind;  // grad dtype | param dtype << 2 (3: none)
  uint32_t reserved;
};

struct ListScalars {
  float b1, omb1, b2, omb2, eps, sqrt_bc2;
  float inv_root, inv_root_low;  // 1 / sqrt(1 - b2^t), and 2^-12 of it
  float scale;       // 1 / loss_scale
  uint32_t key;      // the seed, mixed once
  double step_size;  // lr / (1 - b1^t); a tensor's factor follows
  double lr;
};

inline int64_t adam_blocks(int64_t numel, bool small) {
  const int64_t chunk = small ? kAdamChunk8 : kAdamChunk32;
  return (numel + chunk - 1) / chunk;
}

// Launchers: arguments already validated.  Return hipSuccess or the error.
int launch_adam_table(const zero_adam_tensor_t* tensors, int32_t n, void* table,
                      hipStream_t stream);
int launch_tensors_adam(const zero_adam_list_t* list, const ListScalars& sc,
                        const zero_step_result_t* res, hipStream_t stream);
int launch_adam_moments(const zero_adam_list_t* list, void* m, void* v, bool f32,
                        hipStream_t stream);

}  // namespace zk
