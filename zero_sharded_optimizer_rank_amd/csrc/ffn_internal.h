// Internal interface between the host side of the gated feed-forward block
// (zero_ffn.cpp) and its kernels (zero_ffn.hip, zero_ffn_few.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "zero_internal.h"
#include "zero_shard.h"

namespace zk {

constexpr int64_t kFfnTile = 256;
constexpr int64_t kFfnStep = 64;   // contraction elements a step stages
constexpr int32_t kFfnFew = 64;    // most tokens of the form that streams the weights
constexpr int32_t kFfnLow = 16;    // most tokens whose h is kept in two parts there
constexpr int kFewTile = 128;      // columns of a wave's step there: two lines of a row

// Where things lie in the workspace (byte offsets), and how the work is cut.
struct FfnPlan {
  int64_t hidden_pad, inner_pad;  // row lengths of packed matrices: multiples of 8
  bool few, low;
  bool pack_x, pack_gate, pack_up, pack_down, pack_dy;  // rows that no 16-byte loads fit
  bool small_in, small_out, small_back1, small_back2;  // 128 x 128 tiles, else 256 x 256
  // parts that a product's contraction is cut into; small tiles: any, large: y and dx
  int32_t split_in, split_y, split_dh, split_dw1, split_dx, split_dw2;
  int32_t few_sets_in, few_sets_out;  // few: sets of rows of a workgroup, 2 or 4; both 1: x is
                                      // not shared
  // offsets
  size_t x, w_gate, w_up, w_down, dy, h, h_low, dg, du, acc, total;
};
FfnPlan ffn_plan(const zero_ffn_t* f, const zero_ffn_grads_t* g);

// Launchers: arguments already validated.  Return hipSuccess or the error.
int launch_ffn_forward(const zero_ffn_t* f, const FfnPlan& p, void* ws, void* y, int64_t ldy,
                       const zero_ffn_saved_t* saved, hipStream_t stream);
int launch_ffn_few(const zero_ffn_t* f, const FfnPlan& p, void* ws, void* y, int64_t ldy,
                   const zero_ffn_saved_t* saved, hipStream_t stream);
int launch_ffn_backward(const zero_ffn_t* f, const FfnPlan& p, void* ws,
                        const zero_ffn_saved_t* saved, const zero_ffn_grads_t* g,
                        hipStream_t stream);

}  // namespace zk
