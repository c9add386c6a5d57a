// Internal interface between the host side of the head's loss (zero_head.cpp)
// and its kernels (zero_head.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "zero_internal.h"
#include "zero_shard.h"

namespace zk {

constexpr int64_t kHeadTile = 256;  // token and vocabulary rows are padded to whole tiles
constexpr int64_t kHeadStep = 64;   // contraction elements a step stages

// Where things lie in the workspace (byte offsets), and how the work is cut.
struct HeadPlan {
  int64_t tokens_pad;  // tokens rounded up to a tile
  int64_t hidden_pad;  // hidden rounded up to a step: row length of the packed x (and w)
  int64_t parts;       // softmax partials a token gets (one per kHeadPart vocabulary rows)
  int64_t piece;       // vocabulary rows a piece of the gradient takes (whole tiles)
  int64_t kept;        // first row of the last piece
  int32_t split;       // most ways the hidden gradient's contraction is split (at most 64)
  bool few;            // at most kFewTokens tokens (see zero_head_few.hip)
  bool pack_w;         // w's rows do not start on 16-byte boundaries
  // offsets
  size_t state, sums, index, label, lse, dy, x, xt, w, part, picked, g, logits,
      acc, total;
};
constexpr int64_t kHeadPart = 128;
constexpr int32_t kFewTokens = 64;

struct HeadState {  // at offset `state`
  int32_t valid;
  int32_t ticket;
  int64_t bad;
  float coef;      // c, or NaN
  int32_t split;   // ways dx's contraction is split (not for few tokens)
};

HeadPlan head_plan(const zero_head_t* h, bool grad);

// Launchers: arguments already validated.  Return hipSuccess or the error.
// pack: lse_in is NULL when the loss runs in the same call; token_loss and lse
// (of ignored tokens, where not NULL) and grads' dx rows of theirs are written.
// loss: keep leaves the last piece's exponentials for the gradient; grad: kept
// says that they are there.
int launch_head_pack(const zero_head_t* h, const HeadPlan& p, void* ws, const float* lse_in,
                     float* token_loss, float* lse, const zero_head_grads_t* grads,
                     hipStream_t stream);
int launch_head_loss(const zero_head_t* h, const HeadPlan& p, void* ws, float* token_loss,
                     float* lse, bool keep, zero_loss_result_t* res, hipStream_t stream);
int launch_head_grad(const zero_head_t* h, const HeadPlan& p, void* ws,
                     const zero_head_grads_t* grads, bool kept, hipStream_t stream);

// The same for few tokens: pack() and the logits' partial softmax in one launch
// (the logits stay in the workspace if gradients follow), and the gradients
// (have: the loss ran in the same call).
int launch_few_logits(const zero_head_t* h, const HeadPlan& p, void* ws, const float* lse_in,
                      float* token_loss, float* lse, const zero_head_grads_t* grads,
                      hipStream_t stream);
int launch_few_grads(const zero_head_t* h, const HeadPlan& p, void* ws,
                     const zero_head_grads_t* grads, bool have, hipStream_t stream);

}  // namespace zk
