// Host side of the head's loss: argument checks and the workspace plan.
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "head_internal.h"
#include "host_internal.h"
#include "zero_shard.h"

using namespace zk::host;
using zk::kHeadTile;

namespace {

int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
int64_t clamp(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }
// Largest vocabulary of the form for few tokens, which keeps their fp32 logits
// for the gradient (256 bytes a vocabulary row: 512 MiB).
constexpr int64_t kFewVocab = (int64_t)1 << 21;

bool good_sizes(const zero_head_t* h) {
  return h->tokens >= 0 && h->tokens <= ZERO_HEAD_MAX_TOKENS && h->hidden >= 1 &&
         h->hidden <= ZERO_HEAD_MAX_HIDDEN && h->vocab >= 1 && h->vocab <= ZERO_HEAD_MAX_VOCAB &&
         h->ldx >= h->hidden && h->ldx <= ZERO_HEAD_MAX_HIDDEN && h->ldw >= h->hidden &&
         h->ldw <= ZERO_HEAD_MAX_HIDDEN && (h->dtype == ZERO_F16 || h->dtype == ZERO_BF16) &&
         // one launch takes all tiles of the logits, 512 threads each, of at most 2^32 - 1
         up(h->tokens, kHeadTile) / kHeadTile * (up(h->vocab, kHeadTile) / kHeadTile) <
             ZERO_HEAD_MAX_TILES;
}

int check_head(const zero_head_t* h) {
  if (!h) return fail(ZERO_EINVAL, "head is NULL");
  if (!good_sizes(h))
    return fail(ZERO_EINVAL, "head sizes: tokens %lld hidden %lld vocab %lld ldx %lld ldw %lld "
                "dtype %d", (long long)h->tokens, (long long)h->hidden, (long long)h->vocab,
                (long long)h->ldx, (long long)h->ldw, h->dtype);
  if (!(h->loss_scale > 0.0) || !isfinite(h->loss_scale))
    return fail(ZERO_EINVAL, "loss_scale must be finite and > 0");
  if (!h->w || (h->tokens > 0 && (!h->x || !h->labels)))
    return fail(ZERO_EINVAL, "x, w or labels is NULL");
  if (!aligned(h->x, 2) || !aligned(h->w, 2) || !aligned(h->labels, 8))
    return fail(ZERO_EALIGN, "x and w must be 2-byte, labels 8-byte aligned");
  return ZERO_OK;
}

int check_workspace(const zero_head_t* h, bool grad, void* ws, size_t ws_bytes) {
  if (!ws) return fail(ZERO_EINVAL, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(ZERO_EALIGN, "workspace not 256-byte aligned");
  const size_t need = zk::head_plan(h, grad).total;
  if (ws_bytes < need) return fail(ZERO_ENOSPC, "workspace %zu bytes < %zu", ws_bytes, need);
  return ZERO_OK;
}

int check_loss_out(const float* token_loss, const float* lse, const zero_loss_result_t* res) {
  if (!res) return fail(ZERO_EINVAL, "dev_result is NULL");
  if (!aligned(res, 8)) return fail(ZERO_EALIGN, "dev_result not 8-byte aligned");
  if (!aligned(token_loss, 4) || !aligned(lse, 4))
    return fail(ZERO_EALIGN, "token_loss and lse must be 4-byte aligned");
  return ZERO_OK;
}

size_t span(int64_t rows, int64_t ld, int64_t cols, size_t elem) {
  return rows > 0 ? elem * (size_t)((rows - 1) * ld + cols) : 0;
}

int check_grads(const zero_head_t* h, const zero_head_grads_t* g, const float* lse) {
  if (!g) return fail(ZERO_EINVAL, "grads is NULL");
  if (!g->dw || (h->tokens > 0 && !g->dx)) return fail(ZERO_EINVAL, "dx or dw is NULL");
  if (g->lddx < h->hidden || g->lddw < h->hidden || g->lddx > ZERO_HEAD_MAX_HIDDEN ||
      g->lddw > ZERO_HEAD_MAX_HIDDEN)
    return fail(ZERO_EINVAL, "lddx %lld, lddw %lld", (long long)g->lddx, (long long)g->lddw);
  if (g->dw_dtype != h->dtype && g->dw_dtype != ZERO_F32)
    return fail(ZERO_EINVAL, "dw_dtype %d: the type of w or fp32", g->dw_dtype);
  const size_t ew = g->dw_dtype == ZERO_F32 ? 4 : 2;
  if (!aligned(g->dx, 2) || !aligned(g->dw, ew))
    return fail(ZERO_EALIGN, "dx and dw must be aligned to their elements");
  const int64_t T = h->tokens, V = h->vocab, H = h->hidden;
  struct Range { const void* p; size_t n; const char* name; };
  const Range out[2] = {{g->dx, span(T, g->lddx, H, 2), "dx"}, {g->dw, span(V, g->lddw, H, ew), "dw"}};
  const Range in[4] = {{h->x, span(T, h->ldx, H, 2), "x"}, {h->w, span(V, h->ldw, H, 2), "w"},
                       {h->labels, 8 * (size_t)T, "labels"}, {lse, 4 * (size_t)T, "lse"}};
  for (const Range& o : out)
    for (const Range& i : in)
      if (o.n && i.n && i.p && overlap(o.p, o.n, i.p, i.n))
        return fail(ZERO_EINVAL, "%s overlaps %s", o.name, i.name);
  if (out[0].n && overlap(out[0].p, out[0].n, out[1].p, out[1].n))
    return fail(ZERO_EINVAL, "dx overlaps dw");
  return ZERO_OK;
}

}  // namespace

namespace zk {

HeadPlan head_plan(const zero_head_t* h, bool grad) {
  HeadPlan p{};
  p.hidden_pad = up(h->hidden, kHeadStep);
  p.few = h->tokens <= kFewTokens && h->vocab <= kFewVocab;
  // an empty batch has its join, and its dw to clear: a tile's room at least
  p.tokens_pad = p.few ? kFewTokens : up(h->tokens > 0 ? h->tokens : 1, kHeadTile);
  p.pack_w = !p.few && (h->hidden % 8 != 0 || h->ldw % 8 != 0 || !aligned(h->w, 16));
  const int64_t vocab_pad = up(h->vocab, kHeadTile);
  p.parts = vocab_pad / kHeadPart;
  const int64_t htiles = up(h->hidden, kHeadTile) / kHeadTile;
  if (grad && p.few) {
    // dx: two rounds of the 256 CUs' workgroups (two a CU fit), of at least two stages each
    p.split = (int32_t)clamp((512 + htiles - 1) / htiles, 1, up(h->vocab, 128) / 128);
  } else if (grad) {
    // a piece's block of g stays within 1 GiB: with all 128256 rows of a
    // Llama-3 head up to 4096 tokens go in one piece, whose logits are formed
    // once, and every further doubling of the tokens halves the piece, down to
    // 16 tiles of rows (131072 tokens), whose products still fill the CUs
    int64_t piece = ((int64_t)1 << 29) / p.tokens_pad / kHeadTile * kHeadTile;
    piece = clamp(piece, 16 * kHeadTile, vocab_pad);
    const int64_t pieces = (vocab_pad + piece - 1) / piece;
    p.piece = up((vocab_pad + pieces - 1) / pieces, kHeadTile);
    p.kept = (h->vocab - 1) / p.piece * p.piece;
    // dx: up to four rounds of the 256 CUs (how many is settled on the device,
    // which knows the valid tokens)
    const int64_t tiles = p.tokens_pad / kHeadTile * htiles;
    p.split = (int32_t)clamp((1024 + tiles - 1) / tiles, 1,
                             p.piece / kHeadTile < 64 ? p.piece / kHeadTile : 64);
  }
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t o = at;
    at += (size_t)(bytes + 255) / 256 * 256;
    return o;
  };
  p.state = take(sizeof(HeadState));
  p.sums = take(8 * (p.tokens_pad / 16));
  p.index = take(4 * p.tokens_pad);
  p.label = take(4 * p.tokens_pad);
  p.lse = take(4 * p.tokens_pad);
  p.dy = take(4 * p.tokens_pad);
  p.picked = take(8 * p.tokens_pad);
  p.x = take(p.few ? 0 : 2 * p.tokens_pad * p.hidden_pad);
  p.xt = take(grad && p.few ? 2 * p.tokens_pad * p.hidden_pad : 0);
  p.w = take(p.pack_w ? 2 * h->vocab * p.hidden_pad : 0);
  p.part = take(8 * p.parts * p.tokens_pad);
  if (grad) {
    p.g = take(2 * p.tokens_pad * p.piece);
    p.logits = take(p.few ? 4 * kFewTokens * h->vocab : 0);
    p.acc = take(4 * p.split * p.tokens_pad * p.hidden_pad);
  }
  p.total = at;
  return p;
}

}  // namespace zk

extern "C" {

size_t zero_head_workspace_bytes(const zero_head_t* head, int32_t grad) {
  if (!head || !good_sizes(head)) return 0;
  // A batch of fewer tokens can need more: a piece of g shrinks where the
  // vocabulary takes one piece more, and dx's splits are whole.  The plan
  // changes by the tile, and at kFewTokens.
  zero_head_t h = *head;
  size_t need = 0;
  const auto count = [&](int64_t tokens) {
    h.tokens = tokens < head->tokens ? tokens : head->tokens;
    const size_t n = zk::head_plan(&h, grad != 0).total;
    if (n > need) need = n;
  };
  count(zk::kFewTokens);
  for (int64_t t = 0; t < head->tokens; t += kHeadTile) count(t + kHeadTile);
  return need;
}

int zero_head_loss(const zero_head_t* head, float* token_loss, float* lse, void* workspace,
                   size_t ws_bytes, zero_loss_result_t* dev_result, hipStream_t stream) {
  g_err[0] = 0;
  int rc = check_head(head);
  if (!rc) rc = check_loss_out(token_loss, lse, dev_result);
  if (!rc) rc = check_workspace(head, false, workspace, ws_bytes);
  if (rc) return rc;
  const zk::HeadPlan p = zk::head_plan(head, false);
  int e = zk::launch_head_pack(head, p, workspace, nullptr, token_loss, lse, nullptr, stream);
  if (!e) e = zk::launch_head_loss(head, p, workspace, token_loss, lse, false, dev_result, stream);
  return hip_status(e, "head_loss launch");
}

int zero_head_grad(const zero_head_t* head, const float* lse, const zero_head_grads_t* grads,
                   void* workspace, size_t ws_bytes, hipStream_t stream) {
  g_err[0] = 0;
  int rc = check_head(head);
  if (!rc && head->tokens > 0 && !lse) rc = fail(ZERO_EINVAL, "lse is NULL");
  if (!rc && !aligned(lse, 4)) rc = fail(ZERO_EALIGN, "lse not 4-byte aligned");
  if (!rc) rc = check_grads(head, grads, lse);
  if (!rc) rc = check_workspace(head, true, workspace, ws_bytes);
  if (rc) return rc;
  const zk::HeadPlan p = zk::head_plan(head, true);
  int e = zk::launch_head_pack(head, p, workspace, lse, nullptr, nullptr, grads, stream);
  if (!e) e = zk::launch_head_grad(head, p, workspace, grads, false, stream);
  return hip_status(e, "head_grad launch");
}

int zero_head_loss_grad(const zero_head_t* head, float* token_loss, float* lse,
                        const zero_head_grads_t* grads, void* workspace, size_t ws_bytes,
                        zero_loss_result_t* dev_result, hipStream_t stream) {
  g_err[0] = 0;
  int rc = check_head(head);
  if (!rc) rc = check_loss_out(token_loss, lse, dev_result);
  if (!rc) rc = check_grads(head, grads, lse);
  if (!rc) rc = check_workspace(head, true, workspace, ws_bytes);
  if (rc) return rc;
  const zk::HeadPlan p = zk::head_plan(head, true);
  int e = zk::launch_head_pack(head, p, workspace, nullptr, token_loss, lse, grads, stream);
  if (!e) e = zk::launch_head_loss(head, p, workspace, token_loss, lse, true, dev_result, stream);
  if (!e) e = zk::launch_head_grad(head, p, workspace, grads, true, stream);
  return hip_status(e, "head_loss_grad launch");
}

}  // extern "C"
