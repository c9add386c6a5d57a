// Host side of the gated feed-forward block: argument checks and the workspace
// plan.
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "ffn_internal.h"
#include "host_internal.h"
#include "zero_shard.h"

using namespace zk::host;

namespace {

int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
int64_t tiles(int64_t x, int64_t tile) { return (x + tile - 1) / tile; }

bool good_ld(int64_t ld, int64_t width) { return ld >= width && ld <= ZERO_FFN_MAX_WIDTH; }

bool good_sizes(const zero_ffn_t* f) {
  return f->tokens >= 0 && f->tokens <= ZERO_FFN_MAX_TOKENS && f->hidden >= 1 &&
         f->hidden <= ZERO_FFN_MAX_WIDTH && f->inner >= 1 && f->inner <= ZERO_FFN_MAX_WIDTH &&
         good_ld(f->ldx, f->hidden) && good_ld(f->ld_gate, f->hidden) &&
         good_ld(f->ld_up, f->hidden) && good_ld(f->ld_down, f->inner) &&
         (f->dtype == ZERO_F16 || f->dtype == ZERO_BF16) && f->act >= ZERO_ACT_SILU &&
         f->act <= ZERO_ACT_RELU &&
         // tiles of one launch, 512 threads each, of at most 2^32 - 1
         tiles(f->tokens, 256) * tiles(f->inner, 128) < ZERO_FFN_MAX_TILES &&
         tiles(f->tokens, 256) * tiles(f->hidden, 256) < ZERO_FFN_MAX_TILES &&
         3 * tiles(f->inner, 256) * tiles(f->hidden, 256) < ZERO_FFN_MAX_TILES;
}

int check_ffn(const zero_ffn_t* f) {
  if (!f) return fail(ZERO_EINVAL, "ffn is NULL");
  if (!good_sizes(f))
    return fail(ZERO_EINVAL, "ffn sizes: tokens %lld hidden %lld inner %lld ld %lld %lld %lld %lld "
                "dtype %d act %d", (long long)f->tokens, (long long)f->hidden,
                (long long)f->inner, (long long)f->ldx, (long long)f->ld_gate,
                (long long)f->ld_up, (long long)f->ld_down, f->dtype, f->act);
  if (!f->w_gate || !f->w_up || !f->w_down || (f->tokens > 0 && !f->x))
    return fail(ZERO_EINVAL, "x or a weight is NULL");
  if (!aligned(f->x, 2) || !aligned(f->w_gate, 2) || !aligned(f->w_up, 2) ||
      !aligned(f->w_down, 2))
    return fail(ZERO_EALIGN, "x and the weights must be 2-byte aligned");
  return ZERO_OK;
}

int check_saved(const zero_ffn_t* f, const zero_ffn_saved_t* s) {
  if (s->ld < up(f->inner, 8) || s->ld % 8 || s->ld > ZERO_FFN_MAX_WIDTH)
    return fail(ZERO_EINVAL, "rows of act, slope, low and h %lld apart", (long long)s->ld);
  if (f->tokens > 0 && (!s->act || !s->slope || !s->low || !s->h))
    return fail(ZERO_EINVAL, "act, slope, low or h is NULL");
  if (!aligned(s->act, 16) || !aligned(s->slope, 16) || !aligned(s->low, 16) || !aligned(s->h, 16))
    return fail(ZERO_EALIGN, "act, slope, low and h must be 16-byte aligned");
  return ZERO_OK;
}

struct Range {
  const void* p;
  size_t n;
  const char* name;
};
Range matrix(const void* p, int64_t rows, int64_t ld, int64_t cols, size_t elem, const char* name) {
  return {p, p && rows > 0 ? elem * (size_t)((rows - 1) * ld + cols) : 0, name};
}

// No output over another output, an input or the workspace.
int check_apart(const Range* out, int n_out, const Range* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < i; ++j)
      if (out[i].n && out[j].n && overlap(out[i].p, out[i].n, out[j].p, out[j].n))
        return fail(ZERO_EINVAL, "%s overlaps %s", out[i].name, out[j].name);
    for (int j = 0; j < n_in; ++j)
      if (out[i].n && in[j].n && overlap(out[i].p, out[i].n, in[j].p, in[j].n))
        return fail(ZERO_EINVAL, "%s overlaps %s", out[i].name, in[j].name);
  }
  return ZERO_OK;
}

int check_workspace(size_t need, const void* ws, size_t ws_bytes) {
  if (!ws) return fail(ZERO_EINVAL, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(ZERO_EALIGN, "workspace not 256-byte aligned");
  if (ws_bytes < need) return fail(ZERO_ENOSPC, "workspace %zu bytes < %zu", ws_bytes, need);
  return ZERO_OK;
}

// Rows that 16-byte loads do not fit.
bool ragged(const void* p, int64_t ld, int64_t width) {
  return width % 8 != 0 || ld % 8 != 0 || !aligned(p, 16);
}

// A product's tiles and their stages; small tiles share a CU by two.
struct Work {
  int64_t count, stages;
};
Work work(int64_t rows, int64_t cols, int64_t k, bool small) {
  const int64_t t = small ? 128 : 256;
  return {tiles(rows, t) * tiles(cols, t), tiles(k, zk::kFfnStep)};
}
int64_t places(bool small) { return small ? 512 : 256; }

// Ways to split a contraction whose output has few tiles: up to three quarters of
// a round of them, of at least four stages each (more parts cost more in their
// fp32 sums than idle CUs do: 512 x 4096 x 14336, 32 tiles, in 4 / 6 / 7 / 9 parts 203 /
// 197 / 200 / 216 us a forward pass; 1024 x 1600 x 6400, 28 tiles, in 3 / 5 / 7 / 9 108 / 99
// / 98 / 100).
int32_t split_of(const Work& w, bool small) {
  int64_t s = places(small) * 3 / 4 / (w.count > 0 ? w.count : 1);
  if (s > w.stages / 4) s = w.stages / 4;
  return (int32_t)(s < 1 ? 1 : s);
}
// Parts of dx where other tiles share the launch and fill up behind: a part is about as
// long as what a CU gets of the whole (1024 x 1600 x 6400, 200 stages of 44 a CU, in 3 /
// 4 / 5 / 9 parts 279 / 259 / 266 / 280 us a training pass; 512 x 4096 x 14336, 448 of 112,
// in 3 / 4 / 5 / 6 593 / 562 / 568 / 591).
int32_t split_beside(const Work& w, int64_t other_stages) {
  const int64_t all = w.count * w.stages + other_stages;
  const int64_t s = w.stages * places(false) / (all > 0 ? all : 1);
  const int32_t most = split_of(w, false);
  return (int32_t)(s > most ? most : s < 1 ? 1 : s);
}
// Parts of the products of one launch of small tiles: about as long as what one of
// three quarters of the places gets of the whole, and at least four stages.
int64_t part_length(int64_t all_stages) {
  const int64_t each = tiles(all_stages, places(true) * 3 / 4);
  return each > 4 ? each : 4;
}
int32_t parts_of(const Work& w, int64_t length) {
  const int64_t s = w.stages / length;
  return (int32_t)(s < 1 ? 1 : s > 64 ? 64 : s);
}
int64_t sums_bytes(int64_t rows, int64_t cols, int64_t parts) {
  return parts > 1 ? 4 * parts * up(rows, 256) * up(cols, 256) : 0;
}

}  // namespace

namespace zk {

FfnPlan ffn_plan(const zero_ffn_t* f, const zero_ffn_grads_t* g) {
  FfnPlan p{};
  const int64_t T = f->tokens, H = f->hidden, F = f->inner;
  p.hidden_pad = up(H, 8);
  p.inner_pad = up(F, 8);
  p.few = !g && T <= kFfnFew && H >= 8 && F >= 8;  // whole 16-byte loads
  p.low = p.few && T <= kFfnLow;
  if (!p.few) {
    p.pack_x = ragged(f->x, f->ldx, H);
    p.pack_gate = ragged(f->w_gate, f->ld_gate, H);
    p.pack_up = ragged(f->w_up, f->ld_up, H);
    p.pack_down = ragged(f->w_down, f->ld_down, F);
    p.pack_dy = g && ragged(g->dy, g->lddy, H);
  }
  // Small tiles where the large ones would leave half of the CUs idle (100 x 4096 x 14336,
  // 112 tiles, forward 130 -> 107 us; 1024 x 1600 x 6400, 200 tiles, 88 -> 100), in a
  // backward pass also where a CU's share is short, so that a tile's start and end weigh
  // (300 x 1600 x 6400, training, first launch 168 -> 145 us, second 149 -> 144; 512 x 4096 x
  // 14336 587 -> 607 and 588 -> 706), and for y and the second backward launch of up to one
  // small tile's tokens (y: 100 x 4096 x 14336, forward 111 -> 107, 200 x 4096 x 14336 135 ->
  // 143; training 318 -> 304 and 426 -> 470; 64 x 8192 x 28672 1005 -> 1007).
  const auto all = [](const Work& w) { return w.count * w.stages; };
  Work in = work(2 * F, T, H, false), dh = work(F, T, H, false), dw = work(F, H, T, false);
  Work dx = work(T, H, 2 * F, false);
  p.small_in = in.count < 128;
  p.small_out = T <= 128;
  p.small_back1 = dh.count + dw.count < 128 || all(dh) + all(dw) < 24 * 256;
  p.small_back2 = T <= 128 || dx.count + 2 * dw.count < 128 || all(dx) + 2 * all(dw) < 24 * 256;
  p.split_in = p.split_y = p.split_dh = p.split_dw1 = p.split_dx = p.split_dw2 = 1;
  if (!p.few && !g) {
    p.split_y = split_of(work(T, H, F, p.small_out), p.small_out);
    in = work(2 * F, T, H, true);
    if (p.small_in) p.split_in = parts_of(in, part_length(all(in)));
  }
  // (what a call does not want is counted all the same: the plan does not depend on it)
  if (g && p.small_back1) {
    const Work d = work(F, T, H, true), w = work(F, H, T, true);
    const int64_t length = part_length(all(d) + all(w));
    p.split_dh = parts_of(d, length);
    p.split_dw1 = parts_of(w, length);
  }
  if (g && p.small_back2) {
    const Work d = work(T, H, 2 * F, true), w = work(F, H, T, true);
    const int64_t length = part_length(all(d) + 2 * all(w));
    p.split_dx = parts_of(d, length);
    p.split_dw2 = parts_of(w, length);
  } else if (g) {
    p.split_dx = split_beside(dx, 2 * all(dw));
  }
  if (p.few) {
    // Sets of the first product by the rounds that its workgroups take on the 256 CUs, one a
    // CU; at a tie four, which fetch x half as often (12 tokens, two and four sets: 2048 x
    // 8192 32 and 39 us a forward pass, 4096 x 11008 81 and 63, 8192 x 22016 208 and 232).
    const auto rounds = [&](int64_t sets) { return tiles(tiles(F, 16 * sets), 256) * sets; };
    p.few_sets_in = rounds(2) < rounds(4) ? 2 : 4;
    // Sets of the second: four where its rows are many, so that h is fetched half as often (40
    // and 60 tokens, two and four sets: 8192 x 28672 278 and 270, 303 and 287 us a forward
    // pass; 4096 x 14336 79 and 79, 87 and 85; 2048 x 8192 37 and 38, 41 and 41); with fewer
    // rows either is ahead by a few percent (1024 x 4096 23.5 and 24.4, 26.2 and 26.0; 1600 x
    // 6400 36.2 and 35.4, 39.5 and 38.3; 768 x 2048 22.3 and 22.4, 24.8 and 24.0).
    p.few_sets_out = H >= 2048 ? 4 : 2;
    // Up to 8 tokens' x and h come from the L2 as fast, and the waves need not wait for one
    // another, unless the products are large and the tokens more than 4 (8 tokens, not
    // shared and shared: 768 x 2048 13 and 20 us, 4096 x 8192 49 and 58, 4096 x 14336 82 and
    // 72, 8192 x 28672 284 and 258).  Up to 4 tokens never: one token 71 and 72 at 4096 x 14336,
    // 248 and 259 at 8192 x 28672; at four the 3% of 4096 x 14336 (74.5 and 72.5; 8192 x 28672
    // 258 and 258, 4096 x 11008 60 and 63) are left for the simpler rule.
    if (T <= 4 || (T <= 8 && (H < 2048 || F <= 8192)))
      p.few_sets_in = p.few_sets_out = 1;
    if (p.few_sets_out > 1) {
      const int64_t blocks = tiles(H, 32 * p.few_sets_out), steps = tiles(F, kFewTile);
      const int64_t most = steps * p.few_sets_out / (2 * 8);  // two steps a slice at least
      int64_t s = 256 / blocks;
      if (s > most) s = most;
      p.split_y = (int32_t)(s < 1 ? 1 : s);
    }
  }
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t o = at;
    at += (size_t)(bytes + 255) / 256 * 256;
    return o;
  };
  p.x = take(p.pack_x ? 2 * T * p.hidden_pad : 0);
  p.w_gate = take(p.pack_gate ? 2 * F * p.hidden_pad : 0);
  p.w_up = take(p.pack_up ? 2 * F * p.hidden_pad : 0);
  p.w_down = take(p.pack_down ? 2 * H * p.inner_pad : 0);
  p.dy = take(p.pack_dy ? 2 * T * p.hidden_pad : 0);
  p.h = take(g ? 0 : 2 * T * p.inner_pad);
  p.h_low = take(p.low ? 2 * T * p.inner_pad : 0);
  if (g) {
    p.dg = take(2 * T * p.inner_pad);
    p.du = take(2 * T * p.inner_pad);
  }
  // the launches' sums, one launch's after the other's
  int64_t sums;
  if (p.few) {
    sums = p.split_y > 1 ? 4 * p.split_y * T * p.hidden_pad : 0;
  } else if (!g) {
    const int64_t one = 2 * sums_bytes(F, T, p.split_in), two = sums_bytes(H, T, p.split_y);
    sums = one > two ? one : two;
  } else {
    const int64_t one = sums_bytes(F, T, p.split_dh) + sums_bytes(F, H, p.split_dw1);
    const int64_t two = sums_bytes(H, T, p.split_dx) + 2 * sums_bytes(F, H, p.split_dw2);
    sums = one > two ? one : two;
  }
  p.acc = take(sums);
  p.total = at > 0 ? at : 256;
  return p;
}

}  // namespace zk

extern "C" {

size_t zero_ffn_workspace_bytes(const zero_ffn_t* ffn, const zero_ffn_grads_t* grads) {
  if (!ffn || !good_sizes(ffn) || (grads && !good_ld(grads->lddy, ffn->hidden))) return 0;
  // a batch of fewer tokens may be cut into more parts; the plan changes by the stage
  // of 64
  zero_ffn_t f = *ffn;
  size_t need = 0;
  const auto count = [&](int64_t tokens) {
    f.tokens = tokens < ffn->tokens ? tokens : ffn->tokens;
    const size_t n = zk::ffn_plan(&f, grads).total;
    if (n > need) need = n;
  };
  for (int64_t t = 1; t <= zk::kFfnFew; ++t) count(t);
  for (int64_t t = zk::kFfnFew; t < ffn->tokens; t += zk::kFfnStep) count(t + zk::kFfnStep);
  return need;
}

int zero_ffn_forward(const zero_ffn_t* ffn, void* y, int64_t ldy, const zero_ffn_saved_t* saved,
                     void* workspace, size_t ws_bytes, hipStream_t stream) {
  g_err[0] = 0;
  int rc = check_ffn(ffn);
  if (rc) return rc;
  const int64_t T = ffn->tokens, H = ffn->hidden, F = ffn->inner;
  if (T > 0 && !y) return fail(ZERO_EINVAL, "y is NULL");
  if (!good_ld(ldy, H)) return fail(ZERO_EINVAL, "ldy %lld", (long long)ldy);
  if (!aligned(y, 2)) return fail(ZERO_EALIGN, "y must be 2-byte aligned");
  if (saved) rc = check_saved(ffn, saved);
  if (rc) return rc;
  const zk::FfnPlan p = zk::ffn_plan(ffn, nullptr);
  rc = check_workspace(p.total, workspace, ws_bytes);
  if (rc) return rc;
  const int64_t Fp = p.inner_pad;
  const zero_ffn_saved_t none = {nullptr, nullptr, nullptr, nullptr, 0}, *s = saved ? saved : &none;
  const Range out[6] = {matrix(y, T, ldy, H, 2, "y"), matrix(s->act, T, s->ld, Fp, 2, "act"),
                        matrix(s->slope, T, s->ld, Fp, 2, "slope"),
                        matrix(s->low, T, s->ld, Fp, 2, "low"),
                        matrix(s->h, T, s->ld, Fp, 2, "h"), {workspace, p.total, "workspace"}};
  const Range in[4] = {matrix(ffn->x, T, ffn->ldx, H, 2, "x"),
                       matrix(ffn->w_gate, F, ffn->ld_gate, H, 2, "w_gate"),
                       matrix(ffn->w_up, F, ffn->ld_up, H, 2, "w_up"),
                       matrix(ffn->w_down, H, ffn->ld_down, F, 2, "w_down")};
  rc = check_apart(out, 6, in, 4);
  if (rc || T == 0) return rc;
  const int e = p.few ? zk::launch_ffn_few(ffn, p, workspace, y, ldy, saved, stream)
                      : zk::launch_ffn_forward(ffn, p, workspace, y, ldy, saved, stream);
  return hip_status(e, "ffn_forward launch");
}

int zero_ffn_backward(const zero_ffn_t* ffn, const zero_ffn_saved_t* saved,
                      const zero_ffn_grads_t* g, void* workspace, size_t ws_bytes,
                      hipStream_t stream) {
  g_err[0] = 0;
  int rc = check_ffn(ffn);
  if (rc) return rc;
  const int64_t T = ffn->tokens, H = ffn->hidden, F = ffn->inner;
  if (!saved || !g) return fail(ZERO_EINVAL, "saved or grads is NULL");
  rc = check_saved(ffn, saved);
  if (rc) return rc;
  if (g->dw_dtype != ffn->dtype && g->dw_dtype != ZERO_F32)
    return fail(ZERO_EINVAL, "dw_dtype %d: the type of the weights or fp32", g->dw_dtype);
  if (T > 0 && !g->dy) return fail(ZERO_EINVAL, "dy is NULL");
  if (!good_ld(g->lddy, H) || (g->dx && !good_ld(g->lddx, H)) ||
      (g->dw_gate && !good_ld(g->lddw_gate, H)) || (g->dw_up && !good_ld(g->lddw_up, H)) ||
      (g->dw_down && !good_ld(g->lddw_down, F)))
    return fail(ZERO_EINVAL, "rows of the gradients %lld %lld %lld %lld %lld apart",
                (long long)g->lddy, (long long)g->lddx, (long long)g->lddw_gate,
                (long long)g->lddw_up, (long long)g->lddw_down);
  const size_t ew = g->dw_dtype == ZERO_F32 ? 4 : 2;
  if (!aligned(g->dy, 2) || !aligned(g->dx, 2) || !aligned(g->dw_gate, ew) ||
      !aligned(g->dw_up, ew) || !aligned(g->dw_down, ew))
    return fail(ZERO_EALIGN, "gradients must be aligned to their elements");
  const zk::FfnPlan p = zk::ffn_plan(ffn, g);
  rc = check_workspace(p.total, workspace, ws_bytes);
  if (rc) return rc;
  const int64_t Fp = p.inner_pad;
  const Range out[5] = {matrix(g->dx, T, g->lddx, H, 2, "dx"),
                        matrix(g->dw_gate, F, g->lddw_gate, H, ew, "dw_gate"),
                        matrix(g->dw_up, F, g->lddw_up, H, ew, "dw_up"),
                        matrix(g->dw_down, H, g->lddw_down, F, ew, "dw_down"),
                        {workspace, p.total, "workspace"}};
  const Range in[9] = {matrix(ffn->x, T, ffn->ldx, H, 2, "x"),
                       matrix(ffn->w_gate, F, ffn->ld_gate, H, 2, "w_gate"),
                       matrix(ffn->w_up, F, ffn->ld_up, H, 2, "w_up"),
                       matrix(ffn->w_down, H, ffn->ld_down, F, 2, "w_down"),
                       matrix(g->dy, T, g->lddy, H, 2, "dy"),
                       matrix(saved->act, T, saved->ld, Fp, 2, "act"),
                       matrix(saved->slope, T, saved->ld, Fp, 2, "slope"),
                       matrix(saved->low, T, saved->ld, Fp, 2, "low"),
                       matrix(saved->h, T, saved->ld, Fp, 2, "h")};
  rc = check_apart(out, 5, in, 9);
  if (rc) return rc;
  return hip_status(zk::launch_ffn_backward(ffn, p, workspace, saved, g, stream),
                    "ffn_backward launch");
}

}  // extern "C"
