// The head's loss and gradients for up to 64 tokens (short prompts, single
// tokens).
//
// With so few tokens every product is bound by w: the logits and dx read it
// once each, dw writes as much; the arithmetic (128 operations a weight) is an
// eighth of what the matrix cores do in that time.  So w is never staged for
// reuse: the logits take it from memory straight into fragments, each wave its
// own 32 vocabulary rows, with no barrier in the loop; and since the few large
// elements of g would show a 16-bit rounding in the results, g is taken as the
// sum of two 16-bit values, at twice the products.  The fp32 logits of the
// tokens stay in the workspace (256 bytes a vocabulary row), token-contiguous.
// w's rows may start anywhere; nothing is laid out again.
//
//   k_few_logits  logits, and the partial softmax of 128 vocabulary rows; a few
//                 workgroups of the same launch put the valid tokens in order
//                 and transpose x for the gradients (a launch of their own in
//                 front cost 5 us of 50)
//   (join)        as with many tokens
//   k_few_grads   dw tiles, and dx's partial sums over runs of the vocabulary
//   k_few_dx      those sums joined
#include <stddef.h>

#include <type_traits>

#include "head_device.h"

namespace zk {
namespace {

using namespace dev;

constexpr int kThreads4 = 256;  // four waves
constexpr int kT = kFewTokens;  // 64

// Elements [k, k + 8) of a row of n elements; those past its end are zero.
__device__ __forceinline__ s16x8 row8(const uint16_t* row, int32_t k, int32_t n) {
  u32x4 v = {0, 0, 0, 0};
  if (k + 8 <= n) {
    v = *(const u32x4_a2*)(row + k);
  } else if (k < n) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k + e < n) v[e >> 1] |= (uint32_t)row[k + e] << (16 * (e & 1));
  }
  return __builtin_bit_cast(s16x8, v);
}

struct FewLogits {
  const int64_t* labels;
  const uint16_t *x, *w;
  int64_t ldx, ldw, lddx;
  double loss_scale;
  int32_t tokens, vocab, hidden, hidden_pad, mean;
  const float* lse_in;    // or NULL
  float *token_loss, *lse_out;  // or NULL
  uint16_t *xt, *dx;      // NULL: no gradients
  // in the workspace
  int32_t *index, *label;
  float* lse;
  HeadState* state;
  float2* part;
  double* picked;
  float* logits;          // NULL if no gradients follow
};

// The valid tokens in order: lane i of `ok` takes place popcount(ok below i).
__device__ __forceinline__ int32_t place(uint64_t ok, int lane) {
  return __popcll(ok & ((1ull << lane) - 1));
}

// Workgroups of a launch that take pack() instead of logits.
constexpr int32_t kPacks = kT;

// Workgroup r of kPacks: what token r gets if it takes no part; of the r-th
// valid token the label's logit, in fp64 (its rounding to fp32 would be the
// largest error of a short prompt's loss), and x's transpose for the gradients
// (column r, zero past the last); r = 0, the packed tokens' indices and labels.
template <typename T>
__device__ __forceinline__ void pack(const FewLogits& f) {
  const int lane = threadIdx.x & 63;
  const int64_t y = lane < f.tokens ? f.labels[lane] : -1;
  const uint64_t ok = __ballot(y >= 0 && y < f.vocab), bad = __ballot(y >= f.vocab);
  const int32_t valid = __popcll(ok), r = (int32_t)blockIdx.x;
  if (r == 0 && threadIdx.x < 64) {
    if (ok >> lane & 1) {
      const int32_t at = place(ok, lane);
      f.index[at] = lane;
      f.label[at] = (int32_t)y;
      if (f.lse_in) f.lse[at] = f.lse_in[lane];
    }
    if (lane == 0) {
      double c = f.loss_scale;
      if (f.mean) c /= valid > 0 ? (double)valid : 1.0;
      f.state->valid = valid;
      f.state->ticket = 0;
      f.state->bad = __popcll(bad);
      f.state->coef = bad ? __builtin_nanf("") : (float)c;
    }
  }
  if (r < f.tokens && !(ok >> r & 1)) {
    if (threadIdx.x == 0) {
      const float v = bad >> r & 1 ? __builtin_nanf("") : 0.0f;
      if (f.token_loss) f.token_loss[r] = v;
      if (f.lse_out) f.lse_out[r] = v;
    }
    if (f.dx)
      for (int32_t h = threadIdx.x; h < f.hidden; h += kThreads4)
        f.dx[r * f.lddx + h] = bad >> r & 1 ? kNan16 : 0;
  }
  if (r >= valid && !f.xt) return;
  int32_t src = -1;  // the r-th valid token
  uint64_t m = ok;
  for (int32_t i = 0; m; ++i, m &= m - 1)
    if (i == r) src = __ffsll((unsigned long long)m) - 1;
  const uint16_t* w = f.w + (src >= 0 ? __shfl(y, src) : 0) * f.ldw;
  double dot = 0.0;
  for (int32_t c = threadIdx.x; c < f.hidden_pad / 8; c += kThreads4) {
    s16x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
    if (src >= 0) {
      v = row8(f.x + src * f.ldx, 8 * c, f.hidden);
      const s16x8 u = row8(w, 8 * c, f.hidden);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        dot = __builtin_fma((double)widen<T>((uint16_t)v[e]), (double)widen<T>((uint16_t)u[e]),
                            dot);
    }
    if (f.xt)
#pragma unroll
      for (int e = 0; e < 8; ++e) f.xt[(int64_t)(8 * c + e) * kT + r] = (uint16_t)v[e];
  }
  uint32_t none = 0;
  block_tree<kThreads4>(dot, none);
  if (threadIdx.x == 0 && r < valid) f.picked[r] = dot;
}

// Logits of 128 vocabulary rows, 32 a wave: A = w from memory straight into
// fragments, 128 hidden columns (8 KiB a wave) on their way while the last ones
// are multiplied; B = packed x through LDS, since all four waves read it.
// Bound by memory: 128256 x 4096, one token 168 us (6.2 TB/s), 64 tokens 190
// (5.5); 50257 x 1600, 37 tokens 35 us (4.6).  Behind a call that has written a dw
// of 1 GB, whose lines are still on their way out, 64 tokens take 270 us.
//
// Workgroups start at different columns: rows of 4096 columns lie a power of
// two apart, and all workgroups at the same column would ask the same memory
// channels (64 tokens: 183 against 237 us).  Two waves a SIMD and one set of
// columns on its way: three waves were slower (202 against 190 us), three sets
// too (206).  Only as many 16-token columns as there may be tokens are
// multiplied (37 tokens, 50257 x 1600: 38 -> 35 us).
//
// LONG: rows of eight elements or more.  A piece that passes the row's end is
// then loaded from the row's last eight elements, and what does not belong to
// it is taken out later, without a branch around any load: with branches the
// compiler waits for the newest loads where they join (37 tokens, 50257 x 1600:
// 37.4 against 34.8 us; dx of 50 tokens, 1000 x 72, 10.2 against 6.4).
constexpr int kXTile = 128;
template <typename T, int NJ, bool LONG>
__global__ __launch_bounds__(kThreads4) __attribute__((amdgpu_waves_per_eu(2, 2))) void
k_few_logits(const FewLogits f) {
  constexpr int kTokens = 16 * NJ;
  __shared__ int32_t s_src[kT], s_y[kT];
  __shared__ float s_m[4][kTokens], s_s[4][kTokens];
  // [tokens][128 columns]: 16-byte chunk c of row r lies at c ^ (r & 15)
  __shared__ __attribute__((aligned(1024))) char lx[2][kTokens * kXTile * 2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, q = lane & 15;
  if ((int32_t)blockIdx.x < kPacks) return pack<T>(f);
  const int32_t vocab = f.vocab, hidden = f.hidden, block = (int32_t)blockIdx.x - kPacks;
  const int beyond = (8 - hidden % 8) % 8;
  const int64_t v0 = (int64_t)block * kHeadPart + wave * 32;
  // A load covers 8 rows' whole 128-byte lines: lanes of q < 8 take the first
  // half of row q % 8's, the others the second.  The fragments want lane q to
  // hold row q: two loads of 8 rows each trade halves (lines() below).
  const uint16_t* wr[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t v = v0 + 16 * i + 8 * r + (q & 7);
      wr[i][r] = f.w + (v < vocab ? v : vocab - 1) * f.ldw;  // rows past the end are masked below
    }
  const int32_t wk = 8 * (4 * (q >> 3) + g);
  f32x4 acc[2][NJ];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{};
  // LONG: where to load the piece at column k from, and the piece that the row
  // holds (beyond: the columns of the row's end that lie past it)
  auto inside = [&](int32_t k) { return k + 8 <= hidden ? k : hidden - 8; };
  auto held = [&](s16x8 v, int32_t k) {
    if (k >= hidden) return s16x8{};
    return k + 8 > hidden ? drop_first(v, beyond) : v;
  };
  // a[buffer][i][line][rows 0-7 or 8-15]
  s16x8 a[2][2][2][2], xr[NJ];
  auto fetch_w = [&](s16x8 (&d)[2][2][2], int32_t tile) {
    const int32_t k0 = tile * kXTile + wk;
    if constexpr (LONG) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int l = 0; l < 2; ++l) {
            const int32_t k = inside(k0 + 64 * l);
            d[i][l][r] = __builtin_bit_cast(s16x8, *(const u32x4_a2*)(wr[i][r] + k));
          }
    } else if ((tile + 1) * kXTile <= hidden) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int l = 0; l < 2; ++l)
            d[i][l][r] = __builtin_bit_cast(s16x8, *(const u32x4_a2*)(wr[i][r] + k0 + 64 * l));
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int l = 0; l < 2; ++l) d[i][l][r] = row8(wr[i][r], k0 + 64 * l, hidden);
    }
  };
  // the fragments of a line's two halves: lane q < 8 holds row q of its own
  // first load and gets row q's second half from lane q + 8, and so on
  auto lines = [&](const s16x8 (&d)[2], s16x8 (&f)[2]) {
    const u32x4 lo = __builtin_bit_cast(u32x4, d[0]), hi = __builtin_bit_cast(u32x4, d[1]);
    const bool first = q < 8;
    u32x4 x, y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t give = first ? hi[e] : lo[e];
      const uint32_t got =
          (uint32_t)__builtin_amdgcn_update_dpp(0, (int)give, 0x128, 0xF, 0xF, false);
      x[e] = first ? lo[e] : got;
      y[e] = first ? got : hi[e];
    }
    f[0] = __builtin_bit_cast(s16x8, x);
    f[1] = __builtin_bit_cast(s16x8, y);
  };
  // thread: chunk threadIdx % 16 of rows threadIdx / 16 + 16 k
  const int xc = threadIdx.x & 15, xrow = threadIdx.x >> 4;
  const uint16_t* xp[NJ];
  auto fetch_x = [&](int32_t tile) {
    const int32_t c = tile * kXTile + 8 * xc;
    if constexpr (LONG) {
#pragma unroll
      for (int k = 0; k < NJ; ++k)
        xr[k] = __builtin_bit_cast(s16x8, *(const u32x4_a2*)(xp[k] + inside(c)));
    } else if ((tile + 1) * kXTile <= hidden) {
#pragma unroll
      for (int k = 0; k < NJ; ++k) xr[k] = __builtin_bit_cast(s16x8, *(const u32x4_a2*)(xp[k] + c));
    } else {
#pragma unroll
      for (int k = 0; k < NJ; ++k) xr[k] = row8(xp[k], c, hidden);
    }
  };
  auto store_x = [&](char* d, int32_t tile) {
    if (LONG && (tile + 1) * kXTile > hidden) {
#pragma unroll
      for (int k = 0; k < NJ; ++k) xr[k] = held(xr[k], tile * kXTile + 8 * xc);
    }
#pragma unroll
    for (int k = 0; k < NJ; ++k)
      *(s16x8*)(d + (xrow + 16 * k) * 256 + ((xc ^ xrow) << 4)) = xr[k];
  };
  auto use = [&](s16x8 (&d)[2][2][2], const char* l, int32_t tile) {
    if (LONG && (tile + 1) * kXTile > hidden) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            d[i][n][r] = held(d[i][n][r], tile * kXTile + wk + 64 * n);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      s16x8 f[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) lines(d[i][n], f[i]);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const s16x8 b =
              *(const s16x8*)(l + (16 * j + q) * 256 + (((8 * n + 4 * s + g) ^ q) << 4));
#pragma unroll
          for (int i = 0; i < 2; ++i) acc[i][j] = mfma(T{}, f[i][s], b, acc[i][j]);
        }
    }
  };
  // whole pairs; zeros past the end
  const int32_t tiles = (hidden + 2 * kXTile - 1) / (2 * kXTile) * 2;
  const int32_t from = (int32_t)(blockIdx.x / kXcds) % tiles;  // the XCD's workgroups in turn
  auto tile = [&](int32_t t) { return t + from < tiles ? t + from : t + from - tiles; };
  fetch_w(a[0], tile(0));
  // the packed tokens: where their rows of x are, and their labels
  const int64_t own = lane < f.tokens ? f.labels[lane] : -1;
  const uint64_t ok = __ballot(own >= 0 && own < vocab);
  const int32_t valid = __popcll(ok);
  if (valid == 0) return;
  if (wave == 0) {
    if (lane >= valid) {
      s_src[lane] = 0;  // any row: what its columns hold reaches no result
      s_y[lane] = -1;
    }
    if (ok >> lane & 1) {
      s_src[place(ok, lane)] = lane;
      s_y[place(ok, lane)] = (int32_t)own;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NJ; ++k) xp[k] = f.x + s_src[xrow + 16 * k] * f.ldx;
  fetch_x(tile(0));
  store_x(lx[0], tile(0));
  fetch_x(tile(1));
  // tile t is in LDS, and the buffer of the one before is free
  auto turn = [&] { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
  for (int32_t t = 0; t < tiles - 2; t += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      turn();
      fetch_w(a[1 - h], tile(t + h + 1));
      store_x(lx[1 - h], tile(t + h + 1));
      fetch_x(tile(t + h + 2));
      use(a[h], lx[h], tile(t + h));
    }
  }
  turn();
  fetch_w(a[1], tile(tiles - 1));
  store_x(lx[1], tile(tiles - 1));
  use(a[0], lx[0], tile(tiles - 2));
  turn();
  use(a[1], lx[1], tile(tiles - 1));
  const int32_t rows = (int32_t)(vocab - v0 < 32 ? vocab - v0 : 32);
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int32_t t = 16 * j + q;
    const int64_t y = s_y[t] >= 0 ? s_y[t] - v0 : -1;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 16 * i + 4 * g + e;
        float l = acc[i][j][e];
        if (r >= rows) l = -INFINITY;
        if (f.logits && r < rows) f.logits[(v0 + r) * kT + t] = l;
        if (r == y) l = -INFINITY;  // pack() has it
        acc[i][j][e] = l;
        m = __builtin_elementwise_maximum(m, l);
      }
    m = __builtin_elementwise_maximum(m, __shfl_xor(m, 16));
    m = __builtin_elementwise_maximum(m, __shfl_xor(m, 32));
    m = __builtin_ceilf(m * kLog2e);
    const float shift = (m == -INFINITY ? 0.0f : -m) + g_log2<T>();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s += exp2_fast(__builtin_fmaf(acc[i][j][e], kLog2e, shift));
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (lane < 16) {
      s_m[wave][t] = m;
      s_s[wave][t] = s;
    }
  }
  __syncthreads();
  if (wave == 0 && lane < kTokens) {
    float m = s_m[0][lane], s = s_s[0][lane];
#pragma unroll
    for (int k = 1; k < 4; ++k) join(m, s, s_m[k][lane], s_s[k][lane]);
    f.part[(int64_t)block * kT + lane] = float2{m, s};
  }
}

// The tokens' side of g, in LDS: g's scale less the lse, in base 2 (-inf: no
// token), the label's row, and its element e^-loss - 1 (from the loss of the
// same call, which keeps a small one's digits, or from lse).
struct Tokens {
  float shift[kT], dy[kT];
  int32_t y[kT];
};
template <typename T>
__device__ __forceinline__ float g_of(float l, int32_t v, int32_t vocab, float shift, float dy,
                                      int32_t y) {
  if (shift == -INFINITY || v >= vocab) return 0.0f;  // no token, no row
  return v == y ? dy : exp2_fast(__builtin_fmaf(l, kLog2e, shift));
}

// Eight values into their two 16-bit parts.
template <typename T>
__device__ __forceinline__ void two_parts(const float (&v)[8], s16x8& hi, s16x8& lo) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    hi[e] = (short)narrow<T>(v[e]);
    lo[e] = (short)narrow<T>(v[e] - widen<T>((uint16_t)hi[e]));
  }
}

struct FewGrad {
  const float* logits;
  const uint16_t* w;
  int64_t ldw;
  const uint16_t* xt;
  const int32_t* label;
  const float *lse, *dy;  // dy: e^-loss - 1, or NULL
  const double* picked;
  const HeadState* state;
  float* acc;       // dx's partial sums [split][64][hidden_pad]
  void* dw;
  int64_t lddw;
  int32_t vocab, hidden, hidden_pad;
  int32_t dw_blocks, dw_cols;       // workgroups of dw: 64 rows times dw_cols hidden columns
  int32_t split, run;               // dx: vocabulary rows a split takes (whole stages)
  int32_t accumulate;
};

template <typename T>
__device__ __forceinline__ void load_tokens(const FewGrad& f, Tokens& k) {
  const int t = threadIdx.x;
  if (t < kT) {
    const bool there = t < f.state->valid;
    const float z = there ? f.lse[t] : 0.0f;
    k.shift[t] = there ? g_log2<T>() - z * kLog2e : -INFINITY;
    const float dy =
        there ? (f.dy ? f.dy[t] : expm1f((float)(f.picked[t] - (double)z))) : 0.0f;
    k.dy[t] = dy * g_scale<T>();
    k.y[t] = there ? f.label[t] : -1;
  }
  __syncthreads();
}

// dw of 64 vocabulary rows and dw_cols hidden columns: A = x^T (rows: hidden),
// B = g (rows: vocabulary), contraction over the 64 tokens.  A wave takes 64
// columns at a time; its g stays in registers.
template <typename T, bool F32OUT>
__device__ __forceinline__ void few_dw(const FewGrad& f, const Tokens& tok, char* lds,
                                       int32_t block) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, q = lane & 15;
  const int32_t vblocks = (f.vocab + 63) / 64;
  const int32_t v0 = block % vblocks * 64, h1 = (block / vblocks + 1) * f.dw_cols;
  const float c = f.state->coef / g_scale<T>();
  s16x8 hi[2][4], lo[2][4];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float v[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int32_t row = v0 + 16 * j + q;
      const f32x4* p =
          (const f32x4*)(f.logits + (int64_t)(row < f.vocab ? row : 0) * kT + 32 * s + 8 * g);
      const f32x4 a = p[0], b = p[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[j][e] = a[e];
        v[j][4 + e] = b[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int t = 32 * s + 8 * g + e;
      const float shift = tok.shift[t], dy = tok.dy[t];
      const int32_t y = tok.y[t];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j][e] = g_of<T>(v[j][e], v0 + 16 * j + q, f.vocab, shift, dy, y);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) two_parts<T>(v[j], hi[s][j], lo[s][j]);
  }
  char* mine = lds + wave * 8192;  // 64 rows of 64 columns in 16 bits
  for (int32_t h0 = h1 - f.dw_cols + wave * 64; h0 < h1 && h0 < f.hidden; h0 += 256) {
    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint16_t* p = f.xt + (int64_t)(h0 + 16 * i + q) * kT + 8 * g;
      const s16x8 a0 = *(const s16x8*)p, a1 = *(const s16x8*)(p + 32);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
        d = mfma(T{}, a0, lo[0][j], d);
        d = mfma(T{}, a1, lo[1][j], d);
        d = mfma(T{}, a0, hi[0][j], d);
        acc[i][j] = mfma(T{}, a1, hi[1][j], d) * c;
      }
    }
    if (!F32OUT && !f.accumulate) {
      // through this wave's own LDS (in order within a wave), so that the rows
      // leave in 128-byte pieces; 16-byte chunk k of row r lies at k ^ (r & 7)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4& d = acc[i][j];
          const int r = 16 * j + q, k = 2 * i + (g >> 1);
          *(u32x2*)(mine + r * 128 + ((k ^ (r & 7)) << 4) + (g & 1) * 8) =
              narrow4<T>(d[0], d[1], d[2], d[3]);
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = 8 * k + (lane >> 3);
        const u32x4 d = *(const u32x4*)(mine + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
        const int32_t v = v0 + r, h = h0 + (lane & 7) * 8;
        if (v >= f.vocab || h >= f.hidden) continue;
        uint16_t* o = (uint16_t*)f.dw + (int64_t)v * f.lddw + h;
        if (h + 8 <= f.hidden) {
          *(u32x4_a2*)o = d;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (h + e < f.hidden) o[e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int32_t v = v0 + 16 * j + q;
        if (v >= f.vocab) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t h = h0 + 16 * i + 4 * g;
          const int64_t at = (int64_t)v * f.lddw + h;
          f32x4 d = acc[i][j];
          if constexpr (F32OUT) {
            float* o = (float*)f.dw + at;
            if (h + 4 <= f.hidden) {
              if (f.accumulate) d = *(const f32x4_a4*)o + d;
              *(f32x4_a4*)o = d;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (h + e < f.hidden) o[e] = f.accumulate ? o[e] + d[e] : d[e];
            }
          } else {
            uint16_t* o = (uint16_t*)f.dw + at;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (h + e < f.hidden) o[e] = (uint16_t)narrow<T>(widen<T>(o[e]) + d[e]);
          }
        }
      }
    }
  }
}

// dx's partial sums of 256 hidden columns over one run of the vocabulary, 64
// rows at a time: A = w (columns of memory, staged in LDS), B = g, which the
// workgroup forms in LDS from the logits.  The next rows of w and of the
// logits are on their way while these are multiplied.
template <typename T, bool LONG>
__device__ __forceinline__ void few_dx(const FewGrad& f, const Tokens& tok, char* lds,
                                       int32_t block) {
  using FA = Frags<256, true>;
  using FB = Frags<64, false>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t htiles = (f.hidden + 255) / 256;
  const int32_t h0 = block % htiles * 256, ks = block / htiles;
  const int32_t va = ks * f.run, vb = va + f.run < f.vocab ? va + f.run : f.vocab;
  const float shift = tok.shift[lane], dy = tok.dy[lane];
  const int32_t y = tok.y[lane];
  lds_char* lw = (lds_char*)lds;             // w: [64 rows][256 columns], pairs swizzled
  lds_char* lg = (lds_char*)(lds + 32768);   // g: two parts of [64 tokens][64 rows]
  const FA fa(wave * 64, lane);
  const FB fb(0, lane);
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{};
  s16x8 nw[8];
  float nl[16];
  const int32_t column = h0 + (lane & 31) * 8;
  const int beyond = (8 - f.hidden % 8) % 8;  // of a row's last piece
  auto fetch = [&](int32_t v0) {  // w: rows 8k + wave*2 + lane/32
    const uint16_t* p = f.w + (v0 + wave * 2 + (lane >> 5)) * f.ldw + h0;
    const float* l = f.logits + (int64_t)(v0 + wave * 16) * kT + lane;
    if constexpr (LONG) {
      const int32_t c = column + 8 <= f.hidden ? column : f.hidden - 8;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int32_t v = v0 + 8 * k + wave * 2 + (lane >> 5);
        nw[k] = __builtin_bit_cast(
            s16x8, *(const u32x4_a2*)(f.w + (int64_t)(v < f.vocab ? v : f.vocab - 1) * f.ldw + c));
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int32_t v = v0 + wave * 16 + e;
        nl[e] = f.logits[(int64_t)(v < f.vocab ? v : f.vocab - 1) * kT + lane];
      }
    } else if (v0 + kStage <= vb && h0 + 256 <= f.hidden) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        nw[k] = __builtin_bit_cast(s16x8, *(const u32x4_a2*)(p + 8 * k * f.ldw + (lane & 31) * 8));
#pragma unroll
      for (int e = 0; e < 16; ++e) nl[e] = l[e * kT];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        nw[k] = s16x8{};
        if (v0 + 8 * k + wave * 2 + (lane >> 5) < vb)
          nw[k] = row8(p + 8 * k * f.ldw, (lane & 31) * 8, f.hidden - h0);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) nl[e] = v0 + wave * 16 + e < vb ? l[e * kT] : 0.0f;
    }
  };
  if (va < vb) fetch(va);
  for (int32_t v0 = va; v0 < vb; v0 += kStage) {
    __syncthreads();  // the last rows have been multiplied
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = 8 * k + wave * 2 + (lane >> 5);
      const int c = (lane & 31) ^ ((r & 3) << 2 | (r >> 3 & 1) << 1);
      // what columns past the row's end hold reaches no column of dx
      if (LONG && beyond && column < f.hidden && column + 8 > f.hidden)
        nw[k] = drop_first(nw[k], beyond);
      *(__attribute__((address_space(3))) s16x8*)(lw + r * 512 + c * 16) = nw[k];
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = g_of<T>(nl[8 * p + e], v0 + wave * 16 + 8 * p + e, vb, shift, dy, y);
      s16x8 hi, lo;
      two_parts<T>(v, hi, lo);
      lds_char* o = lg + lane * 128 + (((2 * wave + p) ^ (lane >> 1 & 7)) << 4);
      *(__attribute__((address_space(3))) s16x8*)o = hi;
      *(__attribute__((address_space(3))) s16x8*)(o + 8192) = lo;
    }
    if (v0 + kStage < vb) fetch(v0 + kStage);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      s16x8 a[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = fa.load(lw, i, s);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const s16x8 hi = fb.load(lg, j, s), lo = fb.load(lg + 8192, j, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i][j] = mfma(T{}, a[i], lo, acc[i][j]);
          acc[i][j] = mfma(T{}, a[i], hi, acc[i][j]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int32_t h = h0 + wave * 64 + 16 * i + 4 * (lane >> 4);
      if (h < f.hidden_pad)
        *(f32x4*)(f.acc + ((int64_t)ks * kT + 16 * j + (lane & 15)) * f.hidden_pad + h) = acc[i][j];
    }
}

// Workgroups of dx first: they run longest.  Bound by memory: 64 tokens, 128256 x
// 4096, 440 to 500 us (w read, dw written: 4.2 to 4.8 TB/s), and 8 tokens hardly
// less, since all of this is 64 tokens wide.  A dw in fp32 0.75 ms, accumulated
// 1.24 ms; in 16 bits accumulated, element by element, 2.1 ms.
template <typename T, bool F32OUT, bool LONG>
__global__ __launch_bounds__(kThreads4) void k_few_grads(FewGrad f, int32_t dx_blocks) {
  __shared__ __attribute__((aligned(1024))) char lds[49152];
  __shared__ Tokens tok;
  load_tokens<T>(f, tok);
  if ((int32_t)blockIdx.x < dx_blocks) few_dx<T, LONG>(f, tok, lds, blockIdx.x);
  else few_dw<T, F32OUT>(f, tok, lds, blockIdx.x - dx_blocks);
}

// dx: the splits' sums, 64 lanes of four columns, four waves sharing the splits.
template <typename T>
__global__ __launch_bounds__(kThreads4) void k_few_dx(
    const float* __restrict__ acc, int32_t split, int32_t hidden_pad, int32_t hidden,
    const int32_t* __restrict__ index, const HeadState* __restrict__ state,
    uint16_t* __restrict__ dx, int64_t lddx) {
  __shared__ f32x4 s_sum[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t r = blockIdx.y, h = (blockIdx.x * 64 + lane) * 4;
  if (r >= state->valid) return;
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (h < hidden) {
    const float* p = acc + (int64_t)r * hidden_pad + h;
#pragma unroll 8
    for (int32_t k = wave; k < split; k += 4)
      s += *(const f32x4*)(p + (int64_t)k * kT * hidden_pad);
  }
  s_sum[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || h >= hidden) return;
  s = (s_sum[0][lane] + s_sum[1][lane]) + (s_sum[2][lane] + s_sum[3][lane]);
  const float c = state->coef / g_scale<T>();
  uint16_t* o = dx + (int64_t)index[r] * lddx + h;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (h + e < hidden) o[e] = (uint16_t)narrow<T>(s[e] * c);
}

template <typename T>
int logits_t(const zero_head_t* h, const HeadPlan& p, void* ws, const float* lse_in,
             float* token_loss, float* lse, const zero_head_grads_t* gr, hipStream_t stream) {
  FewLogits f{};
  f.labels = h->labels;
  f.x = (const uint16_t*)h->x;
  f.w = (const uint16_t*)h->w;
  f.ldx = h->ldx;
  f.ldw = h->ldw;
  f.loss_scale = h->loss_scale;
  f.tokens = (int32_t)h->tokens;
  f.vocab = (int32_t)h->vocab;
  f.hidden = (int32_t)h->hidden;
  f.hidden_pad = (int32_t)p.hidden_pad;
  f.mean = h->mean;
  f.lse_in = lse_in;
  f.token_loss = token_loss;
  f.lse_out = lse;
  if (gr) {
    f.xt = at<uint16_t>(ws, p.xt);
    f.dx = (uint16_t*)gr->dx;
    f.lddx = gr->lddx;
    f.logits = at<float>(ws, p.logits);
  }
  f.index = at<int32_t>(ws, p.index);
  f.label = at<int32_t>(ws, p.label);
  f.lse = at<float>(ws, p.lse);
  f.state = at<HeadState>(ws, p.state);
  f.part = at<float2>(ws, p.part);
  f.picked = at<double>(ws, p.picked);
  const int columns = (int)((h->tokens + 15) / 16);
  const auto pick = [&](auto whole) {
    constexpr bool W = decltype(whole)::value;
    return columns <= 1   ? k_few_logits<T, 1, W>
           : columns == 2 ? k_few_logits<T, 2, W>
           : columns == 3 ? k_few_logits<T, 3, W>
                          : k_few_logits<T, 4, W>;
  };
  const auto kernel = h->hidden >= 8 ? pick(std::true_type{}) : pick(std::false_type{});
  hipLaunchKernelGGL(kernel, dim3((uint32_t)(kPacks + (h->vocab + kHeadPart - 1) / kHeadPart)),
                     dim3(kThreads4), 0, stream, f);
  return (int)hipGetLastError();
}

template <typename T>
int grads_t(const zero_head_t* h, const HeadPlan& p, void* ws, const zero_head_grads_t* gr,
            bool have, hipStream_t stream) {
  FewGrad f{};
  f.logits = at<const float>(ws, p.logits);
  f.w = (const uint16_t*)h->w;
  f.ldw = h->ldw;
  f.xt = at<const uint16_t>(ws, p.xt);
  f.label = at<const int32_t>(ws, p.label);
  f.lse = at<const float>(ws, p.lse);
  f.dy = have ? at<const float>(ws, p.dy) : nullptr;
  f.picked = at<const double>(ws, p.picked);
  f.state = at<const HeadState>(ws, p.state);
  f.acc = at<float>(ws, p.acc);
  f.dw = gr->dw;
  f.lddw = gr->lddw;
  f.vocab = (int32_t)h->vocab;
  f.hidden = (int32_t)h->hidden;
  f.hidden_pad = (int32_t)p.hidden_pad;
  f.accumulate = gr->accumulate;
  const int32_t vblocks = (f.vocab + 63) / 64, htiles = (f.hidden + 255) / 256;
  // dw: all columns by one workgroup (g is formed once) unless that leaves CUs idle
  int32_t parts = (1024 + vblocks - 1) / vblocks;
  if (parts > htiles) parts = htiles;
  f.dw_cols = (htiles + parts - 1) / parts * 256;
  f.dw_blocks = vblocks * ((f.hidden + f.dw_cols - 1) / f.dw_cols);
  f.split = p.split;
  f.run = (int32_t)(((h->vocab + p.split - 1) / p.split + kStage - 1) / kStage * kStage);
  const int32_t dx_blocks = h->tokens > 0 ? htiles * f.split : 0;
  const bool f32 = gr->dw_dtype == ZERO_F32;
  const auto kernel = h->hidden >= 8
                          ? (f32 ? k_few_grads<T, true, true> : k_few_grads<T, false, true>)
                          : (f32 ? k_few_grads<T, true, false> : k_few_grads<T, false, false>);
  hipLaunchKernelGGL(kernel, dim3((uint32_t)(dx_blocks + f.dw_blocks)), dim3(kThreads4), 0, stream,
                     f, dx_blocks);
  ZK_LAUNCHED();
  if (h->tokens > 0)
    hipLaunchKernelGGL(k_few_dx<T>, dim3((uint32_t)htiles, (uint32_t)h->tokens), dim3(kThreads4), 0,
                       stream, f.acc, f.split, f.hidden_pad, f.hidden,
                       at<const int32_t>(ws, p.index), f.state, (uint16_t*)gr->dx, gr->lddx);
  return (int)hipGetLastError();
}

}  // namespace

int launch_few_logits(const zero_head_t* h, const HeadPlan& p, void* ws, const float* lse_in,
                      float* token_loss, float* lse, const zero_head_grads_t* gr,
                      hipStream_t stream) {
  return h->dtype == ZERO_BF16 ? logits_t<BF16>(h, p, ws, lse_in, token_loss, lse, gr, stream)
                               : logits_t<FP16>(h, p, ws, lse_in, token_loss, lse, gr, stream);
}

int launch_few_grads(const zero_head_t* h, const HeadPlan& p, void* ws,
                     const zero_head_grads_t* gr, bool have, hipStream_t stream) {
  return h->dtype == ZERO_BF16 ? grads_t<BF16>(h, p, ws, gr, have, stream)
                               : grads_t<FP16>(h, p, ws, gr, have, stream);
}

}  // namespace zk
