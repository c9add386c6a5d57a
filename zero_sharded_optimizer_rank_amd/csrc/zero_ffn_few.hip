// The feed-forward block's forward pass for up to 64 tokens (single tokens,
// short prompts).
//
// Both products are bound by the weights, which are read once: 128 operations a
// weight at 64 tokens.  So no weight is staged: a wave takes 16 rows' pieces
// from memory straight into fragments, 128 columns at a time, the next ones on
// their way while the last are multiplied; x (and h) come from the L2 the same
// way.  A workgroup has 16 rows (of both projections: 16 + 16) and its waves
// share the contraction, so that a projection of 4096 x 14336 gives 3584 waves;
// their sums are joined through LDS in a fixed order, where the activation and
// the rounding are.  Rows may start anywhere.
#include <stddef.h>

#include "ffn_device.h"

namespace zk {
namespace {

using namespace dev;

constexpr int kTile = 128;  // columns of a wave's step: two whole 128-byte lines a row

struct Few {
  const uint16_t *w0, *w1;  // gate and up, or down
  int64_t ldw0, ldw1;
  const uint16_t* x;        // [tokens, k]
  int64_t ldx;
  int32_t rows, k, tokens, act;
  uint16_t* out;            // [tokens, rows], rows ldo apart
  int64_t ldo;
  uint16_t *gate, *up;      // or NULL
  int64_t lds;
  int32_t pad;              // PAIR: columns of h, gate and up; those past the rows are zero
};

// Elements [c, c + 8) of a row of n < 8 elements.
__device__ __forceinline__ s16x8 short_row(const uint16_t* row, int32_t c, int32_t n) {
  return __builtin_bit_cast(s16x8, take8(row + c, c < n ? n - c : 0));
}

template <typename T, int NJ, int WAVES, bool PAIR, bool LONG>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(2, 2))) void
k_ffn_few(const Few a) {
  constexpr int NI = PAIR ? 2 : 1;
  static_assert(NJ <= WAVES, "a thread for every quad");
  __shared__ f32x4 s_sum[WAVES][NI * NJ][64];
  const int lane = threadIdx.x & 63, g = lane >> 4, q = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t r0 = (int32_t)blockIdx.x * 16, k = a.k;
  // A load covers 8 rows' whole 128-byte lines: lanes of q < 8 take the first half
  // of row q % 8's, the others the second; the fragments want lane q to hold row q,
  // so two loads of 8 rows trade halves (fragments()).
  const uint16_t* wr[NI][2];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int32_t r = r0 + 8 * h + (q & 7);
      wr[i][h] = (i ? a.w1 : a.w0) + (int64_t)(r < a.rows ? r : a.rows - 1) * (i ? a.ldw1 : a.ldw0);
    }
  const uint16_t* xr[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int32_t t = 16 * j + q;
    xr[j] = a.x + (int64_t)(t < a.tokens ? t : a.tokens - 1) * a.ldx;
  }
  const int32_t wk = 8 * (4 * (q >> 3) + g);
  const int beyond = (8 - k % 8) % 8;
  // A piece that passes the row's end is loaded from the row's last eight elements;
  // what does not belong to it is taken out before it is used.
  auto inside = [&](int32_t c) { return c + 8 <= k ? c : k - 8; };
  auto load = [&](const uint16_t* row, int32_t c) {
    if constexpr (LONG) return __builtin_bit_cast(s16x8, *(const u32x4_a2*)(row + inside(c)));
    else return short_row(row, c, k);
  };
  auto held = [&](s16x8 v, int32_t c) {
    if (c >= k) return s16x8{};
    return LONG && c + 8 > k ? drop_first(v, beyond) : v;
  };
  f32x4 acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{};
  struct Step {
    s16x8 w[NI][2][2];  // [line][rows 0-7 or 8-15]
    s16x8 x[4][NJ];
  };
  auto fetch = [&](Step& d, int32_t tile) {
    const int32_t c = tile * kTile;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int l = 0; l < 2; ++l)
#pragma unroll
        for (int h = 0; h < 2; ++h) d.w[i][l][h] = load(wr[i][h], c + 64 * l + wk);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < NJ; ++j) d.x[s][j] = load(xr[j], c + 32 * s + 8 * g);
  };
  auto fragments = [&](const s16x8 (&d)[2], s16x8 (&f)[2]) {
    const u32x4 lo = __builtin_bit_cast(u32x4, d[0]), hi = __builtin_bit_cast(u32x4, d[1]);
    const bool first = q < 8;
    u32x4 u, v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t give = first ? hi[e] : lo[e];
      const uint32_t got =
          (uint32_t)__builtin_amdgcn_update_dpp(0, (int)give, 0x128, 0xF, 0xF, false);
      u[e] = first ? lo[e] : got;
      v[e] = first ? got : hi[e];
    }
    f[0] = __builtin_bit_cast(s16x8, u);
    f[1] = __builtin_bit_cast(s16x8, v);
  };
  auto use = [&](Step& d, int32_t tile) {
    const int32_t c = tile * kTile;
    if (c + kTile > k) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int l = 0; l < 2; ++l)
#pragma unroll
          for (int h = 0; h < 2; ++h) d.w[i][l][h] = held(d.w[i][l][h], c + 64 * l + wk);
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < NJ; ++j) d.x[s][j] = held(d.x[s][j], c + 32 * s + 8 * g);
    }
#pragma unroll
    for (int l = 0; l < 2; ++l)
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        s16x8 f[2];
        fragments(d.w[i][l], f);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int j = 0; j < NJ; ++j) acc[i][j] = mfma(T{}, f[s], d.x[2 * l + s][j], acc[i][j]);
      }
  };
  // The wave's steps: every WAVES-th, from another place in each workgroup, since rows
  // of a power of two columns would all ask the same memory channels.  What is
  // fetched past the last one is the last one again, from the cache.
  const int32_t tiles = (k + kTile - 1) / kTile;
  const int32_t count = wave < tiles ? (tiles - wave + WAVES - 1) / WAVES : 0;
  if (count > 0) {
    const int32_t from = (int32_t)(blockIdx.x / kXcds) % count;
    auto tile = [&](int32_t i) {
      i = (i < count ? i : count - 1) + from;
      return (i < count ? i : i - count) * WAVES + wave;
    };
    Step d[2];
    fetch(d[0], tile(0));
    for (int32_t i = 0; i < count; i += 2) {
      fetch(d[1], tile(i + 1));
      use(d[0], tile(i));
      fetch(d[0], tile(i + 2));
      if (i + 1 < count) use(d[1], tile(i + 1));
    }
  }
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) s_sum[wave][i * NJ + j][lane] = acc[i][j];
  __syncthreads();
  if (wave >= NJ) return;
  const int32_t t = 16 * wave + q, r = r0 + 4 * g;
  f32x4 sum[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    sum[i] = s_sum[0][i * NJ + wave][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum[i] += s_sum[w][i * NJ + wave][lane];
  }
  if (t >= a.tokens) return;
  if constexpr (PAIR) {
    if (r >= a.pad) return;
    f32x4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (r + e >= a.rows) sum[0][e] = sum[1][e] = 0.0f;
    with_act(a.act, [&](auto act) {
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = activated(act, sum[0][e]) * sum[1][e];
    });
    *(u32x2*)(a.out + t * a.ldo + r) = narrow4<T>(h[0], h[1], h[2], h[3]);
    if (a.gate) {
      *(u32x2*)(a.gate + t * a.lds + r) = narrow4<T>(sum[0][0], sum[0][1], sum[0][2], sum[0][3]);
      *(u32x2*)(a.up + t * a.lds + r) = narrow4<T>(sum[1][0], sum[1][1], sum[1][2], sum[1][3]);
    }
  } else {
    uint16_t* o = a.out + t * a.ldo + r;
    const u32x2 v = narrow4<T>(sum[0][0], sum[0][1], sum[0][2], sum[0][3]);
    if (r + 4 <= a.rows) {
      *(u32x2_a2*)o = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (r + e < a.rows) o[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
  }
}

template <typename T, int NJ, int WAVES, bool PAIR>
int few_k(const Few& a, hipStream_t stream) {
  const dim3 grid((uint32_t)((a.rows + 15) / 16)), block(64 * WAVES);
  if (a.k >= 8)
    hipLaunchKernelGGL((k_ffn_few<T, NJ, WAVES, PAIR, true>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((k_ffn_few<T, NJ, WAVES, PAIR, false>), grid, block, 0, stream, a);
  return (int)hipGetLastError();
}

template <typename T, int NJ>
int few_j(const Few& in, const Few& out, hipStream_t stream) {
  const int e = few_k<T, NJ, 4, true>(in, stream);
  return e ? e : few_k<T, NJ, 8, false>(out, stream);
}

template <typename T>
int few_t(const zero_ffn_t* f, const FfnPlan& p, void* ws, void* y, int64_t ldy,
          const zero_ffn_saved_t* saved, hipStream_t stream) {
  uint16_t* h = at<uint16_t>(ws, p.h);
  Few in{};
  in.w0 = (const uint16_t*)f->w_gate;
  in.w1 = (const uint16_t*)f->w_up;
  in.ldw0 = f->ld_gate;
  in.ldw1 = f->ld_up;
  in.x = (const uint16_t*)f->x;
  in.ldx = f->ldx;
  in.rows = (int32_t)f->inner;
  in.k = (int32_t)f->hidden;
  in.tokens = (int32_t)f->tokens;
  in.act = f->act;
  in.out = h;
  in.ldo = p.inner_pad;
  in.pad = (int32_t)p.inner_pad;
  if (saved) {
    in.gate = (uint16_t*)saved->gate;
    in.up = (uint16_t*)saved->up;
    in.lds = saved->ld;
  }
  Few out{};
  out.w0 = out.w1 = (const uint16_t*)f->w_down;
  out.ldw0 = out.ldw1 = f->ld_down;
  out.x = h;
  out.ldx = p.inner_pad;
  out.rows = (int32_t)f->hidden;
  out.k = (int32_t)f->inner;
  out.tokens = (int32_t)f->tokens;
  out.out = (uint16_t*)y;
  out.ldo = ldy;
  if (f->tokens <= 16) return few_j<T, 1>(in, out, stream);
  if (f->tokens <= 32) return few_j<T, 2>(in, out, stream);
  return few_j<T, 4>(in, out, stream);
}

}  // namespace

int launch_ffn_few(const zero_ffn_t* f, const FfnPlan& p, void* ws, void* y, int64_t ldy,
                   const zero_ffn_saved_t* saved, hipStream_t stream) {
  return f->dtype == ZERO_BF16 ? few_t<BF16>(f, p, ws, y, ldy, saved, stream)
                               : few_t<FP16>(f, p, ws, y, ldy, saved, stream);
}

}  // namespace zk
