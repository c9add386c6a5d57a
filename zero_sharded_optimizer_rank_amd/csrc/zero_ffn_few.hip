// The feed-forward block's forward pass for up to 64 tokens (single tokens,
// short prompts).
//
// Both products are bound by the weights, which are read once: 128 operations a
// weight at 64 tokens.  So no weight is staged: a wave takes 32 rows' pieces (16
// of each projection) from memory straight into fragments, 128 columns at a time,
// the next ones on their way while the last are multiplied.  Rows may start anywhere.
//   up to 4 or 8 tokens  k_ffn_direct  the waves of a workgroup share the contraction
//   more                 k_ffn_shared  x (and h) go through LDS, and waves of the same
//                                      columns share them: fetched by each wave from the
//                                      L2 they would be twice the weights' bytes at 64
//                                      tokens (4096 x 14336: 184 us a pass, so 87).
//                                      Eight waves are R sets of rows by 8 / R slices of
//                                      the contraction, joined through LDS in a fixed
//                                      order; the second product's, whose rows are few,
//                                      is also split over workgroups (k_ffn_few_join)
// One token of 4096 x 14336 in bf16 takes 66 us (352 MB of weights, 5.3 TB/s), 37 tokens of
// 1600 x 6400 in fp16 30 (61 MB; about 20 of them are the launches' start and end), 22 of
// 8192 x 28672 259 (5.4 TB/s).
//
// With few tokens the outputs are few, and a second rounding on the way to them shows (y
// is off by 2.3e-3 in bf16 where its own rounding alone is 1.7e-3).  Up to 16 tokens h
// therefore is kept in two 16-bit parts, the second what the first one's rounding left:
// without more products up to 8 tokens, whose second parts are the columns that have
// no token, with twice as many of the second product for more, which still wait for the
// weights (16 tokens, 1600 x 6400: 30.4 -> 31.9 us).  From 24 on it would cost 8%.
#include <stddef.h>

#include "ffn_device.h"

namespace zk {
namespace {

using namespace dev;

constexpr int kWaves = 8;

struct Few {
  const uint16_t *w0, *w1;  // PAIR: gate and up; else w0
  int64_t ldw0, ldw1;
  const uint16_t* x;        // [tokens, k]
  int64_t ldx;
  const uint16_t* x_low;    // else: what x's rounding left, or NULL; rows ldx_low apart
  int64_t ldx_low;
  int32_t rows, k, tokens, act, split;
  Kept to;                  // PAIR
  uint16_t* h_low;          // PAIR: what h's rounding leaves, rows pad apart, or NULL
  int32_t pad;              // PAIR: columns of h; those past the rows are zero
  uint16_t* out;            // else, split = 1: [tokens, rows], rows ldo apart
  int64_t ldo;
  float* acc;               // else: [split][tokens][pad]
};

// The piece [c, c + 8) of a row of k >= 8 elements.  One that passes the row's end is
// loaded from the row's last eight elements, without a branch around the load, and
// what does not belong to it is taken out before it is used (held8; beyond: (8 - k %
// 8) % 8).
__device__ __forceinline__ s16x8 row8(const uint16_t* row, int32_t c, int32_t k) {
  return __builtin_bit_cast(s16x8, *(const u32x4_a2*)(row + (c + 8 <= k ? c : k - 8)));
}
__device__ __forceinline__ s16x8 held8(s16x8 v, int32_t c, int32_t k, int beyond) {
  if (c >= k) return s16x8{};
  return c + 8 > k ? drop_first(v, beyond) : v;
}

// A load covers 8 rows' whole 128-byte lines: lanes with q = lane % 16 < 8 take the
// first half of row q % 8's, the others the second; a fragment wants lane q to hold
// row q, so two loads of 8 rows trade halves.
__device__ __forceinline__ void fragments(const s16x8 (&d)[2], s16x8 (&f)[2], bool first) {
  const u32x4 lo = __builtin_bit_cast(u32x4, d[0]), hi = __builtin_bit_cast(u32x4, d[1]);
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
}

// Both projections' sums of four rows r .. of token t: h, and what is kept.  Rows
// past the last give zeros.
template <typename T, typename A>
__device__ __forceinline__ void leave_pair(const Few& a, A act, f32x4 g, f32x4 u, int32_t t,
                                           int32_t r) {
  f32x4 h, v, b;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float slope;
    v[e] = activated(act, g[e], slope);
    b[e] = u[e] * slope;
    h[e] = v[e] * u[e];
    if (r + e >= a.rows) h[e] = v[e] = b[e] = 0.0f;
  }
  if (t >= a.tokens || r >= a.pad) return;
  const int64_t at = t * a.to.ld + r;
  const u32x2 h16 = narrow4<T>(h[0], h[1], h[2], h[3]);
  *(u32x2*)(a.to.h + at) = h16;
  if (a.h_low) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float rest = h[e] - widen<T>(h16[e >> 1] >> (16 * (e & 1)) & 0xFFFFu);
      // infinity and NaN are h's to hand on
      h[e] = __builtin_fabsf(rest) < __builtin_inff() ? rest : 0.0f;
    }
    *(u32x2*)(a.h_low + (int64_t)t * a.pad + r) = narrow4<T>(h[0], h[1], h[2], h[3]);
  }
  if (a.to.act) {
    const Kept4 k = keep4(v, b);
    *(u32x2*)(a.to.act + at) = k.act;
    *(u32x2*)(a.to.slope + at) = k.slope;
    *(u32x2*)(a.to.low + at) = k.low;
  }
}
// Sums over h's two parts.  Where an infinite weight meets a second part of zero that sum
// is NaN; the first part's is what h gives there.
__device__ __forceinline__ float both(float s, float low) {
  return __builtin_fabsf(s) < __builtin_inff() ? s + low : s;
}
// Four columns of an output row that holds n.
template <typename T>
__device__ __forceinline__ void leave4(uint16_t* row, int32_t r, int32_t n, f32x4 s) {
  const u32x2 v = narrow4<T>(s[0], s[1], s[2], s[3]);
  if (r + 4 <= n) {
    *(u32x2_a2*)(row + r) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (r + e < n) row[r + e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
  }
}

// Up to 8 tokens: 16 rows a workgroup (of both projections: 16 + 16), whose waves share
// the contraction; x comes from the L2 straight into fragments.  More than two waves a
// SIMD were slower (one token, 4096 x 14336: two or three 70, four 86 us a forward pass),
// and so were 8 waves for the first product (74).
template <typename T, int WAVES, bool PAIR>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(2, 2))) void
k_ffn_direct(const Few a) {
  constexpr int NI = PAIR ? 2 : 1;
  __shared__ f32x4 s_sum[WAVES][NI][64];
  const int lane = threadIdx.x & 63, g = lane >> 4, q = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t r0 = (int32_t)blockIdx.x * 16, k = a.k;
  const uint16_t* wr[NI][2];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int32_t r = r0 + 8 * h + (q & 7);
      const int64_t at = r < a.rows ? r : a.rows - 1;
      wr[i][h] = i ? a.w1 + at * a.ldw1 : a.w0 + at * a.ldw0;
    }
  // columns 8 to 15 of the product have no token: they take what h's rounding left
  const bool low = !PAIR && q >= 8;
  const int32_t token = (PAIR ? q : q & 7) < a.tokens ? (PAIR ? q : q & 7) : a.tokens - 1;
  const uint16_t* xr = low ? a.x_low + token * a.ldx_low : a.x + token * a.ldx;
  const int32_t wk = 8 * (4 * (q >> 3) + g);
  const int beyond = (8 - k % 8) % 8;
  f32x4 acc[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) acc[i] = f32x4{};
  struct Step {
    s16x8 w[NI][2][2];  // [line][rows 0-7 or 8-15]
    s16x8 x[4];
  };
  auto fetch = [&](Step& d, int32_t tile) {
    const int32_t c = tile * kFewTile;
#pragma unroll
    for (int s = 0; s < 4; ++s) d.x[s] = row8(xr, c + 32 * s + 8 * g, k);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int l = 0; l < 2; ++l)
#pragma unroll
        for (int h = 0; h < 2; ++h) d.w[i][l][h] = row8(wr[i][h], c + 64 * l + wk, k);
  };
  auto use = [&](Step& d, int32_t tile) {
    const int32_t c = tile * kFewTile;
    if (c + kFewTile > k) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int l = 0; l < 2; ++l)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            d.w[i][l][h] = held8(d.w[i][l][h], c + 64 * l + wk, k, beyond);
#pragma unroll
      for (int s = 0; s < 4; ++s) d.x[s] = held8(d.x[s], c + 32 * s + 8 * g, k, beyond);
    }
#pragma unroll
    for (int l = 0; l < 2; ++l)
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        s16x8 f[2];
        fragments(d.w[i][l], f, q < 8);
#pragma unroll
        for (int s = 0; s < 2; ++s) acc[i] = mfma(T{}, f[s], d.x[2 * l + s], acc[i]);
      }
  };
  // The wave's steps: every WAVES-th, from another place in each workgroup, since rows
  // of a power of two columns would all ask the same memory channels.  What is
  // fetched past the last one is the last one again, from the cache.
  const int32_t tiles = (k + kFewTile - 1) / kFewTile;
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
  for (int i = 0; i < NI; ++i) s_sum[wave][i][lane] = acc[i];
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int w = 1; w < WAVES; ++w) acc[i] += s_sum[w][i][lane];
  const int32_t r = r0 + 4 * g;
  if constexpr (PAIR) {
    with_act(a.act, [&](auto act) { leave_pair<T>(a, act, acc[0], acc[1], q, r); });
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)  // lane q + 8's
      acc[0][e] = both(acc[0][e], __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
                                      0, (int)__float_as_uint(acc[0][e]), 0x128, 0xF, 0xF, false)));
    if (q < a.tokens && r < a.rows) leave4<T>(a.out + q * a.ldo, r, a.rows, acc[0]);
  }
}

// More tokens: x goes through LDS.
template <typename T, int NJ, int R, bool PAIR, bool LOW>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2))) void
k_ffn_shared(const Few a) {
  constexpr int NI = 2, S = kWaves / R, XROWS = 16 * NJ * (LOW ? 2 : 1);
  constexpr int XLOADS = XROWS > 4 * R ? XROWS / (4 * R) : 1;
  constexpr int kTileBytes = XROWS * 2 * kFewTile, kSums = kWaves * NI * NJ * 1024;
  constexpr int kLds = 2 * S * kTileBytes > kSums ? 2 * S * kTileBytes : kSums;
  __shared__ __attribute__((aligned(1024))) char lds[kLds];
  const int lane = threadIdx.x & 63, g = lane >> 4, q = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int set = wave % R, slice = wave / R;
  const int32_t k = a.k;
  const int32_t block = (int32_t)(blockIdx.x / (uint32_t)a.split);
  const int32_t part = (int32_t)(blockIdx.x % (uint32_t)a.split);
  const int32_t r0 = (block * R + set) * (PAIR ? 16 : 16 * NI);
  const uint16_t* wr[NI][2];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int32_t r = r0 + (PAIR ? 0 : 16 * i) + 8 * h + (q & 7);
      const int64_t at = r < a.rows ? r : a.rows - 1;
      wr[i][h] = PAIR && i ? a.w1 + at * a.ldw1 : a.w0 + at * a.ldw0;
    }
  const int32_t wk = 8 * (4 * (q >> 3) + g);
  // x: thread of a slice's sets loads chunk % 16 of rows / 16
  const int xt = set * 64 + lane, xc = xt & 15;
  const uint16_t* xr[XLOADS];
#pragma unroll
  for (int n = 0; n < XLOADS; ++n) {
    const int32_t t = (xt >> 4) + 4 * R * n;
    const int32_t own = t % (16 * NJ) < a.tokens ? t % (16 * NJ) : a.tokens - 1;
    xr[n] = LOW && t >= 16 * NJ ? a.x_low + own * a.ldx_low : a.x + own * a.ldx;
  }
  char* const lx = lds + slice * 2 * kTileBytes;
  const int beyond = (8 - k % 8) % 8;
  auto load = [&](const uint16_t* row, int32_t c) { return row8(row, c, k); };
  auto held = [&](s16x8 v, int32_t c) { return held8(v, c, k, beyond); };
  f32x4 acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{};
  f32x4 low[LOW ? NI : 1][LOW ? NJ : 1] = {};  // the second part's
  // [rows][line][rows 0-7 or 8-15]
  s16x8 w[2][NI][2][2], x[2][XLOADS];
  auto fetch_w = [&](s16x8 (&d)[NI][2][2], int32_t tile) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int l = 0; l < 2; ++l)
#pragma unroll
        for (int h = 0; h < 2; ++h) d[i][l][h] = load(wr[i][h], tile * kFewTile + 64 * l + wk);
  };
  auto fetch_x = [&](s16x8 (&xs)[XLOADS], int32_t tile) {
#pragma unroll
    for (int n = 0; n < XLOADS; ++n) xs[n] = load(xr[n], tile * kFewTile + 8 * xc);
  };
  auto store_x = [&](s16x8 (&xs)[XLOADS], char* d, int32_t tile) {
    if ((tile + 1) * kFewTile > k) {
#pragma unroll
      for (int n = 0; n < XLOADS; ++n) xs[n] = held(xs[n], tile * kFewTile + 8 * xc);
    }
#pragma unroll
    for (int n = 0; n < XLOADS; ++n) {
      const int row = (xt >> 4) + 4 * R * n;
      *(s16x8*)(d + row * 256 + ((xc ^ (row & 15)) << 4)) = xs[n];
    }
  };
  auto use = [&](s16x8 (&d)[NI][2][2], const char* l, int32_t tile) {
    if ((tile + 1) * kFewTile > k) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            d[i][n][h] = held(d[i][n][h], tile * kFewTile + 64 * n + wk);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      s16x8 f[NI][2];
#pragma unroll
      for (int i = 0; i < NI; ++i) fragments(d[i][n], f[i], q < 8);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
#pragma unroll
          for (int part = 0; part < (LOW ? 2 : 1); ++part) {
            const int row = 16 * (part * NJ + j) + q;
            const s16x8 b = *(const s16x8*)(l + row * 256 + (((8 * n + 4 * s + g) ^ q) << 4));
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              f32x4& sum = part ? low[LOW ? i : 0][LOW ? j : 0] : acc[i][j];
              sum = mfma(T{}, f[i][s], b, sum);
            }
          }
        }
    }
  };
  // The part's steps are dealt to the slices in turn, and taken from another place in
  // each workgroup, since rows of a power of two columns would all ask the same memory
  // channels.
  const int32_t tiles = (k + kFewTile - 1) / kFewTile;
  const int32_t first = (int32_t)((int64_t)tiles * part / a.split);
  const int32_t own = (int32_t)((int64_t)tiles * (part + 1) / a.split) - first;
  const int32_t steps = (own + S - 1) / S;
  const int32_t from = (int32_t)(blockIdx.x / kXcds) % steps;
  auto place = [&](int32_t t) {  // of step t, within the part
    t = (t < steps ? t : steps - 1) + from;
    return (t < steps ? t : t - steps) * S + slice;
  };
  // a slice without a tile in the last step loads another one again and skips it
  auto tile = [&](int32_t t) {
    const int32_t p = place(t);
    return first + (p < own ? p : own - 1);
  };
  // the buffer of the step before last is free, the next one's is written
  auto turn = [&] { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
  // x is fetched two steps ahead, since it has to go through LDS, the weights one
  // (37 tokens, 1600 x 6400: 36.5 us a forward pass with one step for both, 36.3 with two,
  // 34.9 so; 22 tokens, 8192 x 28672: 261, 266 and 259).
  fetch_x(x[0], tile(0));
  fetch_w(w[0], tile(0));
  fetch_x(x[1], tile(1));
  store_x(x[0], lx, tile(0));
  fetch_x(x[0], tile(2));
  for (int32_t t = 0; t < steps; t += 2) {
    turn();
    fetch_w(w[1], tile(t + 1));
    store_x(x[1], lx + kTileBytes, tile(t + 1));
    fetch_x(x[1], tile(t + 3));
    if (place(t) < own) use(w[0], lx, tile(t));
    if (t + 1 >= steps) break;
    turn();
    fetch_w(w[0], tile(t + 2));
    store_x(x[0], lx, tile(t + 2));
    fetch_x(x[0], tile(t + 4));
    if (place(t + 1) < own) use(w[1], lx + kTileBytes, tile(t + 1));
  }
  if constexpr (LOW) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = both(acc[i][j][e], low[i][j][e]);
  }
  // The slices' sums, in their order; each wave of a set finishes some of its blocks (50
  // tokens, 72 x 200: 17.8 us a forward pass where the first slice did it all, 16.7 so).
  f32x4* const sums = (f32x4*)lds + set * NI * NJ * 64 + lane;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) sums[(slice * R * NI * NJ + i * NJ + j) * 64] = acc[i][j];
  __syncthreads();
  auto sum = [&](int block) {
    f32x4 v = sums[block * 64];
#pragma unroll
    for (int s = 1; s < S; ++s) v += sums[(s * R * NI * NJ + block) * 64];
    return v;
  };
  if constexpr (PAIR) {
    with_act(a.act, [&](auto act) {
#pragma unroll 1
      for (int j = slice; j < NJ; j += S)
        leave_pair<T>(a, act, sum(j), sum(NJ + j), 16 * j + q, r0 + 4 * g);
    });
  } else {
#pragma unroll 1
    for (int n = slice; n < NI * NJ; n += S) {
      const int32_t t = 16 * (n % NJ) + q, r = r0 + 16 * (n / NJ) + 4 * g;
      if (t >= a.tokens || r >= a.rows) continue;
      const f32x4 v = sum(n);
      if (a.split > 1) *(f32x4*)(a.acc + ((int64_t)part * a.tokens + t) * a.pad + r) = v;
      else leave4<T>(a.out + t * a.ldo, r, a.rows, v);
    }
  }
}

// The parts' sums, four columns a thread.
constexpr int kJoinThreads = 64;
template <typename T>
__global__ __launch_bounds__(kJoinThreads) void k_ffn_few_join(
    const float* __restrict__ acc, int32_t split, int32_t tokens, int32_t pad, int32_t rows,
    uint16_t* __restrict__ out, int64_t ldo) {
  const int32_t t = blockIdx.y, r = (int32_t)(blockIdx.x * kJoinThreads + threadIdx.x) * 4;
  if (r >= rows) return;
  const float* p = acc + (int64_t)t * pad + r;
  f32x4 s = *(const f32x4*)p;
#pragma unroll 8
  for (int32_t n = 1; n < split; ++n) s += *(const f32x4*)(p + (int64_t)n * tokens * pad);
  leave4<T>(out + t * ldo, r, rows, s);
}

template <typename T, int NJ, int R, bool PAIR, bool LOW>
int shared_r(const Few& a, hipStream_t stream) {
  const int32_t each = PAIR ? 16 * R : 32 * R;
  hipLaunchKernelGGL((k_ffn_shared<T, NJ, R, PAIR, LOW>),
                     dim3((uint32_t)((a.rows + each - 1) / each * a.split)), dim3(64 * kWaves), 0,
                     stream, a);
  return (int)hipGetLastError();
}

template <typename T, int NJ>
int shared_j(const Few& in, const Few& out, const FfnPlan& p, hipStream_t stream) {
  constexpr bool LOW = 16 * NJ <= kFfnLow;
  int e = p.few_sets_in == 4 ? shared_r<T, NJ, 4, true, false>(in, stream)
                             : shared_r<T, NJ, 2, true, false>(in, stream);
  if (e) return e;
  e = p.few_sets_out == 4 ? shared_r<T, NJ, 4, false, LOW>(out, stream)
                          : shared_r<T, NJ, 2, false, LOW>(out, stream);
  if (e || out.split == 1) return e;
  hipLaunchKernelGGL((k_ffn_few_join<T>),
                     dim3((uint32_t)((out.rows + 4 * kJoinThreads - 1) / (4 * kJoinThreads)),
                          (uint32_t)out.tokens),
                     dim3(kJoinThreads), 0, stream, out.acc, out.split, out.tokens, out.pad,
                     out.rows, out.out, out.ldo);
  return (int)hipGetLastError();
}

template <typename T>
int direct(const Few& in, const Few& out, hipStream_t stream) {
  hipLaunchKernelGGL((k_ffn_direct<T, 4, true>), dim3((uint32_t)((in.rows + 15) / 16)), dim3(256),
                     0, stream, in);
  ZK_LAUNCHED();
  hipLaunchKernelGGL((k_ffn_direct<T, 8, false>), dim3((uint32_t)((out.rows + 15) / 16)),
                     dim3(512), 0, stream, out);
  return (int)hipGetLastError();
}

template <typename T>
int few_t(const zero_ffn_t* f, const FfnPlan& p, void* ws, void* y, int64_t ldy,
          const zero_ffn_saved_t* saved, hipStream_t stream) {
  const Kept to = kept(p, ws, saved);
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
  in.split = 1;
  in.to = to;
  in.pad = (int32_t)p.inner_pad;
  in.h_low = p.low ? at<uint16_t>(ws, p.h_low) : nullptr;
  Few out{};
  out.w0 = (const uint16_t*)f->w_down;
  out.ldw0 = f->ld_down;
  out.x = to.h;
  out.ldx = to.ld;
  out.x_low = in.h_low;
  out.ldx_low = p.inner_pad;
  out.rows = (int32_t)f->hidden;
  out.k = (int32_t)f->inner;
  out.tokens = (int32_t)f->tokens;
  out.split = p.split_y;
  out.pad = (int32_t)p.hidden_pad;
  out.out = (uint16_t*)y;
  out.ldo = ldy;
  out.acc = at<float>(ws, p.acc);
  if (p.few_sets_in == 1) return direct<T>(in, out, stream);
  if (f->tokens <= 16) return shared_j<T, 1>(in, out, p, stream);
  if (f->tokens <= 32) return shared_j<T, 2>(in, out, p, stream);
  if (f->tokens <= 48) return shared_j<T, 3>(in, out, p, stream);
  return shared_j<T, 4>(in, out, p, stream);
}

}  // namespace

int launch_ffn_few(const zero_ffn_t* f, const FfnPlan& p, void* ws, void* y, int64_t ldy,
                   const zero_ffn_saved_t* saved, hipStream_t stream) {
  return f->dtype == ZERO_BF16 ? few_t<BF16>(f, p, ws, y, ldy, saved, stream)
                               : few_t<FP16>(f, p, ws, y, ldy, saved, stream);
}

}  // namespace zk
