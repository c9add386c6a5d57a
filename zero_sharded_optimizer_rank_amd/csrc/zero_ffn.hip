// Gated feed-forward block and its gradients on the matrix cores (see
// zero_ffn_t in zero_shard.h for the formulas).
//
//   forward   k_ffn_in     both projections of a tile at once, activation and
//                          product on the fp32 sums: h leaves in 16 bits, and for
//                          the gradients act(g) and u act'(g)
//             k_ffn_out    y = h Wd^T
//   backward  k_ffn_back1  dh = dy Wd, whose tiles leave as dg and du; dWd = dy^T h
//             k_ffn_back2  dx = dg Wg + du Wu, one contraction over both; dWg, dWu
// What does not wait for one another shares a launch, so that the tiles of one
// fill the CUs that the last round of the other leaves idle.  All products are the
// tiles of ffn_gemm.h (SMALL: 128 x 128) with fp32 sums; every operand is read as it
// lies.
//
// Large products are bound by the matrix cores at the chip's power limit.  4096 tokens of
// 4096 x 14336 in bf16: k_ffn_in 0.79 ms (1.22 PFLOP/s, 67% of its CUs' cycles in matrix
// instructions), k_ffn_out 0.34 (1.42, 82%), k_ffn_back1 0.86 (1.12, 64%), k_ffn_back2 1.43
// (1.34, 76%).  1024 tokens of 1600 x 6400 in fp16, bound by rounds of tiles, their starts
// and their ends: 57 (50%), 37 (50%), 70 (36%) and 95 us (61%), joins 7 each.
#include <stddef.h>

#include "ffn_device.h"
#include "ffn_gemm.h"

namespace zk {
namespace {

using namespace dev;

constexpr int kPackThreads = 256;

// Rows in whole 16-byte pieces: copies for matrices whose rows lie otherwise, since
// loads straight into LDS need 16-byte addresses.  Bound by memory
// (4099 x 14339: 40 us, 5.8 TB/s).
__global__ __launch_bounds__(kPackThreads) void k_ffn_pack(const uint16_t* __restrict__ src,
                                                           int64_t ld, int64_t rows, int32_t cols,
                                                           int32_t pad,
                                                           uint16_t* __restrict__ out) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    u32x4* o = (u32x4*)(out + r * pad);
    const uint16_t* p = src + r * ld;
    for (int32_t c = threadIdx.x; c < pad / 8; c += kPackThreads)
      o[c] = take8(p + 8 * c, cols - 8 * c);
  }
}

// A matrix as the kernels read it; rows in whole 16-byte pieces.
struct Matrix {
  const uint16_t* p;
  int32_t ld;     // elements
  int32_t width;  // of a row, a multiple of 8
};

// Where rows r0 .. of a matrix are an operand along its rows.
__device__ __forceinline__ Operand by_rows(const Matrix& m, int64_t r0, int64_t rows, int most) {
  const int64_t left = rows - r0;
  return Operand{m.p + r0 * m.ld, m.ld * 2, (int32_t)(left < most ? left : most), m.width};
}
// Where columns c0 .. are: the contraction runs over the rows.
__device__ __forceinline__ Operand by_cols(const Matrix& m, int32_t c0, int64_t rows) {
  return Operand{m.p + c0, m.ld * 2, m.width - c0, (int32_t)rows};
}

// Sixteen bytes of a row of n elements from column c on.
__device__ __forceinline__ void store_row(uint16_t* row, int32_t c, int32_t n, u32x4 v) {
  if (c + 8 <= n) {
    *(u32x4_a2*)(row + c) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < n) row[c + e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
  }
}

template <int N>
__device__ __forceinline__ uint32_t tiles_of(int32_t x) { return (uint32_t)((x + N - 1) / N); }

// --- contractions in parts -------------------------------------------------------
// Where a product leaves few tiles its contraction is cut into parts, whose fp32 sums
// are joined by a launch of their own: part i of a tile's element (row, col) lies at
// acc[(i * rows + col) * ld + row].
struct Parts {
  int32_t count;
  int32_t ld;
  int64_t rows;
  float* acc;
};

// A source from contraction index k0 to `end`: nothing is loaded past it.
template <typename S>
struct Ranged {
  S src;
  int32_t k0, end;
  __device__ __forceinline__ int32_t in(int32_t k) const {
    k += k0;
    return k < end ? k : 0x40000000;  // past every operand
  }
  __device__ __forceinline__ const Operand& a0(int32_t& k) const {
    k = in(k);
    return src.a0(k);
  }
  __device__ __forceinline__ const Operand& a1(int32_t& k) const {
    k = in(k);
    return src.a1(k);
  }
  __device__ __forceinline__ const Operand& b(int32_t& k) const {
    k = in(k);
    return src.b(k);
  }
};

// acc = part `part` of the source's `stages` stages.
template <typename G, typename S>
__device__ __forceinline__ void run_part(const S& src, int32_t stages, int32_t part,
                                         int32_t parts, const typename G::Lds& lds,
                                         f32x4 (&acc)[G::MI][G::NJ]) {
  const int32_t s0 = (int32_t)((int64_t)stages * part / parts);
  const int32_t s1 = (int32_t)((int64_t)stages * (part + 1) / parts);
  G::run(Ranged<S>{src, s0 * kStage, s1 * kStage}, (s1 - s0) * kStage, lds, acc);
}

// Blocks [i0, i1) of the tile's rows as a part's sums; r0, c0: the tile's place.
template <typename G>
__device__ __forceinline__ void leave_part(const Parts& p, int32_t part, int32_t r0, int32_t c0,
                                           int i0, int i1, const f32x4 (&acc)[G::MI][G::NJ]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < G::NJ; ++j) {
    float* o = p.acc + ((int64_t)part * p.rows + c0 + G::col(wave, j) + (lane & 15)) * p.ld;
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < G::MI; ++i)
      if (i >= i0 && i < i1)
        *(f32x4*)(o + r0 + G::row(wave, i - i0) + 4 * (lane >> 4)) = acc[i][j];
  }
}
// Four sums, of the row that starts at `at`.
__device__ __forceinline__ f32x4 joined(const Parts& p, int64_t row, int32_t c) {
  const float* q = p.acc + row * p.ld + c;
  f32x4 s = *(const f32x4*)q;
#pragma unroll 4
  for (int32_t i = 1; i < p.count; ++i) s += *(const f32x4*)(q + (int64_t)i * p.rows * p.ld);
  return s;
}
__device__ __forceinline__ int32_t stages_of(int32_t k) { return (k + kStage - 1) / kStage; }

// Rows of blocks [i0, i1) of a tile's sums that lie past the operand's (its row 0 is r0) are
// zero: an infinity in the other operand makes them NaN, and those that fill h's, dg's and
// du's rows up to 8 take part in the next contraction.
template <typename G>
__device__ __forceinline__ void clear_past(int32_t r0, int32_t rows, int i0, int i1,
                                           f32x4 (&acc)[G::MI][G::NJ]) {
  if (r0 + G::kRows <= rows) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < G::MI; ++i) {
    if (i < i0 || i >= i1) continue;
    const int32_t r = r0 + G::row(wave, i - i0) + 4 * (lane >> 4);
#pragma unroll
    for (int j = 0; j < G::NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (r + e >= rows) acc[i][j][e] = 0.0f;
  }
}
// The same of four sums.
__device__ __forceinline__ f32x4 before(int32_t rows, int32_t r, f32x4 s) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (r + e >= rows) s[e] = 0.0f;
  return s;
}

// --- forward -------------------------------------------------------------------
struct PairProduct {
  Operand gate, up, B;
  __device__ __forceinline__ const Operand& a0(int32_t&) const { return gate; }
  __device__ __forceinline__ const Operand& a1(int32_t&) const { return up; }
  __device__ __forceinline__ const Operand& b(int32_t&) const { return B; }
};

// What both projections' sums become: h, and what the gradients need.
template <int ACT>
__device__ __forceinline__ void gated(f32x4 g, f32x4 u, f32x4& h, f32x4& a, f32x4& b) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float slope;
    a[e] = activated(Act<ACT>{}, g[e], slope);
    b[e] = u[e] * slope;
    h[e] = a[e] * u[e];
  }
}

// A tile has the same inner columns of both projections, so that a lane holds g and u
// of the same element.  What the gradients need is formed here, from the fp32
// sums, so that the backward pass has two products an element left to do.  That is 8
// bytes an element to write, by all CUs at a time, at the end of each round of tiles.
template <typename T, int ACT, bool SAVE, bool SMALL>
__global__ __launch_bounds__(SMALL ? 256 : 512) void k_ffn_in(Matrix x, Matrix w_gate, Matrix w_up,
                                                              int32_t tokens, int32_t inner,
                                                              int32_t inner_pad, Kept to,
                                                              Parts parts) {
  using G = typename TileOf<SMALL, T, false, false, true>::G;
  const auto lds = G::shared();
  const uint32_t tt = tiles_of<G::kCols>(tokens);
  int32_t mt, nt;
  if (!tile_of(blockIdx.x, tiles_of<G::kRows>(inner), tt * (uint32_t)parts.count, mt, nt)) return;
  const int32_t f0 = mt * G::kRows, t0 = (int32_t)((uint32_t)nt % tt) * G::kCols;
  const PairProduct src{by_rows(w_gate, f0, inner, G::kRows), by_rows(w_up, f0, inner, G::kRows),
                        by_rows(x, t0, tokens, G::kCols)};
  constexpr int H = G::MI / 2;
  f32x4 acc[G::MI][G::NJ];
  if (SMALL && parts.count > 1) {
    const int32_t part = (int32_t)((uint32_t)nt / tt);
    run_part<G>(src, stages_of(x.width), part, parts.count, lds, acc);
    // both projections' sums side by side
    leave_part<G>(parts, part, f0, t0, 0, H, acc);
    leave_part<G>(parts, part, parts.ld / 2 + f0, t0, H, G::MI, acc);
    return;
  }
  G::run(src, x.width, lds, acc);
  clear_past<G>(f0, inner, 0, H, acc);
  clear_past<G>(f0, inner, H, G::MI, acc);
  auto leave = [&](uint16_t* out, int region) {
    G::take_half(lds, region, [&](int col, int row, u32x4 v) {
      const int32_t t = t0 + col, f = f0 + row;
      if (t < tokens && f < inner_pad) *(u32x4*)(out + (int64_t)t * to.ld + f) = v;
    });
  };
#pragma unroll
  for (int j = 0; j < G::NJ; ++j)
#pragma unroll
    for (int i = 0; i < H; ++i) {
      f32x4 a, b, h;
      gated<ACT>(acc[i][j], acc[H + i][j], h, a, b);
      G::put_half(lds, 0, i, j, narrow4<T>(h[0], h[1], h[2], h[3]));
      if constexpr (SAVE) {
        Kept4 k = keep4(a, b);
        G::put_half(lds, 1, i, j, k.act);
        // formed here, into the sums' registers, and not where they leave
        asm volatile("" : "+v"(k.slope), "+v"(k.low));
        acc[i][j] = f32x4{__uint_as_float(k.slope[0]), __uint_as_float(k.slope[1]),
                          __uint_as_float(k.low[0]), __uint_as_float(k.low[1])};
      }
    }
  __syncthreads();
  leave(to.h, 0);
  if constexpr (SAVE) {
    leave(to.act, 1);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < G::NJ; ++j)
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const f32x4 v = acc[i][j];
        G::put_half(lds, 0, i, j, u32x2{__float_as_uint(v[0]), __float_as_uint(v[1])});
        G::put_half(lds, 1, i, j, u32x2{__float_as_uint(v[2]), __float_as_uint(v[3])});
      }
    __syncthreads();
    leave(to.slope, 0);
    leave(to.low, 1);
  }
}

// The same from the parts' sums, four columns a thread: bound by memory (387 tokens of
// 4096 x 272, 16 parts: 6.5 us, mostly its launch).
template <typename T, int ACT>
__global__ __launch_bounds__(kPackThreads) void k_ffn_in_join(Parts parts, int32_t tokens,
                                                              int32_t inner, int32_t inner_pad,
                                                              Kept to) {
  const int64_t q = (int64_t)blockIdx.x * kPackThreads + threadIdx.x;
  const int64_t t = q / (inner_pad / 4);
  const int32_t f = (int32_t)(q % (inner_pad / 4)) * 4;
  if (t >= tokens) return;
  f32x4 h, a, b;
  gated<ACT>(before(inner, f, joined(parts, t, f)),
             before(inner, f, joined(parts, t, parts.ld / 2 + f)), h, a, b);
  const int64_t at = t * to.ld + f;
  *(u32x2*)(to.h + at) = narrow4<T>(h[0], h[1], h[2], h[3]);
  if (!to.act) return;
  const Kept4 k = keep4(a, b);
  *(u32x2*)(to.act + at) = k.act;
  *(u32x2*)(to.slope + at) = k.slope;
  *(u32x2*)(to.low + at) = k.low;
}

// --- y and dx --------------------------------------------------------------------
// out [tokens, hidden] = B1 A1^T (+ B2 A2^T): A's rows are hidden columns (y: Wd by
// its rows; dx: Wg, Wu by their columns), B is h, dg, du by its rows.  The second
// product follows the first in one contraction.
struct TwoProducts {
  Operand A1, A2, B1, B2;
  int32_t k1;  // where the second product starts (a multiple of a stage)
  __device__ __forceinline__ const Operand& pick(int32_t& k, const Operand& p,
                                                 const Operand& q) const {
    if (k < k1) return p;
    k -= k1;
    return q;
  }
  __device__ __forceinline__ const Operand& a0(int32_t& k) const { return pick(k, A1, A2); }
  __device__ __forceinline__ const Operand& a1(int32_t& k) const { return pick(k, A1, A2); }
  __device__ __forceinline__ const Operand& b(int32_t& k) const { return pick(k, B1, B2); }
};

struct OutArgs {
  Matrix a1, a2, b1, b2;
  int32_t tokens, hidden, inner;
  Parts parts;
  uint16_t* out;
  int64_t ldo;
};

template <typename T, bool DX, bool SMALL>
__device__ __forceinline__ void out_tile(uint32_t block, const OutArgs& o) {
  using G = typename TileOf<SMALL, T, DX, false>::G;
  const auto lds = G::shared();
  const uint32_t ht = tiles_of<G::kRows>(o.hidden);
  int32_t mt, nt;
  if (!tile_of(block, tiles_of<G::kCols>(o.tokens), ht * (uint32_t)o.parts.count, mt, nt)) return;
  const int32_t h0 = (int32_t)((uint32_t)nt % ht) * G::kRows, t0 = mt * G::kCols;
  const int32_t part = (int32_t)((uint32_t)nt / ht), stages = stages_of(o.inner);
  f32x4 acc[G::MI][G::NJ];
  if constexpr (DX) {
    const TwoProducts src{by_cols(o.a1, h0, o.inner), by_cols(o.a2, h0, o.inner),
                          by_rows(o.b1, t0, o.tokens, G::kCols),
                          by_rows(o.b2, t0, o.tokens, G::kCols), stages * kStage};
    run_part<G>(src, 2 * stages, part, o.parts.count, lds, acc);
  } else {
    const OneProduct src{by_rows(o.a1, h0, o.hidden, G::kRows),
                         by_rows(o.b1, t0, o.tokens, G::kCols)};
    run_part<G>(src, stages, part, o.parts.count, lds, acc);
  }
  if (o.parts.count > 1) return leave_part<G>(o.parts, part, h0, t0, 0, G::MI, acc);
  G::transposed(lds, acc, narrow4<T>, [&](int col, int row, u32x4 v) {
    const int32_t t = t0 + col, c = h0 + row;
    if (t < o.tokens && c < o.hidden) store_row(o.out + (int64_t)t * o.ldo, c, o.hidden, v);
  });
}

// y.  One product of T x hidden tiles: few, so its contraction, the longest, is often cut
// into parts (512 tokens of 4099 x 14339: 34 tiles in 5 parts, 101 us, 0.59 PFLOP/s).
template <typename T, bool SMALL>
__global__ __launch_bounds__(SMALL ? 256 : 512) void k_ffn_out(OutArgs o) {
  out_tile<T, false, SMALL>(blockIdx.x, o);
}

// y or dx from the parts' sums, four columns a thread: bound by memory (1024 x 1600, 6 and 4
// parts: 6.6 us, 5.5 TB/s).
template <typename T>
__global__ __launch_bounds__(kPackThreads) void k_ffn_out_join(Parts parts, int32_t tokens,
                                                               int32_t hidden,
                                                               uint16_t* __restrict__ out,
                                                               int64_t ldo) {
  const int32_t quads = (hidden + 3) / 4;
  const int64_t q = (int64_t)blockIdx.x * kPackThreads + threadIdx.x, t = q / quads;
  const int32_t c = (int32_t)(q % quads) * 4;
  if (t >= tokens) return;
  const f32x4 s = joined(parts, t, c);
  uint16_t* o = out + t * ldo + c;
  const u32x2 v = narrow4<T>(s[0], s[1], s[2], s[3]);
  if (c + 4 <= hidden) {
    *(u32x2_a2*)o = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < hidden) o[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
  }
}

// --- backward --------------------------------------------------------------------
struct DhArgs {
  Matrix w_down, dy;
  int32_t tokens, hidden, inner, inner_pad;
  const uint16_t *act, *slope, *low;  // rows ld apart
  int64_t ld;
  uint16_t *dg, *du;                  // rows inner_pad apart
  Parts parts;
};

// dh of four elements becomes dg and du.
template <typename T>
__device__ __forceinline__ void gradients(f32x4 dh, u32x2 act, u32x2 slope, u32x2 low, u32x2& dg,
                                          u32x2& du) {
  f32x4 x, y;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = dh[e] * kept_at<1>(slope, low, e);
    y[e] = dh[e] * kept_at<0>(act, low, e);
  }
  dg = narrow4<T>(x[0], x[1], x[2], x[3]);
  du = narrow4<T>(y[0], y[1], y[2], y[3]);
}

// A tile of dh: A = Wd by its columns (inner), B = dy by its rows; it leaves as dg =
// dh (u act'(g)) and du = dh act(g).  Lane by lane what was kept lies as the sums do,
// eight bytes each; the next few blocks' are on their way while some are multiplied.
// Six bytes an element to read and four to write at a tile's end are why the launch
// reaches 64% of the matrix cores' cycles where k_ffn_out reaches 82%.
template <typename T, bool SMALL>
__device__ __forceinline__ void dh_tile(uint32_t block, const DhArgs& a) {
  using G = typename TileOf<SMALL, T, true, false>::G;
  const auto lds = G::shared();
  const uint32_t tt = tiles_of<G::kCols>(a.tokens);
  int32_t mt, nt;
  if (!tile_of(block, tiles_of<G::kRows>(a.inner), tt * (uint32_t)a.parts.count, mt, nt)) return;
  const int32_t f0 = mt * G::kRows, t0 = (int32_t)((uint32_t)nt % tt) * G::kCols;
  const OneProduct src{by_cols(a.w_down, f0, a.hidden), by_rows(a.dy, t0, a.tokens, G::kCols)};
  f32x4 acc[G::MI][G::NJ];
  if (SMALL && a.parts.count > 1) {
    const int32_t part = (int32_t)((uint32_t)nt / tt);
    run_part<G>(src, stages_of(a.hidden), part, a.parts.count, lds, acc);
    return leave_part<G>(a.parts, part, f0, t0, 0, G::MI, acc);
  }
  G::run(src, a.hidden, lds, acc);
  clear_past<G>(f0, a.inner, 0, G::MI, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int N = 4, kSets = G::MI * G::NJ / N;  // blocks of a set
  u32x2 av[2][N], bv[2][N], lv[2][N];
  auto fetch = [&](int set) {  // what lies past the operands is not stored
    const int j = set * N / G::MI;
    const int32_t t = t0 + G::col(wave, j) + (lane & 15);
    const int64_t row = (int64_t)(t < a.tokens ? t : a.tokens - 1) * a.ld;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int32_t f = f0 + G::row(wave, set * N % G::MI + n) + 4 * (lane >> 4);
      const int64_t at = row + (f < a.inner_pad ? f : 0);
      av[set & 1][n] = *(const u32x2*)(a.act + at);
      bv[set & 1][n] = *(const u32x2*)(a.slope + at);
      lv[set & 1][n] = *(const u32x2*)(a.low + at);
    }
  };
  fetch(0);
#pragma unroll
  for (int set = 0; set < kSets; ++set) {
    if (set + 1 < kSets) fetch(set + 1);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int j = set * N / G::MI, i = set * N % G::MI + n;
      u32x2 x, y;
      gradients<T>(acc[i][j], av[set & 1][n], bv[set & 1][n], lv[set & 1][n], x, y);
      G::put(lds, i, j, x);
      // narrowed here, into a sum's registers, and not where it leaves
      asm volatile("" : "+v"(y));
      acc[i][j][0] = __uint_as_float(y[0]);
      acc[i][j][1] = __uint_as_float(y[1]);
    }
  }
  auto leave = [&](uint16_t* out) {
    __syncthreads();
    G::take(lds, [&](int col, int row, u32x4 v) {
      const int32_t t = t0 + col, f = f0 + row;
      if (t < a.tokens && f < a.inner_pad) *(u32x4*)(out + (int64_t)t * a.inner_pad + f) = v;
    });
  };
  leave(a.dg);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < G::NJ; ++j)
#pragma unroll
    for (int i = 0; i < G::MI; ++i)
      G::put(lds, i, j, u32x2{__float_as_uint(acc[i][j][0]), __float_as_uint(acc[i][j][1])});
  leave(a.du);
}

// The same from the parts' sums, four columns a thread: bound by memory (64 tokens of
// 4096 x 14336, 2 parts: 5 us).
template <typename T>
__global__ __launch_bounds__(kPackThreads) void k_ffn_dh_join(DhArgs a) {
  const int64_t q = (int64_t)blockIdx.x * kPackThreads + threadIdx.x;
  const int64_t t = q / (a.inner_pad / 4);
  const int32_t f = (int32_t)(q % (a.inner_pad / 4)) * 4;
  if (t >= a.tokens) return;
  const int64_t at = t * a.ld + f, to = t * a.inner_pad + f;
  u32x2 x, y;
  gradients<T>(before(a.inner, f, joined(a.parts, t, f)), *(const u32x2*)(a.act + at),
               *(const u32x2*)(a.slope + at), *(const u32x2*)(a.low + at), x, y);
  *(u32x2*)(a.dg + to) = x;
  *(u32x2*)(a.du + to) = y;
}

// One weight's gradient [n, m] = B^T A: row j is column j of B against the columns
// of A, over the tokens.
struct WeightGrad {
  Matrix a, b;
  int32_t m, n, tokens, accumulate;
  uint32_t first;  // its first workgroup
  void* out;
  int64_t ld;
  Parts parts;
};

// Four sums of row n from column m on, into their place.
template <typename T, bool F32OUT>
__device__ __forceinline__ void leave_dw(const WeightGrad& w, int32_t n, int32_t m, f32x4 d) {
  const int64_t at = (int64_t)n * w.ld + m;
  if constexpr (F32OUT) {
    float* o = (float*)w.out + at;
    if (m + 4 <= w.m) {
      if (w.accumulate) d = *(const f32x4_a4*)o + d;
      *(f32x4_a4*)o = d;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (m + e < w.m) o[e] = w.accumulate ? o[e] + d[e] : d[e];
    }
  } else {
    uint16_t* o = (uint16_t*)w.out + at;
    if (m + 4 <= w.m) {
      if (w.accumulate) {
        const u32x2 q = *(const u32x2_a2*)o;
        d += f32x4{widen<T>(q[0] & 0xFFFFu), widen<T>(q[0] >> 16), widen<T>(q[1] & 0xFFFFu),
                   widen<T>(q[1] >> 16)};
      }
      *(u32x2_a2*)o = narrow4<T>(d[0], d[1], d[2], d[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (m + e < w.m)
          o[e] = (uint16_t)narrow<T>(w.accumulate ? widen<T>(o[e]) + d[e] : d[e]);
    }
  }
}

template <typename T, bool F32OUT, bool SMALL>
__device__ __forceinline__ void dw_tile(uint32_t block, const WeightGrad& w) {
  using G = typename TileOf<SMALL, T, true, true>::G;
  const auto lds = G::shared();
  const uint32_t rows = tiles_of<G::kRows>(w.m);
  int32_t mt, nt;
  if (!tile_of(block, tiles_of<G::kCols>(w.n), rows * (uint32_t)w.parts.count, nt, mt)) return;
  const int32_t m0 = (int32_t)((uint32_t)mt % rows) * G::kRows, n0 = nt * G::kCols;
  const OneProduct src{by_cols(w.a, m0, w.tokens), by_cols(w.b, n0, w.tokens)};
  f32x4 acc[G::MI][G::NJ];
  if (SMALL && w.parts.count > 1) {
    const int32_t part = (int32_t)((uint32_t)mt / rows);
    run_part<G>(src, stages_of(w.tokens), part, w.parts.count, lds, acc);
    return leave_part<G>(w.parts, part, m0, n0, 0, G::MI, acc);
  }
  G::run(src, w.tokens, lds, acc);
  if (!F32OUT && !w.accumulate) {
    uint16_t* out = (uint16_t*)w.out;
    G::transposed(lds, acc, narrow4<T>, [&](int col, int row, u32x4 v) {
      const int32_t n = n0 + col, m = m0 + row;
      if (n < w.n && m < w.m) store_row(out + (int64_t)n * w.ld, m, w.m, v);
    });
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < G::NJ; ++j) {
    const int32_t n = n0 + G::col(wave, j) + (lane & 15);
    if (n >= w.n) continue;
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < G::MI; ++i)
      leave_dw<T, F32OUT>(w, n, m0 + G::row(wave, i) + 4 * (lane >> 4), acc[i][j]);
  }
}

// The same from the parts' sums, four columns a thread, bound by memory; the second
// weight's workgroups, if it has any, start at b.first.  For many tokens of narrow blocks
// only: their weights' tiles are few and the contraction, the tokens, long (2000 tokens of
// 24 x 40, 8 parts: 3 us, its launch).
template <typename T, bool F32OUT>
__global__ __launch_bounds__(kPackThreads) void k_ffn_dw_join(WeightGrad a, WeightGrad b) {
  const bool second = blockIdx.x >= b.first;
  const WeightGrad w = second ? b : a;
  const int32_t quads = (w.m + 3) / 4;
  const int64_t q = (int64_t)(blockIdx.x - (second ? b.first : 0u)) * kPackThreads + threadIdx.x;
  const int64_t n = q / quads;
  const int32_t m = (int32_t)(q % quads) * 4;
  if (n < w.n) leave_dw<T, F32OUT>(w, (int32_t)n, m, joined(w.parts, n, m));
}

// Workgroups from w.first on take dWd, those before dh: whichever has the longer
// contraction comes first, so that the shorter tiles fill the last round.
template <typename T, bool F32OUT, bool SMALL>
__global__ __launch_bounds__(SMALL ? 256 : 512) void k_ffn_back1(DhArgs d, uint32_t dh_first,
                                                                 WeightGrad w) {
  const bool weight = w.first > dh_first ? blockIdx.x >= w.first : blockIdx.x < dh_first;
  if (weight) dw_tile<T, F32OUT, SMALL>(blockIdx.x - w.first, w);
  else dh_tile<T, SMALL>(blockIdx.x - dh_first, d);
}

// dx first, whose contraction over both projections is the longest, then dWg and dWu, 2/3
// of the work.
template <typename T, bool F32OUT, bool SMALL>
__global__ __launch_bounds__(SMALL ? 256 : 512) void k_ffn_back2(OutArgs o, WeightGrad g,
                                                                 WeightGrad u) {
  if (blockIdx.x < g.first) return out_tile<T, true, SMALL>(blockIdx.x, o);
  const WeightGrad w = blockIdx.x < u.first ? g : u;
  dw_tile<T, F32OUT, SMALL>(blockIdx.x - w.first, w);
}

// --- launches ----------------------------------------------------------------------
// The matrix as the kernels read it: in place, or laid out in the workspace.
int view(const void* src, int64_t ld, int64_t rows, int64_t cols, bool pack, void* ws, size_t at_,
         hipStream_t stream, Matrix& out) {
  if (!pack) {
    out = Matrix{(const uint16_t*)src, (int32_t)ld, (int32_t)cols};
    return (int)hipSuccess;
  }
  const int32_t pad = (int32_t)((cols + 7) / 8 * 8);
  uint16_t* to = at<uint16_t>(ws, at_);
  out = Matrix{to, pad, pad};
  if (rows == 0) return (int)hipSuccess;
  constexpr int64_t kRows = 1 << 20;  // workgroups at most
  hipLaunchKernelGGL(k_ffn_pack, dim3((uint32_t)(rows < kRows ? rows : kRows)), dim3(kPackThreads),
                     0, stream, (const uint16_t*)src, ld, rows, (int32_t)cols, pad, to);
  return (int)hipGetLastError();
}

uint32_t grid_of(int64_t rows, int64_t cols, int64_t tile, int64_t times = 1) {
  return tile_grid((rows + tile - 1) / tile, (cols + tile - 1) / tile * times);
}
uint32_t quads_grid(int64_t rows, int64_t cols) {
  return (uint32_t)((rows * ((cols + 3) / 4) + kPackThreads - 1) / kPackThreads);
}
// Sums of `parts` parts of cols rows of `rows` columns, at *next floats into acc.
Parts parts_at(void* ws, const FfnPlan& p, int64_t rows, int64_t cols, int32_t parts,
               int64_t* next) {
  Parts q{parts, (int32_t)((rows + 255) / 256 * 256), (cols + 255) / 256 * 256, nullptr};
  if (parts > 1) {
    q.acc = at<float>(ws, p.acc) + *next;
    *next += q.ld * q.rows * parts;
  }
  return q;
}

template <typename T>
int out_join(const OutArgs& o, hipStream_t stream) {
  if (o.parts.count == 1) return (int)hipSuccess;
  hipLaunchKernelGGL((k_ffn_out_join<T>), dim3(quads_grid(o.tokens, o.hidden)),
                     dim3(kPackThreads), 0, stream, o.parts, o.tokens, o.hidden, o.out, o.ldo);
  return (int)hipGetLastError();
}

template <typename T, bool SAVE, bool SMALL>
auto in_kernel(int32_t act) {
  return act == ZERO_ACT_SILU        ? k_ffn_in<T, ZERO_ACT_SILU, SAVE, SMALL>
         : act == ZERO_ACT_GELU      ? k_ffn_in<T, ZERO_ACT_GELU, SAVE, SMALL>
         : act == ZERO_ACT_GELU_TANH ? k_ffn_in<T, ZERO_ACT_GELU_TANH, SAVE, SMALL>
                                     : k_ffn_in<T, ZERO_ACT_RELU, SAVE, SMALL>;
}
template <typename T>
auto in_join_kernel(int32_t act) {
  return act == ZERO_ACT_SILU        ? k_ffn_in_join<T, ZERO_ACT_SILU>
         : act == ZERO_ACT_GELU      ? k_ffn_in_join<T, ZERO_ACT_GELU>
         : act == ZERO_ACT_GELU_TANH ? k_ffn_in_join<T, ZERO_ACT_GELU_TANH>
                                     : k_ffn_in_join<T, ZERO_ACT_RELU>;
}

template <typename T>
int forward_t(const zero_ffn_t* f, const FfnPlan& p, void* ws, void* y, int64_t ldy,
              const zero_ffn_saved_t* saved, hipStream_t stream) {
  Matrix x, wg, wu, wd;
  const int64_t H = f->hidden, F = f->inner, T_ = f->tokens;
  int e = view(f->x, f->ldx, T_, H, p.pack_x, ws, p.x, stream, x);
  if (!e) e = view(f->w_gate, f->ld_gate, F, H, p.pack_gate, ws, p.w_gate, stream, wg);
  if (!e) e = view(f->w_up, f->ld_up, F, H, p.pack_up, ws, p.w_up, stream, wu);
  if (!e) e = view(f->w_down, f->ld_down, H, F, p.pack_down, ws, p.w_down, stream, wd);
  if (e) return e;
  const Kept to = kept(p, ws, saved);
  int64_t next = 0;
  Parts parts = parts_at(ws, p, F, T_, p.split_in, &next);
  if (parts.count > 1) {  // both projections
    parts.ld *= 2;
    next *= 2;
  }
  const auto in = p.small_in ? (saved ? in_kernel<T, true, true>(f->act)
                                      : in_kernel<T, false, true>(f->act))
                             : (saved ? in_kernel<T, true, false>(f->act)
                                      : in_kernel<T, false, false>(f->act));
  const int64_t rows = p.small_in ? 64 : 128;  // of each projection
  hipLaunchKernelGGL(in, dim3(tile_grid((F + rows - 1) / rows,
                                        (T_ + 2 * rows - 1) / (2 * rows) * parts.count)),
                     dim3(p.small_in ? 256 : 512), 0, stream, x, wg, wu, (int32_t)T_, (int32_t)F,
                     (int32_t)p.inner_pad, to, parts);
  ZK_LAUNCHED();
  if (parts.count > 1) {
    hipLaunchKernelGGL(in_join_kernel<T>(f->act), dim3(quads_grid(T_, p.inner_pad)),
                       dim3(kPackThreads), 0, stream, parts, (int32_t)T_, (int32_t)F,
                       (int32_t)p.inner_pad, to);
    ZK_LAUNCHED();
  }
  const Matrix h{to.h, (int32_t)to.ld, (int32_t)p.inner_pad};
  next = 0;  // the sums before have been read by then
  const OutArgs o{wd, wd, h, h, (int32_t)T_, (int32_t)H, (int32_t)F,
                  parts_at(ws, p, H, T_, p.split_y, &next), (uint16_t*)y, ldy};
  const uint32_t blocks = grid_of(T_, H, p.small_out ? 128 : 256, o.parts.count);
  if (p.small_out)
    hipLaunchKernelGGL((k_ffn_out<T, true>), dim3(blocks), dim3(256), 0, stream, o);
  else
    hipLaunchKernelGGL((k_ffn_out<T, false>), dim3(blocks), dim3(512), 0, stream, o);
  ZK_LAUNCHED();
  return out_join<T>(o, stream);
}

template <typename T, bool F32OUT>
int backward_t(const zero_ffn_t* f, const FfnPlan& p, void* ws, const zero_ffn_saved_t* saved,
               const zero_ffn_grads_t* g, hipStream_t stream) {
  Matrix x, wg{}, wu{}, wd, dy;
  const int64_t H = f->hidden, F = f->inner, T_ = f->tokens;
  int e = view(f->x, f->ldx, T_, H, p.pack_x, ws, p.x, stream, x);
  if (!e && g->dx) e = view(f->w_gate, f->ld_gate, F, H, p.pack_gate, ws, p.w_gate, stream, wg);
  if (!e && g->dx) e = view(f->w_up, f->ld_up, F, H, p.pack_up, ws, p.w_up, stream, wu);
  if (!e) e = view(f->w_down, f->ld_down, H, F, p.pack_down, ws, p.w_down, stream, wd);
  if (!e) e = view(g->dy, g->lddy, T_, H, p.pack_dy, ws, p.dy, stream, dy);
  if (e) return e;
  const int32_t Fp = (int32_t)p.inner_pad;
  const Matrix h{(const uint16_t*)saved->h, (int32_t)saved->ld, Fp};
  const Matrix dg{at<uint16_t>(ws, p.dg), Fp, Fp}, du{at<uint16_t>(ws, p.du), Fp, Fp};
  const int64_t tile1 = p.small_back1 ? 128 : 256, tile2 = p.small_back2 ? 128 : 256;
  // tokens 0: nothing but weights' gradients to clear
  const bool weights = T_ > 0 || !g->accumulate;
  const auto weight = [&](const Matrix& a, const Matrix& b, int64_t m, int64_t n, void* out,
                          int64_t ld, int32_t parts, int64_t* next) {
    return WeightGrad{a, b, (int32_t)m, (int32_t)n, (int32_t)T_, g->accumulate, 0,
                      weights ? out : nullptr, ld,
                      parts_at(ws, p, m, n, weights && out ? parts : 1, next)};
  };
  const auto dw_grid = [&](const WeightGrad& w, int64_t tile) {
    return w.out ? grid_of(w.n, w.m, tile, w.parts.count) : 0u;
  };

  const bool through = T_ > 0 && (g->dx || g->dw_gate || g->dw_up);
  int64_t next = 0;
  const DhArgs dh{wd, dy, (int32_t)T_, (int32_t)H, (int32_t)F, Fp, (const uint16_t*)saved->act,
                  (const uint16_t*)saved->slope, (const uint16_t*)saved->low, saved->ld,
                  (uint16_t*)dg.p, (uint16_t*)du.p,
                  parts_at(ws, p, F, T_, through ? p.split_dh : 1, &next)};
  WeightGrad down = weight(h, dy, F, H, g->dw_down, g->lddw_down, p.split_dw1, &next);
  const uint32_t dh_blocks = through ? grid_of(F, T_, tile1, dh.parts.count) : 0;
  const uint32_t down_blocks = dw_grid(down, tile1);
  if (dh_blocks + down_blocks) {
    const bool dh_first = through && H >= T_;
    down.first = dh_first ? dh_blocks : 0;
    if (p.small_back1)
      hipLaunchKernelGGL((k_ffn_back1<T, F32OUT, true>), dim3(dh_blocks + down_blocks), dim3(256),
                         0, stream, dh, dh_first ? 0 : down_blocks, down);
    else
      hipLaunchKernelGGL((k_ffn_back1<T, F32OUT, false>), dim3(dh_blocks + down_blocks), dim3(512),
                         0, stream, dh, dh_first ? 0 : down_blocks, down);
    ZK_LAUNCHED();
  }
  if (dh.parts.count > 1) {
    hipLaunchKernelGGL((k_ffn_dh_join<T>), dim3(quads_grid(T_, Fp)), dim3(kPackThreads), 0, stream,
                       dh);
    ZK_LAUNCHED();
  }
  const auto dw_join = [&](const WeightGrad& a, const WeightGrad& b) {
    const WeightGrad& one = a.parts.count > 1 ? a : b;
    WeightGrad two = b;
    two.first = quads_grid(one.n, one.m);
    const bool both = a.parts.count > 1 && b.parts.count > 1;
    hipLaunchKernelGGL((k_ffn_dw_join<T, F32OUT>),
                       dim3(two.first + (both ? quads_grid(two.n, two.m) : 0u)),
                       dim3(kPackThreads), 0, stream, one, two);
    return (int)hipGetLastError();
  };
  if (down.parts.count > 1) {
    e = dw_join(down, WeightGrad{});
    if (e) return e;
  }

  next = 0;  // the sums before have been read by then
  const bool dx = g->dx && T_ > 0;
  const OutArgs o{wg, wu, dg, du, (int32_t)T_, (int32_t)H, (int32_t)F,
                  parts_at(ws, p, H, T_, dx ? p.split_dx : 1, &next), (uint16_t*)g->dx, g->lddx};
  WeightGrad gate = weight(x, dg, H, F, g->dw_gate, g->lddw_gate, p.split_dw2, &next);
  WeightGrad up = weight(x, du, H, F, g->dw_up, g->lddw_up, p.split_dw2, &next);
  gate.first = dx ? grid_of(T_, H, tile2, o.parts.count) : 0;
  up.first = gate.first + dw_grid(gate, tile2);
  const uint32_t blocks = up.first + dw_grid(up, tile2);
  if (blocks) {
    if (p.small_back2)
      hipLaunchKernelGGL((k_ffn_back2<T, F32OUT, true>), dim3(blocks), dim3(256), 0, stream, o,
                         gate, up);
    else
      hipLaunchKernelGGL((k_ffn_back2<T, F32OUT, false>), dim3(blocks), dim3(512), 0, stream, o,
                         gate, up);
    ZK_LAUNCHED();
  }
  if (gate.parts.count > 1 || up.parts.count > 1) {
    e = dw_join(gate, up);
    if (e) return e;
  }
  return dx ? out_join<T>(o, stream) : (int)hipSuccess;
}

template <typename T>
int backward_o(const zero_ffn_t* f, const FfnPlan& p, void* ws, const zero_ffn_saved_t* saved,
               const zero_ffn_grads_t* g, hipStream_t stream) {
  return g->dw_dtype == ZERO_F32 ? backward_t<T, true>(f, p, ws, saved, g, stream)
                                 : backward_t<T, false>(f, p, ws, saved, g, stream);
}

}  // namespace

int launch_ffn_forward(const zero_ffn_t* f, const FfnPlan& p, void* ws, void* y, int64_t ldy,
                       const zero_ffn_saved_t* saved, hipStream_t stream) {
  return f->dtype == ZERO_BF16 ? forward_t<BF16>(f, p, ws, y, ldy, saved, stream)
                               : forward_t<FP16>(f, p, ws, y, ldy, saved, stream);
}

int launch_ffn_backward(const zero_ffn_t* f, const FfnPlan& p, void* ws,
                        const zero_ffn_saved_t* saved, const zero_ffn_grads_t* g,
                        hipStream_t stream) {
  return f->dtype == ZERO_BF16 ? backward_o<BF16>(f, p, ws, saved, g, stream)
                               : backward_o<FP16>(f, p, ws, saved, g, stream);
}

}  // namespace zk
