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
#include <stddef.h>

#include "ffn_device.h"
#include "ffn_gemm.h"

namespace zk {
namespace {

using namespace dev;

constexpr int kPackThreads = 256;

// Rows in whole 16-byte pieces: copies for matrices whose rows lie otherwise.
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

// --- forward -------------------------------------------------------------------
struct PairProduct {
  Operand gate, up, B;
  __device__ __forceinline__ const Operand& a0(int32_t&) const { return gate; }
  __device__ __forceinline__ const Operand& a1(int32_t&) const { return up; }
  __device__ __forceinline__ const Operand& b(int32_t&) const { return B; }
};

// A tile has the same inner columns of both projections, so that a lane holds g and u
// of the same element.  What the gradients need is formed here, from the fp32
// sums, so that the backward pass has two products an element left to do.
template <typename T, int ACT, bool SAVE, bool SMALL>
__global__ __launch_bounds__(SMALL ? 256 : 512) void k_ffn_in(Matrix x, Matrix w_gate, Matrix w_up,
                                                              int32_t tokens, int32_t inner,
                                                              int32_t inner_pad, Kept to) {
  using G = typename TileOf<SMALL, T, false, false, true>::G;
  const auto lds = G::shared();
  int32_t mt, nt;
  if (!tile_of(blockIdx.x, tiles_of<G::kRows>(inner), tiles_of<G::kCols>(tokens), mt, nt)) return;
  const int32_t f0 = mt * G::kRows, t0 = nt * G::kCols;
  const PairProduct src{by_rows(w_gate, f0, inner, G::kRows), by_rows(w_up, f0, inner, G::kRows),
                        by_rows(x, t0, tokens, G::kCols)};
  constexpr int H = G::MI / 2;
  f32x4 acc[G::MI][G::NJ];
  G::run(src, x.width, lds, acc);
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
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = acc[H + i][j][e];
        float slope;
        a[e] = activated(Act<ACT>{}, acc[i][j][e], slope);
        b[e] = u * slope;
        h[e] = a[e] * u;
      }
      G::put_half(lds, 0, i, j, narrow4<T>(h[0], h[1], h[2], h[3]));
      if constexpr (SAVE) {
        G::put_half(lds, 1, i, j, narrow4<T>(a[0], a[1], a[2], a[3]));
        u32x2 v = narrow4<T>(b[0], b[1], b[2], b[3]);
        // narrowed here, into a sum's registers, and not where it leaves
        asm volatile("" : "+v"(v));
        acc[i][j][0] = __uint_as_float(v[0]);
        acc[i][j][1] = __uint_as_float(v[1]);
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
      for (int i = 0; i < H; ++i)
        G::put_half(lds, 0, i, j,
                    u32x2{__float_as_uint(acc[i][j][0]), __float_as_uint(acc[i][j][1])});
    __syncthreads();
    leave(to.slope, 0);
  }
}

// --- y and dx --------------------------------------------------------------------
// out [tokens, hidden] = B1 A1^T (+ B2 A2^T): A's rows are hidden columns (y: Wd by
// its rows; dx: Wg, Wu by their columns), B is h, dg, du by its rows.  The second
// product follows the first in one contraction.  Where that leaves few tiles it
// is split; the splits' fp32 sums are joined by k_ffn_join.
template <bool TWO>
struct Products {
  Operand A1, A2, B1, B2;
  int32_t k0;       // first contraction index of this workgroup's part
  int32_t k1;       // where the second product starts (a multiple of a stage)
  int32_t end;      // of this part: nothing is loaded past it
  __device__ __forceinline__ const Operand& pick(int32_t& k, const Operand& p,
                                                 const Operand& q) const {
    k += k0;
    if (k >= end) k = 0x40000000;  // past every operand
    if constexpr (!TWO) return p;
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
  int32_t tokens, hidden, inner, split;
  int64_t acc_rows;   // of a split's sums
  int32_t acc_ld;
  float* acc;         // split > 1
  uint16_t* out;      // split = 1
  int64_t ldo;
};

template <typename T, bool DX, bool SMALL>
__device__ __forceinline__ void out_tile(uint32_t block, const OutArgs& o) {
  using G = typename TileOf<SMALL, T, DX, false>::G;
  const auto lds = G::shared();
  const uint32_t ht = tiles_of<G::kRows>(o.hidden);
  int32_t mt, nt;
  if (!tile_of(block, tiles_of<G::kCols>(o.tokens), ht * (uint32_t)o.split, mt, nt)) return;
  const int32_t h0 = (int32_t)((uint32_t)nt % ht) * G::kRows, t0 = mt * G::kCols;
  const int32_t part = (int32_t)((uint32_t)nt / ht);
  const int32_t stages = (o.inner + kStage - 1) / kStage, all = DX ? 2 * stages : stages;
  const int32_t s0 = (int32_t)((int64_t)all * part / o.split);
  const int32_t s1 = (int32_t)((int64_t)all * (part + 1) / o.split);
  Products<DX> src;
  src.A1 = DX ? by_cols(o.a1, h0, o.inner) : by_rows(o.a1, h0, o.hidden, G::kRows);
  src.B1 = by_rows(o.b1, t0, o.tokens, G::kCols);
  if constexpr (DX) {
    src.A2 = by_cols(o.a2, h0, o.inner);
    src.B2 = by_rows(o.b2, t0, o.tokens, G::kCols);
  }
  src.k0 = s0 * kStage;
  src.k1 = stages * kStage;
  src.end = s1 * kStage;
  f32x4 acc[G::MI][G::NJ];
  G::run(src, (s1 - s0) * kStage, lds, acc);
  if (o.split == 1) {
    G::transposed(lds, acc, narrow4<T>, [&](int col, int row, u32x4 v) {
      const int32_t t = t0 + col, c = h0 + row;
      if (t < o.tokens && c < o.hidden) store_row(o.out + (int64_t)t * o.ldo, c, o.hidden, v);
    });
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < G::NJ; ++j) {
    const int32_t t = t0 + G::col(wave, j) + (lane & 15);
    float* p = o.acc + ((int64_t)part * o.acc_rows + t) * o.acc_ld;
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < G::MI; ++i)
      *(f32x4*)(p + h0 + G::row(wave, i) + 4 * (lane >> 4)) = acc[i][j];
  }
}

template <typename T, bool SMALL>
__global__ __launch_bounds__(SMALL ? 256 : 512) void k_ffn_out(OutArgs o) {
  out_tile<T, false, SMALL>(blockIdx.x, o);
}

// The splits' sums, four columns a thread.
template <typename T>
__global__ __launch_bounds__(kPackThreads) void k_ffn_join(const float* __restrict__ acc,
                                                           int32_t split, int64_t acc_rows,
                                                           int32_t acc_ld, int32_t hidden,
                                                           uint16_t* __restrict__ out,
                                                           int64_t ldo) {
  const int64_t t = blockIdx.y;
  const int32_t c = (int32_t)(blockIdx.x * kPackThreads + threadIdx.x) * 4;
  if (c >= hidden) return;
  const float* p = acc + t * acc_ld + c;
  f32x4 s = *(const f32x4*)p;
#pragma unroll 4
  for (int32_t k = 1; k < split; ++k) s += *(const f32x4*)(p + (int64_t)k * acc_rows * acc_ld);
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
  const uint16_t *act, *slope;  // rows ld apart
  int64_t ld;
  uint16_t *dg, *du;            // rows inner_pad apart
};

// A tile of dh: A = Wd by its columns (inner), B = dy by its rows; it leaves as dg =
// dh (u act'(g)) and du = dh act(g).  Lane by lane those lie as the sums do, eight
// bytes each; the next column's are on their way while one is multiplied.
template <typename T, bool SMALL>
__device__ __forceinline__ void dh_tile(uint32_t block, const DhArgs& a) {
  using G = typename TileOf<SMALL, T, true, false>::G;
  const auto lds = G::shared();
  int32_t mt, nt;
  if (!tile_of(block, tiles_of<G::kRows>(a.inner), tiles_of<G::kCols>(a.tokens), mt, nt)) return;
  const int32_t f0 = mt * G::kRows, t0 = nt * G::kCols;
  f32x4 acc[G::MI][G::NJ];
  G::run(by_cols(a.w_down, f0, a.hidden), by_rows(a.dy, t0, a.tokens, G::kCols), a.hidden, lds,
         acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  u32x2 av[2][G::MI], bv[2][G::MI];
  auto fetch = [&](int j) {  // what lies past the operands is not stored
    const int32_t t = t0 + G::col(wave, j) + (lane & 15);
    const int64_t row = (int64_t)(t < a.tokens ? t : a.tokens - 1) * a.ld;
#pragma unroll
    for (int i = 0; i < G::MI; ++i) {
      const int32_t f = f0 + G::row(wave, i) + 4 * (lane >> 4);
      const int64_t at = row + (f < a.inner_pad ? f : 0);
      av[j & 1][i] = *(const u32x2*)(a.act + at);
      bv[j & 1][i] = *(const u32x2*)(a.slope + at);
    }
  };
  fetch(0);
#pragma unroll
  for (int j = 0; j < G::NJ; ++j) {
    if (j + 1 < G::NJ) fetch(j + 1);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < G::MI; ++i) {
      f32x4 x, y;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = acc[i][j][e] * widen<T>((bv[j & 1][i][e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
        y[e] = acc[i][j][e] * widen<T>((av[j & 1][i][e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
      }
      G::put(lds, i, j, narrow4<T>(x[0], x[1], x[2], x[3]));
      u32x2 v = narrow4<T>(y[0], y[1], y[2], y[3]);
      // narrowed here, into a sum's registers, and not where it leaves
      asm volatile("" : "+v"(v));
      acc[i][j][0] = __uint_as_float(v[0]);
      acc[i][j][1] = __uint_as_float(v[1]);
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

// One weight's gradient [n, m] = B^T A: row j is column j of B against the columns
// of A, over the tokens.
struct WeightGrad {
  Matrix a, b;
  int32_t m, n, tokens, accumulate;
  uint32_t first;  // its first workgroup
  void* out;
  int64_t ld;
};

template <typename T, bool F32OUT, bool SMALL>
__device__ __forceinline__ void dw_tile(uint32_t block, const WeightGrad& w) {
  using G = typename TileOf<SMALL, T, true, true>::G;
  const auto lds = G::shared();
  int32_t mt, nt;
  if (!tile_of(block, tiles_of<G::kCols>(w.n), tiles_of<G::kRows>(w.m), nt, mt)) return;
  const int32_t m0 = mt * G::kRows, n0 = nt * G::kCols, accumulate = w.accumulate;
  f32x4 acc[G::MI][G::NJ];
  G::run(by_cols(w.a, m0, w.tokens), by_cols(w.b, n0, w.tokens), w.tokens, lds, acc);
  if (!F32OUT && !accumulate) {
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
    for (int i = 0; i < G::MI; ++i) {
      const int32_t m = m0 + G::row(wave, i) + 4 * (lane >> 4);
      const int64_t at = (int64_t)n * w.ld + m;
      f32x4 d = acc[i][j];
      if constexpr (F32OUT) {
        float* o = (float*)w.out + at;
        if (m + 4 <= w.m) {
          if (accumulate) d = *(const f32x4_a4*)o + d;
          *(f32x4_a4*)o = d;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (m + e < w.m) o[e] = accumulate ? o[e] + d[e] : d[e];
        }
      } else {
        uint16_t* o = (uint16_t*)w.out + at;
        if (m + 4 <= w.m) {
          const u32x2 q = *(const u32x2_a2*)o;
          *(u32x2_a2*)o = narrow4<T>(widen<T>(q[0] & 0xFFFFu) + d[0], widen<T>(q[0] >> 16) + d[1],
                                     widen<T>(q[1] & 0xFFFFu) + d[2], widen<T>(q[1] >> 16) + d[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (m + e < w.m) o[e] = (uint16_t)narrow<T>(widen<T>(o[e]) + d[e]);
        }
      }
    }
  }
}

// Workgroups from w.first on take dWd, those before dh: whichever has the longer
// contraction comes first.
template <typename T, bool F32OUT, bool SMALL>
__global__ __launch_bounds__(SMALL ? 256 : 512) void k_ffn_back1(DhArgs d, uint32_t dh_first,
                                                                 WeightGrad w) {
  const bool weight = w.first > dh_first ? blockIdx.x >= w.first : blockIdx.x < dh_first;
  if (weight) dw_tile<T, F32OUT, SMALL>(blockIdx.x - w.first, w);
  else dh_tile<T, SMALL>(blockIdx.x - dh_first, d);
}

// dx first, then dWg and dWu.
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

OutArgs out_args(const zero_ffn_t* f, const FfnPlan& p, void* ws, Matrix a1, Matrix a2, Matrix b1,
                 Matrix b2, int32_t split, void* out, int64_t ldo) {
  const int64_t ht = (f->hidden + 255) / 256, tt = (f->tokens + 255) / 256;
  return OutArgs{a1, a2, b1, b2, (int32_t)f->tokens, (int32_t)f->hidden, (int32_t)f->inner, split,
                 tt * 256, (int32_t)(ht * 256), at<float>(ws, p.acc), (uint16_t*)out, ldo};
}
uint32_t grid_of(int64_t rows, int64_t cols, int64_t tile, int64_t times = 1) {
  return tile_grid((rows + tile - 1) / tile, (cols + tile - 1) / tile * times);
}

template <typename T>
int join_t(const OutArgs& o, hipStream_t stream) {
  if (o.split == 1) return (int)hipSuccess;
  const int64_t cols = 4 * kPackThreads, most = 65535;
  for (int64_t t0 = 0; t0 < o.tokens; t0 += most) {
    const int64_t n = o.tokens - t0 < most ? o.tokens - t0 : most;
    hipLaunchKernelGGL((k_ffn_join<T>),
                       dim3((uint32_t)((o.hidden + cols - 1) / cols), (uint32_t)n),
                       dim3(kPackThreads), 0, stream, o.acc + t0 * o.acc_ld, o.split, o.acc_rows,
                       o.acc_ld, o.hidden, o.out + t0 * o.ldo, o.ldo);
    ZK_LAUNCHED();
  }
  return (int)hipSuccess;
}

template <typename T, bool SAVE, bool SMALL>
auto in_kernel(int32_t act) {
  return act == ZERO_ACT_SILU        ? k_ffn_in<T, ZERO_ACT_SILU, SAVE, SMALL>
         : act == ZERO_ACT_GELU      ? k_ffn_in<T, ZERO_ACT_GELU, SAVE, SMALL>
         : act == ZERO_ACT_GELU_TANH ? k_ffn_in<T, ZERO_ACT_GELU_TANH, SAVE, SMALL>
                                     : k_ffn_in<T, ZERO_ACT_RELU, SAVE, SMALL>;
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
  const auto in = p.small_in ? (saved ? in_kernel<T, true, true>(f->act)
                                      : in_kernel<T, false, true>(f->act))
                             : (saved ? in_kernel<T, true, false>(f->act)
                                      : in_kernel<T, false, false>(f->act));
  hipLaunchKernelGGL(in, dim3(grid_of(2 * F, T_, p.small_in ? 128 : 256)),
                     dim3(p.small_in ? 256 : 512), 0, stream, x, wg, wu, (int32_t)T_, (int32_t)F,
                     (int32_t)p.inner_pad, to);
  ZK_LAUNCHED();
  const Matrix h{to.h, (int32_t)to.ld, (int32_t)p.inner_pad};
  const OutArgs o = out_args(f, p, ws, wd, wd, h, h, p.split_y, y, ldy);
  const uint32_t blocks = grid_of(T_, H, p.small_out ? 128 : 256, o.split);
  if (p.small_out)
    hipLaunchKernelGGL((k_ffn_out<T, true>), dim3(blocks), dim3(256), 0, stream, o);
  else
    hipLaunchKernelGGL((k_ffn_out<T, false>), dim3(blocks), dim3(512), 0, stream, o);
  ZK_LAUNCHED();
  return join_t<T>(o, stream);
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
  WeightGrad down{h, dy, (int32_t)F, (int32_t)H, (int32_t)T_, g->accumulate, 0, g->dw_down,
                  g->lddw_down};
  WeightGrad gate{x, dg, (int32_t)H, (int32_t)F, (int32_t)T_, g->accumulate, 0, g->dw_gate,
                  g->lddw_gate};
  WeightGrad up{x, du, (int32_t)H, (int32_t)F, (int32_t)T_, g->accumulate, 0, g->dw_up,
                g->lddw_up};
  const DhArgs dh{wd, dy, (int32_t)T_, (int32_t)H, (int32_t)F, Fp, (const uint16_t*)saved->act,
                  (const uint16_t*)saved->slope, saved->ld, (uint16_t*)dg.p, (uint16_t*)du.p};
  const bool through = T_ > 0 && (g->dx || g->dw_gate || g->dw_up);
  const uint32_t dh_blocks = through ? grid_of(F, T_, tile1) : 0;
  const uint32_t down_blocks = weights && down.out ? grid_of(H, F, tile1) : 0;
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
  const OutArgs o = out_args(f, p, ws, wg, wu, dg, du, p.split_dx, g->dx, g->lddx);
  const bool dx = g->dx && T_ > 0;
  gate.first = dx ? grid_of(T_, H, tile2, o.split) : 0;
  up.first = gate.first + (weights && gate.out ? grid_of(F, H, tile2) : 0);
  const uint32_t blocks = up.first + (weights && up.out ? grid_of(F, H, tile2) : 0);
  if (blocks) {
    if (p.small_back2)
      hipLaunchKernelGGL((k_ffn_back2<T, F32OUT, true>), dim3(blocks), dim3(256), 0, stream, o,
                         gate, up);
    else
      hipLaunchKernelGGL((k_ffn_back2<T, F32OUT, false>), dim3(blocks), dim3(512), 0, stream, o,
                         gate, up);
    ZK_LAUNCHED();
  }
  return dx ? join_t<T>(o, stream) : (int)hipSuccess;
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
