// Gated feed-forward block and its gradients on the matrix cores (see
// zero_ffn_t in zero_shard.h for the formulas).
//
//   forward   k_ffn_in    both projections of a tile at once, activation and
//                         product on the fp32 sums: h leaves in 16 bits
//             k_ffn_out   y = h Wd^T
//   backward  k_ffn_dh    dh = dy Wd, whose tile becomes dg, du (and h again, from
//                         the kept g and u) before it leaves
//             k_ffn_dw    the three weights' gradients in one launch
//             k_ffn_out   dx = dg Wg + du Wu, one contraction over both
// All products are 256 x 256 tiles of head_gemm.h with fp32 sums; every operand
// is read as it lies.
#include <stddef.h>

#include "ffn_device.h"

namespace zk {
namespace {

using namespace dev;

constexpr int kGemmThreads = 512;
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

// --- forward -------------------------------------------------------------------
struct PairProduct {
  Operand gate, up, B;
  __device__ __forceinline__ const Operand& a0(int32_t&) const { return gate; }
  __device__ __forceinline__ const Operand& a1(int32_t&) const { return up; }
  __device__ __forceinline__ const Operand& b(int32_t&) const { return B; }
};

// A tile: 128 inner columns of both projections, 256 tokens, so that a lane holds g
// and u of the same element.
template <typename T>
__global__ __launch_bounds__(kGemmThreads) void k_ffn_in(Matrix x, Matrix w_gate, Matrix w_up,
                                                         int32_t tokens, int32_t inner,
                                                         int32_t inner_pad, int32_t act,
                                                         uint16_t* __restrict__ h,
                                                         uint16_t* __restrict__ gate,
                                                         uint16_t* __restrict__ up, int64_t ld) {
  using G = Gemm<T, false, false, true>;
  ZK_GEMM_LDS;
  int32_t mt, nt;
  if (!tile_of(blockIdx.x, (uint32_t)((inner + 127) / 128), (uint32_t)((tokens + 255) / 256), mt,
               nt))
    return;
  const int32_t f0 = mt * 128, t0 = nt * 256;
  const PairProduct src{by_rows(w_gate, f0, inner, 128), by_rows(w_up, f0, inner, 128),
                        by_rows(x, t0, tokens, 256)};
  f32x4 acc[G::MI][G::NJ];
  G::run(src, x.width, lds, acc);
  if (gate) {
    G::transposed(lds, acc, narrow4<T>, [&](int col, int row, u32x4 v) {
      // rows: 64 of g, 64 of u, and again
      const int32_t t = t0 + col, f = f0 + row / 128 * 64 + row % 64;
      if (t < tokens && f < inner_pad)
        *(u32x4*)((row & 64 ? up : gate) + (int64_t)t * ld + f) = v;
    });
    __syncthreads();
  }
  with_act(act, [&](auto a) {
#pragma unroll
    for (int j = 0; j < G::NJ; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = activated(a, acc[i][j][e]) * acc[4 + i][j][e];
        G::put_half(lds, i, j, narrow4<T>(v[0], v[1], v[2], v[3]));
      }
  });
  __syncthreads();
  G::take_half(lds, [&](int col, int row, u32x4 v) {
    const int32_t t = t0 + col, f = f0 + row;
    if (t < tokens && f < inner_pad) *(u32x4*)(h + (int64_t)t * inner_pad + f) = v;
  });
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

template <typename T, bool DX>
__global__ __launch_bounds__(kGemmThreads) void k_ffn_out(Matrix a1, Matrix a2, Matrix b1,
                                                          Matrix b2, int32_t tokens,
                                                          int32_t hidden, int32_t inner,
                                                          int32_t split, int64_t acc_rows,
                                                          int32_t acc_ld,
                                                          float* __restrict__ acc_out,
                                                          uint16_t* __restrict__ out,
                                                          int64_t ldo) {
  using G = Gemm<T, DX, false>;
  ZK_GEMM_LDS;
  const uint32_t ht = (uint32_t)((hidden + 255) / 256);
  int32_t mt, nt;
  if (!tile_of(blockIdx.x, (uint32_t)((tokens + 255) / 256), ht * (uint32_t)split, mt, nt)) return;
  const int32_t h0 = (int32_t)((uint32_t)nt % ht) * 256, t0 = mt * 256;
  const int32_t part = (int32_t)((uint32_t)nt / ht);
  const int32_t stages = (inner + kStage - 1) / kStage, all = DX ? 2 * stages : stages;
  const int32_t s0 = (int32_t)((int64_t)all * part / split);
  const int32_t s1 = (int32_t)((int64_t)all * (part + 1) / split);
  Products<DX> src;
  src.A1 = DX ? by_cols(a1, h0, inner) : by_rows(a1, h0, hidden, 256);
  src.B1 = by_rows(b1, t0, tokens, 256);
  if constexpr (DX) {
    src.A2 = by_cols(a2, h0, inner);
    src.B2 = by_rows(b2, t0, tokens, 256);
  }
  src.k0 = s0 * kStage;
  src.k1 = stages * kStage;
  src.end = s1 * kStage;
  f32x4 acc[G::MI][G::NJ];
  G::run(src, (s1 - s0) * kStage, lds, acc);
  if (split == 1) {
    G::transposed(lds, acc, narrow4<T>, [&](int col, int row, u32x4 v) {
      const int32_t t = t0 + col, c = h0 + row;
      if (t < tokens && c < hidden) store_row(out + (int64_t)t * ldo, c, hidden, v);
    });
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < G::NJ; ++j) {
    const int32_t t = t0 + (wave % 4) * 64 + j * 16 + (lane & 15);
    float* o = acc_out + ((int64_t)part * acc_rows + t) * acc_ld;
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < G::MI; ++i)
      *(f32x4*)(o + h0 + wave / 4 * 128 + 16 * i + 4 * (lane >> 4)) = acc[i][j];
  }
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
// A tile of dh: A = Wd by its columns (inner), B = dy by its rows.  Each lane reads
// g and u of its elements, and the tile leaves as h, dg and du.
template <typename T, int ACT>
__global__ __launch_bounds__(kGemmThreads) void k_ffn_dh(Matrix w_down, Matrix dy, int32_t tokens,
                                                         int32_t hidden, int32_t inner,
                                                         int32_t inner_pad,
                                                         const uint16_t* __restrict__ gate,
                                                         const uint16_t* __restrict__ up,
                                                         int64_t ld, uint16_t* __restrict__ h,
                                                         uint16_t* __restrict__ dg,
                                                         uint16_t* __restrict__ du) {
  using G = Gemm<T, true, false>;
  ZK_GEMM_LDS;
  int32_t mt, nt;
  if (!tile_of(blockIdx.x, (uint32_t)((inner + 255) / 256), (uint32_t)((tokens + 255) / 256), mt,
               nt))
    return;
  const int32_t f0 = mt * 256, t0 = nt * 256;
  f32x4 acc[G::MI][G::NJ];
  G::run(by_cols(w_down, f0, hidden), by_rows(dy, t0, tokens, 256), hidden, lds, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < G::NJ; ++j) {
    const int32_t t = t0 + (wave % 4) * 64 + j * 16 + (lane & 15);
    const int64_t row = (int64_t)(t < tokens ? t : tokens - 1) * ld;
    lds_char* p = G::column(lds, j);
    // 16 loads at a time: more would not fit beside the sums (what lies past the
    // operands is not stored)
    u32x2 gv[G::MI], uv[G::MI];
#pragma unroll
    for (int i = 0; i < G::MI; ++i) {
      const int32_t f = f0 + wave / 4 * 128 + 16 * i + 4 * (lane >> 4);
      gv[i] = *(const u32x2*)(gate + row + (f < inner_pad ? f : 0));
      uv[i] = *(const u32x2*)(up + row + (f < inner_pad ? f : 0));
    }
#pragma unroll
    for (int i = 0; i < G::MI; ++i) {
      f32x4 hh, x, y;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float g = widen<T>((gv[i][e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
        const float u = widen<T>((uv[i][e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
        float slope;
        const float v = activated(Act<ACT>{}, g, slope);
        hh[e] = v * u;
        x[e] = acc[i][j][e] * u * slope;
        y[e] = acc[i][j][e] * v;
      }
      G::put(p, i, j, narrow4<T>(hh[0], hh[1], hh[2], hh[3]));
      u32x2 xs = narrow4<T>(x[0], x[1], x[2], x[3]), ys = narrow4<T>(y[0], y[1], y[2], y[3]);
      // narrowed here, into the sums' registers, and not where they leave
      asm volatile("" : "+v"(xs), "+v"(ys));
      acc[i][j] = f32x4{__uint_as_float(xs[0]), __uint_as_float(xs[1]), __uint_as_float(ys[0]),
                        __uint_as_float(ys[1])};
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }
  auto leave = [&](uint16_t* out) {
    __syncthreads();
    G::take(lds, [&](int col, int row, u32x4 v) {
      const int32_t t = t0 + col, f = f0 + row;
      if (t < tokens && f < inner_pad) *(u32x4*)(out + (int64_t)t * inner_pad + f) = v;
    });
    __syncthreads();
  };
  leave(h);
#pragma unroll
  for (int d = 0; d < 2; ++d) {
#pragma unroll
    for (int j = 0; j < G::NJ; ++j) {
      lds_char* p = G::column(lds, j);
#pragma unroll
      for (int i = 0; i < G::MI; ++i)
        G::put(p, i, j, u32x2{__float_as_uint(acc[i][j][2 * d]),
                              __float_as_uint(acc[i][j][2 * d + 1])});
    }
    leave(d == 0 ? dg : du);
  }
}

// One weight's gradient [n, m] = B^T A: row j is column j of B against the columns
// of A, over the tokens.
struct WeightGrad {
  Matrix a, b;
  int32_t m, n;
  uint32_t first;  // workgroup of its first tile
  void* out;       // NULL: not wanted
  int64_t ld;
};
struct WeightGrads {
  WeightGrad w[3];
};

template <typename T, bool F32OUT>
__global__ __launch_bounds__(kGemmThreads) void k_ffn_dw(WeightGrads all, int32_t tokens,
                                                         int32_t accumulate) {
  using G = Gemm<T, true, true>;
  ZK_GEMM_LDS;
  const int which = blockIdx.x >= all.w[2].first ? 2 : blockIdx.x >= all.w[1].first ? 1 : 0;
  const WeightGrad w = all.w[which];
  int32_t mt, nt;
  if (!tile_of(blockIdx.x - w.first, (uint32_t)((w.n + 255) / 256), (uint32_t)((w.m + 255) / 256),
               nt, mt))
    return;
  const int32_t m0 = mt * 256, n0 = nt * 256;
  f32x4 acc[G::MI][G::NJ];
  G::run(by_cols(w.a, m0, tokens), by_cols(w.b, n0, tokens), tokens, lds, acc);
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
    const int32_t n = n0 + wave % 4 * 64 + j * 16 + (lane & 15);
    if (n >= w.n) continue;
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < G::MI; ++i) {
      const int32_t m = m0 + wave / 4 * 128 + 16 * i + 4 * (lane >> 4);
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

template <typename T, bool DX>
int out_t(const zero_ffn_t* f, const FfnPlan& p, void* ws, Matrix a1, Matrix a2, Matrix b1,
          Matrix b2, int32_t split, void* out, int64_t ldo, hipStream_t stream) {
  const int64_t ht = (f->hidden + 255) / 256, tt = (f->tokens + 255) / 256;
  hipLaunchKernelGGL((k_ffn_out<T, DX>), dim3(tile_grid(tt, ht * split)), dim3(kGemmThreads), 0,
                     stream, a1, a2, b1, b2, (int32_t)f->tokens, (int32_t)f->hidden,
                     (int32_t)f->inner, split, tt * 256, (int32_t)(ht * 256),
                     at<float>(ws, p.acc), (uint16_t*)out, ldo);
  ZK_LAUNCHED();
  if (split == 1) return (int)hipSuccess;
  const int64_t cols = 4 * kPackThreads, most = 65535;
  for (int64_t t0 = 0; t0 < f->tokens; t0 += most) {
    const int64_t n = f->tokens - t0 < most ? f->tokens - t0 : most;
    hipLaunchKernelGGL((k_ffn_join<T>),
                       dim3((uint32_t)((f->hidden + cols - 1) / cols), (uint32_t)n),
                       dim3(kPackThreads), 0, stream,
                       at<const float>(ws, p.acc) + t0 * ht * 256, split, tt * 256,
                       (int32_t)(ht * 256), (int32_t)f->hidden, (uint16_t*)out + t0 * ldo, ldo);
    ZK_LAUNCHED();
  }
  return (int)hipSuccess;
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
  uint16_t* h = at<uint16_t>(ws, p.h);
  hipLaunchKernelGGL((k_ffn_in<T>), dim3(tile_grid((F + 127) / 128, (T_ + 255) / 256)),
                     dim3(kGemmThreads), 0, stream, x, wg, wu, (int32_t)T_, (int32_t)F,
                     (int32_t)p.inner_pad, f->act, h, saved ? (uint16_t*)saved->gate : nullptr,
                     saved ? (uint16_t*)saved->up : nullptr, saved ? saved->ld : 0);
  ZK_LAUNCHED();
  const Matrix hm{h, (int32_t)p.inner_pad, (int32_t)p.inner_pad};
  return out_t<T, false>(f, p, ws, wd, wd, hm, hm, p.split_y, y, ldy, stream);
}

template <typename T>
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
  const Matrix h{at<uint16_t>(ws, p.h), Fp, Fp}, dg{at<uint16_t>(ws, p.dg), Fp, Fp},
      du{at<uint16_t>(ws, p.du), Fp, Fp};
  const int64_t ftiles = (F + 255) / 256, htiles = (H + 255) / 256, ttiles = (T_ + 255) / 256;
  if (T_ > 0) {
    const auto dh = f->act == ZERO_ACT_SILU        ? k_ffn_dh<T, ZERO_ACT_SILU>
                    : f->act == ZERO_ACT_GELU      ? k_ffn_dh<T, ZERO_ACT_GELU>
                    : f->act == ZERO_ACT_GELU_TANH ? k_ffn_dh<T, ZERO_ACT_GELU_TANH>
                                                   : k_ffn_dh<T, ZERO_ACT_RELU>;
    hipLaunchKernelGGL(dh, dim3(tile_grid(ftiles, ttiles)), dim3(kGemmThreads), 0, stream, wd, dy,
                       (int32_t)T_, (int32_t)H, (int32_t)F, Fp, (const uint16_t*)saved->gate,
                       (const uint16_t*)saved->up, saved->ld, (uint16_t*)h.p, (uint16_t*)dg.p,
                       (uint16_t*)du.p);
    ZK_LAUNCHED();
  }
  if (T_ > 0 || !g->accumulate) {
    WeightGrads all;
    all.w[0] = WeightGrad{x, dg, (int32_t)H, (int32_t)F, 0, g->dw_gate, g->lddw_gate};
    all.w[1] = WeightGrad{x, du, (int32_t)H, (int32_t)F, 0, g->dw_up, g->lddw_up};
    all.w[2] = WeightGrad{h, dy, (int32_t)F, (int32_t)H, 0, g->dw_down, g->lddw_down};
    uint32_t blocks = 0;
    const uint32_t each = tile_grid(ftiles, htiles);
    for (WeightGrad& w : all.w) {
      w.first = blocks;
      if (w.out) blocks += each;
    }
    // one that is not wanted has no workgroups: the next one starts where it does
    if (blocks) {
      if (g->dw_dtype == ZERO_F32)
        hipLaunchKernelGGL((k_ffn_dw<T, true>), dim3(blocks), dim3(kGemmThreads), 0, stream, all,
                           (int32_t)T_, g->accumulate);
      else
        hipLaunchKernelGGL((k_ffn_dw<T, false>), dim3(blocks), dim3(kGemmThreads), 0, stream, all,
                           (int32_t)T_, g->accumulate);
      ZK_LAUNCHED();
    }
  }
  if (!g->dx || T_ == 0) return (int)hipSuccess;
  return out_t<T, true>(f, p, ws, wg, wu, dg, du, p.split_dx, g->dx, g->lddx, stream);
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
  return f->dtype == ZERO_BF16 ? backward_t<BF16>(f, p, ws, saved, g, stream)
                               : backward_t<FP16>(f, p, ws, saved, g, stream);
}

}  // namespace zk
