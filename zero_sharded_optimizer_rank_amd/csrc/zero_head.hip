// Loss of a language-model head and its gradients, in pieces of the
// vocabulary (see zero_head_t in zero_shard.h for the formulas).
//
//   1. scan and pack: the valid tokens, in order, become the rows of a packed
//      x (zero-padded to whole tiles), so that ignored tokens cost nothing and
//      whatever their x holds reaches no result;
//   2. loss: logits tile by tile on the matrix cores, transposed (vocabulary
//      rows x token columns) so that a token's logits lie in one lane's
//      registers; the tile leaves only (max, sum of exp) per token and 128
//      vocabulary rows, and the label's logit;
//   3. those partials are joined into lse and the loss;
//   4. gradient, piece by piece: the logits again, turned into
//      g = exp(l - lse) - [v = y] in 16 bits (the type the matrix cores
//      multiply), then dx += g w (fp32 between pieces) and dw = g^T x.
// All four products accumulate in fp32.
#include <stddef.h>

#include "head_gemm.h"
#include "head_internal.h"
#include "zero_device.h"

namespace zk {
namespace {

using namespace dev;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kScanThreads = 1024;
constexpr int kPackThreads = 256;
constexpr int kGemmThreads = 512;
constexpr int kJoinTokens = 64, kJoinWaves = 4;

// g's scale before it is rounded: |p - [v = y]| <= 1, so 2^15 keeps fp16 in
// range and p down to 2^-29 normal; bf16 has fp32's exponents.
template <typename T>
__device__ __forceinline__ constexpr float g_scale();
template <>
__device__ __forceinline__ constexpr float g_scale<BF16>() { return 1.0f; }
template <>
__device__ __forceinline__ constexpr float g_scale<FP16>() { return 32768.0f; }

template <typename T>
__device__ __forceinline__ uint32_t narrow(float x);
template <>
__device__ __forceinline__ uint32_t narrow<BF16>(float x) { return f2bf(x); }
template <>
__device__ __forceinline__ uint32_t narrow<FP16>(float x) { return f2h(x); }
template <typename T>
__device__ __forceinline__ float widen(uint32_t b);
template <>
__device__ __forceinline__ float widen<BF16>(uint32_t b) { return bf2f(b); }
template <>
__device__ __forceinline__ float widen<FP16>(uint32_t b) { return h2f(b); }

// --- 1. scan and pack --------------------------------------------------------
// One workgroup: the valid tokens in order.  index[r] is packed row r's token;
// label and (for the gradient alone) lse likewise.
__global__ __launch_bounds__(kScanThreads) void k_head_scan(
    const int64_t* __restrict__ labels, int32_t tokens, int32_t vocab, double loss_scale,
    int32_t mean, const float* __restrict__ lse_in, int32_t* __restrict__ index,
    int32_t* __restrict__ label, float* __restrict__ lse, HeadState* __restrict__ state) {
  __shared__ int32_t s_count[kScanThreads / 64];
  __shared__ int32_t s_bad;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  int32_t at = 0;  // valid tokens before this round
  for (int32_t t0 = 0; t0 < tokens; t0 += kScanThreads) {
    const int32_t t = t0 + threadIdx.x;
    const int64_t y = t < tokens ? labels[t] : -1;
    const bool ok = y >= 0 && y < vocab;
    if (y >= vocab) atomicAdd(&s_bad, 1);
    const uint64_t mask = __ballot(ok);
    if (lane == 0) s_count[wave] = __popcll(mask);
    __syncthreads();
    int32_t before = at, total = 0;
    for (int w = 0; w < kScanThreads / 64; ++w) {
      if (w < wave) before += s_count[w];
      total += s_count[w];
    }
    if (ok) {
      const int32_t r = before + __popcll(mask & ((1ull << lane) - 1));
      index[r] = t;
      label[r] = (int32_t)y;
      if (lse_in) lse[r] = lse_in[t];
    }
    at += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    double c = loss_scale;
    if (mean) c /= at > 0 ? (double)at : 1.0;
    state->valid = at;
    state->ticket = 0;
    state->bad = s_bad;
    state->coef = s_bad ? __builtin_nanf("") : (float)c;
  }
}

// Eight elements from p, of which the first n exist.
__device__ __forceinline__ u32x4 take8(const uint16_t* p, int64_t n, bool whole16) {
  if (whole16 && n >= 8) return *(const u32x4*)p;
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
  return v;
}

// Packed x: workgroup r copies valid token index[r], zero-padded; rows from
// the valid count to the next whole tile are zero.
__global__ __launch_bounds__(kPackThreads) void k_head_pack_x(
    const uint16_t* __restrict__ x, int64_t ldx, int32_t hidden, int32_t hidden_pad,
    const int32_t* __restrict__ index, const HeadState* __restrict__ state,
    uint16_t* __restrict__ out) {
  const int32_t r = blockIdx.x, valid = state->valid;
  if (r >= (valid + kHeadTile - 1) / kHeadTile * kHeadTile) return;
  u32x4* o = (u32x4*)(out + (int64_t)r * hidden_pad);
  const uint16_t* p = r < valid ? x + (int64_t)index[r] * ldx : nullptr;
  const bool whole16 = ((uintptr_t)p & 15) == 0;
  for (int32_t c = threadIdx.x; c < hidden_pad / 8; c += kPackThreads) {
    u32x4 v = {0, 0, 0, 0};
    if (p) v = take8(p + 8 * c, hidden - 8 * c, whole16);
    o[c] = v;
  }
}

// Packed w, for rows that do not start on 16-byte boundaries.
__global__ __launch_bounds__(kPackThreads) void k_head_pack_w(
    const uint16_t* __restrict__ w, int64_t ldw, int32_t hidden, int32_t hidden_pad,
    uint16_t* __restrict__ out) {
  const int64_t v = blockIdx.x;
  u32x4* o = (u32x4*)(out + v * hidden_pad);
  const uint16_t* p = w + v * ldw;
  const bool whole16 = ((uintptr_t)p & 15) == 0;
  for (int32_t c = threadIdx.x; c < hidden_pad / 8; c += kPackThreads)
    o[c] = take8(p + 8 * c, hidden - 8 * c, whole16);
}

// dx of the tokens that take no part.
__global__ __launch_bounds__(kPackThreads) void k_head_zero_dx(
    const int64_t* __restrict__ labels, int32_t vocab, int32_t hidden, uint16_t* __restrict__ dx,
    int64_t lddx) {
  const int64_t t = blockIdx.x;
  if (labels[t] >= 0 && labels[t] < vocab) return;
  for (int32_t h = threadIdx.x; h < hidden; h += kPackThreads) dx[t * lddx + h] = 0;
}

// --- 2. the logits' tiles ------------------------------------------------------
// A = w (vocabulary rows), B = packed x (token rows), both contiguous along
// the hidden axis.
template <typename T>
struct LogitTile {
  using G = Gemm<T, false, false>;

  static __device__ __forceinline__ bool run(const uint16_t* w, int64_t ldw, int64_t v0,
                                             int32_t vocab, const uint16_t* x, int32_t t0,
                                             int32_t hidden_pad, int32_t K,
                                             f32x16 (&acc)[G::MI][G::NJ]) {
    ZK_GEMM_LDS;
    const int64_t rows = vocab - v0;
    const Operand A{w + v0 * ldw, ldw * 2, (int32_t)(rows < G::BM ? rows : G::BM), K};
    const Operand B{x + (int64_t)t0 * hidden_pad, (int64_t)hidden_pad * 2, G::BN, K};
    G::run(A, B, K, lds, acc);
    return true;
  }
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Loss: (max, sum of exp(l - max)) of every token over each 128 vocabulary
// rows, and the label's logit.
template <typename T>
__global__ __launch_bounds__(kGemmThreads) void k_head_partials(
    const uint16_t* __restrict__ w, int64_t ldw, int32_t vocab, const uint16_t* __restrict__ x,
    int32_t hidden_pad, int32_t K, int32_t tokens_pad, const int32_t* __restrict__ label,
    const HeadState* __restrict__ state, float2* __restrict__ part, float* __restrict__ picked) {
  using L = LogitTile<T>;
  using G = typename L::G;
  static_assert(G::MI * 32 == kHeadPart, "one partial a wave");
  int32_t mt, nt;
  if (!tile_of(blockIdx.x, (uint32_t)((vocab + G::BM - 1) / G::BM),
               (uint32_t)((state->valid + G::BN - 1) / G::BN), mt, nt))
    return;
  const int32_t t0 = nt * G::BN;
  const int64_t v0 = (int64_t)mt * G::BM;
  constexpr int MI = G::MI, NJ = G::NJ;
  f32x16 acc[MI][NJ];
  L::run(w, ldw, v0, vocab, x, t0, hidden_pad, K, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t vw = v0 + (wave / 4) * MI * 32;  // the wave's first vocabulary row
  const int32_t rows = (int32_t)(vocab - vw < MI * 32 ? vocab - vw : MI * 32);
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int32_t t = t0 + (wave % 4) * NJ * 32 + j * 32 + (lane & 31);
    const int64_t y = t < state->valid ? (int64_t)label[t] - vw : -1;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int r = 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        float l = acc[i][j][e];
        if (r >= rows) l = -INFINITY;
        acc[i][j][e] = l;
        m = fmaxf(m, l);
        if (r == y) picked[t] = l;
      }
    m = fmaxf(m, __shfl_xor(m, 32));
    float s = 0.0f;
    if (m > -INFINITY) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) s += exp2_fast((acc[i][j][e] - m) * kLog2e);
    }
    // a row of NaN alone has max -inf: it must not pass for an empty one
    if (!(m > -INFINITY)) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (acc[i][j][e] != acc[i][j][e]) s = acc[i][j][e];
    }
    s += __shfl_xor(s, 32);
    if (lane < 32) part[(vw / kHeadPart) * tokens_pad + t] = float2{m, s};
  }
}

// --- 3. join -------------------------------------------------------------------
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float n = fmaxf(m, m2);
  if (n > -INFINITY)
    s = s * exp2_fast((m - n) * kLog2e) + s2 * exp2_fast((m2 - n) * kLog2e);
  else
    s = s + s2;  // both empty, or NaN
  m = n;
}

// Workgroup b joins the partials of 64 packed rows, kJoinWaves waves sharing
// the vocabulary; the last workgroup to finish sums the losses.
__global__ __launch_bounds__(64 * kJoinWaves) void k_head_join(
    const float2* __restrict__ part, int32_t parts, int32_t tokens_pad,
    const float* __restrict__ picked, const int32_t* __restrict__ index, float* __restrict__ lse,
    float* __restrict__ token_loss, float* __restrict__ lse_out, double* __restrict__ sums,
    int32_t mean, HeadState* __restrict__ state, zero_loss_result_t* __restrict__ res) {
  __shared__ float s_m[kJoinWaves][64], s_s[kJoinWaves][64];
  __shared__ uint32_t s_last;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t valid = state->valid;
  const int32_t r = blockIdx.x * kJoinTokens + lane;
  double loss = 0.0;
  if (r < valid) {
    float m = -INFINITY, s = 0.0f;
    for (int32_t p = wave; p < parts; p += kJoinWaves) {
      const float2 q = part[(int64_t)p * tokens_pad + r];
      join(m, s, q.x, q.y);
    }
    s_m[wave][lane] = m;
    s_s[wave][lane] = s;
  }
  __syncthreads();
  if (wave == 0 && r < valid) {
    float m = s_m[0][lane], s = s_s[0][lane];
    for (int k = 1; k < kJoinWaves; ++k) join(m, s, s_m[k][lane], s_s[k][lane]);
    const float l = m + __logf(s);
    const float d = (m - picked[r]) + __logf(s);
    lse[r] = l;
    if (lse_out) lse_out[index[r]] = l;
    if (token_loss) token_loss[index[r]] = d;
    loss = d;
  }
  if (wave == 0) {
    for (int off = 32; off > 0; off >>= 1) loss += __shfl_xor(loss, off);
    if (lane == 0) {
      sums[blockIdx.x] = loss;
      __threadfence();
      s_last = atomicAdd(&state->ticket, 1) == (int32_t)gridDim.x - 1 ? 1u : 0u;
    }
  }
  __syncthreads();
  if (!s_last || wave != 0) return;
  __threadfence();
  double total = 0.0;
  for (int32_t b = lane; b < (int32_t)gridDim.x; b += 64) total += sums[b];
  for (int off = 32; off > 0; off >>= 1) total += __shfl_xor(total, off);
  if (lane == 0) {
    if (state->bad) total = __builtin_nan("");
    res->loss_sum = total;
    res->loss = (float)(mean ? total / (valid > 0 ? (double)valid : 1.0) : total);
    res->reserved = 0;
    res->valid = valid;
    res->bad = state->bad;
  }
}

// Loss and lse of the tokens that take no part.
__global__ __launch_bounds__(kPackThreads) void k_head_ignored(
    const int64_t* __restrict__ labels, int32_t tokens, int32_t vocab, float* __restrict__ token_loss,
    float* __restrict__ lse) {
  const int32_t t = blockIdx.x * kPackThreads + threadIdx.x;
  if (t >= tokens) return;
  const int64_t y = labels[t];
  if (y >= 0 && y < vocab) return;
  const float v = y < 0 ? 0.0f : __builtin_nanf("");
  if (token_loss) token_loss[t] = v;
  if (lse) lse[t] = v;
}

// --- 4. gradient -----------------------------------------------------------------
// g of a piece: rows are packed tokens, columns the piece's vocabulary rows;
// columns past the vocabulary and rows past the valid tokens are zero.
template <typename T>
__global__ __launch_bounds__(kGemmThreads) void k_head_g(
    const uint16_t* __restrict__ w, int64_t ldw, int32_t vocab, const uint16_t* __restrict__ x,
    int32_t hidden_pad, int32_t K, const int32_t* __restrict__ label,
    const float* __restrict__ lse, const HeadState* __restrict__ state, int64_t piece0,
    int32_t piece, uint16_t* __restrict__ g) {
  using L = LogitTile<T>;
  using G = typename L::G;
  const int32_t valid = state->valid;
  const int32_t left = vocab - piece0 < piece ? (int32_t)(vocab - piece0) : piece;
  int32_t mt, nt;
  if (!tile_of(blockIdx.x, (uint32_t)((left + G::BM - 1) / G::BM),
               (uint32_t)((valid + G::BN - 1) / G::BN), mt, nt))
    return;
  const int32_t t0 = nt * G::BN;
  const int32_t c0 = mt * G::BM;  // column of g
  const int64_t v0 = piece0 + c0;
  constexpr int MI = G::MI, NJ = G::NJ;
  f32x16 acc[MI][NJ];
  L::run(w, ldw, v0, vocab, x, t0, hidden_pad, K, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t cw = c0 + (wave / 4) * MI * 32;
  const int32_t rows = left - cw;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int32_t t = t0 + (wave % 4) * NJ * 32 + j * 32 + (lane & 31);
    const bool there = t < valid;
    const float z = there ? lse[t] : 0.0f;
    const int64_t y = there ? (int64_t)label[t] - piece0 - cw : -1;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = 32 * i + 8 * q + 4 * (lane >> 5);
        uint32_t b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p = exp2_fast((acc[i][j][4 * q + e] - z) * kLog2e);
          if (r + e == y) p -= 1.0f;
          if (!there || r + e >= rows) p = 0.0f;
          b[e] = narrow<T>(p * g_scale<T>());
        }
        *(u32x2*)(g + (int64_t)t * piece + cw + r) = u32x2{b[0] | b[1] << 16, b[2] | b[3] << 16};
      }
  }
}

// dx: A = g (token rows, contiguous along the vocabulary), B = w (contiguous
// along the hidden axis).  Split s of the piece adds into its own fp32 block.
template <typename T>
__global__ __launch_bounds__(kGemmThreads) void k_head_dx(
    const uint16_t* __restrict__ g, int32_t piece, const uint16_t* __restrict__ w, int64_t ldw,
    int32_t vocab_left, int32_t hidden_w, int32_t hidden, int32_t hidden_pad, int32_t tokens_pad,
    int32_t split, int32_t part, int32_t first, const HeadState* __restrict__ state, float* __restrict__ acc_out) {
  using G = Gemm<T, false, true>;
  ZK_GEMM_LDS;
  const uint32_t ht = (uint32_t)((hidden + G::BN - 1) / G::BN);
  int32_t mt, nt;
  if (!tile_of(blockIdx.x, (uint32_t)((state->valid + G::BM - 1) / G::BM), ht * (uint32_t)split,
               mt, nt))
    return;
  const int32_t h0 = nt % ht * G::BN, t0 = mt * G::BM, ks = nt / ht, k0 = ks * part;
  int32_t K = piece - k0 < part ? piece - k0 : part;
  if (K > vocab_left - k0) K = vocab_left - k0;
  // g's columns are zero from the vocabulary's end to the next tile
  const Operand A{g + (int64_t)t0 * piece + k0, (int64_t)piece * 2, G::BM, (K + 7) & ~7};
  const Operand B{w + (int64_t)k0 * ldw + h0, ldw * 2, hidden_w - h0, K};
  constexpr int MI = G::MI, NJ = G::NJ;
  f32x16 acc[MI][NJ];
  G::run(A, B, K, lds, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float* out = acc_out + ((int64_t)ks * tokens_pad + t0 + (wave / 4) * MI * 32) * hidden_pad;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int32_t h = h0 + (wave % 4) * NJ * 32 + j * 32 + (lane & 31);
    if (h >= hidden_pad) continue;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      asm volatile("" ::: "memory");
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int r = 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        float* o = out + (int64_t)r * hidden_pad + h;
        *o = first ? acc[i][j][e] : *o + acc[i][j][e];
      }
    }
  }
}

// dx from the splits' sums.
template <typename T>
__global__ __launch_bounds__(kPackThreads) void k_head_dx_out(
    const float* __restrict__ acc, int32_t split, int32_t tokens_pad, int32_t hidden_pad,
    int32_t hidden, const int32_t* __restrict__ index, const HeadState* __restrict__ state,
    uint16_t* __restrict__ dx, int64_t lddx) {
  const int32_t r = blockIdx.x;
  if (r >= state->valid) return;
  const float c = state->coef / g_scale<T>();
  uint16_t* o = dx + (int64_t)index[r] * lddx;
  for (int32_t h = threadIdx.x; h < hidden; h += kPackThreads) {
    float s = 0.0f;
    for (int32_t k = 0; k < split; ++k) s += acc[((int64_t)k * tokens_pad + r) * hidden_pad + h];
    o[h] = (uint16_t)narrow<T>(s * c);
  }
}

// dw: A = g, B = packed x, both contiguous along their rows; the contraction
// runs over the tokens.
template <typename T, bool F32OUT>
__global__ __launch_bounds__(kGemmThreads) void k_head_dw(
    const uint16_t* __restrict__ g, int32_t piece, const uint16_t* __restrict__ x,
    int32_t hidden_pad, int32_t hidden, int32_t vocab_left, const HeadState* __restrict__ state,
    int32_t accumulate, void* __restrict__ dw, int64_t lddw) {
  using G = Gemm<T, true, true>;
  ZK_GEMM_LDS;
  int32_t mt, nt;
  if (!tile_of(blockIdx.x, (uint32_t)((vocab_left + G::BM - 1) / G::BM),
               (uint32_t)((hidden + G::BN - 1) / G::BN), mt, nt))
    return;
  const int32_t h0 = nt * G::BN, c0 = mt * G::BM;
  const int32_t K = state->valid;
  const float c = state->coef / g_scale<T>();
  const Operand A{g + c0, (int64_t)piece * 2, piece - c0, K};
  const Operand B{x + h0, (int64_t)hidden_pad * 2, hidden_pad - h0, K};
  constexpr int MI = G::MI, NJ = G::NJ;
  f32x16 acc[MI][NJ];
  G::run(A, B, K, lds, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool bad = state->bad != 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int32_t h = h0 + (wave % 4) * NJ * 32 + j * 32 + (lane & 31);
    if (h >= hidden) continue;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      asm volatile("" ::: "memory");
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int32_t v = c0 + (wave / 4) * MI * 32 + 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        if (v >= vocab_left) continue;
        const int64_t at = (int64_t)v * lddw + h;
        // bad labels alone (no valid token) still have to show
        float d = bad ? c : acc[i][j][e] * c;
        if constexpr (F32OUT) {
          float* o = (float*)dw + at;
          *o = accumulate ? *o + d : d;
        } else {
          uint16_t* o = (uint16_t*)dw + at;
          if (accumulate) d += widen<T>(*o);
          *o = (uint16_t)narrow<T>(d);
        }
      }
    }
  }
}

template <typename P>
P* at(void* ws, size_t off) { return (P*)((char*)ws + off); }

#define ZK_LAUNCHED()                              \
  do {                                             \
    const hipError_t e_ = hipGetLastError();       \
    if (e_ != hipSuccess) return (int)e_;          \
  } while (0)

struct WeightView {
  const uint16_t* w;
  int64_t ld;       // elements
  int32_t K;        // contraction length of the logits
  int32_t width;    // columns a row holds
};
WeightView weight_view(const zero_head_t* h, const HeadPlan& p, void* ws) {
  if (p.pack_w)
    return {at<const uint16_t>(ws, p.w), p.hidden_pad, (int32_t)p.hidden_pad,
            (int32_t)p.hidden_pad};
  return {(const uint16_t*)h->w, h->ldw, (int32_t)h->hidden, (int32_t)h->hidden};
}

template <typename T>
int loss_t(const zero_head_t* h, const HeadPlan& p, void* ws, float* token_loss, float* lse,
           zero_loss_result_t* res, hipStream_t stream) {
  const WeightView w = weight_view(h, p, ws);
  HeadState* state = at<HeadState>(ws, p.state);
  if (h->tokens > 0) {
    hipLaunchKernelGGL(k_head_partials<T>,
                       dim3(tile_grid(p.tokens_pad / 256, (h->vocab + 255) / 256)),
                       dim3(kGemmThreads), 0, stream, w.w, w.ld, (int32_t)h->vocab,
                       at<const uint16_t>(ws, p.x), (int32_t)p.hidden_pad, w.K,
                       (int32_t)p.tokens_pad, at<const int32_t>(ws, p.label), state,
                       at<float2>(ws, p.part), at<float>(ws, p.picked));
    ZK_LAUNCHED();
    if (token_loss || lse) {
      hipLaunchKernelGGL(k_head_ignored, dim3((uint32_t)((h->tokens + kPackThreads - 1) / kPackThreads)),
                         dim3(kPackThreads), 0, stream, h->labels, (int32_t)h->tokens,
                         (int32_t)h->vocab, token_loss, lse);
      ZK_LAUNCHED();
    }
  }
  hipLaunchKernelGGL(k_head_join, dim3((uint32_t)(p.tokens_pad / kJoinTokens)),
                     dim3(64 * kJoinWaves), 0, stream, at<const float2>(ws, p.part),
                     (int32_t)(((h->vocab + 255) / 256) * 2), (int32_t)p.tokens_pad,
                     at<const float>(ws, p.picked), at<const int32_t>(ws, p.index),
                     at<float>(ws, p.lse), token_loss, lse, at<double>(ws, p.sums), h->mean, state,
                     res);
  return (int)hipGetLastError();
}

template <typename T>
int grad_t(const zero_head_t* h, const HeadPlan& p, void* ws, const zero_head_grads_t* gr,
           hipStream_t stream) {
  const WeightView w = weight_view(h, p, ws);
  HeadState* state = at<HeadState>(ws, p.state);
  const uint32_t htiles = (uint32_t)((h->hidden + 255) / 256), ttiles = (uint32_t)(p.tokens_pad / 256);
  uint16_t* g = at<uint16_t>(ws, p.g);
  float* acc = at<float>(ws, p.acc);
  const uint16_t* x = at<const uint16_t>(ws, p.x);
  const int32_t part = (int32_t)((p.piece / p.split + kHeadStep - 1) / kHeadStep * kHeadStep);
  for (int64_t v0 = 0; v0 < h->vocab; v0 += p.piece) {
    const int64_t left = h->vocab - v0 < p.piece ? h->vocab - v0 : p.piece;
    const uint32_t vtiles = (uint32_t)((left + 255) / 256);
    if (h->tokens > 0) {
      hipLaunchKernelGGL(k_head_g<T>, dim3(tile_grid(ttiles, vtiles)), dim3(kGemmThreads), 0, stream,
                         w.w, w.ld, (int32_t)h->vocab, x, (int32_t)p.hidden_pad, w.K,
                         at<const int32_t>(ws, p.label), at<const float>(ws, p.lse), state, v0,
                         (int32_t)p.piece, g);
      ZK_LAUNCHED();
      hipLaunchKernelGGL(k_head_dx<T>, dim3(tile_grid(htiles * p.split, ttiles)),
                         dim3(kGemmThreads), 0, stream, g, (int32_t)p.piece, w.w + v0 * w.ld, w.ld,
                         (int32_t)left, w.width, (int32_t)h->hidden, (int32_t)p.hidden_pad,
                         (int32_t)p.tokens_pad, p.split, part, v0 == 0 ? 1 : 0, state, acc);
      ZK_LAUNCHED();
    }
    const size_t ew = gr->dw_dtype == ZERO_F32 ? 4 : 2;
    void* dw = (char*)gr->dw + ew * (size_t)(v0 * gr->lddw);
    if (gr->dw_dtype == ZERO_F32)
      hipLaunchKernelGGL((k_head_dw<T, true>), dim3(tile_grid(htiles, vtiles)), dim3(kGemmThreads), 0,
                         stream, g, (int32_t)p.piece, x, (int32_t)p.hidden_pad,
                         (int32_t)h->hidden, (int32_t)left, state, gr->accumulate, dw, gr->lddw);
    else
      hipLaunchKernelGGL((k_head_dw<T, false>), dim3(tile_grid(htiles, vtiles)), dim3(kGemmThreads), 0,
                         stream, g, (int32_t)p.piece, x, (int32_t)p.hidden_pad,
                         (int32_t)h->hidden, (int32_t)left, state, gr->accumulate, dw, gr->lddw);
    ZK_LAUNCHED();
  }
  if (h->tokens > 0)
    hipLaunchKernelGGL((k_head_dx_out<T>), dim3((uint32_t)h->tokens), dim3(kPackThreads), 0,
                       stream, acc, p.split, (int32_t)p.tokens_pad, (int32_t)p.hidden_pad,
                       (int32_t)h->hidden, at<const int32_t>(ws, p.index), state,
                       (uint16_t*)gr->dx, gr->lddx);
  return (int)hipGetLastError();
}

}  // namespace

int launch_head_pack(const zero_head_t* h, const HeadPlan& p, void* ws, const float* lse_in,
                     const zero_head_grads_t* gr, hipStream_t stream) {
  HeadState* state = at<HeadState>(ws, p.state);
  hipLaunchKernelGGL(k_head_scan, dim3(1), dim3(kScanThreads), 0, stream, h->labels,
                     (int32_t)h->tokens, (int32_t)h->vocab, h->loss_scale, h->mean, lse_in,
                     at<int32_t>(ws, p.index), at<int32_t>(ws, p.label), at<float>(ws, p.lse),
                     state);
  ZK_LAUNCHED();
  if (h->tokens > 0) {
    hipLaunchKernelGGL(k_head_pack_x, dim3((uint32_t)p.tokens_pad), dim3(kPackThreads), 0, stream,
                       (const uint16_t*)h->x, h->ldx, (int32_t)h->hidden, (int32_t)p.hidden_pad,
                       at<const int32_t>(ws, p.index), state, at<uint16_t>(ws, p.x));
    ZK_LAUNCHED();
    if (gr) {
      hipLaunchKernelGGL(k_head_zero_dx, dim3((uint32_t)h->tokens), dim3(kPackThreads), 0, stream,
                         h->labels, (int32_t)h->vocab, (int32_t)h->hidden, (uint16_t*)gr->dx,
                         gr->lddx);
      ZK_LAUNCHED();
    }
  }
  if (p.pack_w) {
    hipLaunchKernelGGL(k_head_pack_w, dim3((uint32_t)h->vocab), dim3(kPackThreads), 0, stream,
                       (const uint16_t*)h->w, h->ldw, (int32_t)h->hidden, (int32_t)p.hidden_pad,
                       at<uint16_t>(ws, p.w));
    ZK_LAUNCHED();
  }
  return (int)hipSuccess;
}

int launch_head_loss(const zero_head_t* h, const HeadPlan& p, void* ws, float* token_loss,
                     float* lse, zero_loss_result_t* res, hipStream_t stream) {
  return h->dtype == ZERO_BF16 ? loss_t<BF16>(h, p, ws, token_loss, lse, res, stream)
                               : loss_t<FP16>(h, p, ws, token_loss, lse, res, stream);
}

int launch_head_grad(const zero_head_t* h, const HeadPlan& p, void* ws,
                     const zero_head_grads_t* gr, hipStream_t stream) {
  return h->dtype == ZERO_BF16 ? grad_t<BF16>(h, p, ws, gr, stream)
                               : grad_t<FP16>(h, p, ws, gr, stream);
}

}  // namespace zk
