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
//   4. gradient, piece by piece: g = exp(l - lse) - [v = y] in 16 bits (the
//      type the matrix cores multiply), then dx += g w (fp32 between pieces)
//      and dw = g^T x.  The piece that the loss formed last has its
//      exponentials in g's block already; the logits of the others are formed
//      again.
// All products accumulate in fp32.
#include <stddef.h>

#include "head_device.h"

namespace zk {
namespace {

using namespace dev;

constexpr int kScanThreads = 1024;
constexpr int kPackThreads = 256;
constexpr int kGemmThreads = 512;
constexpr int kJoinTokens = 16, kJoinWaves = 16, kJoinBatch = 8;

// --- 1. scan and pack --------------------------------------------------------
// Ways to split dx's contraction: the fewest whose tiles come close to filling
// whole rounds of the 256 CUs (a token count that leaves 208 tiles would
// idle a fifth of the chip; eight times as many tiles, a twentieth).  One wave;
// lane l weighs l + 1 ways.
constexpr int32_t kCus = 256;
__device__ __forceinline__ int32_t dx_split(int32_t tiles, int32_t most, int lane) {
  const float c = (float)((tiles * (lane + 1) + kCus - 1) / kCus) / (float)(lane + 1);
  int32_t best = 1;
  float cost = __shfl(c, 0);
  for (int32_t s = 2; s <= most; ++s) {
    const float cs = __shfl(c, s - 1);
    if (cs < 0.97f * cost) {
      cost = cs;
      best = s;
    }
  }
  return best;
}

// One workgroup: the valid tokens in order.  index[r] is packed row r's token;
// label and (for the gradient alone) lse likewise.  Bound by latency: 5 us for
// up to 2048 tokens, 12 us for 8192.
__global__ __launch_bounds__(kScanThreads) void k_head_scan(
    const int64_t* __restrict__ labels, int32_t tokens, int32_t vocab, double loss_scale,
    int32_t mean, int32_t htiles, int32_t most, const float* __restrict__ lse_in,
    int32_t* __restrict__ index, int32_t* __restrict__ label, float* __restrict__ lse,
    HeadState* __restrict__ state) {
  __shared__ int32_t s_count[kScanThreads / 64];
  __shared__ int32_t s_bad;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  int32_t at = 0;  // valid tokens before these
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
  if (wave != 0) return;
  const int32_t ttiles = (int32_t)((at + kHeadTile - 1) / kHeadTile);
  const int32_t split = dx_split(ttiles * htiles, most, lane);
  if (lane == 0) {
    state->split = split;
    double c = loss_scale;
    if (mean) c /= at > 0 ? (double)at : 1.0;
    state->valid = at;
    state->ticket = 0;
    state->bad = s_bad;
    state->coef = s_bad ? __builtin_nanf("") : (float)c;
  }
}

// Workgroup r: packed row r copies valid token index[r], zero-padded (rows from
// the valid count to the next whole tile are zero); and if token r takes no
// part, its loss, lse and dx are written.  Bound by memory: 8192 x 4096, 22 us
// (5.6 TB/s).
__global__ __launch_bounds__(kPackThreads) void k_head_pack_x(
    const uint16_t* __restrict__ x, int64_t ldx, int32_t tokens, int32_t hidden,
    int32_t hidden_pad, int32_t vocab, const int64_t* __restrict__ labels,
    const int32_t* __restrict__ index, const HeadState* __restrict__ state,
    uint16_t* __restrict__ out, float* __restrict__ token_loss, float* __restrict__ lse,
    uint16_t* __restrict__ dx, int64_t lddx) {
  const int32_t r = blockIdx.x, valid = state->valid;
  if (r < tokens) {
    const int64_t y = labels[r];
    if (y < 0 || y >= vocab) {
      if (threadIdx.x == 0) {
        const float v = y < 0 ? 0.0f : __builtin_nanf("");
        if (token_loss) token_loss[r] = v;
        if (lse) lse[r] = v;
      }
      if (dx)
        for (int32_t h = threadIdx.x; h < hidden; h += kPackThreads)
          dx[r * lddx + h] = y < 0 ? 0 : kNan16;
    }
  }
  if (r >= (valid + kHeadTile - 1) / kHeadTile * kHeadTile) return;
  u32x4* o = (u32x4*)(out + (int64_t)r * hidden_pad);
  const uint16_t* p = r < valid ? x + (int64_t)index[r] * ldx : nullptr;
  for (int32_t c = threadIdx.x; c < hidden_pad / 8; c += kPackThreads) {
    u32x4 v = {0, 0, 0, 0};
    if (p) v = take8(p + 8 * c, hidden - 8 * c);
    o[c] = v;
  }
}

// Packed w, for rows that do not start on 16-byte boundaries.
constexpr uint32_t kPackRows = 1 << 20;  // workgroups at most: a launch holds 2^32 threads
__global__ __launch_bounds__(kPackThreads) void k_head_pack_w(
    const uint16_t* __restrict__ w, int64_t ldw, int32_t vocab, int32_t hidden,
    int32_t hidden_pad, uint16_t* __restrict__ out) {
  for (int64_t v = blockIdx.x; v < vocab; v += gridDim.x) {
    u32x4* o = (u32x4*)(out + v * hidden_pad);
    const uint16_t* p = w + v * ldw;
    for (int32_t c = threadIdx.x; c < hidden_pad / 8; c += kPackThreads)
      o[c] = take8(p + 8 * c, hidden - 8 * c);
  }
}

// --- 2. the logits' tiles ------------------------------------------------------
// A = w (vocabulary rows), B = packed x (token rows), both contiguous along
// the hidden axis.
template <typename T>
struct LogitTile {
  using G = Gemm<T, false, false>;

  static __device__ __forceinline__ void run(const uint16_t* w, int64_t ldw, int64_t v0,
                                             int32_t vocab, const uint16_t* x, int32_t t0,
                                             int32_t hidden_pad, int32_t K, const GemmLds& lds,
                                             f32x4 (&acc)[G::MI][G::NJ]) {
    const int64_t rows = vocab - v0;
    const Operand A{w + v0 * ldw, (int32_t)ldw * 2, (int32_t)(rows < G::BM ? rows : G::BM), K};
    const Operand B{x + (int64_t)t0 * hidden_pad, hidden_pad * 2, G::BN, K};
    G::run(A, B, K, lds, acc);
  }
};

// Loss: (m, g_scale sum of 2^(l log2 e - m)) of every token over each 128
// vocabulary rows, m the largest l log2 e rounded up, the label's row left out,
// and the label's logit: a confident token's loss is log(1 + the others' sum),
// whose digits a sum that held the label's 1 would have lost.  Where the
// gradient follows in the same call, the exponentials of the piece of the
// vocabulary that starts at `kept` stay in g's block (rounded to 16 bits):
// k_head_rescale turns them into g without forming those logits again.
// Bound by the matrix cores (busy 75 to 80%, at the chip's power limit): 7373 x
// 128256 x 4096, bf16, 5.5 ms (1410 TFLOP/s); with the exponentials stored, 3277
// tokens 2.62 ms (1320).  1024 x 50257 x 1600, fp16, 0.206 ms (800): 788 tiles on
// 256 CUs, four rounds for three.
template <typename T>
__global__ __launch_bounds__(kGemmThreads) void k_head_partials(
    const uint16_t* __restrict__ w, int64_t ldw, int32_t vocab, const uint16_t* __restrict__ x,
    int32_t hidden_pad, int32_t K, int32_t tokens_pad, const int32_t* __restrict__ label,
    const HeadState* __restrict__ state, float2* __restrict__ part, double* __restrict__ picked,
    int64_t kept, int32_t piece, uint16_t* __restrict__ g) {
  using L = LogitTile<T>;
  using G = typename L::G;
  static_assert(G::MI * 16 == kHeadPart, "one partial a wave");
  int32_t mt, nt;
  if (!tile_of(blockIdx.x, (uint32_t)((vocab + G::BM - 1) / G::BM),
               (uint32_t)((state->valid + G::BN - 1) / G::BN), mt, nt))
    return;
  const int32_t t0 = nt * G::BN;
  const int64_t v0 = (int64_t)mt * G::BM;
  constexpr int MI = G::MI, NJ = G::NJ;
  f32x4 acc[MI][NJ];
  ZK_GEMM_LDS;
  L::run(w, ldw, v0, vocab, x, t0, hidden_pad, K, lds, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t vw = v0 + (wave / 4) * kHeadPart;  // the wave's first vocabulary row
  const int32_t rows = (int32_t)(vocab - vw < kHeadPart ? vocab - vw : kHeadPart);
  const int r0 = 4 * (lane >> 4);  // element (i, e) is row r0 + 16i + e
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int32_t t = t0 + (wave % 4) * 64 + j * 16 + (lane & 15);
    const int64_t y = t < state->valid ? (int64_t)label[t] - vw : -1;
    if (rows < kHeadPart) {  // the vocabulary ends here
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (r0 + 16 * i + e >= rows) acc[i][j][e] = -INFINITY;
    }
    // the element of this lane that is the label's, if one is
    const bool mine = y >= 0 && y < kHeadPart && ((int32_t)y >> 2 & 3) == lane >> 4;
    const int want = mine ? ((int32_t)y >> 4) * 4 + ((int32_t)y & 3) : -1;
    if (__any(mine)) {
      float p = 0.0f;
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool hit = want == 4 * i + e;
          p = hit ? acc[i][j][e] : p;
          acc[i][j][e] = hit ? -INFINITY : acc[i][j][e];
        }
      if (mine) picked[t] = p;
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) m = __builtin_elementwise_maximum(m, acc[i][j][e]);
    m = __builtin_elementwise_maximum(m, __shfl_xor(m, 16));  // NaN if one is
    m = __builtin_elementwise_maximum(m, __shfl_xor(m, 32));
    // in base 2, rounded up to a whole number, so that taking it off is exact;
    // one multiply-add and one exponential a value; rows that are -inf alone give 0
    m = __builtin_ceilf(m * kLog2e);
    const float shift = (m == -INFINITY ? 0.0f : -m) + g_log2<T>();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[i][j][e] = exp2_fast(__builtin_fmaf(acc[i][j][e], kLog2e, shift));
        s += acc[i][j][e];
      }
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (lane < 16) part[(vw / kHeadPart) * tokens_pad + t] = float2{m, s};
  }
  if (g && v0 >= kept) {
    G::transposed(lds, acc, narrow4<T>,
                  [&](int col, int row, u32x4 v) {
                    *(u32x4*)(g + (int64_t)(t0 + col) * piece + (v0 - kept) + row) = v;
                  });
  }
}

// --- 3. join -------------------------------------------------------------------
// Workgroup b joins the partials of 16 packed rows (a line of partials), 64
// strips of the vocabulary side by side; the last workgroup to finish sums the
// losses.  Sums, logarithm and exponential are fp64 from here: few values, and a
// confident token's loss would lose digits in fp32.  Bound by latency: 3277
// tokens x 1002 partials 20 us, 37 x 393 7 us.
__global__ __launch_bounds__(64 * kJoinWaves) void k_head_join(
    const float2* __restrict__ part, int32_t parts, int32_t tokens_pad,
    const double* __restrict__ picked, const int32_t* __restrict__ index, float* __restrict__ lse,
    float* __restrict__ dy, float* __restrict__ token_loss, float* __restrict__ lse_out,
    double* __restrict__ sums, double scale, int32_t mean, HeadState* __restrict__ state,
    zero_loss_result_t* __restrict__ res) {
  constexpr int kStrips = 4 * kJoinWaves;
  __shared__ float s_m[kJoinWaves][kJoinTokens], s_s[kJoinWaves][kJoinTokens];
  __shared__ uint32_t s_last;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t valid = state->valid;
  const int32_t r = blockIdx.x * kJoinTokens + (lane & 15);
  double loss = 0.0;
  float m = -INFINITY, s = 0.0f;
  if (r < valid) {
    for (int32_t p = threadIdx.x >> 4; p < parts; p += kStrips * kJoinBatch) {
      float2 q[kJoinBatch];
#pragma unroll
      for (int k = 0; k < kJoinBatch; ++k) {
        q[k] = float2{-INFINITY, 0.0f};
        if (p + k * kStrips < parts) q[k] = part[(int64_t)(p + k * kStrips) * tokens_pad + r];
      }
#pragma unroll
      for (int k = 0; k < kJoinBatch; ++k) join(m, s, q[k].x, q[k].y);
    }
  }
#pragma unroll
  for (int off = 16; off < 64; off <<= 1) {
    const float m2 = __shfl_xor(m, off), s2 = __shfl_xor(s, off);
    // both sides join in the same order, so that all lanes agree
    const bool low = !(lane & off);
    float a = low ? m : m2, b = low ? s : s2;
    join(a, b, low ? m2 : m, low ? s2 : s);
    m = a;
    s = b;
  }
  if (lane < kJoinTokens) {
    s_m[wave][lane] = m;
    s_s[wave][lane] = s;
  }
  __syncthreads();
  if (wave == 0 && lane < kJoinTokens && r < valid) {
    for (int k = 1; k < kJoinWaves; ++k) join(m, s, s_m[k][lane], s_s[k][lane]);
    // with o the others' sum over the label's exponential: log(1 + o)
    const double y = picked[r], top = (double)m / (double)kLog2e, gap = top - y;
    const double sum = (double)s * scale;
    const double more = gap > 0.0 ? log(sum + exp(-gap)) : log1p(sum * exp(gap));
    double d = gap > 0.0 ? gap + more : more;
    if (!(gap == gap) || y == INFINITY) d = __builtin_nan("");
    // a label at -inf: the loss is infinite, the others' lse is not
    const float l = (float)(y == -INFINITY && d == d ? top + more : y + d);
    lse[r] = l;
    if (lse_out) lse_out[index[r]] = l;
    if (token_loss) token_loss[index[r]] = (float)d;
    dy[r] = (float)expm1(-d);
    loss = (float)d;
  }
  if (wave == 0) {
    for (int off = 8; off > 0; off >>= 1) loss += __shfl_xor(loss, off);
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

// --- 4. gradient -----------------------------------------------------------------
// g of a piece: rows are packed tokens, columns the piece's vocabulary rows;
// columns past the vocabulary and rows past the valid tokens are zero.  Rounded
// once to 16 bits, the type the matrix cores multiply (dx and dw keep 32-bit
// sums).  The label's element is e^-loss - 1 (dy) where the loss ran in the same
// call; from the lse alone (dy NULL) a confident token's loses the digits that
// the fp32 lse has lost.  Bound as k_head_partials: 4096 x 128256 x 4096, bf16,
// 3.18 ms (1350 TFLOP/s).
template <typename T>
__global__ __launch_bounds__(kGemmThreads) void k_head_g(
    const uint16_t* __restrict__ w, int64_t ldw, int32_t vocab, const uint16_t* __restrict__ x,
    int32_t hidden_pad, int32_t K, const int32_t* __restrict__ label,
    const float* __restrict__ lse, const float* __restrict__ dy,
    const HeadState* __restrict__ state, int64_t piece0, int32_t piece,
    uint16_t* __restrict__ g) {
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
  f32x4 acc[MI][NJ];
  ZK_GEMM_LDS;
  L::run(w, ldw, v0, vocab, x, t0, hidden_pad, K, lds, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t cw = c0 + (wave / 4) * kHeadPart;
  const int32_t rows = left - cw;
  const int r0 = 4 * (lane >> 4);  // element (i, e) is row r0 + 16i + e
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int32_t t = t0 + (wave % 4) * 64 + j * 16 + (lane & 15);
    const bool there = t < valid;
    const float z = there ? lse[t] : 0.0f;
    const int64_t y = there ? (int64_t)label[t] - piece0 - cw : -1;
    const bool mine = y >= 0 && y < kHeadPart && ((int32_t)y >> 2 & 3) == lane >> 4;
    const int want = mine ? ((int32_t)y >> 4) * 4 + ((int32_t)y & 3) : -1;
    const float shift = g_log2<T>() - z * kLog2e;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[i][j][e] = exp2_fast(__builtin_fmaf(acc[i][j][e], kLog2e, shift));
    if (__any(mine)) {
      const float at = dy && mine ? dy[t] * g_scale<T>() : 0.0f;
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = dy ? at : acc[i][j][e] - g_scale<T>();
          acc[i][j][e] = want == 4 * i + e ? p : acc[i][j][e];
        }
    }
    if (rows < kHeadPart || !__all(there)) {  // the vocabulary's or the tokens' end
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!there || r0 + 16 * i + e >= rows) acc[i][j][e] = 0.0f;
    }
  }
  G::transposed(lds, acc, narrow4<T>,
                [&](int col, int row, u32x4 v) {
                  *(u32x4*)(g + (int64_t)(t0 + col) * piece + c0 + row) = v;
                });
}

// g of the piece whose exponentials were kept: 2^(l log2 e - m) 2^(m - lse log2
// e) - [v = y], m the reference of the 128 vocabulary rows.  The label's element is
// e^-loss - 1.  A workgroup takes 8 tokens (half a line of partials), a wave
// each, and kRescaleCols columns, all of them loaded before the first is used.
// Bound by memory: 3277 x 128256, 0.29 ms (5.9 TB/s).
constexpr int kRescaleCols = 2048, kRescaleWaves = 8, kRescaleLoads = kRescaleCols / 512;
template <typename T>
__global__ __launch_bounds__(64 * kRescaleWaves) void k_head_rescale(
    uint16_t* __restrict__ g, int32_t piece, int32_t left, const float2* __restrict__ part,
    int32_t part0, int32_t tokens_pad, const int32_t* __restrict__ label, int64_t piece0,
    const float* __restrict__ lse, const float* __restrict__ dy,
    const HeadState* __restrict__ state) {
  const int32_t valid = state->valid;
  const int32_t t = blockIdx.y * kRescaleWaves + (threadIdx.x >> 6);
  if (t >= (valid + kHeadTile - 1) / kHeadTile * kHeadTile) return;
  const int32_t first = (int32_t)blockIdx.x * kRescaleCols, c0 = first + (threadIdx.x & 63) * 8;
  const int32_t end = (left + kHeadTile - 1) / kHeadTile * kHeadTile;  // at most piece
  u32x4* o = (u32x4*)(g + (int64_t)t * piece + c0);
  if (t >= valid) {
#pragma unroll
    for (int k = 0; k < kRescaleLoads; ++k)
      if (c0 + 512 * k < end) o[64 * k] = u32x4{0, 0, 0, 0};
    return;
  }
  u32x4 v[kRescaleLoads];
  float f[kRescaleLoads];
#pragma unroll
  for (int k = 0; k < kRescaleLoads; ++k) {
    const int32_t c = c0 + 512 * k;
    v[k] = u32x4{0, 0, 0, 0};
    f[k] = 0.0f;
    if (c < left) {
      v[k] = o[64 * k];
      f[k] = part[(int64_t)(part0 + c / kHeadPart) * tokens_pad + t].x;
    }
  }
  const float z = lse[t];
  const int64_t y = (int64_t)label[t] - piece0;
  const bool plain = first + kRescaleCols <= left && (y < first || y >= first + kRescaleCols);
#pragma unroll
  for (int k = 0; k < kRescaleLoads; ++k) {
    const int32_t c = c0 + 512 * k;
    const float s = exp2_fast(__builtin_fmaf(-z, kLog2e, f[k]));
    float p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = widen<T>((v[k][e >> 1] >> (16 * (e & 1))) & 0xFFFFu) * s;
    if (!plain) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (c + e == y) p[e] = dy[t] * g_scale<T>();
        if (c + e >= left) p[e] = 0.0f;
      }
      if (c >= end) continue;
    }
    const u32x2 a = narrow4<T>(p[0], p[1], p[2], p[3]), b = narrow4<T>(p[4], p[5], p[6], p[7]);
    o[64 * k] = u32x4{a[0], a[1], b[0], b[1]};
  }
}

// dx: A = w (rows of the tile: hidden columns, contiguous along them), B = g
// (token rows, contiguous along the vocabulary).  Split s of the piece adds
// into its own fp32 block.  Bound by the matrix cores: 3277 x 128256 x 4096,
// bf16, 2.75 ms (1250 TFLOP/s); 1024 x 50257 x 1600, fp16, 0.166 ms (990).
template <typename T>
__global__ __launch_bounds__(kGemmThreads) void k_head_dx(
    const uint16_t* __restrict__ g, int32_t piece, const uint16_t* __restrict__ w, int64_t ldw,
    int32_t vocab_left, int32_t hidden_w, int32_t hidden, int32_t hidden_pad, int32_t tokens_pad,
    int32_t first, const HeadState* __restrict__ state, float* __restrict__ acc_out) {
  using G = Gemm<T, true, false>;
  ZK_GEMM_LDS;
  const uint32_t ht = (uint32_t)((hidden + G::BM - 1) / G::BM);
  const uint32_t tt = (uint32_t)((state->valid + G::BN - 1) / G::BN);
  const int32_t split = state->split;
  const int32_t part = (piece / split + kStage - 1) / kStage * kStage;
  int32_t mt, nt;
  if (!tile_of(blockIdx.x, tt, ht * (uint32_t)split, mt, nt)) return;
  const int32_t h0 = nt % ht * G::BM, t0 = mt * G::BN, ks = nt / ht, k0 = ks * part;
  int32_t K = piece - k0 < part ? piece - k0 : part;
  if (K > vocab_left - k0) K = vocab_left - k0;
  // g's columns are zero from the vocabulary's end to the next tile
  const Operand A{w + (int64_t)k0 * ldw + h0, (int32_t)ldw * 2, hidden_w - h0, K};
  const Operand B{g + (int64_t)t0 * piece + k0, piece * 2, G::BN, (K + 7) & ~7};
  constexpr int MI = G::MI, NJ = G::NJ;
  f32x4 acc[MI][NJ];
  G::run(A, B, K, lds, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int32_t t = t0 + (wave % 4) * 64 + j * 16 + (lane & 15);
    float* out = acc_out + ((int64_t)ks * tokens_pad + t) * hidden_pad;
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int32_t h = h0 + wave / 4 * 128 + 16 * i + 4 * (lane >> 4);
      if (h >= hidden_pad) continue;
      f32x4* o = (f32x4*)(out + h);
      *o = first ? acc[i][j] : *o + acc[i][j];
    }
  }
}

// dx from the splits' sums, four columns a thread.  Bound by memory: 2047 x 8192
// 24 us (4.1 TB/s); 1024 x 1600 of nine splits 17 us.
template <typename T>
__global__ __launch_bounds__(kPackThreads) void k_head_dx_out(
    const float* __restrict__ acc, int32_t tokens_pad, int32_t hidden_pad,
    int32_t hidden, const int32_t* __restrict__ index, const HeadState* __restrict__ state,
    uint16_t* __restrict__ dx, int64_t lddx) {
  const int32_t r = blockIdx.y, valid = state->valid;
  const int32_t h = (blockIdx.x * kPackThreads + threadIdx.x) * 4;
  if (r >= valid || h >= hidden) return;
  const int32_t split = state->split;
  const float c = state->coef / g_scale<T>();
  const float* p = acc + (int64_t)r * hidden_pad + h;
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int32_t k = 0; k < split; ++k)
    s += *(const f32x4*)(p + (int64_t)k * tokens_pad * hidden_pad);
  uint16_t* o = dx + (int64_t)index[r] * lddx + h;
  s *= c;
  if (h + 4 <= hidden) {
    *(u32x2_a2*)o = narrow4<T>(s[0], s[1], s[2], s[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (h + e < hidden) o[e] = (uint16_t)narrow<T>(s[e]);
  }
}

// dw: A = packed x (rows of the tile: hidden columns), B = g (vocabulary
// rows), both contiguous along their rows; the contraction runs over the
// tokens.  Bound by the matrix cores: 3277 x 128256 x 4096, bf16, 2.56 ms (1340
// TFLOP/s); 2047 x 32000 x 8192 0.94 ms (1140).  Only a 16-bit dw that is
// overwritten leaves through LDS in whole lines; the others go out from the
// registers, 8 or 16 bytes of 16 rows at a time: 4096 x 128256 x 4096, bf16 3.2 ms,
// bf16 accumulated 3.6, fp32 3.4, fp32 accumulated 3.7.
template <typename T, bool F32OUT>
__global__ __launch_bounds__(kGemmThreads) void k_head_dw(
    const uint16_t* __restrict__ g, int32_t piece, const uint16_t* __restrict__ x,
    int32_t hidden_pad, int32_t hidden, int32_t vocab_left, const HeadState* __restrict__ state,
    int32_t accumulate, void* __restrict__ dw, int64_t lddw) {
  using G = Gemm<T, true, true>;
  ZK_GEMM_LDS;
  int32_t mt, nt;
  if (!tile_of(blockIdx.x, (uint32_t)((vocab_left + G::BN - 1) / G::BN),
               (uint32_t)((hidden + G::BM - 1) / G::BM), mt, nt))
    return;
  const int32_t h0 = nt * G::BM, c0 = mt * G::BN;
  const int32_t K = state->valid;
  const float c = state->coef / g_scale<T>();
  const Operand A{x + h0, hidden_pad * 2, hidden_pad - h0, K};
  const Operand B{g + c0, piece * 2, piece - c0, K};
  constexpr int MI = G::MI, NJ = G::NJ;
  f32x4 acc[MI][NJ];
  G::run(A, B, K, lds, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (!F32OUT && !accumulate) {
    uint16_t* out = (uint16_t*)dw;
    G::transposed(lds, acc,
                  [c](float p, float q, float r, float s) {
                    return narrow4<T>(p * c, q * c, r * c, s * c);
                  },
                  [&](int col, int row, u32x4 d) {
                    const int32_t v = c0 + col, h = h0 + row;
                    if (v >= vocab_left || h >= hidden) return;
                    uint16_t* o = out + (int64_t)v * lddw + h;
                    if (h + 8 <= hidden) {
                      *(u32x4_a2*)o = d;
                    } else {
#pragma unroll
                      for (int e = 0; e < 8; ++e)
                        if (h + e < hidden) o[e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
                    }
                  });
    return;
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int32_t v = c0 + wave % 4 * 64 + j * 16 + (lane & 15);
    if (v >= vocab_left) continue;
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int32_t h = h0 + wave / 4 * 128 + 16 * i + 4 * (lane >> 4);
      const int64_t at = (int64_t)v * lddw + h;
      f32x4 d = acc[i][j] * c;
      if constexpr (F32OUT) {
        float* o = (float*)dw + at;
        if (h + 4 <= hidden) {
          if (accumulate) d = *(const f32x4_a4*)o + d;
          *(f32x4_a4*)o = d;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (h + e < hidden) o[e] = accumulate ? o[e] + d[e] : d[e];
        }
      } else {
        uint16_t* o = (uint16_t*)dw + at;
        if (h + 4 <= hidden) {
          const u32x2 q = *(const u32x2_a2*)o;
          *(u32x2_a2*)o = narrow4<T>(widen<T>(q[0] & 0xFFFFu) + d[0], widen<T>(q[0] >> 16) + d[1],
                                     widen<T>(q[1] & 0xFFFFu) + d[2], widen<T>(q[1] >> 16) + d[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (h + e < hidden) o[e] = (uint16_t)narrow<T>(widen<T>(o[e]) + d[e]);
        }
      }
    }
  }
}

// kept: the vocabulary row from which the exponentials stay in g's block, or
// none if the loss stands alone.
template <typename T>
int loss_t(const zero_head_t* h, const HeadPlan& p, void* ws, float* token_loss, float* lse,
           bool keep, zero_loss_result_t* res, hipStream_t stream) {
  const WeightView w = weight_view(h, p, ws);
  HeadState* state = at<HeadState>(ws, p.state);
  const int64_t tile = p.few ? kHeadPart : kHeadTile;  // vocabulary rows a workgroup takes
  if (!p.few && h->tokens > 0) {
    hipLaunchKernelGGL(k_head_partials<T>,
                       dim3(tile_grid(p.tokens_pad / 256, (h->vocab + 255) / 256)),
                       dim3(kGemmThreads), 0, stream, w.w, w.ld, (int32_t)h->vocab,
                       at<const uint16_t>(ws, p.x), (int32_t)p.hidden_pad, w.K,
                       (int32_t)p.tokens_pad, at<const int32_t>(ws, p.label), state,
                       at<float2>(ws, p.part), at<double>(ws, p.picked), p.kept,
                       (int32_t)p.piece, keep ? at<uint16_t>(ws, p.g) : nullptr);
    ZK_LAUNCHED();
  }
  const int64_t joins = h->tokens > 0 ? (h->tokens + kJoinTokens - 1) / kJoinTokens : 1;
  hipLaunchKernelGGL(k_head_join, dim3((uint32_t)joins),
                     dim3(64 * kJoinWaves), 0, stream, at<const float2>(ws, p.part),
                     (int32_t)((h->vocab + tile - 1) / tile * tile / kHeadPart),
                     (int32_t)p.tokens_pad,
                     at<const double>(ws, p.picked), at<const int32_t>(ws, p.index),
                     at<float>(ws, p.lse), at<float>(ws, p.dy), token_loss, lse,
                     at<double>(ws, p.sums), 1.0 / (double)g_scale<T>(), h->mean, state, res);
  return (int)hipGetLastError();
}

// One piece of the vocabulary, from row v0: g, then its share of dx and its dw.
// loss_ran: in the same call; its exponentials of the first piece (the last
// of the vocabulary) lie in g's block.
template <typename T>
int piece_t(const zero_head_t* h, const HeadPlan& p, void* ws, const zero_head_grads_t* gr,
            int64_t v0, bool loss_ran, bool first, hipStream_t stream) {
  const WeightView w = weight_view(h, p, ws);
  HeadState* state = at<HeadState>(ws, p.state);
  const uint32_t htiles = (uint32_t)((h->hidden + 255) / 256);
  const uint32_t ttiles = (uint32_t)(p.tokens_pad / 256);
  uint16_t* g = at<uint16_t>(ws, p.g);
  const uint16_t* x = at<const uint16_t>(ws, p.x);
  const int64_t left = h->vocab - v0 < p.piece ? h->vocab - v0 : p.piece;
  const uint32_t vtiles = (uint32_t)((left + 255) / 256);
  const int32_t* label = at<const int32_t>(ws, p.label);
  const float* lse = at<const float>(ws, p.lse);
  if (h->tokens > 0) {
    if (loss_ran && first)
      hipLaunchKernelGGL(k_head_rescale<T>,
                         dim3((uint32_t)((left + kRescaleCols - 1) / kRescaleCols),
                              (uint32_t)(p.tokens_pad / kRescaleWaves)),
                         dim3(64 * kRescaleWaves), 0, stream, g, (int32_t)p.piece, (int32_t)left,
                         at<const float2>(ws, p.part), (int32_t)(v0 / kHeadPart),
                         (int32_t)p.tokens_pad, label, v0, lse, at<const float>(ws, p.dy), state);
    else
      hipLaunchKernelGGL(k_head_g<T>, dim3(tile_grid(ttiles, vtiles)), dim3(kGemmThreads), 0,
                         stream, w.w, w.ld, (int32_t)h->vocab, x, (int32_t)p.hidden_pad, w.K,
                         label, lse, loss_ran ? at<const float>(ws, p.dy) : nullptr, state, v0,
                         (int32_t)p.piece, g);
    ZK_LAUNCHED();
    hipLaunchKernelGGL(k_head_dx<T>, dim3(tile_grid(htiles * p.split, ttiles)),
                       dim3(kGemmThreads), 0, stream, g, (int32_t)p.piece, w.w + v0 * w.ld, w.ld,
                       (int32_t)left, w.width, (int32_t)h->hidden, (int32_t)p.hidden_pad,
                       (int32_t)p.tokens_pad, first ? 1 : 0, state,
                       at<float>(ws, p.acc));
    ZK_LAUNCHED();
  }
  const size_t ew = gr->dw_dtype == ZERO_F32 ? 4 : 2;
  void* dw = (char*)gr->dw + ew * (size_t)(v0 * gr->lddw);
  if (gr->dw_dtype == ZERO_F32)
    hipLaunchKernelGGL((k_head_dw<T, true>), dim3(tile_grid(htiles, vtiles)), dim3(kGemmThreads),
                       0, stream, g, (int32_t)p.piece, x, (int32_t)p.hidden_pad,
                       (int32_t)h->hidden, (int32_t)left, state, gr->accumulate, dw, gr->lddw);
  else
    hipLaunchKernelGGL((k_head_dw<T, false>), dim3(tile_grid(htiles, vtiles)), dim3(kGemmThreads),
                       0, stream, g, (int32_t)p.piece, x, (int32_t)p.hidden_pad,
                       (int32_t)h->hidden, (int32_t)left, state, gr->accumulate, dw, gr->lddw);
  return (int)hipGetLastError();
}

template <typename T>
int grad_t(const zero_head_t* h, const HeadPlan& p, void* ws, const zero_head_grads_t* gr,
           bool kept, hipStream_t stream) {
  // the kept piece lies in g's block: it goes first
  int e = piece_t<T>(h, p, ws, gr, p.kept, kept, true, stream);
  for (int64_t v0 = 0; !e && v0 < p.kept; v0 += p.piece)
    e = piece_t<T>(h, p, ws, gr, v0, kept, false, stream);
  if (e) return e;
  if (h->tokens > 0)
    hipLaunchKernelGGL((k_head_dx_out<T>),
                       dim3((uint32_t)((h->hidden + 4 * kPackThreads - 1) / (4 * kPackThreads)),
                            (uint32_t)h->tokens),
                       dim3(kPackThreads), 0, stream, at<const float>(ws, p.acc),
                       (int32_t)p.tokens_pad, (int32_t)p.hidden_pad, (int32_t)h->hidden,
                       at<const int32_t>(ws, p.index), at<HeadState>(ws, p.state),
                       (uint16_t*)gr->dx, gr->lddx);
  return (int)hipGetLastError();
}

}  // namespace

int launch_head_pack(const zero_head_t* h, const HeadPlan& p, void* ws, const float* lse_in,
                     float* token_loss, float* lse, const zero_head_grads_t* gr,
                     hipStream_t stream) {
  if (p.few) return launch_few_logits(h, p, ws, lse_in, token_loss, lse, gr, stream);
  HeadState* state = at<HeadState>(ws, p.state);
  hipLaunchKernelGGL(k_head_scan, dim3(1), dim3(kScanThreads), 0, stream, h->labels,
                     (int32_t)h->tokens, (int32_t)h->vocab, h->loss_scale, h->mean,
                     (int32_t)((h->hidden + kHeadTile - 1) / kHeadTile), p.split, lse_in,
                     at<int32_t>(ws, p.index), at<int32_t>(ws, p.label), at<float>(ws, p.lse),
                     state);
  ZK_LAUNCHED();
  if (h->tokens > 0) {
    hipLaunchKernelGGL(k_head_pack_x, dim3((uint32_t)p.tokens_pad), dim3(kPackThreads), 0, stream,
                       (const uint16_t*)h->x, h->ldx, (int32_t)h->tokens, (int32_t)h->hidden,
                       (int32_t)p.hidden_pad, (int32_t)h->vocab, h->labels,
                       at<const int32_t>(ws, p.index), state, at<uint16_t>(ws, p.x), token_loss,
                       lse, gr ? (uint16_t*)gr->dx : nullptr, gr ? gr->lddx : 0);
    ZK_LAUNCHED();
  }
  if (p.pack_w) {
    const uint32_t rows = h->vocab < kPackRows ? (uint32_t)h->vocab : kPackRows;
    hipLaunchKernelGGL(k_head_pack_w, dim3(rows), dim3(kPackThreads), 0, stream,
                       (const uint16_t*)h->w, h->ldw, (int32_t)h->vocab, (int32_t)h->hidden,
                       (int32_t)p.hidden_pad, at<uint16_t>(ws, p.w));
    ZK_LAUNCHED();
  }
  return (int)hipSuccess;
}

int launch_head_loss(const zero_head_t* h, const HeadPlan& p, void* ws, float* token_loss,
                     float* lse, bool keep, zero_loss_result_t* res, hipStream_t stream) {
  return h->dtype == ZERO_BF16 ? loss_t<BF16>(h, p, ws, token_loss, lse, keep, res, stream)
                               : loss_t<FP16>(h, p, ws, token_loss, lse, keep, res, stream);
}

int launch_head_grad(const zero_head_t* h, const HeadPlan& p, void* ws,
                     const zero_head_grads_t* gr, bool kept, hipStream_t stream) {
  if (p.few) return launch_few_grads(h, p, ws, gr, kept, stream);
  return h->dtype == ZERO_BF16 ? grad_t<BF16>(h, p, ws, gr, kept, stream)
                               : grad_t<FP16>(h, p, ws, gr, kept, stream);
}

}  // namespace zk
