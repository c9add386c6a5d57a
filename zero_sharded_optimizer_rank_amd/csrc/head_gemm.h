// Matrix-product core of the head's loss: one workgroup computes a BM x BN tile
// of A B^T on gfx950's matrix cores, fp32 accumulators in registers, and hands
// them to an epilogue.
//
// A is M x K and B is N x K.  Each operand lies in memory in one of two ways:
//   rows    element (m, k) at base + m*ld + k: the contraction is contiguous
//   cols    element (m, k) at base + k*ld + m: the tile's rows are contiguous
// so that all three products of the loss (logits: rows x rows; dx: rows x
// cols; dw: cols x cols) read their operands as they lie, with no transposed
// copy.  LDS holds a step of 64 contraction elements of each operand, twice
// (one step is computed while the next arrives); global memory goes straight
// to LDS (16 bytes a lane, no registers), and the lanes pick their global
// addresses so that the LDS image is swizzled and every fragment read is free
// of bank conflicts:
//   rows    128 bytes a row; 16-byte chunk c of row r lies at c ^ (r & 7)
//   cols    2*BM bytes a contraction index k; 32-byte pair p lies at p ^ f(k),
//           f(k) = 2 * ((k & 3) | (k >> 3 & 1) << 2); fragments come back
//           transposed (ds_read_b64_tr_b16)
// Lanes whose element lies outside the operand read zero (buffer bounds), so
// ragged edges cost nothing and nothing outside the operand is touched.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace zk {
namespace dev {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) char lds_char;

struct BF16 {};
struct FP16 {};

__device__ __forceinline__ f32x16 mfma(BF16, s16x8 a, s16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma(FP16, s16x8 a, s16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// One operand of a tile.
struct Operand {
  const void* base;   // element (0, 0) of the tile
  int64_t ld;         // bytes between rows (rows) or contraction indexes (cols)
  int32_t count;      // rows of the tile that exist (rows), or columns from base to
                      // the end of a memory row (cols); multiples of 8 along memory
  int32_t k;          // contraction indexes that exist (rows: a multiple of 8)
};

constexpr int kStep = 64;

// f(k) of the cols layout, from bits 0-1 and bit 3 of k; a tile of 128 rows
// has only 8 pairs a memory row and takes the low part.
template <int R>
__device__ __forceinline__ int swizzle(int k01, int k3) {
  return (2 * (k01 | k3 << 2)) & (R / 16 - 1);
}

// R tile rows staged by `waves` waves; COLS as above.
template <int R, bool COLS, int WAVES>
struct Stage {
  static constexpr int kBytes = R * kStep * 2;
  static constexpr int kLoads = kBytes / (WAVES * 1024);  // 1 KiB wave loads of a wave and step
  static_assert(kLoads * WAVES * 1024 == kBytes, "whole loads");
  static constexpr int kRowBytes = COLS ? R * 2 : kStep * 2;
  static constexpr int kLoadRows = 1024 / kRowBytes;  // memory rows a wave load covers

  // Issue the loads of contraction indexes [k0, k0 + 64) into lds; k0 < o.k.
  static __device__ __forceinline__ void issue(const Operand& o, int32_t k0, lds_char* lds,
                                               int wave, int lane) {
    const int32_t left = o.k - k0;
    if constexpr (!COLS) {
      const char* p = (const char*)o.base + 2 * (int64_t)k0;
      const uint32_t bytes = (uint32_t)((int64_t)(o.count - 1) * o.ld + 2 * (left < kStep ? left : kStep));
      const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)bytes, 0x00020000);
      const int r0 = wave * kLoads * 8 + (lane >> 3);
      const int chunk = (lane & 7) ^ (r0 & 7);
      uint32_t v = (uint32_t)((int64_t)r0 * o.ld) + 16 * chunk;
      if (chunk * 8 >= left) v = 0x80000000u;  // past the contraction's end
      const uint32_t inc = chunk * 8 >= left ? 0u : (uint32_t)(8 * o.ld);
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (__attribute__((address_space(3))) void*)(lds + (wave * kLoads + j) * 1024), 16,
            v + j * inc, 0, 0, 0);
      }
    } else {
      const char* p = (const char*)o.base + (int64_t)k0 * o.ld;
      const int rows = left < kStep ? left : kStep;
      const uint32_t bytes = (uint32_t)((int64_t)(rows - 1) * o.ld + 2 * (int64_t)o.count);
      const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)bytes, 0x00020000);
      constexpr int kChunks = kRowBytes / 16;  // lanes a memory row takes
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int k = (wave * kLoads + j) * kLoadRows + lane / kChunks;
        const int q = lane % kChunks;
        const int f = swizzle<R>(k & 3, (k >> 3) & 1);
        const int chunk = (((q >> 1) ^ f) << 1) | (q & 1);
        const uint32_t v = (uint32_t)((int64_t)k * o.ld) + 16 * chunk;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (__attribute__((address_space(3))) void*)(lds + (wave * kLoads + j) * 1024), 16,
            v, 0, 0, 0);
      }
    }
  }
};

// Fragments of F 32-row blocks, rows r0 .. r0 + 32F of the tile, at
// contraction slice s (16 elements): lane l holds row l % 32, elements
// (l / 32) * 8 .. + 8.
template <int R, bool COLS, int F>
struct Frags {
  int base[F];
  __device__ __forceinline__ Frags(int r0, int lane) {
#pragma unroll
    for (int i = 0; i < F; ++i) {
      if constexpr (!COLS) {
        base[i] = (r0 + i * 32 + (lane & 31)) * (kStep * 2);
      } else {
        const int g = lane >> 4, j = lane & 15;
        const int k = (g >> 1) * 8 + (j >> 2);
        const int f = swizzle<R>(j >> 2, g >> 1);
        const int pair = (r0 >> 4) + 2 * i + (g & 1);
        base[i] = k * (R * 2) + ((pair ^ f) << 5) + (j & 3) * 8;
      }
    }
  }
  __device__ __forceinline__ s16x8 load(const lds_char* lds, int i, int s, int lane) const {
    if constexpr (!COLS) {
      const int chunk = (s * 2 + (lane >> 5)) ^ (lane & 7);
      return *(const __attribute__((address_space(3))) s16x8*)(lds + base[i] + chunk * 16);
    } else {
      typedef __attribute__((address_space(3))) s16x4 lds4;
      const lds_char* p = lds + base[i] + s * 16 * (R * 2);
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p);
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 4 * (R * 2)));
      return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// The tile: WM x WN waves, each MI x NJ blocks of 32 x 32.  acc[i][j][e] of
// lane l is row wm*32*MI + 32i + 8(e/4) + 4(l/32) + e%4, column
// wn*32*NJ + 32j + l%32.
template <typename T, int WM, int WN, int MI, int NJ, bool ACOLS, bool BCOLS>
struct Gemm {
  static constexpr int BM = WM * MI * 32, BN = WN * NJ * 32, WAVES = WM * WN;
  static constexpr int THREADS = 64 * WAVES;
  using SA = Stage<BM, ACOLS, WAVES>;
  using SB = Stage<BN, BCOLS, WAVES>;

  template <int P>
  static __device__ __forceinline__ void fragments(const lds_char* a, const lds_char* b, int s,
                                                   const Frags<BM, ACOLS, MI>& fa,
                                                   const Frags<BN, BCOLS, NJ>& fb, int lane,
                                                   s16x8 (&ra)[2][MI], s16x8 (&rb)[2][NJ]) {
#pragma unroll
    for (int i = 0; i < MI; ++i) ra[P][i] = fa.load(a, i, s, lane);
#pragma unroll
    for (int j = 0; j < NJ; ++j) rb[P][j] = fb.load(b, j, s, lane);
  }

  template <int P>
  static __device__ __forceinline__ void multiply(const s16x8 (&ra)[2][MI], const s16x8 (&rb)[2][NJ],
                                                  f32x16 (&acc)[MI][NJ]) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = mfma(T{}, ra[P][i], rb[P][j], acc[i][j]);
  }

  // Every wave's loads to LDS have landed, and its reads of LDS are done.
  static __device__ __forceinline__ void arrive() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  }

  // One step: cur holds contraction indexes [k0, k0 + 64), next receives the
  // following ones; ra/rb[0] hold cur's slice 0 on entry and next's on exit.
  // The next-but-one step's loads go into cur once every wave has read it.
  static __device__ __forceinline__ void step(const Operand& A, const Operand& B, int32_t k0,
                                              int32_t K, lds_char* ca, lds_char* cb, lds_char* na,
                                              lds_char* nb, int wave,
                                              const Frags<BM, ACOLS, MI>& fa,
                                              const Frags<BN, BCOLS, NJ>& fb, int lane,
                                              s16x8 (&ra)[2][MI], s16x8 (&rb)[2][NJ],
                                              f32x16 (&acc)[MI][NJ]) {
    fragments<1>(ca, cb, 1, fa, fb, lane, ra, rb);
    multiply<0>(ra, rb, acc);
    fragments<0>(ca, cb, 2, fa, fb, lane, ra, rb);
    multiply<1>(ra, rb, acc);
    fragments<1>(ca, cb, 3, fa, fb, lane, ra, rb);
    multiply<0>(ra, rb, acc);
    arrive();  // next has arrived, cur has been read
    if (k0 + kStep < K) fragments<0>(na, nb, 0, fa, fb, lane, ra, rb);
    if (k0 + 2 * kStep < K) {
      SA::issue(A, k0 + 2 * kStep, ca, wave, lane);
      SB::issue(B, k0 + 2 * kStep, cb, wave, lane);
    }
    multiply<1>(ra, rb, acc);
  }

  // acc = A B^T over K >= 0 contraction indexes.  lds: kLds bytes in four
  // separate arrays (kept apart so that waits for loads into one buffer are
  // not taken for reads of the other).
  static __device__ __forceinline__ void run(const Operand& A, const Operand& B, int32_t K,
                                             lds_char* a0, lds_char* b0, lds_char* a1,
                                             lds_char* b1, f32x16 (&acc)[MI][NJ]) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Frags<BM, ACOLS, MI> fa((wave / WN) * MI * 32, lane);
    const Frags<BN, BCOLS, NJ> fb((wave % WN) * NJ * 32, lane);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x16{};
    if (K <= 0) return;
    SA::issue(A, 0, a0, wave, lane);
    SB::issue(B, 0, b0, wave, lane);
    arrive();
    if (K > kStep) {
      SA::issue(A, kStep, a1, wave, lane);
      SB::issue(B, kStep, b1, wave, lane);
    }
    s16x8 ra[2][MI], rb[2][NJ];
    fragments<0>(a0, b0, 0, fa, fb, lane, ra, rb);
    int32_t k0 = 0;
    for (; k0 + kStep < K; k0 += 2 * kStep) {
      step(A, B, k0, K, a0, b0, a1, b1, wave, fa, fb, lane, ra, rb, acc);
      step(A, B, k0 + kStep, K, a1, b1, a0, b0, wave, fa, fb, lane, ra, rb, acc);
    }
    if (k0 < K) step(A, B, k0, K, a0, b0, a1, b1, wave, fa, fb, lane, ra, rb, acc);
  }
};

}  // namespace dev
}  // namespace zk
