// Matrix-product core of the head's loss: one workgroup computes a BM x BN tile
// of A B^T on gfx950's matrix cores, fp32 accumulators in registers, and hands
// them to an epilogue.
//
// A is M x K and B is N x K.  Each operand lies in memory in one of two ways:
//   rows    element (m, k) at base + m*ld + k: the contraction is contiguous
//   cols    element (m, k) at base + k*ld + m: the tile's rows are contiguous
// so that all three products of the loss (logits: rows x rows; dx: rows x
// cols; dw: cols x cols) read their operands as they lie, with no transposed
// copy.  LDS is a ring of four slots of 32 contraction elements of both
// operands; global memory goes straight to LDS (16 bytes a lane, no
// registers), and the lanes pick their global addresses so that the LDS image
// is swizzled and every fragment read is free of bank conflicts:
//   rows    64 bytes a row; 16-byte chunk c of row r lies at c ^ (r >> 2 & 3),
//           so that 16 consecutive rows' chunks c fill the 256 bytes the banks
//           deliver in a cycle
//   cols    2*BM bytes a contraction index k; 32-byte pair p lies at p ^ f(k),
//           f(k) = 2 * ((k & 3) | (k >> 3 & 1) << 2); fragments come back
//           transposed (ds_read_b64_tr_b16)
//
// Eight waves, two on each SIMD.  The second four run one phase behind the
// first: while one wave of a SIMD reads its fragments, the other multiplies,
// so the matrix cores do not wait for LDS or for barriers.  A slot is read in
// two consecutive phases (by either half of the waves), and a wave refills its
// part in its next reading phase, five or six phases before it is read again:
// loads are issued while the other half multiplies, never in front of a
// wave's own products, which would wait for the loads to be accepted.
//
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

// Workgroup -> tile of an nm x nn grid.  Workgroups are dealt to the 8 XCDs in
// turn, each with an L2 of its own: XCD x takes the x-th eighth of the tiles,
// and goes through them kGroup tiles of m at a time, so that the tiles one XCD
// works on at a time share operands.  Launch tile_grid(nm, nn) workgroups, nm
// and nn at most what the kernel passes; those without a tile get false.
constexpr uint32_t kXcds = 8, kGroup = 8;
inline uint32_t tile_grid(int64_t nm, int64_t nn) {
  return (uint32_t)((nm * nn + kXcds - 1) / kXcds * kXcds);
}
__device__ __forceinline__ bool tile_of(uint32_t block, uint32_t nm, uint32_t nn, int32_t& m,
                                        int32_t& n) {
  const uint32_t total = nm * nn, each = (total + kXcds - 1) / kXcds;
  const uint32_t i = block / kXcds, t = block % kXcds * each + i;
  if (i >= each || t >= total) return false;
  const uint32_t g = t / (kGroup * nn), r = t - g * kGroup * nn;
  const uint32_t rows = nm - g * kGroup < kGroup ? nm - g * kGroup : kGroup;
  m = (int32_t)(g * kGroup + r % rows);
  n = (int32_t)(r / rows);
  return true;
}

// One operand of a tile.
struct Operand {
  const void* base;   // element (0, 0) of the tile
  int64_t ld;         // bytes between rows (rows) or contraction indexes (cols)
  int32_t count;      // rows of the tile that exist (rows), or columns from base to
                      // the end of a memory row (cols); multiples of 8 along memory
  int32_t k;          // contraction indexes that exist (rows: a multiple of 8)
};

constexpr int kSlot = 32;   // contraction indexes of an LDS slot
constexpr int kSlots = 4;

// f(k) of the cols layout, from bits 0-1 and bit 3 of k; a tile of 128 rows
// has only 8 pairs a memory row and takes the low part.
template <int R>
__device__ __forceinline__ int swizzle(int k01, int k3) {
  return (2 * (k01 | k3 << 2)) & (R / 16 - 1);
}

// R tile rows staged by WAVES waves; COLS as above.
template <int R, bool COLS, int WAVES>
struct Stage {
  static constexpr int kBytes = R * kSlot * 2;
  static constexpr int kLoads = kBytes / (WAVES * 1024);  // 1 KiB wave loads of a wave and slot
  static_assert(kLoads * WAVES * 1024 == kBytes, "whole loads");

  // Issue the loads of contraction indexes [k0, k0 + 32) into lds; past the
  // contraction's end they read zero.
  static __device__ __forceinline__ void issue(const Operand& o, int32_t k0, lds_char* lds,
                                               int wave, int lane) {
    int32_t left = o.k - k0;
    if (left < 0) left = 0;
    if (left > kSlot) left = kSlot;
    left = __builtin_amdgcn_readfirstlane(left);  // uniform, kept in a scalar register
    lds += wave * kLoads * 1024;
    if constexpr (!COLS) {
      const char* p = (const char*)o.base + 2 * (int64_t)k0;
      const uint32_t bytes = left ? (uint32_t)((int64_t)(o.count - 1) * o.ld + 2 * left) : 0u;
      const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)bytes, 0x00020000);
      const int row = wave * kLoads * 16 + (lane >> 2);
      const int chunk = (lane & 3) ^ ((lane >> 4) & 3);
      const uint32_t inc = (uint32_t)(16 * o.ld);
      const uint32_t v = (uint32_t)((int64_t)row * o.ld) + 16 * chunk;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (__attribute__((address_space(3))) void*)(lds + j * 1024), 16,
            chunk * 8 < left ? v + j * inc : 0x80000000u, 0, 0, 0);
      }
    } else {
      const char* p = (const char*)o.base + (int64_t)k0 * o.ld;
      const uint32_t bytes = left ? (uint32_t)((int64_t)(left - 1) * o.ld + 2 * (int64_t)o.count) : 0u;
      const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)bytes, 0x00020000);
      constexpr int kRowBytes = R * 2, kChunks = kRowBytes / 16, kLoadRows = 1024 / kRowBytes;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int k = (wave * kLoads + j) * kLoadRows + lane / kChunks;
        const int q = lane % kChunks;
        const int f = swizzle<R>(k & 3, (k >> 3) & 1);
        const int chunk = (((q >> 1) ^ f) << 1) | (q & 1);
        const uint32_t v = (uint32_t)((int64_t)k * o.ld) + 16 * chunk;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (__attribute__((address_space(3))) void*)(lds + j * 1024), 16, v, 0, 0, 0);
      }
    }
  }
};

// Fragments of F 32-row blocks, rows r0 .. r0 + 32F of the tile, at slice s
// (16 contraction elements) of a slot: lane l holds row l % 32, elements
// (l / 32) * 8 .. + 8.
template <int R, bool COLS, int F>
struct Frags {
  int base[COLS ? F : 2];
  __device__ __forceinline__ Frags(int r0, int lane) {
    if constexpr (!COLS) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        base[s] = (r0 + (lane & 31)) * (kSlot * 2) +
                  16 * ((s * 2 + (lane >> 5)) ^ ((lane >> 2) & 3));
    } else {
#pragma unroll
      for (int i = 0; i < F; ++i) {
        const int g = lane >> 4, j = lane & 15;
        const int k = (g >> 1) * 8 + (j >> 2);
        const int f = swizzle<R>(j >> 2, g >> 1);
        const int pair = (r0 >> 4) + 2 * i + (g & 1);
        base[i] = k * (R * 2) + ((pair ^ f) << 5) + (j & 3) * 8;
      }
    }
  }
  __device__ __forceinline__ s16x8 load(const lds_char* lds, int i, int s) const {
    if constexpr (!COLS) {
      return *(const __attribute__((address_space(3))) s16x8*)(lds + base[s] + i * 32 * kSlot * 2);
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
  static constexpr int kSlotBytes = (BM + BN) * kSlot * 2;
  static constexpr int kABytes = BM * kSlot * 2;
  static_assert(WAVES == 8, "two halves of four waves");
  using SA = Stage<BM, ACOLS, WAVES>;
  using SB = Stage<BN, BCOLS, WAVES>;

  static __device__ __forceinline__ void issue(const Operand& A, const Operand& B, int32_t slot,
                                               lds_char* lds, int wave, int lane) {
    SA::issue(A, slot * kSlot, lds, wave, lane);
    SB::issue(B, slot * kSlot, lds + kABytes, wave, lane);
  }

  // Slot number `slot`, in ring position `lds`; `ahead` is the position three on.
  static __device__ __forceinline__ void phases(const Operand& A, const Operand& B, int32_t slot,
                                                lds_char* lds, lds_char* ahead, int wave,
                                                const Frags<BM, ACOLS, MI>& fa,
                                                const Frags<BN, BCOLS, NJ>& fb, int lane,
                                                f32x16 (&acc)[MI][NJ]) {
    s16x8 ra[2][MI], rb[2][NJ];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) rb[s][j] = fb.load(lds + kABytes, j, s);
#pragma unroll
      for (int i = 0; i < MI; ++i) ra[s][i] = fa.load(lds, i, s);
    }
    issue(A, B, slot + kSlots - 1, ahead, wave, lane);
    // this wave has read the slot, and its loads of the next one have landed
    // (those of the two after it may be on their way)
    static_assert(2 * (SA::kLoads + SB::kLoads) == 8, "the count below");
    asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = mfma(T{}, ra[s][i], rb[s][j], acc[i][j]);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
  }

  // acc = A B^T over K >= 0 contraction indexes.  s0 .. s3: the ring's slots
  // (separate arrays, so that the compiler does not take a read of one for a
  // reader of loads into another).  On return every wave is done with LDS.
  static __device__ __forceinline__ void run(const Operand& A, const Operand& B, int32_t K,
                                             lds_char* s0, lds_char* s1, lds_char* s2,
                                             lds_char* s3, f32x16 (&acc)[MI][NJ]) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = wave / 4;
    const Frags<BM, ACOLS, MI> fa((wave / WN) * MI * 32, lane);
    const Frags<BN, BCOLS, NJ> fb((wave % WN) * NJ * 32, lane);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x16{};
    if (K <= 0) return;
    issue(A, B, 0, s0, wave, lane);
    issue(A, B, 1, s1, wave, lane);
    issue(A, B, 2, s2, wave, lane);
    asm volatile("s_waitcnt vmcnt(8)\n\ts_barrier" ::: "memory");
    if (half != 0) asm volatile("s_barrier" ::: "memory");  // one phase behind
    const int32_t n = (K + kSlot - 1) / kSlot;
    int32_t t = 0;
    for (; t + kSlots <= n; t += kSlots) {
      phases(A, B, t, s0, s3, wave, fa, fb, lane, acc);
      phases(A, B, t + 1, s1, s0, wave, fa, fb, lane, acc);
      phases(A, B, t + 2, s2, s1, wave, fa, fb, lane, acc);
      phases(A, B, t + 3, s3, s2, wave, fa, fb, lane, acc);
    }
    if (t < n) phases(A, B, t, s0, s3, wave, fa, fb, lane, acc);
    if (t + 1 < n) phases(A, B, t + 1, s1, s0, wave, fa, fb, lane, acc);
    if (t + 2 < n) phases(A, B, t + 2, s2, s1, wave, fa, fb, lane, acc);
    if (half == 0) asm volatile("s_barrier" ::: "memory");
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
};

}  // namespace dev
}  // namespace zk
