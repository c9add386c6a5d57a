// Matrix-product core of the head's loss: one workgroup computes a 256 x 256 tile
// of A B^T on gfx950's matrix cores, fp32 accumulators in registers, and hands
// them to an epilogue.
//
// A is M x K and B is N x K.  Each operand lies in memory in one of two ways:
//   rows    element (m, k) at base + m*ld + k: the contraction is contiguous
//   cols    element (m, k) at base + k*ld + m: the tile's rows are contiguous
// so that all three products of the loss (logits: rows x rows; dx: rows x
// cols; dw: cols x cols) read their operands as they lie, with no transposed
// copy.  LDS holds two stages of 64 contraction elements of both operands,
// each in three parts: the B rows, and two halves of the A rows.  Global
// memory goes straight to LDS (16 bytes a lane, no registers), in whole
// 128-byte lines, and the lanes pick their global addresses so that the LDS
// image is swizzled and every fragment read is free of bank conflicts:
//   rows    128 bytes a row; 16-byte chunk c of row r lies at c ^ (r >> 1 & 7),
//           so that 16 consecutive rows' chunks c fill the 256 bytes the banks
//           deliver in a cycle
//   cols    a contraction index k's elements side by side; 32-byte pair p lies
//           at p ^ (2 * (k & 3) + (k >> 3 & 1)); fragments come back transposed
//           (ds_read_b64_tr_b16)
//
// Eight waves, two on each SIMD.  The second four run one phase behind the
// first: while one wave of a SIMD reads fragments and issues loads, the other
// multiplies, so the matrix cores wait neither for LDS nor for barriers, and
// no product queues behind a load that has yet to be accepted.  A stage takes
// a wave two rounds of (read, multiply): the first reads B and its rows of the
// first A half (and keeps B in registers), the second its rows of the other
// half.  A part is refilled in the round after its last reading, five or six
// phases before it is read again.
//
// The products are 16 x 16 x 32.  On full tiles the chip runs at its power
// limit, not at its issue limit: 32 x 32 x 16 products need 6% fewer cycles but
// held the clock at 1.54 GHz where these run at 1.70 (logits of 7373 x 128256 x
// 4096: 5.99 against 5.77 ms), since they move twice the accumulator bits for
// the same multiplications.
//
// Lanes whose element lies outside the operand read zero (buffer bounds), so
// ragged edges cost nothing and nothing outside the operand is touched.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace zk {
namespace dev {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) char lds_char;

struct BF16 {};
struct FP16 {};

__device__ __forceinline__ f32x4 mfma(BF16, s16x8 a, s16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(FP16, s16x8 a, s16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
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
  int32_t ld;         // bytes between rows (rows) or contraction indexes (cols); at most 2^22,
                      // so that offsets within a tile fit 32 bits
  int32_t count;      // rows of the tile that exist (rows), or columns from base to
                      // the end of a memory row (cols); multiples of 8 along memory
  int32_t k;          // contraction indexes that exist (rows: a multiple of 8)
};

constexpr int kStage = 64;  // contraction indexes of a stage

// R tile rows (columns of memory if COLS) staged by eight waves.  HALF 0 or 1:
// R = 128 of the tile's 256 rows, local row r is row r / 64 * 128 + 64 * HALF +
// r % 64; HALF < 0: all rows.
template <int R, bool COLS, int HALF>
struct Part {
  static constexpr int kBytes = R * kStage * 2;
  static constexpr int kLoads = kBytes / (8 * 1024);  // 1 KiB loads of a wave
  static_assert(kLoads * 8 * 1024 == kBytes && (HALF < 0 || R == 128), "whole loads");

  // Issue the loads of contraction indexes [k0, k0 + 64) into lds; past the
  // contraction's end they read zero.
  static __device__ __forceinline__ void issue(const Operand& o, int32_t k0, lds_char* lds,
                                               int wave, int lane) {
    int32_t left = o.k - k0;
    if (left < 0) left = 0;
    if (left > kStage) left = kStage;
    left = __builtin_amdgcn_readfirstlane(left);  // uniform, kept in a scalar register
    lds += wave * kLoads * 1024;
    if constexpr (!COLS) {
      const char* p = (const char*)o.base + 2 * (int64_t)k0;
      const int32_t bytes = left > 0 ? (o.count - 1) * o.ld + 2 * left : 0;
      const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, bytes, 0x00020000);
      int row = wave * kLoads * 8;
      if constexpr (HALF >= 0) row = row / 64 * 128 + 64 * HALF + row % 64;
      const int chunk = (lane & 7) ^ ((lane >> 4) & 3);
      const uint32_t v = (uint32_t)((row + (lane >> 3)) * o.ld), inc = 8u * (uint32_t)o.ld;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int c = chunk ^ ((j & 1) << 2);  // the 8 rows of every second load have bit 3 set
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (__attribute__((address_space(3))) void*)(lds + j * 1024), 16,
            c * 8 < left ? v + j * inc + 16 * c : 0x80000000u, 0, 0, 0);
      }
    } else {
      const char* p = (const char*)o.base + (int64_t)k0 * o.ld;
      const int32_t bytes = left > 0 ? (left - 1) * o.ld + 2 * o.count : 0;
      const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, bytes, 0x00020000);
      constexpr int kRowBytes = R * 2, kChunks = kRowBytes / 16, kLoadRows = 1024 / kRowBytes;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int k = (wave * kLoads + j) * kLoadRows + lane / kChunks;
        const int q = (lane % kChunks) ^ ((k & 3) << 2 | (k >> 3 & 1) << 1);
        const int col = HALF < 0 ? 16 * q : (q >> 3) * 256 + 128 * HALF + 16 * (q & 7);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (__attribute__((address_space(3))) void*)(lds + j * 1024), 16,
            (uint32_t)(k * o.ld + col), 0, 0, 0);
      }
    }
  }
};

// Fragments of four 16-row blocks, local rows r0 .. r0 + 64 of a part, at slice
// s (32 contraction elements) of a stage: lane l holds row l % 16, elements
// (l / 16) * 8 .. + 8.
template <int R, bool COLS>
struct Frags {
  int base[COLS ? 4 : 2];
  __device__ __forceinline__ Frags(int r0, int lane) {
    const int g = lane >> 4, j = lane & 15;
    if constexpr (!COLS) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        base[s] = (r0 + j) * (kStage * 2) + 16 * ((s * 4 + g) ^ (j >> 1));
    } else {
      const int k = g * 8 + (j >> 2), f = (j >> 2) << 1 | (g & 1);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        base[i] = k * (R * 2) + ((((r0 >> 4) + i) ^ f) << 5) + (j & 3) * 8;
    }
  }
  __device__ __forceinline__ s16x8 load(const lds_char* lds, int i, int s) const {
    if constexpr (!COLS) {
      return *(const __attribute__((address_space(3))) s16x8*)(lds + base[s] + i * 16 * kStage * 2);
    } else {
      typedef __attribute__((address_space(3))) s16x4 lds4;
      const lds_char* p = lds + base[i] + s * 32 * (R * 2);
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p);
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 4 * (R * 2)));
      return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// The stages' memory: separate arrays, so that the compiler does not take a
// read of one for a reader of loads into another.
#define ZK_GEMM_LDS                                                                       \
  __shared__ __attribute__((aligned(1024))) char lds_a00[16384], lds_a10[16384],           \
      lds_b0[32768], lds_a01[16384], lds_a11[16384], lds_b1[32768];                        \
  const GemmLds lds{{(lds_char*)lds_a00, (lds_char*)lds_a10, (lds_char*)lds_b0},           \
                    {(lds_char*)lds_a01, (lds_char*)lds_a11, (lds_char*)lds_b1}}
struct StageLds {
  lds_char *a0, *a1, *b;
};
struct GemmLds {
  StageLds even, odd;
};

// The 256 x 256 tile: 2 x 4 waves, each 8 x 4 blocks of 16 x 16.
// acc[i][j][e] of lane l is row wm*128 + 16i + 4(l/16) + e, column wn*64 + 16j
// + l%16, wm = wave / 4, wn = wave % 4.
template <typename T, bool ACOLS, bool BCOLS>
struct Gemm {
  static constexpr int BM = 256, BN = 256, THREADS = 512, MI = 8, NJ = 4;
  using A0 = Part<128, ACOLS, 0>;
  using A1 = Part<128, ACOLS, 1>;
  using SB = Part<256, BCOLS, -1>;
  using FA = Frags<128, ACOLS>;
  using FB = Frags<256, BCOLS>;

  template <int HALF>
  static __device__ __forceinline__ void multiply(const s16x8 (&ra)[2][4], const s16x8 (&rb)[2][4],
                                                  f32x4 (&acc)[MI][NJ]) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[4 * HALF + i][j] = mfma(T{}, ra[s][i], rb[s][j], acc[4 * HALF + i][j]);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
  }

  // End of a reading phase: this wave has read what it came for, and its loads
  // of the part that the next round reads have landed; the 8 issued since may
  // be on their way.
  static __device__ __forceinline__ void turn() {
    static_assert(A1::kLoads + A0::kLoads + SB::kLoads == 8, "loads in flight");
    asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }

  static __device__ __forceinline__ void stage(const Operand& A, const Operand& B, int32_t k0,
                                               const StageLds& here, const StageLds& other,
                                               int wave, int lane, const FA& fa, const FB& fb,
                                               f32x4 (&acc)[MI][NJ]) {
    s16x8 ra[2][4], rb[2][4];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        rb[s][i] = fb.load(here.b, i, s);
        ra[s][i] = fa.load(here.a0, i, s);
      }
    A1::issue(A, k0 + kStage, other.a1, wave, lane);
    turn();
    multiply<0>(ra, rb, acc);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) ra[s][i] = fa.load(here.a1, i, s);
    A0::issue(A, k0 + 2 * kStage, here.a0, wave, lane);
    SB::issue(B, k0 + 2 * kStage, here.b, wave, lane);
    turn();
    multiply<1>(ra, rb, acc);
  }

  // acc = A B^T over K >= 0 contraction indexes.  On return every wave is done
  // with LDS.
  static __device__ __forceinline__ void run(const Operand& A, const Operand& B, int32_t K,
                                             const GemmLds& lds, f32x4 (&acc)[MI][NJ]) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const FA fa(wave / 4 * 64, lane);
    const FB fb(wave % 4 * 64, lane);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{};
    if (K <= 0) return;
    A0::issue(A, 0, lds.even.a0, wave, lane);
    SB::issue(B, 0, lds.even.b, wave, lane);
    A1::issue(A, 0, lds.even.a1, wave, lane);
    A0::issue(A, kStage, lds.odd.a0, wave, lane);
    SB::issue(B, kStage, lds.odd.b, wave, lane);
    asm volatile("s_waitcnt vmcnt(8)\n\ts_barrier" ::: "memory");
    if (wave >= 4) asm volatile("s_barrier" ::: "memory");  // one phase behind
    int32_t k0 = 0;
    for (; k0 + kStage < K; k0 += 2 * kStage) {
      stage(A, B, k0, lds.even, lds.odd, wave, lane, fa, fb, acc);
      stage(A, B, k0 + kStage, lds.odd, lds.even, wave, lane, fa, fb, acc);
    }
    if (k0 < K) stage(A, B, k0, lds.even, lds.odd, wave, lane, fa, fb, acc);
    if (wave < 4) asm volatile("s_barrier" ::: "memory");
    // loads past the contraction's end (zeros) may still be on their way
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
  }

  // The tile in 16 bits through LDS, so that it leaves in whole lines: pack(a,
  // b, c, d) narrows four values that follow one another along the rows,
  // store(col, row, v) gets eight of them (16 bytes) of a tile column, 32
  // lanes side by side.  A column's 16-byte chunk c lies at c ^ (col % 32).
  // Call after run, by all waves.
  template <typename Pack, typename Store>
  static __device__ __forceinline__ void transposed(const GemmLds& lds, const f32x4 (&acc)[MI][NJ],
                                                    Pack pack, Store store) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int col = j % 2 * 16 + (lane & 15);
      lds_char* p = columns(lds, wave % 4 * 2 + j / 2) + col * 512 + (lane >> 4 & 1) * 8;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const f32x4& v = acc[i][j];
        const int chunk = wave / 4 * 16 + 2 * i + (lane >> 5);
        *(__attribute__((address_space(3))) u32x2*)(p + ((chunk ^ col) << 4)) =
            pack(v[0], v[1], v[2], v[3]);
      }
    }
    __syncthreads();
    const int r = lane & 31, hi = lane >> 5;
    const lds_char* p = columns(lds, wave);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int col = 2 * k + hi;
      store(wave * 32 + col, r * 8,
            *(const __attribute__((address_space(3))) u32x4*)(p + col * 512 + ((r ^ col) << 4)));
    }
  }

 private:
  // 16 KiB of LDS for 32 of the tile's columns.
  static __device__ __forceinline__ lds_char* columns(const GemmLds& l, int block) {
    switch (block) {
      case 0: return l.even.a0;
      case 1: return l.even.a1;
      case 2: return l.odd.a0;
      case 3: return l.odd.a1;
      case 4: return l.even.b;
      case 5: return l.even.b + 16384;
      case 6: return l.odd.b;
      default: return l.odd.b + 16384;
    }
  }
};

}  // namespace dev
}  // namespace zk
