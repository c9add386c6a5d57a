// The feed-forward block's two tile sizes: the 256 x 256 tile of head_gemm.h, and
// one of 128 x 128 for products with few tiles.
//
// The small tile has four waves and half of a CU's LDS and registers, so that two
// workgroups share a CU: one multiplies while the other loads its first stages or
// writes its tile out, which a single 256 x 256 tile a CU leaves idle.  A wave's 64 x
// 64 block needs as many LDS reads for each multiplication as two thirds of the
// matrix cores' rate allow, so large products keep the large tile.
#pragma once

#include "head_gemm.h"

namespace zk {
namespace dev {

struct SmallLds {
  lds_char* stage[2];  // A in 16 KiB, then B
};
// One array for all of a kernel's products.
__device__ __forceinline__ GemmLds large_lds() {
  ZK_GEMM_LDS;
  return lds;
}
__device__ __forceinline__ SmallLds small_lds() {
  __shared__ __attribute__((aligned(1024))) char even[32768], odd[32768];
  return SmallLds{{(lds_char*)even, (lds_char*)odd}};
}

// What both sizes offer:
//   kRows, kCols, kThreads   of a tile (PAIR: kRows of each of two products)
//   MI, NJ                   blocks of 16 x 16 of a wave; PAIR: the first MI / 2 rows of
//                            blocks are the first product's, the others the second's
//   row(wave, i), col(wave, j)  where block (i, j) starts in the tile; lane l has rows
//                            + 4 (l / 16) .. + 4 of column + l % 16
//   run, put, take           see Gemm; put_half, take_half: PAIR
template <typename T, bool ACOLS, bool BCOLS, bool PAIR = false>
struct Large : Gemm<T, ACOLS, BCOLS, PAIR> {
  using G = Gemm<T, ACOLS, BCOLS, PAIR>;
  static constexpr int kRows = PAIR ? 128 : 256, kCols = 256, kThreads = 512;
  using Lds = GemmLds;
  static __device__ __forceinline__ Lds shared() { return large_lds(); }
  static __device__ __forceinline__ int row(int wave, int i) {
    return PAIR ? wave / 4 * 64 + 16 * i : wave / 4 * 128 + 16 * i;
  }
  static __device__ __forceinline__ int col(int wave, int j) { return wave % 4 * 64 + 16 * j; }
  static __device__ __forceinline__ void put(const Lds& lds, int i, int j, u32x2 v) {
    G::put(G::column(lds, j), i, j, v);
  }
};

// 2 x 2 waves.  acc[i][j][e] of lane l is row wm*64 + 16i + 4(l/16) + e, column
// wn*64 + 16j + l%16, wm = wave / 2, wn = wave % 2; PAIR: acc[i][j] is row wm*32 +
// 16i + ... of the first product, acc[2 + i][j] of the second (i < 2).
template <typename T, bool ACOLS, bool BCOLS, bool PAIR = false>
struct Small {
  static constexpr int kRows = PAIR ? 64 : 128, kCols = 128, kThreads = 256, MI = 4, NJ = 4;
  static constexpr int kWaves = 4;
  using Lds = SmallLds;
  using SA = Part<PAIR ? 64 : 128, ACOLS, -1, kWaves>;
  using SB = Part<128, BCOLS, -1, kWaves>;
  using FA = Frags<PAIR ? 64 : 128, ACOLS>;
  using FB = Frags<128, BCOLS>;
  static constexpr int kB = 16384;  // where B starts in a stage

  static __device__ __forceinline__ Lds shared() { return small_lds(); }
  static __device__ __forceinline__ int row(int wave, int i) {
    return wave / 2 * (PAIR ? 32 : 64) + 16 * i;
  }
  static __device__ __forceinline__ int col(int wave, int j) { return wave % 2 * 64 + 16 * j; }

  template <typename S>
  static __device__ __forceinline__ void issue(const S& src, int32_t k0, lds_char* lds, int wave,
                                               int lane) {
    int32_t k = k0;
    const Operand& a = src.a0(k);
    SA::issue(a, k, lds, wave, lane);
    if constexpr (PAIR) {
      k = k0;
      const Operand& a2 = src.a1(k);
      SA::issue(a2, k, lds + SA::kBytes, wave, lane);
    }
    k = k0;
    const Operand& b = src.b(k);
    SB::issue(b, k, lds + kB, wave, lane);
  }

  // One stage, which has landed: all fragments into registers, then the stage after the
  // next into its place, then the products.
  template <typename S>
  static __device__ __forceinline__ void stage(const S& src, int32_t k0, lds_char* here, int wave,
                                               int lane, const FA& fa, const FB& fb,
                                               f32x4 (&acc)[MI][NJ]) {
    s16x8 ra[2][MI], rb[2][NJ];
    static_assert(SA::kLoads * (PAIR ? 2 : 1) + SB::kLoads == 8, "loads in flight");
    asm volatile("s_waitcnt vmcnt(8)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) rb[s][j] = fb.load(here + kB, j, s);
#pragma unroll
      for (int i = 0; i < MI; ++i)
        ra[s][i] = PAIR ? fa.load(here + i / 2 * SA::kBytes, i % 2, s) : fa.load(here, i, s);
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    issue(src, k0 + 2 * kStage, here, wave, lane);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = mfma(T{}, ra[s][i], rb[s][j], acc[i][j]);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  }

  static __device__ __forceinline__ void run(const Operand& A, const Operand& B, int32_t K,
                                             const Lds& lds, f32x4 (&acc)[MI][NJ]) {
    run(OneProduct{A, B}, K, lds, acc);
  }
  // acc = A B^T over K >= 0 contraction indexes.  On return every wave is done
  // with LDS.
  template <typename S>
  static __device__ __forceinline__ void run(const S& src, int32_t K, const Lds& lds,
                                             f32x4 (&acc)[MI][NJ]) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const FA fa(wave / 2 * (PAIR ? 32 : 64), lane);
    const FB fb(wave % 2 * 64, lane);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{};
    if (K <= 0) return;
    issue(src, 0, lds.stage[0], wave, lane);
    issue(src, kStage, lds.stage[1], wave, lane);
    int32_t k0 = 0;
    for (; k0 + kStage < K; k0 += 2 * kStage) {
      stage(src, k0, lds.stage[0], wave, lane, fa, fb, acc);
      stage(src, k0 + kStage, lds.stage[1], wave, lane, fa, fb, acc);
    }
    if (k0 < K) stage(src, k0, lds.stage[0], wave, lane, fa, fb, acc);
    // loads past the contraction's end (zeros) may still be on their way
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
  }

  // The tile in 16 bits through LDS, as Gemm's: a column takes 256 bytes, its chunk c
  // at c ^ (col % 16), and 16 lanes.
  static __device__ __forceinline__ void put(const Lds& lds, int i, int j, u32x2 v) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = col(wave, j) + (lane & 15);
    const int chunk = wave / 2 * 8 + 2 * i + (lane >> 5);
    lds_char* p = lds.stage[0] + c * 256 + (lane >> 4 & 1) * 8;
    *(__attribute__((address_space(3))) u32x2*)(p + ((chunk ^ (c & 15)) << 4)) = v;
  }
  template <typename Store>
  static __device__ __forceinline__ void take(const Lds& lds, Store store) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = wave * 32 + 4 * k + (lane >> 4);
      store(c, r * 8,
            *(const __attribute__((address_space(3))) u32x4*)(lds.stage[0] + c * 256 +
                                                              ((r ^ (c & 15)) << 4)));
    }
  }
  template <typename Pack, typename Store>
  static __device__ __forceinline__ void transposed(const Lds& lds, const f32x4 (&acc)[MI][NJ],
                                                    Pack pack, Store store) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const f32x4& v = acc[i][j];
        put(lds, i, j, pack(v[0], v[1], v[2], v[3]));
      }
    __syncthreads();
    take(lds, store);
  }
  // PAIR: 64 rows (i < 2); a column takes 128 bytes, its chunk c at c ^ (col % 8),
  // and 8 lanes.  Region 0 or 1: 16 KiB each.
  static __device__ __forceinline__ void put_half(const Lds& lds, int region, int i, int j,
                                                  u32x2 v) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = col(wave, j) + (lane & 15);
    const int chunk = wave / 2 * 4 + 2 * i + (lane >> 5);
    lds_char* p = lds.stage[region] + c * 128 + (lane >> 4 & 1) * 8;
    *(__attribute__((address_space(3))) u32x2*)(p + ((chunk ^ (c & 7)) << 4)) = v;
  }
  template <typename Store>
  static __device__ __forceinline__ void take_half(const Lds& lds, int region, Store store) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 7;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = wave * 32 + 8 * k + (lane >> 3);
      store(c, r * 8,
            *(const __attribute__((address_space(3))) u32x4*)(lds.stage[region] + c * 128 +
                                                              ((r ^ (c & 7)) << 4)));
    }
  }
};

template <bool SMALL, typename T, bool ACOLS, bool BCOLS, bool PAIR = false>
struct TileOf {
  using G = Large<T, ACOLS, BCOLS, PAIR>;
};
template <typename T, bool ACOLS, bool BCOLS, bool PAIR>
struct TileOf<true, T, ACOLS, BCOLS, PAIR> {
  using G = Small<T, ACOLS, BCOLS, PAIR>;
};

}  // namespace dev
}  // namespace zk
