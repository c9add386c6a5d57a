// Device helpers shared by the head's kernels (zero_head.hip, zero_head_few.hip).
#pragma once

#include "head_gemm.h"
#include "head_internal.h"
#include "zero_device.h"

namespace zk {
namespace dev {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// g's scale before it is rounded: |p - [v = y]| <= 1, so 2^15 keeps fp16 in
// range and p down to 2^-29 normal; bf16 has fp32's exponents.
template <typename T>
__host__ __device__ constexpr float g_scale();
template <>
__host__ __device__ constexpr float g_scale<BF16>() { return 1.0f; }
template <>
__host__ __device__ constexpr float g_scale<FP16>() { return 32768.0f; }

template <typename T>
__device__ __forceinline__ constexpr float g_log2() { return g_scale<T>() == 1.0f ? 0.0f : 15.0f; }

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

constexpr uint16_t kNan16 = 0x7FFF;  // NaN in either type

// Four consecutive vocabulary rows of a token into g's type.
template <typename T>
__device__ __forceinline__ u32x2 narrow4(float a, float b, float c, float d) {
  return u32x2{narrow<T>(a) | narrow<T>(b) << 16, narrow<T>(c) | narrow<T>(d) << 16};
}

// What the 16-bit value of x leaves.
template <typename T>
__device__ __forceinline__ float second(float x) { return x - widen<T>(narrow<T>(x)); }

// 16 and 8 bytes at any element's address: global loads and stores need no more
// than element alignment on gfx950.
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

// Eight elements from p, of which the first n exist.
__device__ __forceinline__ u32x4 take8(const uint16_t* p, int64_t n) {
  if (n >= 8) return *(const u32x4_a2*)p;
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
  return v;
}

// Without its first n (1 to 7) elements; zeros follow the others.
__device__ __forceinline__ s16x8 drop_first(s16x8 v, int n) {
  typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
  u64x2 q = __builtin_bit_cast(u64x2, v);
  if (n >= 4) q = u64x2{q[1], 0};
  const int bits = 16 * (n & 3);
  if (bits) q = u64x2{q[0] >> bits | q[1] << (64 - bits), q[1] >> bits};
  return __builtin_bit_cast(s16x8, q);
}

// (m, s) stands for s 2^m.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float n = __builtin_elementwise_maximum(m, m2);
  if (n == -INFINITY) return;  // both empty: s = s2 = 0
  s = s * exp2_fast(m - n) + s2 * exp2_fast(m2 - n);
  m = n;
}

template <typename P>
P* at(void* ws, size_t off) { return (P*)((char*)ws + off); }

#define ZK_LAUNCHED()                              \
  do {                                             \
    const hipError_t e_ = hipGetLastError();       \
    if (e_ != hipSuccess) return (int)e_;          \
  } while (0)

// w as the kernels read it: in place, or laid out in the workspace.
struct WeightView {
  const uint16_t* w;
  int64_t ld;       // elements
  int32_t K;        // contraction length of the logits
  int32_t width;    // columns a row holds
};
inline WeightView weight_view(const zero_head_t* h, const HeadPlan& p, void* ws) {
  if (p.pack_w)
    return {at<const uint16_t>(ws, p.w), p.hidden_pad, (int32_t)p.hidden_pad,
            (int32_t)p.hidden_pad};
  return {(const uint16_t*)h->w, h->ldw, (int32_t)h->hidden, (int32_t)h->hidden};
}

}  // namespace dev
}  // namespace zk
