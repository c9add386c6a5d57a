// Device helpers shared by the feed-forward block's kernels (zero_ffn.hip,
// zero_ffn_few.hip): the activations.
#pragma once

#include "ffn_internal.h"
#include "head_device.h"

namespace zk {
namespace dev {

// Where h goes, and what is kept for the gradients (or NULL): act(g) and b = u act'(g)
// in 24 bits each, their upper 16 apart and the lower 8 together.  Rounded to the 16-bit
// type they would be a third rounding on the way to dx, dWg and dWu (relative error
// against 64 bits 2.9e-3 in place of 2.3e-3 in bf16), and end at 65504 in fp16.
struct Kept {
  uint16_t *h, *act, *slope, *low;
  int64_t ld;  // between their rows
};
inline Kept kept(const FfnPlan& p, void* ws, const zero_ffn_saved_t* s) {
  if (s)
    return Kept{(uint16_t*)s->h, (uint16_t*)s->act, (uint16_t*)s->slope, (uint16_t*)s->low, s->ld};
  return Kept{at<uint16_t>(ws, p.h), nullptr, nullptr, nullptr, p.inner_pad};
}

// Four elements of act(g) and of b as they are kept.  Rounding could only lose a NaN of all
// ones: an operand's 16 bits and the instructions' own NaNs leave the lower bits zero.
struct Kept4 {
  u32x2 act, slope, low;
};
__device__ __forceinline__ Kept4 keep4(f32x4 a, f32x4 b) {
  Kept4 k;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t x[2], y[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // rounded to 24 bits
      x[e] = __float_as_uint(a[2 * w + e]) + 0x80u;
      y[e] = __float_as_uint(b[2 * w + e]) + 0x80u;
    }
    k.act[w] = __builtin_amdgcn_perm(x[1], x[0], 0x07060302u);
    k.slope[w] = __builtin_amdgcn_perm(y[1], y[0], 0x07060302u);
    // byte 1 of x0, y0, x1, y1
    k.low[w] = __builtin_amdgcn_perm(y[0], x[0], 0x0C0C0501u) |
               __builtin_amdgcn_perm(y[1], x[1], 0x05010C0Cu);
  }
  return k;
}
// Element e of act (WHICH = 0) or b (1).
template <int WHICH>
__device__ __forceinline__ float kept_at(u32x2 high, u32x2 low, int e) {
  const uint32_t sel = (e & 1 ? 0x0706020Cu : 0x0504000Cu) + (WHICH ? 0x100u : 0u);
  return __uint_as_float(__builtin_amdgcn_perm(high[e >> 1], low[e >> 1], sel));
}

template <int A>
struct Act {};

// fn(Act<act>), one branch for the whole wave.
template <typename Fn>
__device__ __forceinline__ void with_act(int32_t act, Fn fn) {
  switch (act) {
    case ZERO_ACT_SILU: return fn(Act<ZERO_ACT_SILU>{});
    case ZERO_ACT_GELU: return fn(Act<ZERO_ACT_GELU>{});
    case ZERO_ACT_GELU_TANH: return fn(Act<ZERO_ACT_GELU_TANH>{});
    default: return fn(Act<ZERO_ACT_RELU>{});
  }
}

// 1 / (1 + e^-x): exponential and reciprocal of one unit in the last place each.
__device__ __forceinline__ float logistic(float x) {
  return __builtin_amdgcn_rcpf(1.0f + exp2_fast(-kLog2e * x));
}

// The normal distribution's function and its density.  With z = |g| / sqrt 2 and t =
// 1 / (1 + z / 2), e^(z^2) erfc(z) / t is smooth on 0 < t <= 1; the polynomial was
// fitted to it (largest relative error with these coefficients 8.3e-8 for z up to 10).
// In fp32 the function is off by at most 3.6e-7 (1 + z^2) of itself, since the
// exponential's argument is rounded (8e-6 at |g| = 9, where it is 1e-19), and by
// 1.7e-7 absolutely.
__device__ __forceinline__ float normal(float g, float& density) {
  const float z = 0.70710678118654752f * __builtin_fabsf(g);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.5f, z, 1.0f));
  constexpr float k[9] = {0.28208643f, 0.28237531f, 0.24310374f,  0.20268694f, -0.026625827f,
                          0.27806741f, -0.48720014f, 0.28457508f, -0.059068985f};
  float r = k[8];
#pragma unroll
  for (int i = 7; i >= 0; --i) r = __builtin_fmaf(r, t, k[i]);
  const float e = exp2_fast(-kLog2e * z * z), tail = 0.5f * t * r * e;
  density = 0.3989422804014327f * e;
  return g > 0.0f ? 1.0f - tail : tail;
}

// act(g), and its slope.  (1 + tanh z) / 2 is the logistic function of 2z.
constexpr float kGeluTanh = 1.5957691216057308f;  // 2 sqrt(2 / pi)
template <int A>
__device__ __forceinline__ float activated(Act<A>, float g, float& slope) {
  if constexpr (A == ZERO_ACT_SILU) {
    const float s = logistic(g), a = g * s;
    slope = s + a * (1.0f - s);
    return a;
  } else if constexpr (A == ZERO_ACT_GELU) {
    float density;
    const float c = normal(g, density);
    slope = c + g * density;
    return g * c;
  } else if constexpr (A == ZERO_ACT_GELU_TANH) {
    // held finite: beyond, s is 0 or 1, and 0 times an infinite slope of z would be NaN
    const float q = __builtin_fminf(0.044715f * g * g, 0x1p100f);
    const float s = logistic(kGeluTanh * (g + g * q)), a = g * s;
    slope = s + a * (1.0f - s) * (kGeluTanh * (1.0f + 3.0f * q));
    return a;
  } else {
    slope = g > 0.0f ? 1.0f : 0.0f;
    return g < 0.0f ? 0.0f : g;  // a NaN stays one
  }
}
}  // namespace dev
}  // namespace zk
