// AdamW over a list of tensors in one launch, moments in 32 or in 8 bits.
//
//   gc = (g s) c;  m = b1 m + (1-b1) gc;  v = b2 v + (1-b2) gc^2
//   p = p (1 - lr wd) - (m / (sqrt(v) / sqrt(1-b2^t) + eps)) lr / (1-b1^t)
//
// the shard update's sequence, one rounding an operation.  Every element is
// read and written once: 28 bytes with 16-bit gradients and parameters and
// 32-bit moments, 16 with 8-bit ones.  GPT-2 1.5B, 582 tensors: 6.9 ms with fp16
// gradients and 32 bits (6.3 TB/s), 4.75 ms with fp32 gradients and 8 (5.9).
//
// The list lies in a device table: one launch takes all tensors, whatever
// their number, and a graph can hold it.  A wave finds its workgroup's tensor
// by one load for up to 64 tensors, two for up to 4096 (its lanes look at 64
// places of the list at once).
//
// 8-bit moments.  A value keeps the sign, the exponent and 3 bits of the
// fraction, fp32's pattern cut at bit 20; what is stored is that pattern less a
// base that 128 neighbouring elements share, so that 8 bits hold it:
//   v  codes 0..255, 32 octaves below the block's largest value
//   m  sign and codes 0..127, 16 octaves
// The base is 8 times an exponent, one byte a block; a scale that is a power of
// two costs nothing in precision, since the elements are floats themselves.  A v
// that is not zero stays at least the smallest code: rounded to zero it
// would leave eps alone under m.
//
// The cut rounds stochastically: b2 = 0.999 moves v by a thousandth a step, and
// to nearest everything under half of an eighth would be lost, so that v could
// grow but never fall.  The random bits are a hash of (seed, tensor,
// element), so equal calls give equal bits and nothing is kept for them.
#include <stddef.h>

#include "adam_internal.h"
#include "zero_device.h"

namespace zk {
namespace {

using namespace dev;

constexpr int kMomentBlock = ZERO_ADAM_BLOCK;
static_assert(kMomentBlock == 128, "a block is 32 lanes' quads");
constexpr int kNone = 3;  // no parameter

template <typename T>
using gptr = __attribute__((address_space(1))) T*;
// Vectors at their element's alignment: global accesses need no more.
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));

// A 32-bit mixing function: xor-shift, multiply, twice, constants of low bias
// found by search (published as "lowbias32", C. Wellons, 2018).
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x7FEB352Du;
  x = (x ^ (x >> 15)) * 0x846CA68Bu;
  return x ^ (x >> 16);
}

// Largest i < n with first[i] <= b, for the whole wave (n >= 1, first[0] = 0).
__device__ __forceinline__ int32_t find_entry(gptr<const uint32_t> first, int32_t n, uint32_t b) {
  const int32_t lane = (int32_t)(threadIdx.x & 63);
  int32_t lo = 0;
  while (n > 64) {
    const int32_t step = (n + 63) / 64, i = lane * step;
    const bool below = i < n && first[lo + (i < n ? i : 0)] <= b;
    const int32_t k = __popcll(__ballot(below)) - 1;  // first does not fall
    lo += k * step;
    n = n - k * step < step ? n - k * step : step;
  }
  const bool below = lane < n && first[lo + (lane < n ? lane : 0)] <= b;
  return __builtin_amdgcn_readfirstlane(lo + __popcll(__ballot(below)) - 1);
}

// Four elements i .. i + 4 of which the first n exist (n = 4 where FULL).
template <bool FULL>
__device__ __forceinline__ f32x4 load_f32(gptr<const float> p, int64_t i, int n) {
  if constexpr (FULL) return __builtin_nontemporal_load((gptr<const f32x4_a4>)(p + i));
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) x[e] = p[i + e];
  return x;
}
template <bool FULL>
__device__ __forceinline__ void store_f32(gptr<float> p, int64_t i, int n, f32x4 x) {
  if constexpr (FULL) {
    __builtin_nontemporal_store(x, (gptr<f32x4_a4>)(p + i));
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) p[i + e] = x[e];
}
template <bool FULL>
__device__ __forceinline__ u32x2 load_16(gptr<const uint16_t> p, int64_t i, int n) {
  if constexpr (FULL) return __builtin_nontemporal_load((gptr<const u32x2_a2>)(p + i));
  u32x2 x = {0, 0};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) x[e >> 1] |= (uint32_t)p[i + e] << (16 * (e & 1));
  return x;
}
template <bool FULL>
__device__ __forceinline__ void store_16(gptr<uint16_t> p, int64_t i, int n, u32x2 x) {
  if constexpr (FULL) {
    __builtin_nontemporal_store(x, (gptr<u32x2_a2>)(p + i));
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) p[i + e] = (uint16_t)(x[e >> 1] >> (16 * (e & 1)));
}
// Codes are 4-byte aligned (a tensor's start, and i a multiple of 4).
template <bool FULL>
__device__ __forceinline__ uint32_t load_8(gptr<const uint8_t> p, int64_t i, int n) {
  if constexpr (FULL) return __builtin_nontemporal_load((gptr<const uint32_t>)(p + i));
  uint32_t x = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) x |= (uint32_t)p[i + e] << (8 * e);
  return x;
}
template <bool FULL>
__device__ __forceinline__ void store_8(gptr<uint8_t> p, int64_t i, int n, uint32_t x) {
  if constexpr (FULL) {
    __builtin_nontemporal_store(x, (gptr<uint32_t>)(p + i));
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) p[i + e] = (uint8_t)(x >> (8 * e));
}

// Gradients as they lie (16-bit ones in the first two words).
template <int GD, bool FULL>
__device__ __forceinline__ f32x4 load_grad(gptr<const void> p, int64_t i, int n) {
  if constexpr (GD == ZERO_F32) return load_f32<FULL>((gptr<const float>)p, i, n);
  const u32x2 x = load_16<FULL>((gptr<const uint16_t>)p, i, n);
  return f32x4{__uint_as_float(x[0]), __uint_as_float(x[1]), 0.0f, 0.0f};
}
template <int GD>
__device__ __forceinline__ float grad_of(f32x4 x, int e) {
  if constexpr (GD == ZERO_F32) return x[e];
  else
    return to_f32<GD == ZERO_BF16 ? Fmt::BF16 : Fmt::F16>(
        (__float_as_uint(x[e >> 1]) >> (16 * (e & 1))) & 0xFFFFu);
}

// The base of a block, in patterns, from its exponent.
constexpr int kOctavesM = 16, kOctavesV = 32;
template <int OCTAVES>
__device__ __forceinline__ uint32_t base_of(uint32_t exp) {
  return 8 * __builtin_elementwise_sub_sat(exp, (uint32_t)(OCTAVES - 1));
}
// Byte e of four codes; base: the block's, in the pattern's place (<< 20).
__device__ __forceinline__ float decode_m(uint32_t codes, int e, uint32_t base) {
  const uint32_t a = codes >> (8 * e) & 0x7Fu;
  const uint32_t x = a ? (a << 20) + base : 0u;
  return __uint_as_float(x | (codes << (24 - 8 * e) & 0x80000000u));
}
__device__ __forceinline__ float decode_v(uint32_t codes, int e, uint32_t base) {
  const uint32_t a = codes >> (8 * e) & 0xFFu;
  return __uint_as_float(a ? (a << 20) + base : 0u);
}
// fp32's pattern without sign, with 3 fraction bits, rounded up where the bits
// below and the random ones (bits 4 to 19) overflow.  A NaN stays one, whatever its
// sign and payload: without the sign the addition cannot pass 32 bits.
__device__ __forceinline__ uint32_t cut(float x, uint32_t random) {
  const uint32_t pattern = __float_as_uint(x) & 0x7FFFFFFFu;
  const uint32_t p = (pattern + ((random & 0xFFFF0u) | 8u)) >> 20;
  return p < 0x7FFu ? p : 0x7FFu;
}

// The larger of both 16-bit halves over the 32 lanes of a block.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t,
                            __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                      __builtin_bit_cast(u16x2, b)));
}
template <int N>
__device__ __forceinline__ uint32_t rotated(uint32_t x) {  // within 16 lanes
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + N, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
  x = max2(x, rotated<8>(x));
  x = max2(x, rotated<4>(x));
  x = max2(x, rotated<2>(x));
  x = max2(x, rotated<1>(x));
  return max2(x, (uint32_t)__shfl_xor((int)x, 16));
}

struct TensorScalars {
  float step_size, decay, c;
};

template <bool SMALL>
constexpr int kThreadsOf = SMALL ? kAdamThreads8 : kAdamThreads32;
template <bool SMALL>
constexpr int kQuadsOf = SMALL ? kAdamQuads8 : kAdamQuads32;
template <bool SMALL>
constexpr int32_t kChunkOf = (int32_t)(SMALL ? kAdamChunk8 : kAdamChunk32);

// One workgroup's elements [at, at + len) of a tensor; FULL: len is a whole chunk.
template <int GD, bool SMALL, bool FULL>
__device__ __forceinline__ void update_chunk(const AdamEntry& t, int64_t at, int32_t len,
                                             uint32_t key, const ListScalars& sc,
                                             const TensorScalars& ts) {
  constexpr int kQuads = kQuadsOf<SMALL>, kThreads = kThreadsOf<SMALL>;
  const gptr<const void> grad = (gptr<const void>)t.grad;
  const gptr<float> master = (gptr<float>)t.master;
  const int out = (int)(t.kind >> 2 & 3);
  f32x4 g[kQuads], p[kQuads], m[kQuads], v[kQuads];
  uint32_t m8[kQuads], v8[kQuads], mb[kQuads], vb[kQuads];
#pragma unroll
  for (int k = 0; k < kQuads; ++k) {
    const int32_t r = 4 * (int32_t)(threadIdx.x + k * kThreads);
    const int n = FULL ? 4 : len - r;
    const int64_t i = at + r;
    g[k] = load_grad<GD, FULL>(grad, i, n);
    p[k] = load_f32<FULL>(master, i, n);
    if constexpr (SMALL) {
      m8[k] = load_8<FULL>((gptr<const uint8_t>)t.m, i, n);
      v8[k] = load_8<FULL>((gptr<const uint8_t>)t.v, i, n);
      const int64_t b = FULL || n > 0 ? i / kMomentBlock : 0;  // a block's lanes alike, or none
      mb[k] = ((gptr<const uint8_t>)t.m_exp)[b];
      vb[k] = ((gptr<const uint8_t>)t.v_exp)[b];
    } else {
      m[k] = load_f32<FULL>((gptr<const float>)t.m, i, n);
      v[k] = load_f32<FULL>((gptr<const float>)t.v, i, n);
    }
  }
#pragma unroll
  for (int k = 0; k < kQuads; ++k) {
    const int32_t r = 4 * (int32_t)(threadIdx.x + k * kThreads);
    const int n = FULL ? 4 : len - r;
    const int64_t i = at + r;
    if constexpr (SMALL) {
      mb[k] = base_of<kOctavesM>(mb[k]) << 20;
      vb[k] = base_of<kOctavesV>(vb[k]) << 20;
    }
    // the random bits' counter: i runs on from a multiple of 4, within one key
    const uint32_t count = key + (uint32_t)i % (1u << kKeyShift);
    uint32_t pm[4], pv[4], top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float mm, vv, pp = p[k][e];
      if constexpr (SMALL) {
        mm = decode_m(m8[k], e, mb[k]);
        vv = decode_v(v8[k], e, vb[k]);
      } else {
        mm = m[k][e];
        vv = v[k][e];
      }
      const float gc = (grad_of<GD>(g[k], e) * sc.scale) * ts.c;
      mm = sc.b1 * mm + sc.omb1 * gc;
      vv = sc.b2 * vv + sc.omb2 * (gc * gc);
      float u;
      if constexpr (SMALL) {
        // the instruction's root of what fp32 holds with fewer bits is zero, so small
        // ones are raised by 2^24; large ones would pass fp32's range
        const bool low = vv < 1.0f;
        const float den = __builtin_amdgcn_sqrtf(low ? vv * 0x1p24f : vv) *
                              (low ? sc.inv_root_low : sc.inv_root) + sc.eps;
        u = mm * __builtin_amdgcn_rcpf(den);
      } else {
        u = mm / (__builtin_sqrtf(vv) / sc.sqrt_bc2 + sc.eps);
      }
      pp = pp * ts.decay - u * ts.step_size;
      asm volatile("" : "+v"(pp));  // rounded to fp32 before it is cast
      p[k][e] = pp;
      m[k][e] = mm;
      v[k][e] = vv;
      if constexpr (SMALL) {
        const uint32_t random = mix(count + (uint32_t)e);
        pm[e] = cut(mm, random << 4);
        pv[e] = cut(vv, random >> 12);
        if (FULL || e < n) top = max2(top, pm[e] | pv[e] << 16);
      }
    }
    if constexpr (SMALL) {
      top = block_max(top);
      const uint32_t em = (top & 0xFFFFu) >> 3, ev = top >> 19;
      const uint32_t bm = base_of<kOctavesM>(em), bv = base_of<kOctavesV>(ev);
      uint32_t cm = 0, cv = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a = __builtin_elementwise_sub_sat(pm[e], bm);
        const uint32_t b = __builtin_elementwise_sub_sat(pv[e], bv);
        const uint32_t bits = __float_as_uint(v[k][e]), least = bits < 1u ? bits : 1u;
        cm |= a << (8 * e) | (__float_as_uint(m[k][e]) >> (24 - 8 * e) & 0x80u << (8 * e));
        cv |= (b > least ? b : least) << (8 * e);  // a v that is not zero keeps a code
      }
      store_8<FULL>((gptr<uint8_t>)t.m, i, n, cm);
      store_8<FULL>((gptr<uint8_t>)t.v, i, n, cv);
      if (threadIdx.x % 32 == 0 && (FULL || n > 0)) {
        ((gptr<uint8_t>)t.m_exp)[i / kMomentBlock] = (uint8_t)em;
        ((gptr<uint8_t>)t.v_exp)[i / kMomentBlock] = (uint8_t)ev;
      }
    } else {
      store_f32<FULL>((gptr<float>)t.m, i, n, m[k]);
      store_f32<FULL>((gptr<float>)t.v, i, n, v[k]);
    }
    store_f32<FULL>(master, i, n, p[k]);
    if (out == ZERO_F32) {
      store_f32<FULL>((gptr<float>)t.param, i, n, p[k]);
    } else if (out == ZERO_F16) {
      store_16<FULL>((gptr<uint16_t>)t.param, i, n,
                     u32x2{f2h(p[k][0]) | f2h(p[k][1]) << 16, f2h(p[k][2]) | f2h(p[k][3]) << 16});
    } else if (out == ZERO_BF16) {
      store_16<FULL>((gptr<uint16_t>)t.param, i, n,
                     u32x2{f2bf(p[k][0]) | f2bf(p[k][1]) << 16,
                           f2bf(p[k][2]) | f2bf(p[k][3]) << 16});
    }
  }
}

template <int GD, bool SMALL>
__device__ __forceinline__ void update(const AdamEntry& t, int64_t at, uint32_t key,
                                       const ListScalars& sc, const TensorScalars& ts) {
  const int64_t left = t.numel - at;
  if (left >= kChunkOf<SMALL>)
    update_chunk<GD, SMALL, true>(t, at, kChunkOf<SMALL>, key, sc, ts);
  else
    update_chunk<GD, SMALL, false>(t, at, (int32_t)left, key, sc, ts);
}

template <bool SMALL>
__global__ __launch_bounds__(kThreadsOf<SMALL>) void k_tensors_adam(
    const AdamEntry* __restrict__ entries, const uint32_t* __restrict__ first, int32_t n,
    uint32_t b0, ListScalars sc, const zero_step_result_t* __restrict__ res) {
  TensorScalars ts{0.0f, 0.0f, 1.0f};
  if (res) {
    if (res->skip) return;
    ts.c = res->clip_coef;
  }
  const uint32_t b = b0 + blockIdx.x;
  const int32_t i = find_entry((gptr<const uint32_t>)first, n, b);
  const AdamEntry t = entries[i];
  const int64_t at = (int64_t)(b - first[i]) * kChunkOf<SMALL>;
  ts.step_size = (float)(sc.step_size * t.lr_scale);
  ts.decay = (float)(1.0 - sc.lr * (t.lr_scale * t.weight_decay));
  const uint32_t key = mix(mix(sc.key + (uint32_t)i) + (uint32_t)(at >> kKeyShift));
  switch (t.kind & 3u) {
    case ZERO_F32: return update<ZERO_F32, SMALL>(t, at, key, sc, ts);
    case ZERO_F16: return update<ZERO_F16, SMALL>(t, at, key, sc, ts);
    case ZERO_BF16: return update<ZERO_BF16, SMALL>(t, at, key, sc, ts);
  }
}

// The values of 8-bit moments, tensor i's from its offset; bf16 holds them
// exactly (3 fraction bits, fp32's exponents).
template <bool F32, bool FULL>
__device__ __forceinline__ void read_chunk(const AdamEntry& t, int64_t at, int32_t len,
                                           gptr<void> m, gptr<void> v) {
#pragma unroll
  for (int k = 0; k < kAdamQuads8; ++k) {
    const int32_t r = 4 * (int32_t)(threadIdx.x + k * kAdamThreads8);
    const int n = FULL ? 4 : len - r;
    if (!FULL && n <= 0) continue;
    const int64_t i = at + r, o = t.offset + i;
    const uint32_t m8 = load_8<FULL>((gptr<const uint8_t>)t.m, i, n);
    const uint32_t v8 = load_8<FULL>((gptr<const uint8_t>)t.v, i, n);
    const int64_t b = i / kMomentBlock;
    const uint32_t mb = base_of<kOctavesM>(((gptr<const uint8_t>)t.m_exp)[b]) << 20;
    const uint32_t vb = base_of<kOctavesV>(((gptr<const uint8_t>)t.v_exp)[b]) << 20;
    f32x4 x, y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = decode_m(m8, e, mb);
      y[e] = decode_v(v8, e, vb);
    }
    if constexpr (F32) {
      store_f32<FULL>((gptr<float>)m, o, n, x);
      store_f32<FULL>((gptr<float>)v, o, n, y);
    } else {
      auto top = [](f32x4 a) {
        return u32x2{__float_as_uint(a[0]) >> 16 | (__float_as_uint(a[1]) & 0xFFFF0000u),
                     __float_as_uint(a[2]) >> 16 | (__float_as_uint(a[3]) & 0xFFFF0000u)};
      };
      store_16<FULL>((gptr<uint16_t>)m, o, n, top(x));
      store_16<FULL>((gptr<uint16_t>)v, o, n, top(y));
    }
  }
}

template <bool F32>
__global__ __launch_bounds__(kAdamThreads8) void k_adam_moments(
    const AdamEntry* __restrict__ entries, const uint32_t* __restrict__ first, int32_t n,
    uint32_t b0, void* __restrict__ m, void* __restrict__ v) {
  const uint32_t b = b0 + blockIdx.x;
  const int32_t i = find_entry((gptr<const uint32_t>)first, n, b);
  const AdamEntry t = entries[i];
  const int64_t at = (int64_t)(b - first[i]) * kAdamChunk8, left = t.numel - at;
  if (left >= kAdamChunk8)
    read_chunk<F32, true>(t, at, (int32_t)kAdamChunk8, (gptr<void>)m, (gptr<void>)v);
  else
    read_chunk<F32, false>(t, at, (int32_t)left, (gptr<void>)m, (gptr<void>)v);
}

// Part of the table by way of the kernel arguments (4 KiB).
constexpr int kTablePart = 32;
struct TablePart {
  AdamEntry e[kTablePart];
  uint32_t first[2][kTablePart];
};
static_assert(sizeof(TablePart) <= 3968, "kernel arguments");
__global__ __launch_bounds__(64) void k_adam_table(TablePart part, int32_t n, int32_t all,
                                                   AdamEntry* __restrict__ entries,
                                                   uint32_t* __restrict__ first) {
  const int i = (int)threadIdx.x;
  if (i >= n) return;
  entries[i] = part.e[i];
  first[i] = part.first[0][i];
  first[all + i] = part.first[1][i];
}

const uint32_t* firsts(const zero_adam_list_t* l, bool small) {
  return (const uint32_t*)((const AdamEntry*)l->table + l->n_tensors) + (small ? l->n_tensors : 0);
}

template <bool SMALL>
int adam_launch(const zero_adam_list_t* l, int64_t blocks, const ListScalars& sc,
                const zero_step_result_t* res, hipStream_t stream) {
  return launch_segments(blocks, kAdamLaunch / kChunkOf<SMALL>, [&](int64_t b0, int64_t nb) {
    hipLaunchKernelGGL((k_tensors_adam<SMALL>), dim3((uint32_t)nb), dim3(kThreadsOf<SMALL>),
                       SMALL ? 0 : kAdamLds32, stream, (const AdamEntry*)l->table,
                       firsts(l, SMALL), l->n_tensors, (uint32_t)b0, sc, res);
  });
}

}  // namespace

int launch_adam_table(const zero_adam_tensor_t* tensors, int32_t n, void* table,
                      hipStream_t stream) {
  AdamEntry* entries = (AdamEntry*)table;
  uint32_t* first = (uint32_t*)(entries + n);
  uint32_t blocks[2] = {0, 0};
  int64_t offset = 0;
  for (int32_t i0 = 0; i0 < n; i0 += kTablePart) {
    const int32_t m = n - i0 < kTablePart ? n - i0 : kTablePart;
    TablePart part{};
    for (int32_t i = 0; i < m; ++i) {
      const zero_adam_tensor_t& t = tensors[i0 + i];
      const bool small = t.moment_bits == 8;
      const uint32_t out = t.param ? (uint32_t)t.param_dtype : (uint32_t)kNone;
      part.e[i] = AdamEntry{t.grad, t.master, t.m, t.v, t.m_exp, t.v_exp, t.param, t.numel, offset,
                            t.weight_decay, t.lr_scale, (uint32_t)t.grad_dtype | out << 2, 0u};
      part.first[0][i] = blocks[0];
      part.first[1][i] = blocks[1];
      blocks[small] += (uint32_t)adam_blocks(t.numel, small);
      offset += (t.numel + kMomentBlock - 1) / kMomentBlock * kMomentBlock;
    }
    hipLaunchKernelGGL(k_adam_table, dim3(1), dim3(64), 0, stream, part, m, n, entries + i0,
                       first + i0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
  }
  return (int)hipSuccess;
}

int launch_tensors_adam(const zero_adam_list_t* l, const ListScalars& sc,
                        const zero_step_result_t* res, hipStream_t stream) {
  ListScalars mixed = sc;
  mixed.key = mix(sc.key);
  const int e = adam_launch<false>(l, l->blocks32, mixed, res, stream);
  return e ? e : adam_launch<true>(l, l->blocks8, mixed, res, stream);
}

int launch_adam_moments(const zero_adam_list_t* l, void* m, void* v, bool f32,
                        hipStream_t stream) {
  return launch_segments(l->blocks8, kAdamLaunch / kAdamChunk8, [&](int64_t b0, int64_t nb) {
    hipLaunchKernelGGL(f32 ? k_adam_moments<true> : k_adam_moments<false>, dim3((uint32_t)nb),
                       dim3(kAdamThreads8), 0, stream, (const AdamEntry*)l->table,
                       firsts(l, true), l->n_tensors, (uint32_t)b0, m, v);
  });
}

}  // namespace zk
