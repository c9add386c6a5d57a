// Gradient norm and clip over a list of tensors.
//
// Norm: S_i = sum_j x_ij^2 for every tensor, the total, its root and the clip
// coefficient; one read of every element, so the bound is HBM.  A square of an
// fp32 (or 16-bit) value is exact in fp64 and the sums are fp64, so neither
// the length of the list nor the range of bf16 costs digits; the fp64 work is
// one conversion and one fused multiply-add an element, well under what the
// vector units do in the time the element takes to arrive.  The list travels
// in the kernel arguments, kNormBatch tensors a launch: gradient tensors move
// from step to step, and a table in device memory would cost a copy each time.
// 4.02 GB in one fp32 tensor 580 us (6.9 TB/s), 3.12 GB in 582 fp16 tensors, three
// launches, 470 us (6.6).
//
// The sums keep one order: chunk by chunk, thread t of a chunk's workgroup
// takes its 16-byte pieces t, t + T, ... in turn, the workgroup's threads are
// added in a fixed tree, a tensor's chunks and then the tensors likewise.
// Pieces are counted from the tensor's start whatever its address, so two
// tensors with equal values have equal sums.
//
// Clip: y = cast((x * s) * c), one read and one write of every element, bound by
// HBM: 582 tensors from fp32 to fp16, 9.3 GB, 1.56 ms (6.0 TB/s).
#include <stddef.h>

#include "tensors_internal.h"
#include "zero_device.h"

namespace zk {
namespace {

using namespace dev;

constexpr int kNormThreads = 256;
constexpr int kClipThreads = 256;
// Elements a clip workgroup takes: short workgroups, since the stores of one
// overlap the loads of the next (16384 / 8192 / 4096: GPT-2's list from fp32 to
// fp16 1.67 / 1.63 / 1.57 ms).
constexpr int64_t kClipChunk = 4096;
// Entries that fit the 4 KiB of kernel arguments beside the other arguments.
constexpr int kNormBatch = 195;
constexpr int kClipBatch = 139;
// Partials of a tensor that one thread adds in turn.
constexpr int64_t kAlone = 4;
constexpr int kDtypeShift = 60;  // a numel's top bits hold the type(s)

struct NormBatch {
  const void* src[kNormBatch];
  uint64_t numel[kNormBatch];   // | dtype << kDtypeShift
  uint32_t first[kNormBatch];   // first chunk of the tensor within this launch
};
struct ClipBatch {
  const void* src[kClipBatch];
  void* dst[kClipBatch];
  uint64_t numel[kClipBatch];   // | (src dtype | dst dtype << 2) << kDtypeShift
  uint32_t first[kClipBatch];
};
static_assert(sizeof(NormBatch) <= 3904 && sizeof(ClipBatch) <= 3904, "kernel arguments");

struct TensorRecord {
  int64_t first;  // first chunk of the tensor in the whole list
  int64_t chunks;
};

// 16 bytes at any element's address: global loads and stores need no more
// than element alignment on gfx950.
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
// Pointers out of the argument table are generic; typed as global memory the
// accesses need not wait on both memory counters.
template <typename T>
using gptr = __attribute__((address_space(1))) T*;
template <bool NT = true>
__device__ __forceinline__ u32x4 load16(const char* p) {
  if constexpr (NT) return __builtin_nontemporal_load((gptr<const u32x4_a2>)p);
  else return *(gptr<const u32x4_a2>)p;
}
__device__ __forceinline__ void store16(u32x4 v, char* p) {
  __builtin_nontemporal_store(v, (gptr<u32x4_a2>)p);
}

template <int D>
__device__ __forceinline__ constexpr int per16() { return D == ZERO_F32 ? 4 : 8; }

// Element e of a 16-byte piece, and one element in memory.
template <int D>
__device__ __forceinline__ float piece_elem(u32x4 v, int e) {
  if constexpr (D == ZERO_F32) return __uint_as_float(v[e]);
  else
    return to_f32<D == ZERO_BF16 ? Fmt::BF16 : Fmt::F16>((v[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
}
template <int D>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if constexpr (D == ZERO_F32) return ((gptr<const float>)p)[i];
  else return to_f32<D == ZERO_BF16 ? Fmt::BF16 : Fmt::F16>(((gptr<const uint16_t>)p)[i]);
}
template <int D>
__device__ __forceinline__ void store_elem(void* p, int64_t i, float x) {
  if constexpr (D == ZERO_F32) ((gptr<float>)p)[i] = x;
  else ((gptr<uint16_t>)p)[i] = (uint16_t)from_f32<D == ZERO_BF16 ? Fmt::BF16 : Fmt::F16>(x);
}

// Largest i < n with first[i] <= b (n >= 1, first[0] = 0).
__device__ __forceinline__ int find_tensor(const uint32_t* first, int n, uint32_t b) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= b) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Sum of one thread's squares over elements [0, len) of a chunk.  FINITE: inf
// and NaN count zero and set bad.
template <int D, bool FINITE, bool NT>
__device__ __forceinline__ double chunk_squares(const void* base, int64_t at, int64_t len,
                                                uint32_t& bad) {
  constexpr int E = per16<D>(), U = 4;
  const char* p = (const char*)base + at * (D == ZERO_F32 ? 4 : 2);
  const int64_t pieces = len / E;
  double s = 0.0;
  auto add = [&](float x) {
    if constexpr (FINITE) s += sq_or_zero(x, bad);
    else s = __builtin_fma((double)x, (double)x, s);
  };
  int64_t i = threadIdx.x;
  for (; i + (U - 1) * kNormThreads < pieces; i += U * kNormThreads) {
    u32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u] = load16<NT>(p + 16 * (i + u * kNormThreads));
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < E; ++e) add(piece_elem<D>(v[u], e));
  }
  for (; i < pieces; i += kNormThreads) {
    const u32x4 v = load16<NT>(p + 16 * i);
#pragma unroll
    for (int e = 0; e < E; ++e) add(piece_elem<D>(v, e));
  }
  const int64_t j = pieces * E + threadIdx.x;
  if (j < len) add(load_elem<D>(base, at + j));
  return s;
}

template <int D>
__device__ __forceinline__ double chunk_sum(const void* base, int64_t at, int64_t len, bool again,
                                            uint32_t& bad) {
  double s = again ? chunk_squares<D, false, false>(base, at, len, bad)
                   : chunk_squares<D, false, true>(base, at, len, bad);
  // finite elements cannot overflow fp64: a sum that is not finite has met an
  // inf or NaN, and is taken again without them
  if (!__builtin_isfinite(s)) s = chunk_squares<D, true, true>(base, at, len, bad);
  return s;
}

// Values first, first + step, ... of get(0..count).
template <typename Get>
__device__ __forceinline__ void strided_sum(int64_t first, int64_t step, int64_t count, double& x,
                                            uint32_t& bad, Get get) {
  x = 0.0;
  bad = 0;
#pragma unroll 8
  for (int64_t j = first; j < count; j += step) {
    const Partial pt = get(j);
    x += __longlong_as_double((long long)pt.lo);
    bad |= (uint32_t)(pt.hi >> 63);
  }
}

// FINISH: the list's last launch, of few short tensors: its last workgroup does
// what k_tensors_finalize<1> would, in its order.
template <bool FINISH>
__global__ __launch_bounds__(kNormThreads) void k_tensors_norm(
    NormBatch nb, int32_t n, int32_t t0, int64_t chunk0, int64_t chunk, int64_t again, int32_t arm,
    int32_t all, TensorRecord* __restrict__ records, Partial* __restrict__ partials,
    uint32_t* __restrict__ ticket, double* __restrict__ tensor_sq, FinalizeArgs fa,
    zero_step_result_t* __restrict__ res) {
  __shared__ uint32_t s_last;
  const uint32_t b = blockIdx.x;
  if (arm && b == 0 && threadIdx.x == 0) *ticket = 0u;
  const int i = find_tensor(nb.first, n, b);
  const int64_t numel = (int64_t)(nb.numel[i] & ((1ull << kDtypeShift) - 1));
  const int dtype = (int)(nb.numel[i] >> kDtypeShift);
  const int64_t c = (int64_t)(b - nb.first[i]), at = c * chunk;
  const int64_t len = numel - at < chunk ? numel - at : chunk;
  if (c == 0 && threadIdx.x == 0)
    records[t0 + i] = TensorRecord{chunk0 + nb.first[i], numel ? (numel - 1) / chunk + 1 : 1};
  uint32_t bad = 0;
  double s;
  const bool keep = chunk0 + b >= again;
  if (dtype == ZERO_F32) s = chunk_sum<ZERO_F32>(nb.src[i], at, len, keep, bad);
  else if (dtype == ZERO_F16) s = chunk_sum<ZERO_F16>(nb.src[i], at, len, keep, bad);
  else s = chunk_sum<ZERO_BF16>(nb.src[i], at, len, keep, bad);
  block_tree<kNormThreads>(s, bad);
  if (threadIdx.x == 0)
    partials[chunk0 + b] = Partial{(uint64_t)__double_as_longlong(s),
                                   (uint64_t)(bad ? 1u : 0u) << 63};
  if constexpr (FINISH) {
    if (threadIdx.x == 0) {
      __threadfence();  // the workgroup's record and partial, before the ticket
      s_last = atomicAdd(ticket, 1u) == gridDim.x - 1 ? 1u : 0u;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    s = 0.0;
    bad = 0;
    for (int32_t t = threadIdx.x; t < all; t += kNormThreads) {
      const TensorRecord r = records[t];
      double x;
      uint32_t inf;
      strided_sum(0, 1, r.chunks, x, inf, [&](int64_t j) { return partials[r.first + j]; });
      if (tensor_sq) tensor_sq[t] = (x * fa.inv64) * fa.inv64;
      s += x;
      bad |= inf;
    }
    block_tree<kNormThreads>(s, bad);
    if (threadIdx.x == 0) finalize_bf16_into(s, bad, fa, res);
  }
}

// Each G threads sum one tensor's partials (G = 1, a wave or the workgroup: the
// launcher picks by the longest tensor, so that short tensors do not take a
// workgroup each); the last workgroup to finish (ticket) sums the tensors and
// finalizes.
template <int G>
constexpr int kFinalThreads = G > kNormThreads ? G : kNormThreads;
template <int G>
__global__ __launch_bounds__(kFinalThreads<G>) void k_tensors_finalize(
    const Partial* __restrict__ partials, const TensorRecord* __restrict__ records,
    Partial* __restrict__ sums, int32_t n, double* __restrict__ tensor_sq,
    uint32_t* __restrict__ ticket, FinalizeArgs fa, zero_step_result_t* __restrict__ res) {
  constexpr int TB = kFinalThreads<G>;
  __shared__ uint32_t s_last;
  double x = 0.0;
  uint32_t bad = 0;
  const int32_t i = (int32_t)(blockIdx.x * (TB / G) + threadIdx.x / G);
  if (i < n) {
    const TensorRecord r = records[i];
    strided_sum(threadIdx.x % G, G, r.chunks, x, bad, [&](int64_t j) { return partials[r.first + j]; });
  }
  if constexpr (G == 64) {
    for (unsigned int d = 1; d < 64; d <<= 1) {
      x += __longlong_as_double((long long)shfl_down_bits((uint64_t)__double_as_longlong(x), d));
      bad |= (uint32_t)__shfl_xor((int)bad, (int)d);
    }
  } else if constexpr (G == TB) {
    block_tree<TB>(x, bad);
  }
  if (i < n && threadIdx.x % G == 0) {
    if (tensor_sq) tensor_sq[i] = (x * fa.inv64) * fa.inv64;
    if (n > 1)
      sums[i] = Partial{(uint64_t)__double_as_longlong(x), (uint64_t)(bad ? 1u : 0u) << 63};
  }
  if (n > 1) {
    // Every wave waits until its sums are in the XCD's L2; one write-back of
    // that then stands before the ticket.  A fence in every storing thread would
    // be a write-back a wave: 582 tensors 19.5 us, with this 10.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      s_last = gridDim.x == 1 || atomicAdd(ticket, 1u) == gridDim.x - 1 ? 1u : 0u;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    strided_sum(threadIdx.x, TB, n, x, bad, [&](int64_t j) { return sums[j]; });
    block_tree<TB>(x, bad);
  }
  if (threadIdx.x == 0) finalize_bf16_into(x, bad, fa, res);
}

// (x * s) * c, each product rounded to fp32.  The barrier keeps the second
// product apart from the cast: the compiler would otherwise fold both into the
// mixed-precision multiply, whose fp16 result skips the fp32 rounding.
__device__ __forceinline__ float clipped(float x, float s, float c) {
  float y = (x * s) * c;
  asm volatile("" : "+v"(y));
  return y;
}

// One clip workgroup's elements [at, at + len) of a tensor.
template <int SD, int DD>
__device__ __forceinline__ void clip_chunk(const void* src, void* dst, int64_t at, int64_t len,
                                           float s, float c) {
  // a piece is 8 elements: 16 bytes of a 16-bit side, two 16-byte halves of an
  // fp32 side
  const int64_t pieces = len >> 3;
  const char* ps = (const char*)src + at * (SD == ZERO_F32 ? 4 : 2);
  char* pd = (char*)dst + at * (DD == ZERO_F32 ? 4 : 2);
  for (int64_t i = threadIdx.x; i < pieces; i += kClipThreads) {
    float x[8];
    if constexpr (SD == ZERO_F32) {
      const u32x4 a = load16(ps + 32 * i);
      const u32x4 b = load16(ps + 32 * i + 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = __uint_as_float(a[e]);
        x[4 + e] = __uint_as_float(b[e]);
      }
    } else {
      const u32x4 a = load16(ps + 16 * i);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = piece_elem<SD>(a, e);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = clipped(x[e], s, c);
    if constexpr (DD == ZERO_F32) {
      u32x4 a, b;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = __float_as_uint(x[e]);
        b[e] = __float_as_uint(x[4 + e]);
      }
      store16(a, pd + 32 * i);
      store16(b, pd + 32 * i + 16);
    } else {
      constexpr Fmt F = DD == ZERO_BF16 ? Fmt::BF16 : Fmt::F16;
      u32x4 a;
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] = from_f32<F>(x[2 * e]) | (from_f32<F>(x[2 * e + 1]) << 16);
      store16(a, pd + 16 * i);
    }
  }
  const int64_t j = (pieces << 3) + threadIdx.x;
  if (j < len) store_elem<DD>(dst, at + j, clipped(load_elem<SD>(src, at + j), s, c));
}

template <int SD>
__device__ __forceinline__ void clip_to(int dd, const void* src, void* dst, int64_t at,
                                        int64_t len, float s, float c) {
  if (dd == ZERO_F32) clip_chunk<SD, ZERO_F32>(src, dst, at, len, s, c);
  else if (dd == ZERO_F16) clip_chunk<SD, ZERO_F16>(src, dst, at, len, s, c);
  else clip_chunk<SD, ZERO_BF16>(src, dst, at, len, s, c);
}

// What a clip that finishes the norm by itself needs (all: tensors of the list).
struct Finish {
  const Partial* partials;
  const TensorRecord* records;
  double* tensor_sq;
  FinalizeArgs fa;
};

// The sums of k_tensors_finalize, in its order (WIDE: <64>, else <1>), by every
// workgroup for itself: n at most kClipThreads tensors of few partials in all.
template <bool WIDE>
__device__ __forceinline__ void finish_norm(const Finish& f, int32_t n, zero_step_result_t* res) {
  __shared__ double s_x[kClipThreads];
  __shared__ uint32_t s_bad[kClipThreads];
  double x = 0.0;
  uint32_t bad = 0;
  const int32_t t = (int32_t)threadIdx.x;
  if constexpr (WIDE) {
    for (int32_t i = t >> 6; i < n; i += kClipThreads / 64) {
      const TensorRecord r = f.records[i];
      strided_sum(t & 63, 64, r.chunks, x, bad, [&](int64_t j) { return f.partials[r.first + j]; });
      for (unsigned int d = 1; d < 64; d <<= 1) {
        x += __longlong_as_double((long long)shfl_down_bits((uint64_t)__double_as_longlong(x), d));
        bad |= (uint32_t)__shfl_xor((int)bad, (int)d);
      }
      if ((t & 63) == 0) {
        s_x[i] = x;
        s_bad[i] = bad;
      }
    }
    __syncthreads();
    x = t < n ? s_x[t] : 0.0;
    bad = t < n ? s_bad[t] : 0u;
  } else if (t < n) {
    const TensorRecord r = f.records[t];
    strided_sum(0, 1, r.chunks, x, bad, [&](int64_t j) { return f.partials[r.first + j]; });
  }
  if (blockIdx.x == 0 && t < n && f.tensor_sq)
    f.tensor_sq[t] = (x * f.fa.inv64) * f.fa.inv64;
  block_tree<kClipThreads>(x, bad);
  if (t == 0) finalize_bf16_into(x, bad, f.fa, res);
}

enum { kClipAlone, kClipFinish, kClipFinishWide };
template <int MODE>
__global__ __launch_bounds__(kClipThreads) void k_tensors_clip(
    ClipBatch cb, int32_t n, uint32_t last, float s, Finish f,
    zero_step_result_t* __restrict__ res) {
  __shared__ zero_step_result_t s_res;
  if constexpr (MODE != kClipAlone) {
    finish_norm<MODE == kClipFinishWide>(f, n, &s_res);
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x == 0) *res = s_res;
  }
  const zero_step_result_t* got = MODE == kClipAlone ? res : &s_res;
  if (got->skip) return;
  const float c = got->clip_coef;
  const uint32_t b = last - blockIdx.x;
  const int i = find_tensor(cb.first, n, b);
  const int64_t numel = (int64_t)(cb.numel[i] & ((1ull << kDtypeShift) - 1));
  const int sd = (int)(cb.numel[i] >> kDtypeShift) & 3;
  const int dd = (int)(cb.numel[i] >> (kDtypeShift + 2));
  if (cb.src[i] == cb.dst[i] && s == 1.0f && c == 1.0f) return;  // in place: same type
  const int64_t at = (int64_t)(b - cb.first[i]) * kClipChunk;
  const int64_t len = numel - at < kClipChunk ? numel - at : kClipChunk;
  if (len <= 0) return;
  if (sd == ZERO_F32) clip_to<ZERO_F32>(dd, cb.src[i], cb.dst[i], at, len, s, c);
  else if (sd == ZERO_F16) clip_to<ZERO_F16>(dd, cb.src[i], cb.dst[i], at, len, s, c);
  else clip_to<ZERO_BF16>(dd, cb.src[i], cb.dst[i], at, len, s, c);
}

}  // namespace

namespace {

// Workspace: ticket | records [n] | sums [n] | partials [chunks].  clip: a clip
// of the list follows; finish: and that clip finalizes.
int norm_launches(const zero_tensor_t* tensors, int32_t n, const TensorLayout& l,
                  double* tensor_sq, void* workspace, bool clip, bool finish,
                  const FinalizeArgs& fa, zero_step_result_t* res, hipStream_t stream) {
  const int64_t chunk = kTensorChunk << l.shift;
  uint32_t* ticket = (uint32_t*)workspace;
  TensorRecord* records = (TensorRecord*)((char*)workspace + kTicketBytes);
  Partial* sums = (Partial*)(records + n);
  Partial* partials = sums + n;
  // Where a clip follows, it starts with the list's end: the last kAgainBytes
  // are read so that they stay in the last-level cache (256 MB, shared with what
  // the clip writes); the rest passes by.  Llama-3 block, 436 MB: the clip 148 ->
  // 130 us; all of it read so, the norm would take 8 us longer.
  constexpr int64_t kAgainBytes = (int64_t)192 << 20;
  int64_t again = l.chunks;
  if (clip) {
    int64_t bytes = 0;
    for (int32_t i = n - 1; i >= 0 && bytes < kAgainBytes; --i) {
      const int64_t per = chunk * (tensors[i].src_dtype == ZERO_F32 ? 4 : 2);
      const int64_t nc = tensors[i].numel ? (tensors[i].numel - 1) / chunk + 1 : 1;
      const int64_t want = (kAgainBytes - bytes + per - 1) / per;
      again -= nc < want ? nc : want;
      bytes += (nc < want ? nc : want) * per;
    }
  }
  int64_t chunk0 = 0;
  // as few launches as the table allows, of equally many tensors: a short last
  // launch would leave CUs idle
  const int32_t launches = (n + kNormBatch - 1) / kNormBatch;
  const int32_t batch = launches ? (n + launches - 1) / launches : 1;
  // The last launch's last workgroup can finish a list of few short tensors,
  // where launches are what costs; the first has set its ticket.
  const bool fused = launches > 1 && n <= 4 * kNormThreads && l.longest <= kAlone;
  for (int32_t t0 = 0; t0 < n; t0 += batch) {
    const int32_t m = n - t0 < batch ? n - t0 : batch;
    NormBatch nb;
    int64_t blocks = 0;
    for (int32_t i = 0; i < m; ++i) {
      const zero_tensor_t& t = tensors[t0 + i];
      nb.src[i] = t.src;
      nb.numel[i] = (uint64_t)t.numel | (uint64_t)t.src_dtype << kDtypeShift;
      nb.first[i] = (uint32_t)blocks;
      blocks += t.numel ? (t.numel - 1) / chunk + 1 : 1;
    }
    const bool last = fused && t0 + batch >= n;
    hipLaunchKernelGGL(last ? k_tensors_norm<true> : k_tensors_norm<false>, dim3((uint32_t)blocks),
                       dim3(kNormThreads), 0, stream, nb, m, t0, chunk0, chunk, again,
                       t0 == 0 ? 1 : 0, n, records, partials, ticket, tensor_sq, fa, res);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    chunk0 += blocks;
  }
  if (fused || finish) return (int)hipSuccess;
  auto finalize = [&](auto kernel, int group, int threads) {
    const int64_t blocks = ((int64_t)n * group + threads - 1) / threads;
    hipLaunchKernelGGL(kernel, dim3(blocks > 0 ? (uint32_t)blocks : 1u), dim3(threads), 0, stream,
                       partials, records, sums, n, tensor_sq, ticket, fa, res);
  };
  // a thread takes up to kAlone partials in turn, a wave 32 a lane; 290 one-chunk
  // tensors take 5 us by threads, 12 us by workgroups (and their ticket)
  if (l.longest <= kAlone) finalize(k_tensors_finalize<1>, 1, kNormThreads);
  else if (l.longest <= 2048) finalize(k_tensors_finalize<64>, 64, kNormThreads);
  else finalize(k_tensors_finalize<1024>, 1024, 1024);
  return (int)hipGetLastError();
}

// The list is gone through backwards: what the norm has read last may still
// lie in the last-level cache.
int clip_launches(const zero_tensor_t* tensors, int32_t n, float scale, int mode, const Finish& f,
                  zero_step_result_t* res, hipStream_t stream) {
  const auto kernel = mode == kClipAlone    ? k_tensors_clip<kClipAlone>
                      : mode == kClipFinish ? k_tensors_clip<kClipFinish>
                                            : k_tensors_clip<kClipFinishWide>;
  constexpr int64_t kMaxBlocks = (int64_t)1 << 23;  // of one launch: 2^31 threads
  const int32_t launches = (n + kClipBatch - 1) / kClipBatch;
  const int32_t batch = launches ? (n + launches - 1) / launches : 1;
  for (int32_t t1 = n; t1 > 0;) {
    ClipBatch cb;
    int32_t t0 = t1;
    int64_t blocks = 0;
    while (t0 > 0 && t1 - t0 < batch) {
      const int64_t nb = (tensors[t0 - 1].numel + kClipChunk - 1) / kClipChunk;
      if (nb > UINT32_MAX - kMaxBlocks) return (int)hipErrorInvalidValue;
      if (t0 < t1 && blocks + nb > kMaxBlocks) break;
      --t0;
      blocks += nb;
    }
    uint32_t first = 0;
    for (int32_t m = 0; m < t1 - t0; ++m) {
      const zero_tensor_t& t = tensors[t0 + m];
      cb.src[m] = t.src;
      cb.dst[m] = t.dst;
      cb.numel[m] = (uint64_t)t.numel | (uint64_t)(t.src_dtype | t.dst_dtype << 2) << kDtypeShift;
      cb.first[m] = first;
      first += (uint32_t)((t.numel + kClipChunk - 1) / kClipChunk);
    }
    for (int64_t b1 = blocks; b1 > 0; b1 -= kMaxBlocks) {
      hipLaunchKernelGGL(kernel, dim3((uint32_t)(b1 < kMaxBlocks ? b1 : kMaxBlocks)),
                         dim3(kClipThreads), 0, stream, cb, t1 - t0, (uint32_t)(b1 - 1), scale, f,
                         res);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return (int)e;
    }
    t1 = t0;
  }
  return (int)hipSuccess;
}

}  // namespace

int launch_tensors_norm(const zero_tensor_t* tensors, int32_t n, double* tensor_sq,
                        void* workspace, const FinalizeArgs& fa, zero_step_result_t* res,
                        hipStream_t stream) {
  return norm_launches(tensors, n, tensor_layout(tensors, n), tensor_sq, workspace, false, false,
                       fa, res, stream);
}

int launch_tensors_clip(const zero_tensor_t* tensors, int32_t n, float scale,
                        const zero_step_result_t* res, hipStream_t stream) {
  return clip_launches(tensors, n, scale, kClipAlone, Finish{}, (zero_step_result_t*)res, stream);
}

// A small list's clip, of one launch, finishes the norm itself: up to
// kFinishChunks chunks the launch that this saves costs more than every
// workgroup's loads of all partials (a call, fp32 to fp16, finished apart against
// in the clip: 1 tensor of 64 chunks 13.3 / 10.0 us, 9 of 192 16.3 / 14.3, 64
// of 256 18.1 / 15.2, 139 of 256 18.5 / 15.8; beyond, 64 of 320 21.2 / 35.2, 9 of
// 512 23.2 / 25.5, 139 of 1024 41 / 143).
int launch_tensors_norm_clip(const zero_tensor_t* tensors, int32_t n, double* tensor_sq,
                             void* workspace, const FinalizeArgs& fa, float scale,
                             zero_step_result_t* res, hipStream_t stream) {
  const TensorLayout l = tensor_layout(tensors, n);
  constexpr int64_t kFinishChunks = 256;
  bool any = false;
  for (int32_t i = 0; i < n && !any; ++i) any = tensors[i].numel > 0;
  const bool finish = any && n <= kClipBatch && l.chunks <= kFinishChunks;
  static_assert(kClipBatch <= kClipThreads, "a thread for every tensor");
  const int e = norm_launches(tensors, n, l, tensor_sq, workspace, true, finish, fa, res, stream);
  if (e) return e;
  if (!finish)
    return clip_launches(tensors, n, scale, kClipAlone, Finish{}, res, stream);
  const TensorRecord* records = (const TensorRecord*)((char*)workspace + kTicketBytes);
  const Finish f{(const Partial*)(records + n) + n, records, tensor_sq, fa};
  return clip_launches(tensors, n, scale, l.longest <= kAlone ? kClipFinish : kClipFinishWide, f,
                       res, stream);
}

}  // namespace zk
