// Device helpers shared by the kernels of the softmax-attention layer.
#pragma once

#include "gdn2_attn_launch.h"
#include "gdn2_device.h"

namespace gdn2 {

// Largest n in [0, N) with key(n) <= x, for a key that does not decrease and key(0) <= x: a
// 64-way search, every lane of the wave with the same x (N <= 64: one round of loads). A key
// that does decrease (a bad table) still ends, with some n in range.
template <typename F>
__device__ __forceinline__ int wave_search(int N, long x, F key) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) >> 6;
    const int i = lo + lane * step;
    const int cnt = __popcll(__ballot(i < hi && key(i < hi ? i : lo) <= x));
    lo += (cnt > 0 ? cnt - 1 : 0) * step;
    hi = lo + step < hi ? lo + step : hi;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// A word that no one writes during the launch, at a wave-uniform address: a scalar load, which a
// wave waits for apart from its vector loads (those return in order).
template <typename T>
__device__ __forceinline__ T scalar_load(const T* p, long i) {
  typedef const __attribute__((address_space(4))) T* P;
  return reinterpret_cast<P>(reinterpret_cast<uintptr_t>(p))[i];
}

__device__ __forceinline__ int clamped_offset(const int* cu, int n, int T) {
  const int c = cu[n];
  return c < 0 ? 0 : c > T ? T : c;
}

// The new tokens of sequence n: rows [first, first + count) of the token axis, the first of
// them at position len - count (negative positions hold no token).
struct SeqSpan {
  int first, count, len;
};
__device__ __forceinline__ SeqSpan seq_span(const CacheView& c, int n) {
  SeqSpan s;
  if (c.cu_seqlens == nullptr) {
    s.first = n * c.T;
    s.count = c.T;
  } else {
    s.first = clamped_offset(c.cu_seqlens, n, c.T);
    s.count = clamped_offset(c.cu_seqlens, n + 1, c.T) - s.first;
    if (s.count < 0) s.count = 0;
  }
  s.len = c.seq_lens[n];
  if (s.len < 0) s.len = 0;
  return s;
}

// Packed batches: sequence n owns the units of `per` tokens from floor(cu[n] / per) + extra n
// on; for a non-decreasing table the ranges are disjoint.
__device__ __forceinline__ int packed_unit_seq(const CacheView& c, int unit, int per, int extra) {
  return wave_search(c.N, unit, [&](int n) {
    return (long)(clamped_offset(c.cu_seqlens, n, c.T) / per) + (long)extra * n;
  });
}

}  // namespace gdn2
