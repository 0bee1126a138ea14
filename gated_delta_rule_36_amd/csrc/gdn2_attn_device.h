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

// Sum and maximum over the LANES (8 or 16) adjacent lanes of a row, in every lane: DPP steps
// (quad permutations, then the half-row and row mirrors), no trip through LDS.
template <int CTRL>
__device__ __forceinline__ float dpp_f(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, false));
}
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
  x += dpp_f<0xB1>(x);   // quad_perm [1,0,3,2]
  x += dpp_f<0x4E>(x);   // quad_perm [2,3,0,1]
  x += dpp_f<0x141>(x);  // row_half_mirror
  if constexpr (LANES == 16) x += dpp_f<0x140>(x);  // row_mirror
  return x;
}
// Maximum over lanes l, l ^ 16, l ^ 32, l ^ 48, and over l, l ^ 32.
__device__ __forceinline__ float max_halves(float x) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float max_rows(float x) {
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return max_halves(fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1])));
}
__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, dpp_f<0xB1>(x));
  x = fmaxf(x, dpp_f<0x4E>(x));
  x = fmaxf(x, dpp_f<0x141>(x));
  x = fmaxf(x, dpp_f<0x140>(x));
  return max_rows(x);
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
__device__ __forceinline__ SeqSpan seq_span(const CacheView& c, int n) {  // n: wave-uniform
  SeqSpan s;
  s.len = scalar_load(c.seq_lens, n);
  if (c.cu_seqlens == nullptr) {
    s.first = n * c.T;
    s.count = c.T;
  } else {
    const int a = scalar_load(c.cu_seqlens, n), b = scalar_load(c.cu_seqlens, n + 1);
    s.first = a < 0 ? 0 : a > c.T ? c.T : a;
    s.count = (b < 0 ? 0 : b > c.T ? c.T : b) - s.first;
    if (s.count < 0) s.count = 0;
  }
  if (s.len < 0) s.len = 0;
  return s;
}

// Packed batches: the sequence with the largest key(offset, n) <= x (n its index, offset its first
// row), and its span. Up to 64 sequences come in with one round of loads, a lane each.
template <typename F>
__device__ __forceinline__ int packed_span(const CacheView& c, long x, SeqSpan& s, F key) {
  if (c.N > 64) {
    const int n = wave_search(c.N, x, [&](int i) {
      return key(clamped_offset(c.cu_seqlens, i, c.T), i);
    });
    s = seq_span(c, n);
    return n;
  }
  const int lane = threadIdx.x & 63, i = lane < c.N ? lane : c.N - 1;
  const int first = clamped_offset(c.cu_seqlens, i, c.T);
  const int next = clamped_offset(c.cu_seqlens, i + 1, c.T);
  const int len = c.seq_lens[i];
  const int cnt = __popcll(__ballot(lane < c.N && key(first, i) <= x));
  const int n = __builtin_amdgcn_readfirstlane(cnt > 0 ? cnt - 1 : 0);
  s.first = __builtin_amdgcn_readlane(first, n);
  s.count = __builtin_amdgcn_readlane(next, n) - s.first;
  s.len = __builtin_amdgcn_readlane(len, n);
  if (s.count < 0) s.count = 0;
  if (s.len < 0) s.len = 0;
  return n;
}

// The same value, known to be wave-uniform to the compiler, which loses sight of it where paths
// join (bounds held in vector registers turn uniform branches into masked code).
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ SeqSpan uniform(const SeqSpan& s) {
  return SeqSpan{uniform(s.first), uniform(s.count), uniform(s.len)};
}

}  // namespace gdn2
