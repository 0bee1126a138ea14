// Eight channels at a time, for the kernels around the mixer: rows that are read once or written once
// go past the caches' retention (non-temporal).
#pragma once

#include "gdn2_device.h"

namespace gdn2 {

template <typename T>
__device__ __forceinline__ void store8_stream(T* p, const float* f) {
  if constexpr (sizeof(T) == 2) {
    bf16x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = static_cast<bf16>(f[i]);
    __builtin_nontemporal_store(v, reinterpret_cast<bf16x8*>(p));
  } else {
    __builtin_nontemporal_store(f4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f4*>(p));
    __builtin_nontemporal_store(f4{f[4], f[5], f[6], f[7]}, reinterpret_cast<f4*>(p) + 1);
  }
}
__device__ __forceinline__ void load8f(const float* p, float* f) {
  const f4 x = reinterpret_cast<const f4*>(p)[0], y = reinterpret_cast<const f4*>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) { f[i] = x[i]; f[4 + i] = y[i]; }
}

__device__ __forceinline__ void load_stream(Vec8<bf16>& r, const bf16* p) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  r.r = __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u4*>(p)));
}
__device__ __forceinline__ void load_stream(Vec8<float>& r, const float* p) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  r.r0 = __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u4*>(p)));
  r.r1 = __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u4*>(p) + 1));
}

}  // namespace gdn2
