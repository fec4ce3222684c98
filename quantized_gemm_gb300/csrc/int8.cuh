// What the CUDA-core forms of the 8-bit product share.
#pragma once

#include "kernels.h"

namespace qg {

// y = T((acc * a_scale) * b_scale + bias), each step rounded in fp32.
template <typename O>
__device__ __forceinline__ O finish8(float acc, float sa, float sb, float bias) {
  return from_f32<O>(__fadd_rn(__fmul_rn(__fmul_rn(acc, sa), sb), bias));
}
template <typename O>
__device__ __forceinline__ float bias_at(const Int8Args& a, int64_t n) {
  return a.bias ? to_f32(static_cast<const O*>(a.bias)[n * a.bias_s]) : 0.f;
}

// 4 bytes at any address, read in aligned words that each hold one of them.
__device__ __forceinline__ uint32_t bytes4(const int8_t* p) {
  const uint32_t sh = ((uint32_t)reinterpret_cast<uintptr_t>(p) & 3u) * 8;
  const uint32_t* w = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)3);
  const uint32_t lo = __ldg(w), hi = sh ? __ldg(w + 1) : 0u;
  return __funnelshift_r(lo, hi, sh);
}

}  // namespace qg
