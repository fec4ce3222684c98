// What the forms of the 8-bit product share.
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

// Four int8 values as two f16 pairs, exactly: the byte with its sign bit flipped goes
// into the mantissa of 1024, from which 1024 + 128 is subtracted.
__device__ __forceinline__ void halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const uint32_t l = __byte_perm(u, 0x64u, 0x4140u), h = __byte_perm(u, 0x64u, 0x4342u);
  const uint32_t c = 0x64806480u;                // 1152 twice
  const __half2 dl = __hsub2(*reinterpret_cast<const __half2*>(&l), *reinterpret_cast<const __half2*>(&c));
  const __half2 dh = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&c));
  lo = *reinterpret_cast<const uint32_t*>(&dl);
  hi = *reinterpret_cast<const uint32_t*>(&dh);
}

// 4 x 4 bytes turned: byte j of t[i] is byte i of w[j].
__device__ __forceinline__ void turn4(const uint32_t (&w)[4], uint32_t (&t)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
  const uint32_t d = __byte_perm(w[0], w[1], 0x7362), e = __byte_perm(w[2], w[3], 0x7362);
  t[0] = __byte_perm(a, b, 0x5410);
  t[1] = __byte_perm(a, b, 0x7632);
  t[2] = __byte_perm(d, e, 0x5410);
  t[3] = __byte_perm(d, e, 0x7632);
}

}  // namespace qg
