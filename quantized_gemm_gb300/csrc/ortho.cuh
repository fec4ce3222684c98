// What the two forms of the orthogonalised update share: the norm over fp32's
// whole range and the division by it.
#pragma once

#include "kernels.h"

namespace qg {

// Sums of squares over the whole range of fp32: values of 2^50 and more, and of
// less than 2^-60, are squared after a shift by 2^-80 and 2^80.
struct Squares {
  float mid = 0.f, big = 0.f, small = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float ax = fabsf(x);
    if (ax < 1.1258999e+15f && (ax >= 8.6736174e-19f || ax == 0.f)) {
      mid = fmaf(x, x, mid);
    } else if (ax < 1.f) {
      const float y = x * 1.2089258e+24f;
      small = fmaf(y, y, small);
    } else {                         // infinities and NaN too
      const float y = x * 8.2718061e-25f;
      big = fmaf(y, y, big);
    }
  }
  // A group of values: where the largest lies in [2^-30, 2^50) all squares add up as
  // they are (one below 2^-60 is lost, which is nothing beside the largest's).
  template <int E>
  __device__ __forceinline__ void add(const float (&x)[E]) {
    float top = 0.f;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      top = fmaxf(top, fabsf(x[j]));
      nan |= x[j] != x[j];
    }
    if (top < 1.1258999e+15f && top >= 9.3132257e-10f && !nan) {
#pragma unroll
      for (int j = 0; j < E; ++j) mid = fmaf(x[j], x[j], mid);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) add(x[j]);
    }
  }
  // Over a warp, in fp32; the sums then meet in fp64, which one lane of each warp
  // does (fp64 runs at 1/64 of fp32's rate here).
  __device__ __forceinline__ void join_warp() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mid += __shfl_xor_sync(0xffffffffu, mid, o);
      big += __shfl_xor_sync(0xffffffffu, big, o);
      small += __shfl_xor_sync(0xffffffffu, small, o);
    }
  }
  __device__ __forceinline__ double total() const {
    return (double)mid + (double)big * 1.4615016373309029e+48 + (double)small * 6.8422776578360209e-49;   // 2^160, 2^-160
  }
};

// d = |X|_F + eps as m 2^k: a product with the rounded 1 / d where that is in
// fp32's middle range (k = 0; its rounding scales the whole matrix by 1 + 2^-24 at
// most), a division by m in [1, 2) otherwise.  An infinite d (only infinite values give
// one) counts as NaN, so that the whole matrix becomes NaN, not only those values.
struct Divisor {
  float m, r;
  int k;
  Divisor() = default;
  __device__ __forceinline__ explicit Divisor(double t) {
    m = t < 1e300 ? (float)t : __uint_as_float(0x7FFFFFFFu);
    k = 0;
    if ((!(t < 1e30) || !(t > 1e-30)) && t > 0. && t < 1e300) {      // not zero, infinite or NaN
      const double f = frexp(t, &k);
      m = (float)(2. * f);
      --k;
    }
    r = __frcp_rn(m);
    if (k == 0 && !(r < 3e38f && r > 1e-37f)) k = kAlways;      // a zero or NaN divisor divides
  }
  static constexpr int kAlways = 1 << 20;
  __device__ __forceinline__ float divide(float x) const {
    return k == 0 ? x * r : __fdiv_rn(k == kAlways ? x : scalbnf(x, -k), m);
  }
};

// Small matrices, one cluster each (ortho_small.cu).
bool ortho_small_pays(const OrthoArgs& args);
mm_status launch_ortho_small(const OrthoArgs& args, cudaStream_t stream);

}  // namespace qg
