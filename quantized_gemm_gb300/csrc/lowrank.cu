// Per-row low-rank adapters beside a shared projection (mm_lowrank_matmul) and
// their gradients (mm_lowrank_matmul_grad) on the CUDA cores, for every type
// and stride:
//
//   shrink   z[m, r]      = s_g * sum_c x[m, c] a[g, c, r]     g = adapter of row m
//   expand   y[m, n]      = sum_r z[m, r] b[g, r, n]
//   outer    out[g, c, r] = sum over the rows m of adapter g of x[m, c] z[m, r]
//
// z stays fp32; every sum is fp32 in a fixed order.
#include "kernels.h"

namespace qg {

namespace {

__device__ __forceinline__ int64_t adapter_of(const LowRankArgs& l, int64_t m) {
  const int64_t g = load_index(l.idx, m * l.idx_s, l.ind64);
  if (g >= 0 && g < l.G) return g;
  if (g != -1) atomicOr(l.status, kStatusIndexRange);
  return -1;
}

// One block per row and 32 ranks: 8 warps share the sum over c.  Lanes run
// over r when r is the nearer dimension of a, over c otherwise.
template <typename T>
__global__ void __launch_bounds__(256)
    shrink_kernel(const LowRankArgs l, const T* x, int64_t x_rs, int64_t x_cs, int64_t C, const T* a, int64_t a_gs,
                  int64_t a_cs, int64_t a_rs, float* z, int lanes_r) {
  pdl_begin();
  __shared__ float part[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r0 = (int64_t)blockIdx.x * 32;
  for (int64_t m = blockIdx.y; m < l.M; m += gridDim.y) {
    const int64_t g = adapter_of(l, m);
    const T* xr = x + m * x_rs;
    const T* ag = a + (g < 0 ? 0 : g) * a_gs;
    float mine = 0.f;     // lane's rank (r0 + lane), this warp's share
    if (g >= 0) {
      if (lanes_r) {
        const int64_t r = r0 + lane;
        if (r < l.R)
          for (int64_t c = warp; c < C; c += 8)
            mine = __fmaf_rn(to_f32(xr[c * x_cs]), to_f32(ag[c * a_cs + r * a_rs]), mine);
      } else {
        for (int j = 0; j < 32 && r0 + j < l.R; ++j) {
          float v = 0.f;
          for (int64_t c = warp * 32 + lane; c < C; c += 256)
            v = __fmaf_rn(to_f32(xr[c * x_cs]), to_f32(ag[c * a_cs + (r0 + j) * a_rs]), v);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          if (lane == j) mine = v;
        }
      }
    }
    part[warp][lane] = mine;
    __syncthreads();
    if (warp == 0 && r0 + lane < l.R) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) v += part[w][lane];
      z[m * l.R + r0 + lane] = g < 0 ? 0.f : (l.scales ? v * l.scales[g * l.scales_s] : v);
    }
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(256)
    expand_kernel(const LowRankArgs l, const float* z, const T* b, int64_t b_gs, int64_t b_rs, int64_t b_ns,
                  int64_t N, T* y) {
  pdl_begin();
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  for (int64_t m = blockIdx.y; m < l.M; m += gridDim.y) {
    const int64_t g = adapter_of(l, m);
    float v = 0.f;
    if (g >= 0) {
      const T* bg = b + g * b_gs + n * b_ns;
      for (int64_t r = 0; r < l.R; ++r) v = __fmaf_rn(z[m * l.R + r], to_f32(bg[r * b_rs]), v);
    }
    y[m * N + n] = from_f32<T>(v);
  }
}

constexpr int kOuterR = 16;

template <typename T>
__global__ void __launch_bounds__(128)
    outer_kernel(const LowRankArgs l, const T* x, int64_t x_rs, int64_t x_cs, int64_t C, const float* z, T* out,
                 int64_t o_gs, int64_t o_cs, int64_t o_rs) {
  pdl_begin();
  const int64_t c = (int64_t)blockIdx.x * 128 + threadIdx.x;
  const int64_t r0 = (int64_t)blockIdx.z * kOuterR;
  for (int64_t g = blockIdx.y; g < l.G; g += gridDim.y) {
    float acc[kOuterR];
#pragma unroll
    for (int j = 0; j < kOuterR; ++j) acc[j] = 0.f;
    for (int64_t m = 0; m < l.M; ++m) {
      if (adapter_of(l, m) != g) continue;
      const float xv = c < C ? to_f32(x[m * x_rs + c * x_cs]) : 0.f;
#pragma unroll
      for (int j = 0; j < kOuterR; ++j)
        if (r0 + j < l.R) acc[j] = __fmaf_rn(xv, z[m * l.R + r0 + j], acc[j]);
    }
    if (c < C) {
#pragma unroll
      for (int j = 0; j < kOuterR; ++j)
        if (r0 + j < l.R) out[g * o_gs + c * o_cs + (r0 + j) * o_rs] = from_f32<T>(acc[j]);
    }
  }
}

unsigned rows_y(int64_t n) { return (unsigned)(n < 65535 ? n : 65535); }

template <typename T>
mm_status shrink_typed(const LowRankArgs& l, const void* x, int64_t x_rs, int64_t x_cs, int64_t C, const void* a,
                       int64_t a_gs, int64_t a_cs, int64_t a_rs, float* z, cudaStream_t stream) {
  const dim3 grid((unsigned)((l.R + 31) / 32), rows_y(l.M));
  return launch_pdl(shrink_kernel<T>, grid, dim3(256), 0, stream, l, static_cast<const T*>(x), x_rs, x_cs, C,
                    static_cast<const T*>(a), a_gs, a_cs, a_rs, z, (int)(a_rs <= a_cs)) == cudaSuccess ? MM_OK
                                                                                                      : MM_ERR_CUDA;
}

template <typename T>
mm_status expand_typed(const LowRankArgs& l, const float* z, const void* b, int64_t b_gs, int64_t b_rs, int64_t b_ns,
                       int64_t N, void* y, cudaStream_t stream) {
  const dim3 grid((unsigned)((N + 255) / 256), rows_y(l.M));
  return launch_pdl(expand_kernel<T>, grid, dim3(256), 0, stream, l, z, static_cast<const T*>(b), b_gs, b_rs, b_ns, N,
                    static_cast<T*>(y)) == cudaSuccess ? MM_OK : MM_ERR_CUDA;
}

template <typename T>
mm_status outer_typed(const LowRankArgs& l, const void* x, int64_t x_rs, int64_t x_cs, int64_t C, const float* z,
                      void* out, int64_t o_gs, int64_t o_cs, int64_t o_rs, cudaStream_t stream) {
  const dim3 grid((unsigned)((C + 127) / 128), rows_y(l.G), (unsigned)((l.R + kOuterR - 1) / kOuterR));
  return launch_pdl(outer_kernel<T>, grid, dim3(128), 0, stream, l, static_cast<const T*>(x), x_rs, x_cs, C, z,
                    static_cast<T*>(out), o_gs, o_cs, o_rs) == cudaSuccess ? MM_OK : MM_ERR_CUDA;
}

}  // namespace

#define QG_BY_TYPE(fn, ...)                                      \
  switch (l.dtype) {                                             \
    case MM_BF16: return fn<__nv_bfloat16>(l, __VA_ARGS__);      \
    case MM_F16: return fn<__half>(l, __VA_ARGS__);              \
    default: return fn<float>(l, __VA_ARGS__);                   \
  }

mm_status launch_lowrank_shrink(const LowRankArgs& l, const void* x, int64_t x_rs, int64_t x_cs, int64_t C,
                                const void* a, int64_t a_gs, int64_t a_cs, int64_t a_rs, float* z,
                                cudaStream_t stream) {
  if (l.M == 0 || l.R == 0) return MM_OK;
  QG_BY_TYPE(shrink_typed, x, x_rs, x_cs, C, a, a_gs, a_cs, a_rs, z, stream)
}

mm_status launch_lowrank_expand(const LowRankArgs& l, const float* z, const void* b, int64_t b_gs, int64_t b_rs,
                                int64_t b_ns, int64_t N, void* y, cudaStream_t stream) {
  if (l.M == 0 || N == 0) return MM_OK;
  QG_BY_TYPE(expand_typed, z, b, b_gs, b_rs, b_ns, N, y, stream)
}

mm_status launch_lowrank_outer(const LowRankArgs& l, const void* x, int64_t x_rs, int64_t x_cs, int64_t C,
                               const float* z, void* out, int64_t o_gs, int64_t o_cs, int64_t o_rs,
                               cudaStream_t stream) {
  if (l.G == 0 || C == 0 || l.R == 0) return MM_OK;
  QG_BY_TYPE(outer_typed, x, x_rs, x_cs, C, z, out, o_gs, o_cs, o_rs, stream)
}

#undef QG_BY_TYPE

}  // namespace qg
