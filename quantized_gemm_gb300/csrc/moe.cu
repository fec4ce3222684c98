// Mixture-of-experts layer for a few tokens (mm_moe_layer) on the CUDA cores:
// the form that takes every type and stride.
//
//   h[t, s]  = act(x[t] Wg[e]) * (x[t] Wu[e])           e = indices[t, s]
//   out[t]   = sum_s weights[t, s] * (h[t, s] Wd[e])
//
// One pass computes h (fp32, in the workspace), one the weighted sum, every
// sum in fp32 in a fixed order.  Each pick reads its expert's weights anew.
#include "moe.cuh"

namespace qg {

namespace {

constexpr int kMoeThreads = 128;
constexpr int kMoeChunk = 512;     // x or h values staged at a time

// Expert of pick (t, s): -1 for none; an index past [-1, G) counts as none and is recorded.
__device__ __forceinline__ int64_t pick_of(const MoeArgs& a, int64_t t, int64_t s, unsigned* status) {
  const int64_t e = load_index(a.gi, t * a.gi_ts + s * a.gi_ss, a.ind64);
  if (e >= 0 && e < a.G) return e;
  if (e != -1) atomicOr(status, kStatusIndexRange);
  return -1;
}

template <typename T>
__global__ void __launch_bounds__(kMoeThreads) moe_hidden_kernel(const MoeArgs a, float* h, unsigned* status) {
  pdl_begin();
  __shared__ float xs[kMoeChunk];
  const int64_t f = (int64_t)blockIdx.x * kMoeThreads + threadIdx.x;
  for (int64_t pick = blockIdx.y; pick < a.tokens * a.S; pick += gridDim.y) {
    const int64_t t = pick / a.S;
    const int64_t e = pick_of(a, t, pick - t * a.S, status);
    if (e < 0) continue;
    const T* x = static_cast<const T*>(a.x) + t * a.x_rs;
    const T* wg = static_cast<const T*>(a.wg) + e * a.wg_gs + f * a.wg_fs;
    const T* wu = a.wu ? static_cast<const T*>(a.wu) + e * a.wu_gs + f * a.wu_fs : nullptr;
    float g = 0.f, u = 0.f;
    for (int64_t k0 = 0; k0 < a.K; k0 += kMoeChunk) {
      const int n = (int)min((int64_t)kMoeChunk, a.K - k0);
      __syncthreads();
      for (int i = threadIdx.x; i < n; i += kMoeThreads) xs[i] = to_f32(x[(k0 + i) * a.x_cs]);
      __syncthreads();
      if (f < a.F)
        for (int i = 0; i < n; ++i) {
          g = __fmaf_rn(xs[i], to_f32(wg[(k0 + i) * a.wg_ks]), g);
          if (wu) u = __fmaf_rn(xs[i], to_f32(wu[(k0 + i) * a.wu_ks]), u);
        }
    }
    if (f < a.F) h[pick * a.F + f] = wu ? activate(g, a.act) * u : activate(g, a.act);
  }
}

template <typename T>
__global__ void __launch_bounds__(kMoeThreads) moe_combine_kernel(const MoeArgs a, const float* h, unsigned* status) {
  pdl_begin();
  __shared__ float hs[kMoeChunk];
  const int64_t n = (int64_t)blockIdx.x * kMoeThreads + threadIdx.x;
  for (int64_t t = blockIdx.y; t < a.tokens; t += gridDim.y) {
    float out = 0.f;
    for (int64_t s = 0; s < a.S; ++s) {
      const int64_t e = pick_of(a, t, s, status);
      if (e < 0) continue;
      const T* wd = static_cast<const T*>(a.wd) + e * a.wd_gs + n * a.wd_ns;
      const float* hr = h + (t * a.S + s) * a.F;
      float acc = 0.f;
      for (int64_t f0 = 0; f0 < a.F; f0 += kMoeChunk) {
        const int m = (int)min((int64_t)kMoeChunk, a.F - f0);
        __syncthreads();
        for (int i = threadIdx.x; i < m; i += kMoeThreads) hs[i] = hr[f0 + i];
        __syncthreads();
        if (n < a.N)
          for (int i = 0; i < m; ++i) acc = __fmaf_rn(hs[i], to_f32(wd[(f0 + i) * a.wd_fs]), acc);
      }
      const float w = a.ew ? static_cast<const float*>(a.ew)[t * a.ew_ts + s * a.ew_ss] : 1.f;
      out = __fmaf_rn(w, acc, out);
    }
    if (n < a.N) static_cast<T*>(a.out)[t * a.N + n] = from_f32<T>(out);
  }
}

template <typename T>
mm_status launch_typed(const MoeArgs& a, float* h, unsigned* status, cudaStream_t stream) {
  const int64_t bf = (a.F + kMoeThreads - 1) / kMoeThreads, bn = (a.N + kMoeThreads - 1) / kMoeThreads;
  if (bf > 0x7fffffffLL || bn > 0x7fffffffLL) return MM_ERR_UNSUPPORTED;
  const int64_t picks = a.tokens * a.S;
  if (bf > 0 && picks > 0 &&
      launch_pdl(moe_hidden_kernel<T>, dim3((unsigned)bf, (unsigned)min(picks, (int64_t)65535)), dim3(kMoeThreads), 0,
                 stream, a, h, status) != cudaSuccess)
    return MM_ERR_CUDA;
  return launch_pdl(moe_combine_kernel<T>, dim3((unsigned)bn, (unsigned)min(a.tokens, (int64_t)65535)),
                    dim3(kMoeThreads), 0, stream, a, (const float*)h, status) == cudaSuccess ? MM_OK : MM_ERR_CUDA;
}

}  // namespace

mm_status launch_simt_moe(const MoeArgs& a, float* h, unsigned* status, cudaStream_t stream) {
  switch (a.dtype) {
    case MM_BF16: return launch_typed<__nv_bfloat16>(a, h, status, stream);
    case MM_F16: return launch_typed<__half>(a, h, status, stream);
    default: return launch_typed<float>(a, h, status, stream);
  }
}

}  // namespace qg
