// Per-row low-rank adapters beside a shared projection (mm_lowrank_matmul) and
// their gradients (mm_lowrank_matmul_grad) on the CUDA cores, for every type
// and stride:
//
//   shrink   z[m, r]      = s_g * sum_c x[m, c] a[g, c, r]     g = adapter of row m
//   expand   y[m, n]      = sum_r z[m, r] b[g, r, n]
//   outer    out[g, c, r] = sum over the rows m of adapter g of x[m, c] z[m, r]
//
// z stays fp32; every sum is fp32 in a fixed order.  The expansion's y is T in Y
// itself or, for few rows, an fp32 array (kFloatPartRows, kernels.h).
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
    expand_kernel(const LowRankArgs l, const float* z, int64_t z_ld, const T* b, int64_t b_gs, int64_t b_rs, int64_t b_ns,
                  int64_t N, T* y, int y_f32) {
  pdl_begin();
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  for (int64_t m = blockIdx.y; m < l.M; m += gridDim.y) {
    const int64_t g = adapter_of(l, m);
    float v = 0.f;
    if (g >= 0) {
      const T* bg = b + g * b_gs + n * b_ns;
      for (int64_t r = 0; r < l.R; ++r) v = __fmaf_rn(z[m * z_ld + r], to_f32(bg[r * b_rs]), v);
    }
    if (y_f32) reinterpret_cast<float*>(y)[m * N + n] = v;
    else y[m * N + n] = from_f32<T>(v);
  }
}

// ------------------------------------------------------------------ few rows (16-bit types)
//
// A decode batch: each row has its own adapter, so the bound is reading the
// adapters once.  Every row is cut into kSplit shares of c, one block each,
// so that one row's adapter streams through kSplit SMs; a share's sums stay
// apart in zp[share][m][r] and the expansion adds them in share order.
// Rows of one adapter read it from L2 again, which costs less than sorting
// rows while there are few of them (lowrank_few_rows).  (Reading an adapter
// once for four neighbouring rows was slower below 512 rows, and above for
// rows of different adapters.)
//
// 61 rows of 4096 x 14336, rank 32, 48 adapters: 42 us for the three launches,
// 159 MB (3.8 TB/s): shrink about 11, the expansion 9 under the projection's
// 27.  One row of 4096 x 4096, rank 16: 12 us (2.9 TB/s), most of it the three
// launches' latency.

constexpr int kSplit = 8;
constexpr int kFewThreads = 128;

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = to_f32(e[j]);
}

// a with r contiguous: a thread takes 8 ranks of every (128 / octets)-th c.
template <typename T>
__device__ __forceinline__ void shrink_share_r(const T* x, int64_t x_cs, const T* a, int64_t a_cs, int64_t c0,
                                               int64_t c1, int oct, float (&acc)[8]) {
  // lanes of an octet column: threads oct_id + i * oct
  const int o = threadIdx.x % oct, step = kFewThreads / oct;
  const int first = threadIdx.x / oct;
  if (first >= step) return;
  constexpr int kAhead = 8;
  for (int64_t c = c0 + first; c < c1; c += (int64_t)step * kAhead) {
    uint4 u[kAhead];
    float xv[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t ci = c + (int64_t)i * step;
      u[i] = make_uint4(0u, 0u, 0u, 0u);
      xv[i] = 0.f;
      if (ci < c1) {
        u[i] = *reinterpret_cast<const uint4*>(a + ci * a_cs + o * 8);
        xv[i] = to_f32(x[ci * x_cs]);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (c + (int64_t)i * step >= c1) break;     // nothing was read: 0 * x must not make a NaN
      float f[8];
      unpack8<T>(u[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = __fmaf_rn(xv[i], f[j], acc[j]);
    }
  }
}

// Block (share, row): ranks in passes of 64 (a with r contiguous) or one rank
// per warp at a time (a with c contiguous).
template <typename T, bool CC>
__global__ void __launch_bounds__(kFewThreads)
    shrink_rows_kernel(const LowRankArgs l, const T* x, int64_t x_rs, int64_t x_cs, int64_t C, const T* a, int64_t a_gs,
                       int64_t a_ld, float* zp) {
  pdl_begin();
  __shared__ float part[kFewThreads][9];
  const int64_t m = blockIdx.y;
  const int share = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t g = adapter_of(l, m);
  float* z = zp + ((int64_t)share * l.M + m) * l.R;
  if (g < 0) {
    for (int64_t r = threadIdx.x; r < l.R; r += kFewThreads) z[r] = 0.f;
    return;
  }
  const int64_t per = ((C + kSplit - 1) / kSplit + 7) / 8 * 8;
  const int64_t c0 = min(C, share * per), c1 = min(C, c0 + per);
  const float scale = l.scales ? l.scales[g * l.scales_s] : 1.f;
  const T* xr = x + m * x_rs;
  const T* ag = a + g * a_gs;
  if constexpr (!CC) {
    for (int64_t r0 = 0; r0 < l.R; r0 += 64) {
      const int oct = (int)min((int64_t)8, (l.R - r0) / 8);     // R is a multiple of 8
      float acc[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = 0.f;
      shrink_share_r<T>(xr, x_cs, ag + r0, a_ld, c0, c1, oct, acc);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) part[threadIdx.x][j] = acc[j];
      __syncthreads();
      const int step = kFewThreads / oct;
      if (threadIdx.x < oct * 8) {
        const int o = threadIdx.x / 8, j = threadIdx.x % 8;
        float v = 0.f;
        for (int i = 0; i < step; ++i) v += part[o + i * oct][j];
        z[r0 + threadIdx.x] = v * scale;
      }
    }
  } else {
    // four ranks at a time share the reads of x
    for (int64_t r0 = warp * 4; r0 < l.R; r0 += 16) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      for (int64_t c = c0 + lane * 8; c < c1; c += 256) {
        uint4 u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = *reinterpret_cast<const uint4*>(ag + min(r0 + j, l.R - 1) * a_ld + c);
        float xv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) xv[i] = to_f32(xr[(c + i) * x_cs]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float f[8];
          unpack8<T>(u[j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[j] = __fmaf_rn(xv[i], f[i], acc[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
        if (lane == j && r0 + j < l.R) z[r0 + j] = acc[j] * scale;
      }
    }
  }
}

// Block (1024 columns, row): a thread takes 8 columns (b with n contiguous) or
// walks columns with r contiguous; the row's z is the sum of its shares.
// Only z depends on the launch before: the adapter's first rows are read, and
// the next launch let in, ahead of the wait for it (that launch began after
// all earlier work was complete).
constexpr int kExpandMaxR = 1024;

template <typename T, bool NC>
__global__ void __launch_bounds__(kFewThreads)
    expand_rows_kernel(const LowRankArgs l, const float* zp, const T* b, int64_t b_gs, int64_t b_ld, int64_t N, T* y,
                       int yvec, int y_f32) {
  pdl_trigger();
  __shared__ float zs[kExpandMaxR];
  const int64_t m = blockIdx.y;
  const int64_t g = adapter_of(l, m);
  const int R = (int)l.R;
  const T* bg = b + (g < 0 ? 0 : g) * b_gs;
  T* yr = y + m * N;
  const int64_t n8 = ((int64_t)blockIdx.x * kFewThreads + threadIdx.x) * 8;
  constexpr int kAhead = 8;
  uint4 u[kAhead];
  auto read = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) u[i] = *reinterpret_cast<const uint4*>(bg + (int64_t)min(r0 + i, R - 1) * b_ld + n8);
  };
  const bool live = NC && n8 < N && g >= 0;
  if (live) read(0);
  pdl_wait();
  for (int r = threadIdx.x; r < R; r += kFewThreads) {
    float v = 0.f;
#pragma unroll
    for (int s = 0; s < kSplit; ++s) v += __ldcg(zp + ((int64_t)s * l.M + m) * R + r);
    zs[r] = v;
  }
  __syncthreads();
  if constexpr (NC) {
    if (n8 >= N) return;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    for (int r0 = 0; live && r0 < R; r0 += kAhead) {
      if (r0) read(r0);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (r0 + i >= R) break;
        float f[8];
        unpack8<T>(u[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = __fmaf_rn(zs[r0 + i], f[j], acc[j]);
      }
    }
    if (y_f32) {                                               // N is a multiple of 8
      float4* to = reinterpret_cast<float4*>(reinterpret_cast<float*>(y) + m * N + n8);
      to[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      to[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      return;
    }
    uint4 o;
    T* e = reinterpret_cast<T*>(&o);
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = from_f32<T>(acc[j]);
    if (yvec) {
      *reinterpret_cast<uint4*>(yr + n8) = o;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (n8 + j < N) yr[n8 + j] = e[j];
    }
  } else {
    for (int64_t n = (int64_t)blockIdx.x * kFewThreads * 8 + threadIdx.x;
         n < min(N, ((int64_t)blockIdx.x + 1) * kFewThreads * 8); n += kFewThreads) {
      float acc = 0.f;
      if (g >= 0) {
        const T* bn = bg + n * b_ld;
#pragma unroll 4
        for (int r0 = 0; r0 < R; r0 += 8) {                    // R is a multiple of 8
          float f[8];
          unpack8<T>(*reinterpret_cast<const uint4*>(bn + r0), f);
#pragma unroll
          for (int j = 0; j < 8; ++j) acc = __fmaf_rn(zs[r0 + j], f[j], acc);
        }
      }
      if (y_f32) reinterpret_cast<float*>(y)[m * N + n] = acc;
      else yr[n] = from_f32<T>(acc);
    }
  }
}

bool vec8(const void* p, int64_t gs, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && gs % 8 == 0 && ld % 8 == 0;
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
mm_status expand_typed(const LowRankArgs& l, const float* z, int64_t z_ld, const void* b, int64_t b_gs, int64_t b_rs, int64_t b_ns,
                       int64_t N, void* y, int y_f32, cudaStream_t stream) {
  const dim3 grid((unsigned)((N + 255) / 256), rows_y(l.M));
  return launch_pdl(expand_kernel<T>, grid, dim3(256), 0, stream, l, z, z_ld, static_cast<const T*>(b), b_gs, b_rs, b_ns, N,
                    static_cast<T*>(y), y_f32) == cudaSuccess ? MM_OK : MM_ERR_CUDA;
}

template <typename T>
mm_status outer_typed(const LowRankArgs& l, const void* x, int64_t x_rs, int64_t x_cs, int64_t C, const float* z,
                      void* out, int64_t o_gs, int64_t o_cs, int64_t o_rs, cudaStream_t stream) {
  const dim3 grid((unsigned)((C + 127) / 128), rows_y(l.G), (unsigned)((l.R + kOuterR - 1) / kOuterR));
  return launch_pdl(outer_kernel<T>, grid, dim3(128), 0, stream, l, static_cast<const T*>(x), x_rs, x_cs, C, z,
                    static_cast<T*>(out), o_gs, o_cs, o_rs) == cudaSuccess ? MM_OK : MM_ERR_CUDA;
}

template <typename T>
mm_status few_typed(const LowRankArgs& l, const LowRankFew& f, float* zp, cudaStream_t stream) {
  const T* x = static_cast<const T*>(f.x);
  const T* a = static_cast<const T*>(f.a);
  const T* b = static_cast<const T*>(f.b);
  const dim3 gs(kSplit, (unsigned)l.M);
  cudaError_t e;
  if (f.a_rs == 1)
    e = launch_pdl(shrink_rows_kernel<T, false>, gs, dim3(kFewThreads), 0, stream, l, x, f.x_rs, f.x_cs, f.C, a, f.a_gs,
                   f.a_cs, zp);
  else
    e = launch_pdl(shrink_rows_kernel<T, true>, gs, dim3(kFewThreads), 0, stream, l, x, f.x_rs, f.x_cs, f.C, a, f.a_gs,
                   f.a_rs, zp);
  if (e != cudaSuccess) return MM_ERR_CUDA;
  const dim3 ge((unsigned)((f.N + kFewThreads * 8 - 1) / (kFewThreads * 8)), (unsigned)l.M);
  T* y = static_cast<T*>(f.y);
  const int yvec = f.N % 8 == 0 && reinterpret_cast<uintptr_t>(y) % 16 == 0;
  if (f.b_ns == 1)
    e = launch_pdl(expand_rows_kernel<T, true>, ge, dim3(kFewThreads), 0, stream, l, (const float*)zp, b, f.b_gs, f.b_rs,
                   f.N, y, yvec, f.y_f32);
  else
    e = launch_pdl(expand_rows_kernel<T, false>, ge, dim3(kFewThreads), 0, stream, l, (const float*)zp, b, f.b_gs, f.b_ns,
                   f.N, y, yvec, f.y_f32);
  return e == cudaSuccess ? MM_OK : MM_ERR_CUDA;
}

}  // namespace

// 16-byte reads of a along whichever of its dimensions has unit stride, and of
// b likewise; whole octets of that dimension (c and n rows are read past their
// end by no one: C and N are multiples of 8).
bool lowrank_few_supported(const LowRankArgs& l, const LowRankFew& f) {
  if (l.dtype != MM_BF16 && l.dtype != MM_F16) return false;
  if (l.M < 1 || !lowrank_few_rows(l.M, l.G) || l.R < 1 || l.R > kExpandMaxR || l.G < 1 || f.C < 1 || f.N < 1) return false;
  const bool a_r = f.a_rs == 1 && l.R % 8 == 0 && vec8(f.a, f.a_gs, f.a_cs);
  const bool a_c = f.a_rs != 1 && f.a_cs == 1 && f.C % 8 == 0 && vec8(f.a, f.a_gs, f.a_rs);
  const bool b_n = f.b_ns == 1 && f.N % 8 == 0 && vec8(f.b, f.b_gs, f.b_rs);
  const bool b_r = f.b_ns != 1 && f.b_rs == 1 && l.R % 8 == 0 && vec8(f.b, f.b_gs, f.b_ns);
  return (a_r || a_c) && (b_n || b_r);
}

size_t lowrank_few_bytes(const LowRankArgs& l) { return (size_t)kSplit * (size_t)l.M * (size_t)l.R * sizeof(float); }

mm_status launch_lowrank_few(const LowRankArgs& l, const LowRankFew& f, float* zp, cudaStream_t stream) {
  return l.dtype == MM_F16 ? few_typed<__half>(l, f, zp, stream) : few_typed<__nv_bfloat16>(l, f, zp, stream);
}

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

mm_status launch_lowrank_expand(const LowRankArgs& l, const float* z, int64_t z_ld, const void* b, int64_t b_gs,
                                int64_t b_rs, int64_t b_ns, int64_t N, void* y, int y_f32, cudaStream_t stream) {
  if (l.M == 0 || N == 0) return MM_OK;
  QG_BY_TYPE(expand_typed, z, z_ld, b, b_gs, b_rs, b_ns, N, y, y_f32, stream)
}

mm_status launch_lowrank_outer(const LowRankArgs& l, const void* x, int64_t x_rs, int64_t x_cs, int64_t C,
                               const float* z, void* out, int64_t o_gs, int64_t o_cs, int64_t o_rs,
                               cudaStream_t stream) {
  if (l.G == 0 || C == 0 || l.R == 0) return MM_OK;
  QG_BY_TYPE(outer_typed, x, x_rs, x_cs, C, z, out, o_gs, o_cs, o_rs, stream)
}

#undef QG_BY_TYPE

}  // namespace qg
