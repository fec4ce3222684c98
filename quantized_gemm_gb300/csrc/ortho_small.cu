// The orthogonalised update of small matrices (mm_orthogonalize): all steps in one
// launch, one cluster of up to 8 CTAs per matrix, in fp32 on the CUDA cores.
//
// With the smaller side m along i and the longer along j, a CTA holds a slab of
// columns j of X in shared memory for the whole call.  A step is
//   P = sum over the slab of x_j x_j^T     (a 16 x 16 grid of threads, TI x TI sums each)
//   A = sum of the cluster's P             (each CTA adds a share of the rows, in rank
//                                           order, and writes it to every CTA)
//   B = b A + c A A                        (each CTA a share of the rows, written to all)
//   x_j <- a x_j + B x_j                   (in place, 16 TJ columns at a time)
// with a cluster barrier before each of the middle two and before the last.  Bound:
// the multiply-adds of one SM for the slab, and the three barriers a step; as 15
// launches of the chain of products a 61 x 1000 matrix took 250 us.
#include <cmath>
#include <cstring>

#include "ortho.cuh"
#include "tc_ptx.cuh"

namespace qg {

namespace {

constexpr int kThreads = 256, kSide = 16;        // a 16 x 16 grid of threads
constexpr int kMaxCluster = 8;
constexpr int kSmemMost = 226 * 1024;

struct SmallArgs {
  int m, n;                          // the smaller and the longer side
  int cols;                          // columns of a CTA's slab
  BatchMap bm;
  MatView x;
  int64_t x_is, x_js;                // strides of x along i and j
  int64_t o_is, o_js, o_step;        // of the dense output
  void* out;
  int tall;                          // neighbours in memory lie along i
  int steps;
  float eps, scale;
  float coef[3 * MM_ORTHO_MAX_STEPS];
};

template <int TI> constexpr int kPitch = kSide * TI + 4;      // floats: 16-byte rows, shifted banks

__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <int W>
__device__ __forceinline__ void load_row(const float* p, float (&v)[W]) {
  if constexpr (W == 2) {
    const float2 f = *reinterpret_cast<const float2*>(p);
    v[0] = f.x; v[1] = f.y;
  } else {
#pragma unroll
    for (int q = 0; q < W / 4; ++q) {
      const float4 f = *reinterpret_cast<const float4*>(p + 4 * q);
      v[4 * q] = f.x; v[4 * q + 1] = f.y; v[4 * q + 2] = f.z; v[4 * q + 3] = f.w;
    }
  }
}

template <typename T, int TI>
__global__ void __launch_bounds__(kThreads) ortho_small_kernel(const __grid_constant__ SmallArgs a, const int cluster) {
  pdl_begin();
  extern __shared__ __align__(16) float sm[];
  constexpr int P = kPitch<TI>, MP = kSide * TI, TJ = 4;
  float* S = sm;                                 // [MP][P] partial sums, then B
  float* A = sm + MP * P;                        // [MP][P]
  float* X = A + MP * P;                         // [cols, rounded up to 64][P]: X[j][i], zeros past m and n
  __shared__ double part[kThreads / 32 + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % (unsigned)cluster);
  const int64_t b = blockIdx.x / (unsigned)cluster;
  const int j0 = rank * a.cols, nc = max(0, min(a.cols, a.n - j0));
  const int ncp = (nc + 63) / 64 * 64;

  // The slab, and its sum of squares.
  const T* x = static_cast<const T*>(a.x.ptr) + batch_offset(a.bm, a.x.bstride, b);
  for (int e = tid; e < ncp * P; e += kThreads) X[e] = 0.f;
  __syncthreads();
  Squares sq;
  const int inner = a.tall ? a.m : nc, outer = a.tall ? nc : a.m;
  for (int o = warp; o < outer; o += kThreads / 32) {
#pragma unroll 4
    for (int q = lane; q < inner; q += 32) {
      const int i = a.tall ? q : o, j = a.tall ? o : q;
      const float v = to_f32(x[i * a.x_is + (j0 + j) * a.x_js]);
      sq.add(v);
      X[j * P + i] = v;
    }
  }
  double t = sq.total();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (lane == 0) part[warp] = t;
  __syncthreads();
  if (tid == 0) {
    t = 0.;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) t += part[w];
    part[kThreads / 32] = t;
  }
  __syncthreads();
  ptx::cluster_sync();
  t = 0.;
  for (int r = 0; r < cluster; ++r) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];"
                 : "=d"(v)
                 : "r"(ptx::mapa_shared(ptx::smem_u32(&part[kThreads / 32]), (uint32_t)r))
                 : "memory");
    t += v;
  }
  const Divisor d(sqrt(t) + (double)a.eps);
  for (int e = tid; e < nc * MP; e += kThreads) {
    const int j = e / MP, i = e % MP;
    if (i < a.m) X[j * P + i] = d.divide(X[j * P + i]);
  }
  __syncthreads();

  const int ti = tid / kSide * TI, tj = tid % kSide;
  // The rows of A and B that this CTA makes.
  const int share = (a.m + cluster - 1) / cluster, row0 = rank * share, rows = max(0, min(share, a.m - row0));
  for (int step = 0; step < a.steps; ++step) {
    const float ca = a.coef[3 * step], cb = a.coef[3 * step + 1], cc = a.coef[3 * step + 2];
    {
      float acc[TI][TI] = {};
      const float *u = X + ti, *w = X + tj * TI;
#pragma unroll 2
      for (int j = 0; j < nc; ++j, u += P, w += P) {
        float p[TI], q[TI];
        load_row<TI>(u, p);
        load_row<TI>(w, q);
#pragma unroll
        for (int r = 0; r < TI; ++r)
#pragma unroll
          for (int c = 0; c < TI; ++c) acc[r][c] = fmaf(p[r], q[c], acc[r][c]);
      }
#pragma unroll
      for (int r = 0; r < TI; ++r)
#pragma unroll
        for (int c = 0; c < TI; ++c) S[(ti + r) * P + tj * TI + c] = acc[r][c];
    }
    ptx::cluster_sync();
    for (int e = tid; e < rows * MP; e += kThreads) {
      const int at = (row0 + e / MP) * P + e % MP;
      const uint32_t s = ptx::smem_u32(S + at), to = ptx::smem_u32(A + at);
      float v = 0.f;
      for (int r = 0; r < cluster; ++r) v += ld_cluster(ptx::mapa_shared(s, (uint32_t)r));
      for (int r = 0; r < cluster; ++r) st_cluster(ptx::mapa_shared(to, (uint32_t)r), v);
    }
    ptx::cluster_sync();
    for (int e = tid; e < rows * MP; e += kThreads) {
      const int row = row0 + e / MP, c = e % MP;
      float v = 0.f;
#pragma unroll 8
      for (int k = 0; k < a.m; ++k) v = fmaf(A[row * P + k], A[k * P + c], v);
      v = fmaf(cc, v, cb * A[row * P + c]);
      const uint32_t to = ptx::smem_u32(S + row * P + c);
      for (int r = 0; r < cluster; ++r) st_cluster(ptx::mapa_shared(to, (uint32_t)r), v);
    }
    ptx::cluster_sync();
    // 64 columns at a time: this thread TI of i and TJ of j.
    for (int c0 = 0; c0 < nc; c0 += kSide * TJ) {
      float acc[TJ][TI] = {};
      const float* xj = X + (c0 + tj * TJ) * P;
      for (int k = 0; k < a.m; k += 4) {         // X is zero past m, and S finite there where A is
        float xv[TJ][4];
#pragma unroll
        for (int q = 0; q < TJ; ++q) load_row<4>(xj + q * P + k, xv[q]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float bv[TI];
          load_row<TI>(S + (k + e) * P + ti, bv);
#pragma unroll
          for (int q = 0; q < TJ; ++q)
#pragma unroll
            for (int r = 0; r < TI; ++r) acc[q][r] = fmaf(bv[r], xv[q][e], acc[q][r]);
        }
      }
      float old[TJ][TI];
#pragma unroll
      for (int q = 0; q < TJ; ++q) load_row<TI>(xj + q * P + ti, old[q]);
      __syncthreads();
#pragma unroll
      for (int q = 0; q < TJ; ++q)
#pragma unroll
        for (int r = 0; r < TI; ++r)
          X[(c0 + tj * TJ + q) * P + ti + r] = ti + r < a.m ? fmaf(ca, old[q][r], acc[q][r]) : 0.f;
    }
    __syncthreads();
  }

  T* out = static_cast<T*>(a.out) + b * a.o_step;
  for (int o = warp; o < outer; o += kThreads / 32) {
#pragma unroll 4
    for (int q = lane; q < inner; q += 32) {
      const int i = a.tall ? q : o, j = a.tall ? o : q;
      out[i * a.o_is + (j0 + j) * a.o_js] = from_f32<T>(a.scale * X[j * P + i]);
    }
  }
  ptx::cluster_sync();                           // no CTA leaves while its shared memory is read
}

int side_tile(int64_t m) { return m <= 32 ? 2 : m <= 64 ? 4 : 8; }
// Shared memory of a CTA with `cols` columns.
int64_t small_bytes(int64_t m, int64_t cols) {
  const int64_t mp = kSide * side_tile(m), p = mp + 4;
  return 4 * (2 * mp * p + (cols + 63) / 64 * 64 * p);
}
// CTAs per matrix: 8 while the clusters fit the SMs at once, fewer for larger
// stacks, but enough for the slabs to fit.  0: none.
int small_cluster(const OrthoArgs& o) {
  const int64_t m = o.M < o.N ? o.M : o.N, n = o.M < o.N ? o.N : o.M;
  if (m > kSide * 8) return 0;
  int c = kMaxCluster;
  while (c > 1 && (c * 16 > n || (o.bm.count * c > sm_count_public() && small_bytes(m, (n + c / 2 - 1) / (c / 2)) <= kSmemMost)))
    c /= 2;
  return small_bytes(m, (n + c - 1) / c) <= kSmemMost ? c : 0;
}

template <typename T, int TI>
cudaError_t run(const SmallArgs& a, int cluster, int64_t count, size_t smem, cudaStream_t stream) {
  const auto kernel = ortho_small_kernel<T, TI>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(count * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, cluster);
}

template <typename T>
cudaError_t by_side(const SmallArgs& a, int cluster, int64_t count, size_t smem, cudaStream_t stream) {
  switch (side_tile(a.m)) {
    case 2: return run<T, 2>(a, cluster, count, smem, stream);
    case 4: return run<T, 4>(a, cluster, count, smem, stream);
    default: return run<T, 8>(a, cluster, count, smem, stream);
  }
}

}  // namespace

bool ortho_small_pays(const OrthoArgs& o) {
  const int64_t m = o.M < o.N ? o.M : o.N, n = o.M < o.N ? o.N : o.M;
  return small_cluster(o) > 0 && o.bm.count < (1ll << 27) &&
         (double)m * (double)m * (double)n * (double)o.bm.count <= kOrthoSmallWork;
}

mm_status launch_ortho_small(const OrthoArgs& o, cudaStream_t stream) {
  SmallArgs a;
  memset(&a, 0, sizeof(a));
  const bool tall = o.M > o.N;
  a.m = (int)(tall ? o.N : o.M);
  a.n = (int)(tall ? o.M : o.N);
  const int cluster = small_cluster(o);
  a.cols = (a.n + cluster - 1) / cluster;
  a.bm = o.bm;
  a.x = o.x;
  a.x_is = tall ? o.x.cs : o.x.rs;
  a.x_js = tall ? o.x.rs : o.x.cs;
  a.o_is = tall ? 1 : o.N;
  a.o_js = tall ? o.N : 1;
  a.o_step = o.M * o.N;
  a.out = o.out;
  a.tall = tall;
  a.steps = o.steps;
  a.eps = o.eps;
  a.scale = o.scale;
  for (int i = 0; i < 3 * o.steps; ++i) a.coef[i] = o.coef[i];
  const size_t smem = (size_t)small_bytes(a.m, a.cols);
  const cudaError_t e = o.dtype == MM_F32    ? by_side<float>(a, cluster, o.bm.count, smem, stream)
                        : o.dtype == MM_BF16 ? by_side<__nv_bfloat16>(a, cluster, o.bm.count, smem, stream)
                                             : by_side<__half>(a, cluster, o.bm.count, smem, stream);
  return e == cudaSuccess ? MM_OK : MM_ERR_CUDA;
}

}  // namespace qg
