// The orthogonalised update of small matrices (mm_orthogonalize): all steps in one
// launch, one cluster of up to 8 CTAs per matrix, in fp32 on the CUDA cores.
//
// With the smaller side m along i and the longer along j, a CTA holds a slab of
// columns j of X in shared memory for the whole call.  A step is
//   P = sum over the slab of x_j x_j^T     (the lower half in E x E blocks, a thread each,
//                                           over slices of the slab that are added in order)
//   A = sum of the cluster's P             (each CTA adds a share of the rows, in rank
//                                           order, and writes it to every CTA)
//   B = b A + c A A                        (each CTA a share of the rows, written to all)
//   x_j <- a x_j + B x_j                   (in place, 64 columns at a time)
// with a cluster barrier before each of the middle two and before the last.  Bound:
// the multiply-adds and shared-memory reads of one SM for the slab (4 x 4 blocks
// of a full P read twice as much per multiply-add: 69 us for 61 x 1000), and the
// barriers.  61 x 1000 takes 62 us, as 17 launches of the chain of products 177.
#include <cmath>
#include <cstring>

#include "ortho.cuh"
#include "tc_ptx.cuh"

namespace qg {

namespace {

// Sizes by the side MP that m is padded to (32, 64, 128).
template <int MP>
struct Side {
  static constexpr int kThreads = MP <= 64 ? 256 : 512;
  static constexpr int kPitch = MP + 4;                          // floats: 16-byte rows, shifted banks
  static constexpr int E = MP <= 32 ? 4 : 8;                     // P: blocks of E x E, its lower half
  static constexpr int kBlocks = (MP / E) * (MP / E + 1) / 2;
  static constexpr int kSlices = kThreads / kBlocks;             // 7, 7, 3
  static constexpr int TI = MP <= 32 ? 4 : 8;                    // x_j: a thread's rows
  static constexpr int kTeam = MP / TI * 16;                     // threads of 64 columns
  // S and A, which take turns with the slices' sums of P (floats).
  static constexpr int kSums = kSlices * kBlocks * E * E, kMats = 2 * MP * kPitch;
  static constexpr int kHead = kSums > kMats ? kSums : kMats;
};
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

__device__ __forceinline__ void st_cluster(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

template <int W>
__device__ __forceinline__ void load_row(const float* p, float (&v)[W]) {
#pragma unroll
  for (int q = 0; q < W / 4; ++q) {
    const float4 f = *reinterpret_cast<const float4*>(p + 4 * q);
    v[4 * q] = f.x; v[4 * q + 1] = f.y; v[4 * q + 2] = f.z; v[4 * q + 3] = f.w;
  }
}
template <int W>
__device__ __forceinline__ void store_row(float* p, const float (&v)[W]) {
#pragma unroll
  for (int q = 0; q < W / 4; ++q)
    *reinterpret_cast<float4*>(p + 4 * q) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
}

// x_j <- a x_j + B x_j of TJ columns 16 apart, rows ti.. of them a thread.
template <typename Z, int TJ>
__device__ __forceinline__ void update(const float* S, float* xj, int ti, int m, float ca, int team) {
  constexpr int P = Z::kPitch, TI = Z::TI;
  float acc[TJ][TI] = {};
#pragma unroll 2
  for (int k = 0; k < m; k += 4) {               // X and S are zero past m
    float xv[TJ][4];
#pragma unroll
    for (int q = 0; q < TJ; ++q) load_row<4>(xj + q * 16 * P + k, xv[q]);
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
#pragma unroll
  for (int q = 0; q < TJ; ++q) {
    float old[TI];
    load_row<TI>(xj + q * 16 * P + ti, old);
#pragma unroll
    for (int r = 0; r < TI; ++r) acc[q][r] = ti + r < m ? fmaf(ca, old[r], acc[q][r]) : 0.f;
  }
  asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(Z::kTeam) : "memory");   // the team's columns have been read
#pragma unroll
  for (int q = 0; q < TJ; ++q) store_row<TI>(xj + q * 16 * P + ti, acc[q]);
}

template <typename T, int MP>
__global__ void __launch_bounds__(Side<MP>::kThreads, 1) ortho_small_kernel(const __grid_constant__ SmallArgs a,
                                                                         const int cluster) {
  pdl_begin();
  using Z = Side<MP>;
  extern __shared__ __align__(16) float sm[];
  constexpr int P = Z::kPitch, kThreads = Z::kThreads, E = Z::E, TI = Z::TI;
  float* S = sm;                                 // [MP][P] partial sums, then B
  float* A = sm + MP * P;                        // [MP][P]
  float* X = sm + Z::kHead;                      // [cols, rounded up to 64][P]: X[j][i], zeros past m and n
  __shared__ double part[kThreads / 32 + 1];
  __shared__ Divisor whole;
  __shared__ uint16_t blocks[Z::kBlocks];        // a block's first row and column of P
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % (unsigned)cluster);
  const int64_t b = blockIdx.x / (unsigned)cluster;
  const int j0 = rank * a.cols, nc = max(0, min(a.cols, a.n - j0));
  const int ncp = (nc + 63) / 64 * 64;

  // The slab, and its sum of squares.  Neighbouring threads take neighbours in
  // memory, 16 values of a thread in flight.
  const T* x = static_cast<const T*>(a.x.ptr) + batch_offset(a.bm, a.x.bstride, b);
  for (int e = tid * 4; e < ncp * P; e += kThreads * 4) *reinterpret_cast<float4*>(X + e) = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  Squares sq;
  const int inner = a.tall ? a.m : nc, total = a.m * nc;
  const auto place = [&](int e, int& i, int& j) {
    const int o = e / inner, q = e - o * inner;
    i = a.tall ? q : o;
    j = a.tall ? o : q;
  };
  constexpr int kFlight = 16;
  for (int e0 = tid; e0 < total; e0 += kFlight * kThreads) {
    float v[kFlight];
    int at[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int e = e0 + u * kThreads;
      at[u] = -1;
      v[u] = 0.f;
      if (e < total) {
        int i, j;
        place(e, i, j);
        at[u] = j * P + i;
        v[u] = to_f32(x[i * a.x_is + (j0 + j) * a.x_js]);
      }
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
      if (at[u] >= 0) {
        sq.add(v[u]);
        X[at[u]] = v[u];
      }
  }
  sq.join_warp();
  if (lane == 0) part[warp] = sq.total();
  __syncthreads();
  if (tid == 0) {
    double t = 0.;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) t += part[w];
    part[kThreads / 32] = t;
  }
  ptx::cluster_sync();
  if (tid == 0) {
    double t = 0.;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      double v = 0.;
      if (r < cluster)
        asm volatile("ld.shared::cluster.f64 %0, [%1];"
                     : "=d"(v)
                     : "r"(ptx::mapa_shared(ptx::smem_u32(&part[kThreads / 32]), (uint32_t)r))
                     : "memory");
      t += v;
    }
    whole = Divisor(sqrt(t) + (double)a.eps);
  }
  __syncthreads();
  const Divisor d = whole;
  for (int e = tid; e < nc * (MP / 4); e += kThreads) {
    const int j = e / (MP / 4), i = e % (MP / 4) * 4;
    if (i >= a.m) continue;
    float v[4];
    load_row<4>(X + j * P + i, v);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = i + q < a.m ? d.divide(v[q]) : 0.f;
    store_row<4>(X + j * P + i, v);
  }
  __syncthreads();

  // This thread's block of P, and its slice of the slab.
  const int slice = tid / Z::kBlocks;
  int bi = 0, bj = tid % Z::kBlocks;
  while (bj > bi) bj -= ++bi;
  if (slice == 0) blocks[tid] = (uint16_t)(bi * E * 256 + bj * E);   // (read after barriers)
  const int jb = slice < Z::kSlices ? slice * nc / Z::kSlices : 0, je = slice < Z::kSlices ? (slice + 1) * nc / Z::kSlices : 0;
  // Its block of x_j: TI of i and every 16th j (neighbouring rows of X shift the banks by 4).
  const int team = tid / Z::kTeam, ti = tid % Z::kTeam / 16 * TI, tj = tid % 16;
  // The rows of A and B that this CTA makes; A's rows up to the next multiple of 4
  // are read too (times zeros) and are made by the last CTA.
  const int m4 = (a.m + 3) / 4 * 4, share = (m4 / 2 + cluster - 1) / cluster * 2, row0 = rank * share,
            rows = max(0, min(share, m4 - row0));
  for (int step = 0; step < a.steps; ++step) {
    const float ca = a.coef[3 * step], cb = a.coef[3 * step + 1], cc = a.coef[3 * step + 2];
    {
      float acc[E][E] = {};
#pragma unroll 2
      for (int j = jb; j < je; ++j) {
        float p[E], q[E];
        load_row<E>(X + j * P + bi * E, p);
        load_row<E>(X + j * P + bj * E, q);
#pragma unroll
        for (int r = 0; r < E; ++r)
#pragma unroll
          for (int c = 0; c < E; ++c) acc[r][c] = fmaf(p[r], q[c], acc[r][c]);
      }
      // The slices' sums, an element of all blocks side by side, in the place of S and
      // A; then their sum in order, for both halves of P.
      if (slice < Z::kSlices) {
#pragma unroll
        for (int e = 0; e < E * E; ++e) sm[(slice * E * E + e) * Z::kBlocks + tid - slice * Z::kBlocks] = acc[e / E][e % E];
      }
      __syncthreads();
      constexpr int kAll = E * E * Z::kBlocks, kMine = (kAll + kThreads - 1) / kThreads;
      float v[kMine];
#pragma unroll
      for (int u = 0; u < kMine; ++u) {
        const int e = tid + u * kThreads;
        v[u] = 0.f;
        if (e < kAll) {
#pragma unroll
          for (int r = 0; r < Z::kSlices; ++r) v[u] += sm[r * kAll + e];
        }
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kMine; ++u) {
        const int e = tid + u * kThreads;
        if (e < kAll) {
          const int at = blocks[e % Z::kBlocks], y = at / 256 + e / Z::kBlocks / E, z = at % 256 + e / Z::kBlocks % E;
          S[y * P + z] = v[u];
          S[z * P + y] = v[u];
        }
      }
    }
    ptx::cluster_sync();
    for (int e = tid; e < rows * (MP / 4); e += kThreads) {
      const int at = (row0 + e / (MP / 4)) * P + e % (MP / 4) * 4;
      const uint32_t from = ptx::smem_u32(S + at), to = ptx::smem_u32(A + at);
      float4 u[kMaxCluster], v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) u[r] = r < cluster ? ptx::lds128_cluster(ptx::mapa_shared(from, (uint32_t)r)) : v;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) v = make_float4(v.x + u[r].x, v.y + u[r].y, v.z + u[r].z, v.w + u[r].w);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < cluster) st_cluster(ptx::mapa_shared(to, (uint32_t)r), v);
    }
    ptx::cluster_sync();
    for (int e = tid; e < (rows + 1) / 2 * (MP / 4); e += kThreads) {     // two rows, four columns
      const int row = row0 + e / (MP / 4) * 2, c = e % (MP / 4) * 4;
      float v[2][4] = {}, w[2][4] = {};
#pragma unroll 2
      for (int k = 0; k < a.m; k += 4) {         // A is zero past m
        float f[2][4], q[4][4];
#pragma unroll
        for (int y = 0; y < 2; ++y) load_row<4>(A + (row + y) * P + k, f[y]);
#pragma unroll
        for (int u = 0; u < 4; ++u) load_row<4>(A + (k + u) * P + c, q[u]);
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[y][j] = fmaf(f[y][1], q[1][j], fmaf(f[y][0], q[0][j], v[y][j]));
            w[y][j] = fmaf(f[y][3], q[3][j], fmaf(f[y][2], q[2][j], w[y][j]));
          }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float o[4];
        load_row<4>(A + (row + y) * P + c, o);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = fmaf(cc, v[y][j] + w[y][j], cb * o[j]);
        const uint32_t to = ptx::smem_u32(S + (row + y) * P + c);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < cluster) st_cluster(ptx::mapa_shared(to, (uint32_t)r), make_float4(o[0], o[1], o[2], o[3]));
      }
    }
    ptx::cluster_sync();
    for (int c0 = team * 64; c0 < nc; c0 += kThreads / Z::kTeam * 64) {
      float* xj = X + (c0 + tj) * P;
      if (nc - c0 <= 16) update<Z, 1>(S, xj, ti, a.m, ca, team);
      else if (nc - c0 <= 32) update<Z, 2>(S, xj, ti, a.m, ca, team);
      else update<Z, 4>(S, xj, ti, a.m, ca, team);
    }
    __syncthreads();
  }

  T* out = static_cast<T*>(a.out) + b * a.o_step;
#pragma unroll 4
  for (int e = tid; e < total; e += kThreads) {
    int i, j;
    place(e, i, j);
    out[i * a.o_is + (j0 + j) * a.o_js] = from_f32<T>(a.scale * X[j * P + i]);
  }
  ptx::cluster_sync();                           // no CTA leaves while its shared memory is read
}

int padded_side(int64_t m) { return m <= 32 ? 32 : m <= 64 ? 64 : 128; }
// Shared memory of a CTA with `cols` columns.
int64_t small_bytes(int64_t m, int64_t cols) {
  const int64_t mp = padded_side(m), p = mp + 4;
  const int64_t head = mp == 32 ? Side<32>::kHead : mp == 64 ? Side<64>::kHead : Side<128>::kHead;
  return 4 * (head + (cols + 63) / 64 * 64 * p);
}
// CTAs per matrix: 8 while the clusters fit the SMs at once, fewer for larger
// stacks, but enough for the slabs to fit.  0: none.
int small_cluster(const OrthoArgs& o) {
  const int64_t m = o.M < o.N ? o.M : o.N, n = o.M < o.N ? o.N : o.M;
  if (m > 128) return 0;
  int c = kMaxCluster;
  while (c > 1 && (c * 32 > n || (o.bm.count * c > sm_count_public() && small_bytes(m, (n + c / 2 - 1) / (c / 2)) <= kSmemMost)))
    c /= 2;
  return small_bytes(m, (n + c - 1) / c) <= kSmemMost ? c : 0;
}

template <typename T, int MP>
cudaError_t run(const SmallArgs& a, int cluster, int64_t count, size_t smem, cudaStream_t stream) {
  const auto kernel = ortho_small_kernel<T, MP>;
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
  cfg.blockDim = dim3(Side<MP>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, cluster);
}

template <typename T>
cudaError_t by_side(const SmallArgs& a, int cluster, int64_t count, size_t smem, cudaStream_t stream) {
  switch (padded_side(a.m)) {
    case 32: return run<T, 32>(a, cluster, count, smem, stream);
    case 64: return run<T, 64>(a, cluster, count, smem, stream);
    default: return run<T, 128>(a, cluster, count, smem, stream);
  }
}

}  // namespace

bool ortho_small_pays(const OrthoArgs& o) {
  const int64_t m = o.M < o.N ? o.M : o.N, n = o.M < o.N ? o.N : o.M;
  return small_cluster(o) > 0 && o.bm.count < (1ll << 27) &&
         (m <= 64 || (double)m * (double)m * (double)n * (double)o.bm.count <= kOrthoSmallWork);
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
