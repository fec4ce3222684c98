// The 8-bit product (mm_int8_matmul) for up to kInt8LooseRows rows of A whose
// operands are not 16-byte aligned along k: weights [N, K] at any address, and
// weights [K, N].  Both read B once, as it lies, and multiply by dp4a; A passes
// through shared memory in chunks, zeros past K, so that whatever else a word of B
// holds is multiplied by zero.
//
// Bound: memory, then dp4a.  us for 4095 x 14336 (59 MB) as [N, K] and as [K, N], here
// and by a copy of the weights and the streaming kernel:
//   1 row 13.6 35, 21.5 48    2 rows 15.6 35, 21.6 48    4 rows 21.6 35, 26.6 48    8 rows 41.6 35, 42 48
#include "int8.cuh"
#include "tc_ptx.cuh"

namespace qg {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunk = 1024, kWords = kChunk / 4;      // k, and words of a row of A, in shared memory

__device__ __forceinline__ void put(const Int8Args& a, int64_t m, int64_t n, float acc) {
  const float sa = __ldg(a.sa + m * a.sa_s), sb = __ldg(a.sb + n * a.sb_s);
  const int64_t at = m * a.N + n;
  if (a.out_dtype == MM_F32) static_cast<float*>(a.y)[at] = finish8<float>(acc, sa, sb, bias_at<float>(a, n));
  else if (a.out_dtype == MM_BF16)
    static_cast<__nv_bfloat16*>(a.y)[at] = finish8<__nv_bfloat16>(acc, sa, sb, bias_at<__nv_bfloat16>(a, n));
  else static_cast<__half*>(a.y)[at] = finish8<__half>(acc, sa, sb, bias_at<__half>(a, n));
}

// A[:, k0 .. k0 + kChunk) below `end`, as words of four k.
template <int M>
__device__ __forceinline__ void stage(const Int8Args& a, int64_t k0, int64_t end, int (&sA)[M][kWords]) {
  static_assert(kWords == kThreads, "a word of each row a thread");
  const int64_t k = k0 + 4 * threadIdx.x;
  const int8_t* p = a.a + k * a.a_cs;
  uint32_t v[M];
  if (a.a_cs == 1 && k + 4 <= end) {
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = m < a.M ? bytes4(p + m * a.a_rs) : 0u;
  } else {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      v[m] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (m < a.M && k + j < end) v[m] |= (uint32_t)(uint8_t)__ldg(p + m * a.a_rs + j * a.a_cs) << (8 * j);
    }
  }
#pragma unroll
  for (int m = 0; m < M; ++m) sA[m][threadIdx.x] = (int)v[m];
}

// ------------------------------------------------------------------ columns contiguous along k, at any address
//
// A warp owns two columns; a lane reads every 32nd aligned word and takes the bytes
// that its word of the column lacks from the next lane.
template <int M>
__global__ void __launch_bounds__(kThreads) int8_few_shifted_kernel(const Int8Args a) {
  pdl_begin();
  constexpr int kCols = kInt8FewCols, kSteps = kWords / 32;
  __shared__ int sA[M][kWords];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n0 = ((int64_t)blockIdx.x * kWarps + warp) * kCols;
  const uint32_t* b[kCols];
  uint32_t sh[kCols];
  int64_t words[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.b + (n0 + c < a.N ? n0 + c : a.N - 1) * a.b_ns);
    b[c] = reinterpret_cast<const uint32_t*>(at & ~(uintptr_t)3);
    sh[c] = ((uint32_t)at & 3u) * 8;
    words[c] = ((int64_t)(at & 3) + a.K + 3) / 4;
  }
  int acc[M][kCols] = {};
  for (int64_t k0 = 0; k0 < a.K; k0 += kChunk) {
    const int64_t first = k0 / 4 + lane;
    uint32_t w[kCols][kSteps + 1];               // (the last: the word after the chunk, in lane 0)
#pragma unroll
    for (int c = 0; c < kCols; ++c)
#pragma unroll
      for (int i = 0; i <= kSteps; ++i)
        w[c][i] = first + 32 * i < words[c] && (i < kSteps || lane == 0) ? __ldg(b[c] + first + 32 * i) : 0u;
    __syncthreads();                             // the chunk before has been read
    stage<M>(a, k0, a.K, sA);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      uint32_t y[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const uint32_t next = __shfl_sync(0xffffffffu, lane == 0 ? w[c][i + 1] : w[c][i], (lane + 1) & 31);
        y[c] = __funnelshift_r(w[c][i], next, sh[c]);
      }
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int x = sA[m][32 * i + lane];
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[m][c] = __dp4a(x, (int)y[c], acc[m][c]);
      }
    }
  }
  // Sums over the lanes; lane m * kCols + c keeps output (m, n0 + c).
  float mine = 0.f;
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      float v = (float)acc[m][c];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == m * kCols + c) mine = v;
    }
  const int64_t m = lane / kCols, n = n0 + lane % kCols;
  if (m < a.M && n < a.N) put(a, m, n, mine);
}

// ------------------------------------------------------------------ rows contiguous along n
//
// A lane owns four columns, a warp 128; the warps of a block, and the blocks of a
// cluster, share k in groups of four rows, whose 4 x 4 bytes a lane turns.  The
// sums, exact in int32 (K < 2^17), meet in shared memory, then over the cluster.
template <int M, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) int8_few_turned_kernel(const Int8Args a, const int64_t per, const int split) {
  pdl_begin();
  constexpr int kFlight = M == 1 ? 8 : 4;        // groups of a warp in flight
  __shared__ int sA[M][kWords];
  __shared__ __align__(16) int sums[kWarps][M][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = (int)blockIdx.y;
  const int64_t n = (int64_t)blockIdx.x * 128 + lane * 4, begin = rank * per, end = begin + per < a.K ? begin + per : a.K;
  const bool whole = n + 4 <= a.N;
  const auto load = [&](const int8_t* p) {
    uint32_t v = 0;
    if (whole) {
      v = VEC ? __ldg(reinterpret_cast<const uint32_t*>(p)) : bytes4(p);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < a.N) v |= (uint32_t)(uint8_t)__ldg(p + j) << (8 * j);
    }
    return v;
  };
  uint32_t w[kFlight][4];
  const auto fetch = [&](int64_t k0, int g0) {
    const int left = (int)(end - k0 < kChunk ? end - k0 : kChunk);
    const int8_t* p = a.b + k0 * a.b_ks + n;
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int k = 4 * (g0 + u * kWarps) + r;
        w[u][r] = k < left ? load(p + k * a.b_ks) : 0u;
      }
  };
  int acc[M][4] = {};
  if (begin < end) fetch(begin, warp);
  for (int64_t k0 = begin; k0 < end; k0 += kChunk) {
    __syncthreads();                             // the chunk before has been read
    stage<M>(a, k0, end, sA);
    __syncthreads();
    const int groups = (int)((end - k0 < kChunk ? end - k0 : kChunk) + 3) / 4;
    for (int g0 = warp; g0 < groups; g0 += kFlight * kWarps) {
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        if (g0 + u * kWarps >= groups) break;
        uint32_t y[4];
        turn4(w[u], y);
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const int x = sA[m][g0 + u * kWarps];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[m][j] = __dp4a(x, (int)y[j], acc[m][j]);
        }
      }
      if (g0 + kFlight * kWarps < groups) fetch(k0, g0 + kFlight * kWarps);
      else if (k0 + kChunk < end) fetch(k0 + kChunk, warp);
    }
  }
#pragma unroll
  for (int m = 0; m < M; ++m)
    *reinterpret_cast<int4*>(&sums[warp][m][lane * 4]) = make_int4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
  __syncthreads();
  for (int e = threadIdx.x; e < M * 128; e += kThreads) {
    int v = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += sums[i][e / 128][e % 128];
    sums[0][e / 128][e % 128] = v;               // (read and written by this thread alone)
  }
  ptx::cluster_sync();
  const int width = 128 / split;                 // columns that this block finishes
  for (int e = threadIdx.x; e < M * width; e += kThreads) {
    const int m = e / width, c = rank * width + e % width;
    const uint32_t at = ptx::smem_u32(&sums[0][m][c]);
    int v = 0;
    for (int r = 0; r < split; ++r) {
      int x;
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(ptx::mapa_shared(at, (uint32_t)r)) : "memory");
      v += x;
    }
    const int64_t col = (int64_t)blockIdx.x * 128 + c;
    if (m < a.M && col < a.N) put(a, m, col, (float)v);
  }
  ptx::cluster_sync();                           // no block leaves while its sums are read
}

template <int M>
cudaError_t run_shifted(const Int8Args& a, cudaStream_t stream) {
  const int64_t blocks = (a.N + kWarps * kInt8FewCols - 1) / (kWarps * kInt8FewCols);
  return launch_pdl(int8_few_shifted_kernel<M>, dim3((unsigned)blocks), dim3(kThreads), 0, stream, a);
}

// As many blocks a cluster as leave each 128 of k and are resident at once.
template <int M>
cudaError_t run_turned(const Int8Args& a, cudaStream_t stream) {
  const int64_t tiles = (a.N + 127) / 128;
  int split = 8;
  while (split > 1 && (a.K < 128 * split || tiles * split > 4 * (int64_t)sm_count_public())) split /= 2;
  const int64_t per = ((a.K + split - 1) / split + 3) / 4 * 4;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = (unsigned)split;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)tiles, (unsigned)split);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const bool vec = a.b_ks % 4 == 0 && (reinterpret_cast<uintptr_t>(a.b) & 3) == 0;
  return vec ? cudaLaunchKernelEx(&cfg, int8_few_turned_kernel<M, true>, a, per, split)
             : cudaLaunchKernelEx(&cfg, int8_few_turned_kernel<M, false>, a, per, split);
}

// Rows of A in the next power of two, zeros past M.
template <int M>
cudaError_t run(const Int8Args& a, cudaStream_t stream) {
  return a.b_ks == 1 ? run_shifted<M>(a, stream) : run_turned<M>(a, stream);
}

}  // namespace

bool int8_few_supported(const Int8Args& a) {
  return int8_few_aligned(a) || (a.M <= kInt8LooseRows && a.K >= 1 &&
                                 ((a.b_ks == 1 && a.K <= kInt8FewDepth) || (a.b_ns == 1 && a.K < (1 << 17))));
}

mm_status launch_int8_few(const Int8Args& a, cudaStream_t stream) {
  if (int8_few_aligned(a)) return launch_int8_few_aligned(a, stream);
  const cudaError_t e = a.M <= 1 ? run<1>(a, stream) : a.M <= 2 ? run<2>(a, stream) : run<4>(a, stream);
  return e == cudaSuccess ? MM_OK : MM_ERR_CUDA;
}

}  // namespace qg
