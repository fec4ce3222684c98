// Rows to int8 with a scale each (mm_quantize_rows), and the CUDA-core parts of
// the 8-bit product (mm_int8_matmul): the form for a few aligned rows (others are
// in int8_few.cu), the form for every stride, and the copies that the tensor-core
// products multiply.
#include "int8.cuh"
#include "tc_ptx.cuh"

namespace qg {

namespace {

// ------------------------------------------------------------------ quantisation of rows
//
// s = amax / 127 and q = rint(x / s), each one rounded fp32 operation (ties to
// even).  Bound: memory (a row is read once, held in registers between its
// maximum and its quotients).  16384 rows of 4096 bf16 (201 MB): 35.5 us, 5.7 TB/s.

// |x| as unsigned bits, whose order is the values'; NaN is above infinity.
template <typename T> struct AbsBits;
template <> struct AbsBits<float> {
  static constexpr uint32_t kInf = 0x7F800000u;
  static __device__ __forceinline__ uint32_t max(uint32_t m, uint32_t w) { return ::max(m, w & 0x7FFFFFFFu); }
  static __device__ __forceinline__ uint32_t join(uint32_t m) { return m; }
  static __device__ __forceinline__ float value(uint32_t m) { return __uint_as_float(m); }
};
template <> struct AbsBits<__nv_bfloat16> {     // two values per word
  static constexpr uint32_t kInf = 0x7F80u;
  static __device__ __forceinline__ uint32_t max(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }
  static __device__ __forceinline__ uint32_t join(uint32_t m) { return ::max(m & 0xFFFFu, m >> 16); }
  static __device__ __forceinline__ float value(uint32_t m) { return __uint_as_float(m << 16); }
};
template <> struct AbsBits<__half> {
  static constexpr uint32_t kInf = 0x7C00u;
  static __device__ __forceinline__ uint32_t max(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }
  static __device__ __forceinline__ uint32_t join(uint32_t m) { return ::max(m & 0xFFFFu, m >> 16); }
  static __device__ __forceinline__ float value(uint32_t m) { return __half2float(__ushort_as_half((uint16_t)m)); }
};
template <typename T>
__device__ __forceinline__ uint32_t one_abs(T x);
template <> __device__ __forceinline__ uint32_t one_abs(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
template <> __device__ __forceinline__ uint32_t one_abs(__nv_bfloat16 x) { return __bfloat16_as_ushort(x) & 0x7FFFu; }
template <> __device__ __forceinline__ uint32_t one_abs(__half x) { return __half_as_ushort(x) & 0x7FFFu; }

// A row's scale from its largest |x|: NaN for a row that holds an infinity or NaN.
struct RowScale {
  float s, r;        // the scale and its rounded reciprocal
  bool fast;         // a normal scale whose reciprocal is normal
  bool zero;         // every q is 0: a row of zeros, a scale that underflows to 0, or a NaN scale
};
template <typename T>
__device__ __forceinline__ RowScale row_scale(uint32_t amax) {
  RowScale o;
  o.s = amax >= AbsBits<T>::kInf ? __uint_as_float(0x7FFFFFFFu) : __fdiv_rn(AbsBits<T>::value(amax), 127.f);
  o.r = __frcp_rn(o.s);
  o.fast = o.s >= 1.17549435e-38f && o.s < 8.50705917e+37f;      // [2^-126, 2^126)
  o.zero = !(o.s > 0.f);
  return o;
}
__device__ __forceinline__ int32_t quotient(float x, const RowScale& k) {
  if (k.zero) return 0;
  return (int32_t)fminf(fmaxf(rintf(__fdiv_rn(x, k.s)), -127.f), 127.f);
}

// Four quotients as the bytes of a word.  x * RN(1/s) differs from the rounded
// quotient by less than 2^-21 |q| <= 2^-14, so where it lies more than that from
// a half-integer both round to the same integer; `off` collects the distance
// from the nearest integer, and the caller divides where it comes near 1/2.
// Adding 1.5 * 2^23 rounds to an integer, ties to even, and leaves it in the low
// byte.  (|q| <= 127 needs no clamp: x * r <= 127 (1 + 2^-22).)
__device__ __forceinline__ uint32_t quotients4(float x0, float x1, float x2, float x3, float r, float& off) {
  constexpr float kMagic = 12582912.0f;
  const float q0 = __fmul_rn(x0, r), q1 = __fmul_rn(x1, r), q2 = __fmul_rn(x2, r), q3 = __fmul_rn(x3, r);
  const float t0 = __fadd_rn(q0, kMagic), t1 = __fadd_rn(q1, kMagic), t2 = __fadd_rn(q2, kMagic),
              t3 = __fadd_rn(q3, kMagic);
  off = fmaxf(off, fmaxf(fmaxf(fabsf(q0 - __fsub_rn(t0, kMagic)), fabsf(q1 - __fsub_rn(t1, kMagic))),
                         fmaxf(fabsf(q2 - __fsub_rn(t2, kMagic)), fabsf(q3 - __fsub_rn(t3, kMagic)))));
  const uint32_t lo = __byte_perm(__float_as_uint(t0), __float_as_uint(t1), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(t2), __float_as_uint(t3), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

template <typename T> constexpr int kElems = 16 / (int)sizeof(T);     // values per 16-byte piece

template <typename T>
__device__ __forceinline__ void piece_floats(const uint4& u, float (&x)[kElems<T>]) {
  const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
  for (int j = 0; j < kElems<T>; ++j) x[j] = to_f32(e[j]);
}

template <typename T>
__device__ __forceinline__ void store_quotients(const uint4& u, const RowScale& k, int8_t* dst) {
  constexpr int E = kElems<T>;
  float x[E];
  piece_floats<T>(u, x);
  uint32_t w[E / 4];
  float off = 0.f;
#pragma unroll
  for (int j = 0; j < E / 4; ++j) w[j] = quotients4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3], k.r, off);
  if (!k.fast || !(off < 0.5f - 6.1035156e-05f)) {      // 2^-14
#pragma unroll
    for (int j = 0; j < E / 4; ++j) {
      w[j] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[j] |= ((uint32_t)quotient(x[4 * j + e], k) & 0xFFu) << (8 * e);
    }
  }
  if constexpr (E == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(dst) = w[0];
}

// TPR threads own a row of up to TPR * NV pieces of 16 bytes, held in registers;
// longer rows (LONG) are read twice, the second time mostly from the L2.
constexpr int kQuantThreads = 128;
template <typename T, int TPR, int NV, bool LONG>
__global__ void __launch_bounds__(TPR < kQuantThreads ? kQuantThreads : TPR)
    quantize_rows_kernel(const QuantizeArgs a) {
  pdl_begin();
  constexpr int kThreads = TPR < kQuantThreads ? kQuantThreads : TPR, kRowsPer = kThreads / TPR;
  __shared__ uint32_t part[kThreads / 32];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * kRowsPer + threadIdx.x / TPR;
  const bool live = row < a.M;
  const int64_t np = a.K / kElems<T>;                    // pieces
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + (live ? row : 0) * a.x_rs);
  uint4 u[NV];
  uint32_t m = 0;
  for (int64_t base = 0; base < np; base += TPR * NV) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t p = base + v * TPR + t;
      u[v] = live && p < np ? __ldg(src + p) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
      m = AbsBits<T>::max(AbsBits<T>::max(AbsBits<T>::max(AbsBits<T>::max(m, u[v].x), u[v].y), u[v].z), u[v].w);
    if (!LONG) break;
  }
  m = __reduce_max_sync(0xffffffffu, AbsBits<T>::join(m));
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) m = max(m, part[threadIdx.x / TPR * (TPR / 32) + w]);
  }
  if (!live) return;
  const RowScale k = row_scale<T>(m);
  if (t == 0) a.scales[row] = k.s;
  int8_t* dst = a.q + row * a.K;
  for (int64_t base = 0; base < np; base += TPR * NV) {
    if (LONG) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int64_t p = base + v * TPR + t;
        if (p < np) u[v] = __ldg(src + p);
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t p = base + v * TPR + t;
      if (p < np) store_quotients<T>(u[v], k, dst + p * kElems<T>);
    }
    if (!LONG) break;
  }
}

// Any strides and lengths: a block per row, element by element.
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_any_kernel(const QuantizeArgs a) {
  pdl_begin();
  __shared__ uint32_t part[8];
  const T* src = static_cast<const T*>(a.x) + (int64_t)blockIdx.x * a.x_rs;
  uint32_t m = 0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < a.K; i += 256) m = max(m, one_abs<T>(src[i * a.x_cs]));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max(m, part[w]);
  const RowScale k = row_scale<T>(m);
  if (threadIdx.x == 0) a.scales[blockIdx.x] = k.s;
  int8_t* dst = a.q + (int64_t)blockIdx.x * a.K;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < a.K; i += 256) dst[i] = (int8_t)quotient(to_f32(src[i * a.x_cs]), k);
}

// Rows that lie closer together than a row's elements (the columns of a row-major
// matrix, weights [K, N] seen as [N, K]): a block takes 32 rows, lane = row for
// the reads, and turns 32 x 64 tiles in shared memory for the writes.
constexpr int kTurn = 64;
template <typename T>
__global__ void __launch_bounds__(256) quantize_columns_kernel(const QuantizeArgs a) {
  pdl_begin();
  __shared__ uint32_t part[8][32];
  __shared__ int8_t tile[32][kTurn + 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * 32 + lane;
  const bool live = row < a.M;
  const T* src = static_cast<const T*>(a.x) + (live ? row : 0) * a.x_rs;
  uint32_t m = 0;
#pragma unroll 8
  for (int64_t i = warp; i < a.K; i += 8) m = max(m, one_abs<T>(src[i * a.x_cs]));
  part[warp][lane] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max(m, part[w][lane]);
  const RowScale k = row_scale<T>(m);
  if (warp == 0 && live) a.scales[row] = k.s;
  const int64_t first = (int64_t)blockIdx.x * 32;
  for (int64_t k0 = 0; k0 < a.K; k0 += kTurn) {
    float x[kTurn / 8];
#pragma unroll
    for (int j = 0; j < kTurn / 8; ++j) {
      const int64_t i = k0 + warp + 8 * j;
      x[j] = i < a.K ? to_f32(src[i * a.x_cs]) : 0.f;
    }
    __syncthreads();       // the tile before has been written out
#pragma unroll
    for (int j = 0; j < kTurn / 8; ++j) tile[lane][warp + 8 * j] = (int8_t)quotient(x[j], k);
    __syncthreads();
    for (int e = threadIdx.x; e < 32 * kTurn; e += 256) {
      const int r = e / kTurn, c = e % kTurn;
      if (first + r < a.M && k0 + c < a.K) a.q[(first + r) * a.K + k0 + c] = tile[r][c];
    }
  }
}

template <typename T>
mm_status run_quantize(const QuantizeArgs& a, cudaStream_t stream) {
  const bool vec = a.x_cs == 1 && a.K % kElems<T> == 0 && (a.x_rs * sizeof(T)) % 16 == 0 &&
                   (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && (reinterpret_cast<uintptr_t>(a.q) & 7) == 0;
  cudaError_t e;
  if (vec) {
    // Four pieces a thread; as many threads as the row then needs.
    const int64_t np = a.K / kElems<T>;
    const auto rows = [&](int per) { return dim3((unsigned)((a.M + per - 1) / per)); };
    if (np <= 32 * 4) e = launch_pdl(quantize_rows_kernel<T, 32, 4, false>, rows(4), dim3(128), 0, stream, a);
    else if (np <= 128 * 4) e = launch_pdl(quantize_rows_kernel<T, 128, 4, false>, rows(1), dim3(128), 0, stream, a);
    else if (np <= 512 * 4) e = launch_pdl(quantize_rows_kernel<T, 512, 4, false>, rows(1), dim3(512), 0, stream, a);
    else e = launch_pdl(quantize_rows_kernel<T, 512, 4, true>, rows(1), dim3(512), 0, stream, a);
  } else if (a.x_rs < a.x_cs && a.M > 1) {
    e = launch_pdl(quantize_columns_kernel<T>, dim3((unsigned)((a.M + 31) / 32)), dim3(256), 0, stream, a);
  } else {
    e = launch_pdl(quantize_rows_any_kernel<T>, dim3((unsigned)a.M), dim3(256), 0, stream, a);
  }
  return e == cudaSuccess ? MM_OK : MM_ERR_CUDA;
}

// ------------------------------------------------------------------ a few rows
//
// Up to kInt8FewRows rows of A against B whose columns are contiguous along k: B
// streams once.  A warp owns kCols columns; its lanes split k in 16-byte pieces,
// hold kDeep pieces of each column in flight and multiply them with the rows of A
// (from the L1) by dp4a, exactly: a lane adds fewer than 2^17 products of at most
// 2^14, and the lanes' sums are added as floats.  Bound: memory; one row
// by 4096 x 14336 (59 MB): 10.7 us, 5.5 TB/s.

template <typename O, int M>
__global__ void __launch_bounds__(256) int8_few_kernel(const Int8Args a) {
  constexpr int kCols = kInt8FewCols, kDeep = 8;
  const int lane = threadIdx.x & 31;
  const int64_t n0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kCols;
  pdl_begin();
  if (n0 >= a.N) return;
  const uint4* b[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c)
    b[c] = reinterpret_cast<const uint4*>(a.b + (n0 + c < a.N ? n0 + c : n0) * a.b_ns);
  const int pieces = (int)(a.K >> 4);
  int acc[M][kCols] = {};
  const auto load = [&](int p, uint4 (&w)[kCols]) {
#pragma unroll
    for (int c = 0; c < kCols; ++c)
      asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[c].x), "=r"(w[c].y), "=r"(w[c].z), "=r"(w[c].w)
                   : "l"(b[c] + p));
  };
  const auto multiply = [&](int p, const uint4 (&w)[kCols]) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(a.a + m * a.a_rs) + p);
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        int s = acc[m][c];
        s = __dp4a((int)x.x, (int)w[c].x, s);
        s = __dp4a((int)x.y, (int)w[c].y, s);
        s = __dp4a((int)x.z, (int)w[c].z, s);
        acc[m][c] = __dp4a((int)x.w, (int)w[c].w, s);
      }
    }
  };
  int p0 = lane;
  for (; p0 - lane + 32 * kDeep <= pieces; p0 += 32 * kDeep) {
    uint4 w[kDeep][kCols];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) load(p0 + 32 * d, w[d]);
#pragma unroll
    for (int d = 0; d < kDeep; ++d) multiply(p0 + 32 * d, w[d]);
  }
#pragma unroll 4
  for (; p0 < pieces; p0 += 32) {
    uint4 w[kCols];
    load(p0, w);
    multiply(p0, w);
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
  const int m = lane / kCols;
  const int64_t n = n0 + lane % kCols;
  if (m < M && n < a.N)
    static_cast<O*>(a.y)[m * a.N + n] =
        finish8<O>(mine, __ldg(a.sa + m * a.sa_s), __ldg(a.sb + n * a.sb_s), bias_at<O>(a, n));
}

template <typename O>
mm_status run_few(const Int8Args& a, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.N + 8 * kInt8FewCols - 1) / (8 * kInt8FewCols)));
  cudaError_t e = cudaErrorInvalidValue;
  switch (a.M) {
    case 1: e = launch_pdl(int8_few_kernel<O, 1>, grid, dim3(256), 0, stream, a); break;
    case 2: e = launch_pdl(int8_few_kernel<O, 2>, grid, dim3(256), 0, stream, a); break;
    case 3: e = launch_pdl(int8_few_kernel<O, 3>, grid, dim3(256), 0, stream, a); break;
    case 4: e = launch_pdl(int8_few_kernel<O, 4>, grid, dim3(256), 0, stream, a); break;
    case 5: e = launch_pdl(int8_few_kernel<O, 5>, grid, dim3(256), 0, stream, a); break;
    case 6: e = launch_pdl(int8_few_kernel<O, 6>, grid, dim3(256), 0, stream, a); break;
    case 7: e = launch_pdl(int8_few_kernel<O, 7>, grid, dim3(256), 0, stream, a); break;
    case 8: e = launch_pdl(int8_few_kernel<O, 8>, grid, dim3(256), 0, stream, a); break;
    default: break;
  }
  return e == cudaSuccess ? MM_OK : MM_ERR_CUDA;
}

// ------------------------------------------------------------------ every stride
//
// 32 x 32 outputs per block of 256 threads, K through shared memory in slabs of
// 32; a slab's sum is exact in int32 and the slabs add up in int64.
template <typename O>
__global__ void __launch_bounds__(256) int8_any_kernel(const Int8Args a) {
  pdl_begin();
  __shared__ __align__(4) int8_t sA[32][36], sB[32][36];  // [row][k], [column][k]; read in words
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * 32, n0 = (int64_t)blockIdx.x * 32;
  const bool a_k = a.a_cs <= a.a_rs, b_k = a.b_ks <= a.b_ns;       // which way neighbours lie
  long long acc[2][2] = {};
  for (int64_t k0 = 0; k0 < a.K; k0 += 32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = threadIdx.x + 256 * i, fast = e & 31, slow = e >> 5;
      const int ra = a_k ? slow : fast, ka = a_k ? fast : slow, rb = b_k ? slow : fast, kb = b_k ? fast : slow;
      sA[ra][ka] = m0 + ra < a.M && k0 + ka < a.K ? a.a[(m0 + ra) * a.a_rs + (k0 + ka) * a.a_cs] : (int8_t)0;
      sB[rb][kb] = n0 + rb < a.N && k0 + kb < a.K ? a.b[(n0 + rb) * a.b_ns + (k0 + kb) * a.b_ks] : (int8_t)0;
    }
    __syncthreads();
    int s[2][2] = {};
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      int x[2], w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i] = *reinterpret_cast<const int*>(&sA[ty + 16 * i][k]);
        w[i] = *reinterpret_cast<const int*>(&sB[tx + 16 * i][k]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) s[i][j] = __dp4a(x[i], w[j], s[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] += s[i][j];
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < a.M && n < a.N)
        static_cast<O*>(a.y)[m * a.N + n] =
            finish8<O>((float)acc[i][j], a.sa[m * a.sa_s], a.sb[n * a.sb_s], bias_at<O>(a, n));
    }
}

template <typename O>
mm_status run_any(const Int8Args& a, cudaStream_t stream) {
  const int64_t gx = (a.N + 31) / 32, gy = (a.M + 31) / 32;
  // blockIdx.y is limited to 65535: bands of rows
  for (int64_t y0 = 0; y0 < gy; y0 += 65535) {
    Int8Args b = a;
    b.a += y0 * 32 * a.a_rs;
    b.sa += y0 * 32 * a.sa_s;
    b.y = static_cast<O*>(a.y) + y0 * 32 * a.N;
    b.M = a.M - y0 * 32;
    const int64_t h = gy - y0 < 65535 ? gy - y0 : 65535;
    if (b.M > h * 32) b.M = h * 32;
    if (launch_pdl(int8_any_kernel<O>, dim3((unsigned)gx, (unsigned)h), dim3(256), 0, stream, b) != cudaSuccess)
      return MM_ERR_CUDA;
  }
  return MM_OK;
}

// ------------------------------------------------------------------ copies of operands
//
// int8 values are exact in f16.  A row of an f16 copy is `ld` values (a multiple of
// 8, zeros past `cols`), of a copy in bytes a multiple of 16; 16 values a thread.
// Bound: memory, 1 byte read and 2 or 1 written per value.  Sources of any
// alignment are read in aligned words (each holds a byte that is wanted) and
// shifted; a copy in bytes of one whose rows are neighbours (rs = 1) is turned in tiles
// of 128 x 128 through shared memory.  (Byte by byte, 4096 x 14336 took 160 us.)  The f16
// copy of such rows, tokens given as a transpose, is gathered byte by byte: 1024 x 4096
// 16 us more than rows, 16384 x 4096 390.

// 16 bytes at any address.
__device__ __forceinline__ uint4 bytes16(const int8_t* p) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  if ((at & 15) == 0) return __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t sh = ((uint32_t)at & 3u) * 8;
  const uint32_t* w = reinterpret_cast<const uint32_t*>(at & ~(uintptr_t)3);
  const uint32_t w0 = __ldg(w), w1 = __ldg(w + 1), w2 = __ldg(w + 2), w3 = __ldg(w + 3), w4 = sh ? __ldg(w + 4) : 0u;
  return make_uint4(__funnelshift_r(w0, w1, sh), __funnelshift_r(w1, w2, sh), __funnelshift_r(w2, w3, sh),
                    __funnelshift_r(w3, w4, sh));
}

// A copy in bytes of a source whose rows are neighbours (rs = 1): 4 x 4 bytes a step.
constexpr int kTile = 128;
__device__ void turn_bytes(const Int8Copy& c, int64_t block) {
  __shared__ uint32_t tile[kTile][kTile / 4 + 1];      // [row][4 columns], words XORed with row / 32: no bank conflicts
  const int64_t across = (c.ld + kTile - 1) / kTile;
  const int64_t r0 = block / across * kTile, c0 = block % across * kTile;
  const int g = threadIdx.x & 31;
  const int64_t r = r0 + 4 * g;
#pragma unroll
  for (int i = 0; i < kTile / 32; ++i) {
    const int kq = (threadIdx.x >> 5) + 8 * i;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t k = c0 + 4 * kq + j;
      w[j] = 0;
      if (k < c.cols) {
        const int8_t* p = c.src + k * c.cs + r;
        if (r + 4 <= c.rows) {
          w[j] = bytes4(p);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (r + e < c.rows) w[j] |= (uint32_t)(uint8_t)__ldg(p + e) << (8 * e);
        }
      }
    }
    uint32_t t[4];
    turn4(w, t);
#pragma unroll
    for (int j = 0; j < 4; ++j) tile[4 * g + j][kq ^ (g >> 3)] = t[j];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kTile * kTile / 16 / 256; ++i) {
    const int e = threadIdx.x + 256 * i, row = e / (kTile / 16), q = e % (kTile / 16) * 4, x = row >> 5;
    if (r0 + row >= c.rows || c0 + 4 * q >= c.ld) continue;
    const uint32_t* t = tile[row];
    *reinterpret_cast<uint4*>(static_cast<int8_t*>(c.dst) + (r0 + row) * c.ld + c0 + 4 * q) =
        make_uint4(t[q ^ x], t[(q + 1) ^ x], t[(q + 2) ^ x], t[(q + 3) ^ x]);
  }
}
__host__ __device__ __forceinline__ bool turned(const Int8Copy& c) { return c.bytes && c.rs == 1 && c.cs != 1; }

__global__ void __launch_bounds__(256) int8_copy_kernel(const Int8Copy A, const Int8Copy B, const int64_t blocks_a) {
  pdl_begin();               // the product may start: it waits for this grid where it reads a copy
  const bool first = (int64_t)blockIdx.x < blocks_a;
  const Int8Copy& c = first ? A : B;
  if (turned(c)) return turn_bytes(c, (int64_t)blockIdx.x - (first ? 0 : blocks_a));
  const int64_t per_row = (c.ld + 15) / 16;
  const int64_t e = ((int64_t)blockIdx.x - (first ? 0 : blocks_a)) * 256 + threadIdx.x;
  if (e >= per_row * c.rows) return;
  const int64_t r = e < (1ll << 32) ? (int64_t)((uint32_t)e / (uint32_t)per_row) : e / per_row, c0 = (e - r * per_row) * 16;
  const int8_t* src = c.src + r * c.rs + c0 * c.cs;
  uint4 u;
  if (c.cs == 1 && c0 + 16 <= c.cols) {
    u = bytes16(src);
  } else {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (c0 + j < c.cols) w[j >> 2] |= (uint32_t)(uint8_t)__ldg(src + j * c.cs) << (8 * (j & 3));
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (c.bytes) {
    *reinterpret_cast<uint4*>(static_cast<int8_t*>(c.dst) + r * c.ld + c0) = u;
    return;
  }
  uint4 o[2];
  halves(u.x, o[0].x, o[0].y);
  halves(u.y, o[0].z, o[0].w);
  halves(u.z, o[1].x, o[1].y);
  halves(u.w, o[1].z, o[1].w);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__half*>(c.dst) + r * c.ld + c0);
  dst[0] = o[0];
  if (c0 + 8 < c.ld) dst[1] = o[1];
}

}  // namespace

mm_status launch_quantize_rows(const QuantizeArgs& a, cudaStream_t stream) {
  switch (a.dtype) {
    case MM_F32: return run_quantize<float>(a, stream);
    case MM_BF16: return run_quantize<__nv_bfloat16>(a, stream);
    default: return run_quantize<__half>(a, stream);
  }
}

bool int8_few_aligned(const Int8Args& a) {
  // (8191 pieces a lane at most: 8192 products sums of -128 * -128 pass int32.)
  return a.M <= kInt8FewRows && a.K % 16 == 0 && a.K >= 16 && a.K <= kInt8FewDepth && a.a_cs == 1 && a.b_ks == 1 &&
         a.b_ns % 16 == 0 && (a.M == 1 || a.a_rs % 16 == 0) && (reinterpret_cast<uintptr_t>(a.a) & 15) == 0 &&
         (reinterpret_cast<uintptr_t>(a.b) & 15) == 0 && a.N < (1ll << 31);
}

mm_status launch_int8_few_aligned(const Int8Args& a, cudaStream_t stream) {
  switch (a.out_dtype) {
    case MM_F32: return run_few<float>(a, stream);
    case MM_BF16: return run_few<__nv_bfloat16>(a, stream);
    default: return run_few<__half>(a, stream);
  }
}

mm_status launch_int8_any(const Int8Args& a, cudaStream_t stream) {
  switch (a.out_dtype) {
    case MM_F32: return run_any<float>(a, stream);
    case MM_BF16: return run_any<__nv_bfloat16>(a, stream);
    default: return run_any<__half>(a, stream);
  }
}

mm_status launch_int8_copies(const Int8Copy& A, const Int8Copy& B, cudaStream_t stream) {
  const auto blocks = [](const Int8Copy& c) {
    return turned(c) ? (c.rows + kTile - 1) / kTile * ((c.ld + kTile - 1) / kTile)
                     : ((c.ld + 15) / 16 * c.rows + 255) / 256;
  };
  const int64_t na = blocks(A), nb = blocks(B);
  if (na + nb >= (1ll << 31)) return MM_ERR_UNSUPPORTED;
  return launch_pdl(int8_copy_kernel, dim3((unsigned)(na + nb)), dim3(256), 0, stream, A, B, na) == cudaSuccess
             ? MM_OK
             : MM_ERR_CUDA;
}

}  // namespace qg
