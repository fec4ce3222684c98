// The orthogonalised update (mm_orthogonalize): a matrix is divided by its
// Frobenius norm and driven towards the nearest orthogonal one by the odd
// polynomial X <- a X + (b A + c A A) X, A = X X^T (Newton-Schulz), on the side
// with fewer rows (A = X^T X and X <- a X + X (b A + c A A) for a tall matrix).
//
// This file holds the norm, the division and the chain of products.
#include <cmath>
#include <cstring>

#include "api_internal.h"
#include "kernels.h"
#include "ortho.cuh"
#include "tc.h"

namespace qg {

namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ norm and division
//
// Both kernels walk a matrix in pieces of 16 bytes (VEC: rows contiguous, a
// whole number of aligned pieces) or elements; block (b, c) takes share c of
// matrix b.  Bound: memory, each reads X once.

struct NormArgs {
  int64_t M, N, count;               // matrices
  BatchMap bm;
  MatView x;
  int chunks;                        // shares of a matrix
  FastDiv fd_row;                    // pieces (or elements) of a row
  double* part;                      // [count][chunks] sums of squares
  float eps;
  float* s;                          // [count][M][ld], the divided matrix,
  __half* h;                         // that times `up` as f16 [count][M][ld] (NULL: not wanted) and, `rest` further, what that leaves (0: not wanted)
  int64_t ld, rest;
  float up;
};

template <typename T, bool VEC>
__device__ __forceinline__ void walk_share(const NormArgs& a, int64_t b, int chunk, int64_t& first, int64_t& last) {
  constexpr int E = VEC ? 16 / (int)sizeof(T) : 1;
  const int64_t pieces = a.M * (a.N / E);
  first = pieces * chunk / a.chunks;
  last = pieces * (chunk + 1) / a.chunks;
}

template <typename T, bool VEC, typename F>
__device__ __forceinline__ void walk(const NormArgs& a, F&& f) {
  constexpr int E = VEC ? 16 / (int)sizeof(T) : 1;
  const int64_t b = blockIdx.x / a.chunks;
  const int chunk = (int)(blockIdx.x - b * a.chunks);
  int64_t first, last;
  walk_share<T, VEC>(a, b, chunk, first, last);
  const T* x = static_cast<const T*>(a.x.ptr) + batch_offset(a.bm, a.x.bstride, b);
  const uint32_t per_row = a.fd_row.d;
  const auto place = [&](int64_t i, uint32_t& r, int64_t& c) {
    r = i < (1ll << 32) ? fast_div((uint32_t)i, a.fd_row) : (uint32_t)(i / per_row);
    c = (i - (int64_t)r * per_row) * E;
  };
  const auto load = [&](uint32_t r, int64_t c, T (&e)[E]) {
    if constexpr (VEC) *reinterpret_cast<uint4*>(e) = __ldg(reinterpret_cast<const uint4*>(x + r * a.x.rs + c));
    else e[0] = x[r * a.x.rs + c * a.x.cs];
  };
  // (Loads that the calls of f stand between are not moved together by the compiler.)
  constexpr int kTogether = 4;
  int64_t i = first + threadIdx.x;
  for (; i + (kTogether - 1) * kThreads < last; i += kTogether * kThreads) {
    uint32_t r[kTogether];
    int64_t c[kTogether];
    __align__(16) T e[kTogether][E];
#pragma unroll
    for (int q = 0; q < kTogether; ++q) {
      place(i + q * kThreads, r[q], c[q]);
      load(r[q], c[q], e[q]);
    }
#pragma unroll
    for (int q = 0; q < kTogether; ++q) f(b, r[q], c[q], e[q]);
  }
  for (; i < last; i += kThreads) {
    uint32_t r;
    int64_t c;
    __align__(16) T e[E];
    place(i, r, c);
    load(r, c, e);
    f(b, r, c, e);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) norm_kernel(const NormArgs a) {
  pdl_begin();
  __shared__ double part[kThreads / 32];
  Squares q;
  walk<T, VEC>(a, [&](int64_t, uint32_t, int64_t, const auto& e) {
    constexpr int E = sizeof(e) / sizeof(T);
    float v[E];
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = to_f32(e[j]);
    q.add(v);
  });
  q.join_warp();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = q.total();
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v += part[w];
    a.part[blockIdx.x] = v;
  }
}

// |X|_F + eps from the shares' sums.
__device__ __forceinline__ Divisor load_divisor(const NormArgs& a, int64_t b) {
  __shared__ Divisor d;
  if (threadIdx.x < 32) {
    double v = 0.;
    for (int c = threadIdx.x; c < a.chunks; c += 32) v += a.part[b * a.chunks + c];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (threadIdx.x == 0) d = Divisor(sqrt(v) + (double)a.eps);
  }
  __syncthreads();
  return d;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) divide_kernel(const NormArgs a) {
  pdl_begin();
  const Divisor d = load_divisor(a, blockIdx.x / a.chunks);
  walk<T, VEC>(a, [&](int64_t b, uint32_t r, int64_t c, const auto& e) {
    constexpr int E = sizeof(e) / sizeof(T);
    const int64_t at = (b * a.M + r) * a.ld + c;          // ld is a multiple of 8, c of E
    float v[E];
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = d.divide(to_f32(e[j]));
    if (a.h) {
      __align__(16) __half h[E], l[E];
#pragma unroll
      for (int j = 0; j < E; ++j) {
        h[j] = __float2half_rn(a.up * v[j]);
        l[j] = __float2half_rn(a.up * v[j] - __half2float(h[j]));
      }
      if constexpr (E == 8) {
        *reinterpret_cast<uint4*>(a.h + at) = *reinterpret_cast<const uint4*>(h);
        if (a.rest) *reinterpret_cast<uint4*>(a.h + a.rest + at) = *reinterpret_cast<const uint4*>(l);
      } else if constexpr (E == 4) {
        *reinterpret_cast<uint2*>(a.h + at) = *reinterpret_cast<const uint2*>(h);
        if (a.rest) *reinterpret_cast<uint2*>(a.h + a.rest + at) = *reinterpret_cast<const uint2*>(l);
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) {
          a.h[at + j] = h[j];
          if (a.rest) a.h[a.rest + at + j] = l[j];
        }
      }
    }
    if constexpr (E == 8) {                               // 32 bytes a lane: whole sectors
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a.s + at), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                   "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                   : "memory");
    } else if constexpr (E == 4) {
      *reinterpret_cast<float4*>(a.s + at) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) a.s[at + j] = v[j];
    }
  });
}

// out = T(scale * S): S [count][M][ld], out dense.
template <typename T>
__global__ void __launch_bounds__(kThreads) round_kernel(const float* s, int64_t rows, int64_t N, int64_t ld,
                                                         float scale, T* out) {
  pdl_begin();
  const int64_t n = rows * N, step = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += step) {
    const int64_t r = i / N;
    out[i] = from_f32<T>(scale * s[r * ld + (i - r * N)]);
  }
}

int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
// Shares per matrix: four blocks per SM over all matrices, at least 4096 elements each.
int norm_chunks(int64_t M, int64_t N, int64_t count) {
  const int64_t want = (4 * (int64_t)sm_count_public() + count - 1) / count;
  const int64_t most = (M * N + 4095) / 4096;
  const int64_t n = want < most ? want : most;
  return (int)(n < 1 ? 1 : n);
}

template <typename T>
mm_status run_norm(const OrthoArgs& o, NormArgs a, cudaStream_t stream) {
  constexpr int E = 16 / (int)sizeof(T);
  bool vec = o.x.cs == 1 && o.N % E == 0 && (o.x.rs % E == 0 || o.M == 1) && (reinterpret_cast<uintptr_t>(o.x.ptr) & 15) == 0;
  for (int d = 0; d < o.bm.nb; ++d) vec = vec && (o.x.bstride[d] % E == 0 || o.bm.shape[d] == 1);
  // Rows that follow one another without a gap, here and in the copy, are one row.
  if (vec && a.ld == o.N && (o.x.rs == o.N || o.M == 1) && o.M * o.N < (1ll << 31)) {
    a.N = o.M * o.N;
    a.ld = a.N;
    a.M = 1;
  }
  a.fd_row = make_fastdiv((uint32_t)(vec ? a.N / E : a.N));
  const int64_t blocks = o.bm.count * a.chunks;
  if (blocks >= (1ll << 31)) return MM_ERR_UNSUPPORTED;
  const dim3 g((unsigned)blocks), t(kThreads);
  cudaError_t e = vec ? launch_pdl(norm_kernel<T, true>, g, t, 0, stream, a)
                      : launch_pdl(norm_kernel<T, false>, g, t, 0, stream, a);
  if (e == cudaSuccess)
    e = vec ? launch_pdl(divide_kernel<T, true>, g, t, 0, stream, a) : launch_pdl(divide_kernel<T, false>, g, t, 0, stream, a);
  return e == cudaSuccess ? MM_OK : MM_ERR_CUDA;
}

template <typename T>
mm_status run_round(const OrthoArgs& o, const float* s, int64_t ld, cudaStream_t stream) {
  const int64_t rows = o.bm.count * o.M, want = (rows * o.N + 4 * kThreads - 1) / (4 * kThreads);
  const int64_t most = 8 * (int64_t)sm_count_public();
  return launch_pdl(round_kernel<T>, dim3((unsigned)(want < most ? want : most)), dim3(kThreads), 0, stream, s, rows,
                    o.N, ld, o.scale, static_cast<T*>(o.out)) == cudaSuccess
             ? MM_OK
             : MM_ERR_CUDA;
}

// ------------------------------------------------------------------ the chain in fp32

struct FloatPlan {
  int64_t m, ld, ldm;               // the smaller side; row pitches of X and of A, B
  int chunks;
  size_t part, s[2], a, b, bytes;   // offsets in the workspace
};
FloatPlan plan_float(const OrthoArgs& o) {
  FloatPlan p;
  p.m = o.M < o.N ? o.M : o.N;
  p.ld = round_up(o.N, 8);
  p.ldm = round_up(p.m, 4);
  p.chunks = norm_chunks(o.M, o.N, o.bm.count);
  const size_t x = align256((size_t)o.bm.count * o.M * p.ld * 4), sq = align256((size_t)o.bm.count * p.m * p.ldm * 4);
  p.part = 0;
  p.s[0] = align256((size_t)o.bm.count * p.chunks * 8);
  p.s[1] = p.s[0] + x;
  p.a = p.s[1] + x;
  p.b = p.a + sq;
  p.bytes = p.b + sq;
  return p;
}

// A batch of `count` products C = alpha A B + beta C0 of matrices `*_step` apart.
GemmArgs batched(int dtype, int64_t count, int64_t M, int64_t N, int64_t K) {
  GemmArgs g;
  memset(&g, 0, sizeof(g));
  g.dtype = dtype;
  g.M = M; g.N = N; g.K = K;
  g.bm.nb = 1;
  for (int d = 0; d < kMaxBatchDims; ++d) g.bm.shape[d] = 1;
  g.bm.shape[0] = g.bm.count = count;
  g.alpha = 1.f;
  return g;
}
MatView view(const void* p, int64_t step, int64_t rs, int64_t cs) {
  MatView v;
  memset(&v, 0, sizeof(v));
  v.ptr = p;
  v.bstride[0] = step;
  v.rs = rs;
  v.cs = cs;
  return v;
}

// The products of the chain go by the policy as MatMul's do, without the few-row kernels.
mm_status product(const GemmArgs& g, cudaStream_t st) {
  const int path = choose(tc_gemm_supported(g), tensor_pays_dense(g.dtype, g.M, g.N, g.K, g.bm.count));
  return run_dense_on(path, g, st);
}

NormArgs norm_args(const OrthoArgs& o, int chunks, void* part, int64_t ld) {
  NormArgs n;
  memset(&n, 0, sizeof(n));
  n.M = o.M; n.N = o.N; n.count = o.bm.count;
  n.bm = o.bm; n.x = o.x;
  n.chunks = chunks;
  n.part = static_cast<double*>(part);
  n.eps = o.eps;
  n.ld = ld;
  return n;
}
mm_status divide(const OrthoArgs& o, const NormArgs& n, cudaStream_t st) {
  return o.dtype == MM_F32    ? run_norm<float>(o, n, st)
         : o.dtype == MM_BF16 ? run_norm<__nv_bfloat16>(o, n, st)
                              : run_norm<__half>(o, n, st);
}

mm_status run_float(const OrthoArgs& o, void* ws, cudaStream_t st) {
  const FloatPlan p = plan_float(o);
  uint8_t* w = static_cast<uint8_t*>(ws);
  NormArgs n = norm_args(o, p.chunks, w + p.part, p.ld);
  n.s = reinterpret_cast<float*>(w + p.s[0]);
  mm_status s = divide(o, n, st);
  const bool tall = o.M > o.N;
  const int64_t xs = o.M * p.ld, as = p.m * p.ldm;
  float *A = reinterpret_cast<float*>(w + p.a), *B = reinterpret_cast<float*>(w + p.b);
  int cur = 0;
  for (int i = 0; i < o.steps && s == MM_OK; ++i) {
    const float *X = reinterpret_cast<float*>(w + p.s[cur]), *k = o.coef + 3 * i;
    GemmArgs g = batched(MM_F32, o.bm.count, p.m, p.m, tall ? o.M : o.N);
    g.a = tall ? view(X, xs, 1, p.ld) : view(X, xs, p.ld, 1);
    g.b = tall ? view(X, xs, p.ld, 1) : view(X, xs, 1, p.ld);
    g.y = view(A, as, p.ldm, 1);
    if ((s = product(g, st)) != MM_OK) return s;
    g = batched(MM_F32, o.bm.count, p.m, p.m, p.m);
    g.a = g.b = g.c = view(A, as, p.ldm, 1);
    g.y = view(B, as, p.ldm, 1);
    g.alpha = k[2];
    g.beta = k[1];
    if ((s = product(g, st)) != MM_OK) return s;
    g = batched(MM_F32, o.bm.count, o.M, o.N, p.m);
    g.a = tall ? view(X, xs, p.ld, 1) : view(B, as, p.ldm, 1);
    g.b = tall ? view(B, as, p.ldm, 1) : view(X, xs, p.ld, 1);
    g.c = view(X, xs, p.ld, 1);
    g.beta = k[0];
    cur ^= 1;
    if (i + 1 == o.steps && o.dtype == MM_F32) {        // straight into the output
      g.alpha = o.scale;
      g.beta = k[0] * o.scale;
      g.y = view(o.out, o.M * o.N, o.N, 1);
      return product(g, st);
    }
    g.y = view(w + p.s[cur], xs, p.ld, 1);
    s = product(g, st);
  }
  if (s != MM_OK) return s;
  const float* X = reinterpret_cast<float*>(w + p.s[cur]);
  s = o.dtype == MM_F32    ? run_round<float>(o, X, p.ld, st)
      : o.dtype == MM_BF16 ? run_round<__nv_bfloat16>(o, X, p.ld, st)
                           : run_round<__half>(o, X, p.ld, st);
  return o.steps == 0 ? finish(s, MM_PATH_SIMT) : s;     // (the products have said theirs)
}

// ------------------------------------------------------------------ the chain on the tensor cores
//
// The products' operands are f16 (11 bits; X, A and B each rounded once a step),
// their sums fp32.  What is rounded to 11 bits only enters the correction (b A + c A A) X;
// a X itself comes from the state, which is fp32, since the iteration magnifies small
// singular values by a in every step and the state's rounding with them (a state rounded
// to 11 bits: off by 4e-2 for matrices with a few strong directions), and since X_0 is
// as small as the norm is beside eps, matrix by matrix.  A value that is too small for
// the operands (below 2^-39 of the array's bound) lacks its correction, which is as small
// beside a X.  Each array has a power of two of its own, the largest that cannot
// overflow: the singular values start at 1 at most and the polynomial's maximum bounds
// every later step's, so that f16's range is used from the top.
// A and B are symmetric: only the lower triangle's tiles are computed.
//
// fp32 and f16 matrices, and bf16 ones up to kHalfSide, take the same chain with
// every operand split into two f16 values (22 bits) and three products each.
// (Three tf32 products of fp32 operands took 1.49 ms for
// 2048 x 2048 and were off by 1.8e-5: their additions truncate, 3 K / 8 times a sum;
// see kSymF.)  An f16 result would be off by 2.1e-3 with 11-bit operands, ten times
// its own rounding; a bf16 one is off by 1.2 to 1.4 times its rounding from 512 rows
// on, by up to 1.6 times below, where the launches cost more than the products
// (us for 512 x 512, 256 x 256, 8 of 512 x 1000: 148 113 204, split 178 126 267).

double power_below(double x) {
  if (x > 0x1p60) return 0x1p60;         // infinite where the array is zeros
  return std::ldexp(1., (int)std::floor(std::log2(x)));
}
// The largest |f| of f(s) = s (a + b s^2 + c s^4) on [0, u], and of b l + c l^2 on [0, u^2].
double odd_bound(double a, double b, double c, double u) {
  const auto f = [&](double s) { return std::fabs(s * (a + s * s * (b + s * s * c))); };
  double most = f(u);
  const double qa = 5. * c, qb = 3. * b, disc = qb * qb - 4. * qa * a;
  if (disc >= 0.) {
    for (int sign = -1; sign <= 1; sign += 2) {
      const double t = qa != 0. ? (-qb + sign * std::sqrt(disc)) / (2. * qa) : qb != 0. ? -a / qb : -1.;
      if (t > 0. && t < u * u) most = std::fmax(most, f(std::sqrt(t)));
    }
  }
  return most;
}
double even_bound(double b, double c, double u) {
  const auto f = [&](double l) { return std::fabs(l * (b + l * c)); };
  double most = f(u * u);
  const double l = c != 0. ? -b / (2. * c) : -1.;
  if (l > 0. && l < u * u) most = std::fmax(most, f(l));
  return most;
}

struct HalfScales { double x, a, b; };       // powers of two of X, A, B in a step
constexpr double kHalfTop = 32768.;
constexpr double kSlack = 1.02;              // what the roundings may add to a bound
// False where the bounds leave the range that the scales cover, and where a step's
// product outweighs a X by so much that it counts for singular values whose squares are
// lost in the operands: those below 2^-20 of the bound u are, and for s = 2^-20 u the
// correction (b s^2 + c s^4) X is at most 2^-28 of a X under this limit.
bool half_scales(const OrthoArgs& o, HalfScales (&k)[MM_ORTHO_MAX_STEPS + 1]) {
  double u = kSlack;
  for (int i = 0; i < o.steps; ++i) {
    const float* c = o.coef + 3 * i;
    const double u2 = u * u, even = kSlack * even_bound(c[1], c[2], u);
    if ((u != 0. && !(u > 1e-6 && u < 1e6)) || !(even < 1e18)) return false;
    if (std::fabs(c[0]) < 0x1p-12 * (std::fabs(c[1]) + std::fabs(c[2]) * u2) * u2) return false;
    k[i].x = power_below(kHalfTop / u);
    k[i].a = power_below(kHalfTop / u2);
    k[i].b = power_below(kHalfTop / even);
    u = kSlack * odd_bound(c[0], c[1], c[2], u);
  }
  k[o.steps] = {1., 1., 1.};
  return true;
}

constexpr int64_t kHalfSide = 512;
bool split_operands(const OrthoArgs& o) { return o.dtype != MM_BF16 || o.M <= kHalfSide || o.N <= kHalfSide; }

// Products whose sum the tensor cores keep before it is added up in fp32.  Their
// truncation shrinks every step by some 2^-25 an addition, which shows where a fp32
// result is hardly blurred by small singular values: longer matrices.  From 1024 rows on
// fp32 sums are off by so much themselves that 256 is enough.
// Error relative to fp32 sums' at 256, 128 and 64: 600 x 1000 1.9 and 1.1, 333 x 777 2.3
// and 1.35, 1800 x 220 3.0, 1.8 and 1.2; 300 x 420 1.85, 512 x 512 0.9 at 256.  A segment
// costs a hand-over: 8 of 512 x 1000 277 us at 256 and 297 at 128.  From 1024 on, at 256
// and at what the rule below 1024 would take, with us: 1024 x 4096 1.14 435, 0.58 535;
// 1024 x 8192 1.54 747, 0.49 1340; 1100 x 8000 0.81 842, 0.27 1490; 2048 x 6144 0.52 1139,
// 0.30 1445; 9000 x 1500 0.48 1146, 0.21 2020; 2048 x 2048 0.58 511.
int segment_of(const OrthoArgs& o) {
  const int64_t m = o.M < o.N ? o.M : o.N, n = o.M < o.N ? o.N : o.M;
  if (o.dtype != MM_F32 || m >= 1024 || 5 * n < 6 * m) return 256;
  return n < 6 * m ? 128 : 64;
}

struct HalfPlan {
  int64_t m, ld, ldm;
  int chunks;
  size_t part, x[2], a, b, s, bytes;
};
HalfPlan plan_half(const OrthoArgs& o) {
  HalfPlan p;
  p.m = o.M < o.N ? o.M : o.N;
  p.ld = round_up(o.N, 8);
  p.ldm = round_up(p.m, 8);
  p.chunks = norm_chunks(o.M, o.N, o.bm.count);
  const size_t size = split_operands(o) ? 4 : 2;       // of an operand's value
  const size_t x = align256((size_t)o.bm.count * o.M * p.ld * size), sq = align256((size_t)o.bm.count * p.m * p.ldm * size);
  p.part = 0;
  p.x[0] = align256((size_t)o.bm.count * p.chunks * 8);
  p.x[1] = p.x[0] + x;
  p.a = p.x[1] + x;
  p.b = p.a + sq;
  p.s = p.b + sq;
  p.bytes = p.s + align256((size_t)o.bm.count * o.M * p.ld * 4);
  return p;
}

// Matrices whose Gram product is worth the tensor cores.
bool half_chain(const OrthoArgs& o) {
  const int64_t m = o.M < o.N ? o.M : o.N, n = o.M < o.N ? o.N : o.M;
  return choose(m > 1, tensor_pays(m, m, n, o.bm.count)) == MM_PATH_TENSOR;
}

mm_status run_half(const OrthoArgs& o, const HalfScales* k, void* ws, cudaStream_t st) {
  unsigned* status = device_status_ptr();
  if (!status) return MM_ERR_CUDA;
  const HalfPlan p = plan_half(o);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const int64_t xs = o.M * p.ld, as = p.m * p.ldm;
  NormArgs n = norm_args(o, p.chunks, w + p.part, p.ld);
  n.h = reinterpret_cast<__half*>(w + p.x[0]);
  const bool split = split_operands(o);
  const int segment = segment_of(o);
  float* S = reinterpret_cast<float*>(w + p.s);
  n.rest = split ? o.bm.count * xs : 0;
  n.up = (float)k[0].x;
  n.s = S;
  mm_status s = divide(o, n, st);
  const bool tall = o.M > o.N;
  void *A = w + p.a, *B = w + p.b;
  for (int i = 0; i < o.steps && s == MM_OK; ++i) {
    const void* X = w + p.x[i & 1];
    const double a = o.coef[3 * i], b = o.coef[3 * i + 1], c = o.coef[3 * i + 2];
    OrthoProduct g;
    memset(&g, 0, sizeof(g));
    g.sym = 1;
    g.split = split;
    g.segment = segment;
    g.y_dtype = MM_F16;
    g.M = g.N = p.m;
    g.K = tall ? o.M : o.N;
    g.count = o.bm.count;
    g.a = g.b = X;
    g.a_step = g.b_step = xs;
    g.a_rs = g.b_cs = tall ? 1 : p.ld;
    g.a_cs = g.b_rs = tall ? p.ld : 1;
    g.y = A; g.y_rs = p.ldm; g.y_step = as;
    g.alpha = (float)(k[i].a / (k[i].x * k[i].x));
    if ((s = launch_tc_ortho(g, status, st)) != MM_OK) return s;
    g.K = p.m;
    g.a = g.b = g.c = A;
    g.a_step = g.b_step = g.c_step = as;
    g.a_rs = g.b_cs = g.c_rs = p.ldm;
    g.a_cs = g.b_rs = 1;
    g.y = B;
    g.alpha = (float)(k[i].b * c / (k[i].a * k[i].a));
    g.beta = (float)(k[i].b * b / k[i].a);
    if ((s = launch_tc_ortho(g, status, st)) != MM_OK) return s;
    memset(&g, 0, sizeof(g));
    g.M = o.M; g.N = o.N; g.K = p.m;
    g.count = o.bm.count;
    g.a = tall ? X : B; g.a_step = tall ? xs : as; g.a_rs = tall ? p.ld : p.ldm; g.a_cs = 1;
    g.b = tall ? B : X; g.b_step = tall ? as : xs; g.b_rs = tall ? p.ldm : p.ld; g.b_cs = 1;
    const bool last = i + 1 == o.steps;
    const double up = last ? (double)o.scale : 1.;      // the state holds X itself
    g.split = split;
    g.segment = segment;
    g.last = last;
    g.s32 = S; g.s_rs = p.ld; g.s_step = xs;
    g.up = (float)k[i + 1].x;
    g.alpha = (float)(up / (k[i].b * k[i].x));
    g.beta = (float)(up * a);
    g.y_dtype = last ? o.dtype : MM_F16;
    g.y = last ? o.out : w + p.x[(i + 1) & 1];
    g.y_rs = last ? o.N : p.ld;
    g.y_step = last ? o.M * o.N : xs;
    s = launch_tc_ortho(g, status, st);
  }
  return finish(s, MM_PATH_TENSOR);
}

bool ortho_small(const OrthoArgs& o) { return path_policy() != MM_PATH_TENSOR && ortho_small_pays(o); }

}  // namespace

size_t ortho_workspace_bytes(const OrthoArgs& o) {
  // The coefficients are not known yet: room for either chain of 16-bit matrices.
  if (ortho_small(o)) return 0;
  const size_t f = plan_float(o).bytes;
  if (!half_chain(o)) return f;
  const size_t h = plan_half(o).bytes;
  return h > f ? h : f;
}

mm_status launch_ortho(const OrthoArgs& o, void* workspace, cudaStream_t stream) {
  if (ortho_small(o)) return finish(launch_ortho_small(o, stream), MM_PATH_SIMT);
  HalfScales k[MM_ORTHO_MAX_STEPS + 1];
  if (o.steps > 0 && half_chain(o) && half_scales(o, k)) return run_half(o, k, workspace, stream);
  return run_float(o, workspace, stream);
}

}  // namespace qg
