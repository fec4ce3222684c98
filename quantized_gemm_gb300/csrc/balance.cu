// The router's balance loss, the picks per expert (mm_route_balance) and the
// loss's gradient (mm_route_balance_grad).
//
// With p[t, g] the softmax of row t over the experts that can be picked, c[g]
// the picks of expert g, C their sum, T' the rows that have any such expert and
// P[g] = sum_t p[t, g] / T':
//   loss = G sum_g (c[g] / C) P[g]
//   dl[t, j] = dloss (G / T') p[t, j] (c[j] / C - sum_g (c[g] / C) p[t, g])
// A logit of -inf or NaN takes no part (p = 0); a maximum of +inf takes the
// limit, as in mm_route_topk.
//
// Both directions read the logits once and are bound by memory.  A row belongs
// to LPR neighbouring lanes, lane i holding columns [i*V, i*V + V); a lane keeps
// the same columns for every row of its warp, so the column sums (forward) and
// the shares c/C (gradient) stay in its registers.  kRows rows are loaded before
// any is used.  Column sums leave a block through shared memory, one partial
// per block, and a second launch, one cluster, adds the partials in a fixed
// order; picks are integers, counted with shared-memory atomics, whose order
// does not matter.
#include "kernels.h"
#include "tc_ptx.cuh"

namespace qg {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRows = 4;
constexpr int kFinalBlocks = 8;      // the cluster of the second launch

// exp(l - top), with the limit for an infinite top.  The difference is rounded
// once and the function is off by 2 ulp and by |l - top| 2^-23: 3e-6 where the
// result still matters (l - top > -20).
__device__ __forceinline__ float share_of(float l, float top) { return l == top ? 1.f : __expf(l - top); }

template <int LPR>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int LPR>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// V neighbouring values of a row as loaded: raw 16-byte pieces where the row
// allows it, otherwise one element at a time (`fill` past the end).
template <typename T, int V>
struct Piece {
  static constexpr int kPer = 16 / sizeof(T), kVecs = V / kPer;
  static_assert(V % kPer == 0, "whole 16-byte pieces");
  uint4 u[kVecs];
  __device__ __forceinline__ void load(const T* row, int64_t cs, int c0, int n, bool vec, float fill) {
    if (vec && c0 + V <= n) {
#pragma unroll
      for (int q = 0; q < kVecs; ++q) u[q] = __ldg(reinterpret_cast<const uint4*>(row + c0) + q);
    } else {
      T* e = reinterpret_cast<T*>(u);
#pragma unroll
      for (int j = 0; j < V; ++j) e[j] = c0 + j < n ? row[(c0 + j) * cs] : from_f32<T>(fill);
    }
  }
  __device__ __forceinline__ float at(int j) const { return to_f32(reinterpret_cast<const T*>(u)[j]); }
};

// e[j] = exp(l[j] - top) and 1 / sum; false for a row without any expert.
template <typename T, int LPR, int V>
__device__ __forceinline__ bool softmax_row(const Piece<T, V>& l, float (&e)[V], float* inv) {
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < V; ++j) top = fmaxf(top, l.at(j));       // fmaxf drops NaN
  top = lanes_max<LPR>(top);
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float x = l.at(j);
    e[j] = x > -INFINITY ? share_of(x, top) : 0.f;             // false for NaN
    sum += e[j];
  }
  sum = lanes_sum<LPR>(sum);
  *inv = sum > 0.f ? 1.f / sum : 0.f;
  return sum > 0.f;
}

// Partials of a block: psum [G] f32, then picks [G] i32, then rows that take
// part and picks in all.
template <typename T, int LPR, int V>
__global__ void __launch_bounds__(kThreads) balance_partial_kernel(const BalanceArgs a, const int vec, float* psum,
                                                                   int32_t* cnt, unsigned* status) {
  pdl_wait();
  extern __shared__ float sh[];                                // [kWarps][G] column sums, then [G + 2] counts
  int32_t* hist = reinterpret_cast<int32_t*>(sh + kWarps * a.G);
  const int G = (int)a.G, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < G + 2; i += kThreads) hist[i] = 0;
  __syncthreads();
  // picks
  int mine = 0;
  bool bad = false;
  const int64_t picks = a.rows * a.k;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < picks; i += (int64_t)gridDim.x * kThreads) {
    const int64_t off = a.i_cs == 1 && a.i_rs == a.k ? i : (i / a.k) * a.i_rs + (i % a.k) * a.i_cs;
    const int64_t g = load_index(a.indices, off, a.ind64);
    if (g >= 0 && g < G) {
      atomicAdd(hist + (int)g, 1);
      ++mine;
    } else if (g != -1) {
      bad = true;
    }
  }
  if (bad) atomicOr(status, kStatusIndexRange);
  // column sums
  constexpr int kPerWarp = 32 / LPR;
  const int sub = lane / LPR, l = lane % LPR, c0 = l * V;
  const T* logits = static_cast<const T*>(a.logits);
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.f;
  int alive = 0;
  const int64_t step = (int64_t)gridDim.x * kWarps * kPerWarp;
  for (int64_t r0 = ((int64_t)blockIdx.x * kWarps + warp) * kPerWarp; r0 < a.rows; r0 += step * kRows) {
    Piece<T, V> p[kRows];
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      const int64_t r = r0 + q * step + sub;
      p[q].load(logits + (r < a.rows ? r : 0) * a.l_rs, a.l_cs, c0, G, vec, -INFINITY);
    }
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      float e[V], inv;
      const bool any = softmax_row<T, LPR, V>(p[q], e, &inv);
      if (r0 + q * step + sub >= a.rows) continue;
      if (any && l == 0) ++alive;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = fmaf(e[j], inv, acc[j]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    alive += __shfl_xor_sync(0xffffffffu, alive, o);
    mine += __shfl_xor_sync(0xffffffffu, mine, o);
  }
  if (lane == 0) {
    atomicAdd(hist + G, alive);
    atomicAdd(hist + G + 1, mine);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);   // the warp's row groups
    if (sub == 0 && c0 + j < G) sh[warp * G + c0 + j] = acc[j];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < G; c += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sh[w * G + c];
    psum[(int64_t)blockIdx.x * G + c] = s;
  }
  for (int c = threadIdx.x; c < G + 2; c += kThreads) cnt[(int64_t)blockIdx.x * (G + 2) + c] = hist[c];
}

// One cluster: block b finishes columns [b*w, b*w + w), a warp per column, its
// lanes adding the blocks' partials; the first block adds the blocks' parts of the loss.
__global__ void __launch_bounds__(1024) __cluster_dims__(kFinalBlocks, 1, 1)
    balance_final_kernel(const int G, const int nb, const float* psum, const int32_t* cnt, float* loss, int32_t* counts,
                         float* mean) {
  pdl_wait();
  __shared__ float part[32];
  __shared__ int tot[2][32];
  __shared__ float mine;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = (int)ptx::cluster_ctarank();
  // Rows and picks in all: every block adds them for itself.
  int rows = 0, picks = 0;
  for (int b = threadIdx.x; b < nb; b += 1024) {
    rows += __ldg(cnt + (int64_t)b * (G + 2) + G);
    picks += __ldg(cnt + (int64_t)b * (G + 2) + G + 1);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    rows += __shfl_xor_sync(0xffffffffu, rows, o);
    picks += __shfl_xor_sync(0xffffffffu, picks, o);
  }
  if (lane == 0) { tot[0][warp] = rows; tot[1][warp] = picks; }
  __syncthreads();
  rows = __reduce_add_sync(0xffffffffu, tot[0][lane]);
  picks = __reduce_add_sync(0xffffffffu, tot[1][lane]);
  const float inv_rows = rows > 0 ? 1.f / (float)rows : 0.f, inv_picks = picks > 0 ? 1.f / (float)picks : 0.f;
  // 32 neighbouring columns at a time: lane = column for the reads, warps share the blocks.
  __shared__ float ps[32][33];
  __shared__ int cs[32][33];
  float lsum = 0.f;
  for (int c0 = rank * 32; c0 < G; c0 += kFinalBlocks * 32) {
    float s = 0.f;
    int n = 0;
    if (c0 + lane < G) {
#pragma unroll 4
      for (int b = warp; b < nb; b += 32) {
        s += __ldg(psum + (int64_t)b * G + c0 + lane);
        n += __ldg(cnt + (int64_t)b * (G + 2) + c0 + lane);
      }
    }
    __syncthreads();
    ps[lane][warp] = s;
    cs[lane][warp] = n;
    __syncthreads();
    s = ps[warp][lane];
    n = cs[warp][lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    const int c = c0 + warp;
    if (lane == 0 && c < G) {
      const float m = s * inv_rows;
      mean[c] = m;
      counts[c] = n;
      lsum = fmaf((float)n * inv_picks, m, lsum);
    }
  }
  if (lane == 0) part[warp] = lsum;
  __syncthreads();
  if (warp == 0) {
    const float v = lanes_sum<32>(part[lane]);
    if (lane == 0) mine = v;
  }
  ptx::cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    float v = 0.f;
    for (int r = 0; r < kFinalBlocks; ++r) {
      float x;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(ptx::mapa_shared(ptx::smem_u32(&mine), r)) : "memory");
      v += x;
    }
    *loss = (float)G * v;
    counts[G] = rows;
  }
  ptx::cluster_sync();       // no block leaves before its part has been read
}

template <typename T, int LPR, int V>
__global__ void __launch_bounds__(kThreads) balance_grad_kernel(const BalanceGradArgs a, const int vec, const int bvec,
                                                                const int ovec) {
  pdl_begin();
  constexpr int kPerWarp = 32 / LPR, kGradRows = V >= 16 ? 2 : kRows;
  const int G = (int)a.G, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / LPR, l = lane % LPR, c0 = l * V;
  // The shares c / C of this lane's columns; a row's lanes hold all of them.
  float share[V];
  int total = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int n = c0 + j < G ? __ldg(a.counts + (c0 + j) * a.counts_s) : 0;
    total += n;
    share[j] = (float)n;
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int rows_in = __ldg(a.counts + G * a.counts_s);
  const float scale = total > 0 ? 1.f / (float)total : 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) share[j] *= scale;
  const float coef = rows_in > 0 ? __ldg(a.dloss) * ((float)G / (float)rows_in) : 0.f;
  const T* logits = static_cast<const T*>(a.logits);
  const T* base = static_cast<const T*>(a.base);
  T* out = static_cast<T*>(a.out);
  const int64_t step = (int64_t)gridDim.x * kWarps * kPerWarp;
  for (int64_t r0 = ((int64_t)blockIdx.x * kWarps + warp) * kPerWarp; r0 < a.rows; r0 += step * kGradRows) {
    Piece<T, V> p[kGradRows], pb[kGradRows];
#pragma unroll
    for (int q = 0; q < kGradRows; ++q) {
      const int64_t r = r0 + q * step + sub, rr = r < a.rows ? r : 0;
      p[q].load(logits + rr * a.l_rs, a.l_cs, c0, G, vec, -INFINITY);
      if (base) pb[q].load(base + rr * a.b_rs, a.b_cs, c0, G, bvec, 0.f);
    }
#pragma unroll
    for (int q = 0; q < kGradRows; ++q) {
      const int64_t r = r0 + q * step + sub;
      float e[V], inv;
      softmax_row<T, LPR, V>(p[q], e, &inv);
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        e[j] *= inv;
        dot = fmaf(share[j], e[j], dot);
      }
      dot = lanes_sum<LPR>(dot);
      if (r >= a.rows) continue;
      Piece<T, V> o;
      T* oe = reinterpret_cast<T*>(o.u);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        // a column that takes no part has a gradient of zero, whatever dloss is
        const float d = e[j] > 0.f ? coef * e[j] * (share[j] - dot) : 0.f;
        oe[j] = from_f32<T>(base ? pb[q].at(j) + d : d);
      }
      T* dst = out + r * (int64_t)G + c0;
      if (ovec && c0 + V <= G) {
#pragma unroll
        for (int v = 0; v < Piece<T, V>::kVecs; ++v) reinterpret_cast<uint4*>(dst)[v] = o.u[v];
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (c0 + j < G) dst[j] = oe[j];
      }
    }
  }
}

template <typename T>
int vec_ok(const void* p, int64_t rs, int64_t cs) {
  return cs == 1 && (rs * sizeof(T)) % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

// Lanes per row and values per lane for G experts: whole 16-byte pieces, a full
// warp from 16 lanes on.
template <typename T, typename F>
mm_status by_width(int64_t G, F&& f) {
  constexpr int P = 16 / sizeof(T);
  if (G <= 4 * P) return f(std::integral_constant<int, 4>(), std::integral_constant<int, P>());
  if (G <= 8 * P) return f(std::integral_constant<int, 8>(), std::integral_constant<int, P>());
  if (G <= 16 * P) return f(std::integral_constant<int, 16>(), std::integral_constant<int, P>());
  if (G <= 32 * P) return f(std::integral_constant<int, 32>(), std::integral_constant<int, P>());
  if (G <= 64 * P) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 2 * P>());
  if (G <= 128 * P) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 4 * P>());
  return f(std::integral_constant<int, 32>(), std::integral_constant<int, 32>());
}

// Blocks for `rows` rows: enough for one round of kRows rows a warp, at most `per_sm` per SM.
int64_t row_blocks(int64_t rows, int rows_per_block, int per_sm) {
  const int64_t want = (rows + rows_per_block - 1) / rows_per_block, most = (int64_t)sm_count_public() * per_sm;
  return want < 1 ? 1 : want < most ? want : most;
}

constexpr int kPartialPerSm = 3;

template <typename T>
mm_status run_partial(const BalanceArgs& a, void* ws, unsigned* status, cudaStream_t stream) {
  const int64_t nb = balance_partial_blocks(a.rows);
  float* psum = static_cast<float*>(ws);
  int32_t* cnt = reinterpret_cast<int32_t*>(psum + nb * a.G);
  const size_t smem = (size_t)(kWarps * a.G + a.G + 2) * 4;
  return by_width<T>(a.G, [&](auto lpr, auto v) {
    return launch_pdl(balance_partial_kernel<T, lpr(), v()>, dim3((unsigned)nb), dim3(kThreads), smem, stream, a,
                      vec_ok<T>(a.logits, a.l_rs, a.l_cs), psum, cnt, status) == cudaSuccess
               ? MM_OK
               : MM_ERR_CUDA;
  });
}

template <typename T>
mm_status run_grad(const BalanceGradArgs& a, cudaStream_t stream) {
  return by_width<T>(a.G, [&](auto lpr, auto v) {
    const int64_t nb = row_blocks(a.rows, kWarps * (32 / lpr()), 6);
    return launch_pdl(balance_grad_kernel<T, lpr(), v()>, dim3((unsigned)nb), dim3(kThreads), 0, stream, a,
                      vec_ok<T>(a.logits, a.l_rs, a.l_cs), a.base ? vec_ok<T>(a.base, a.b_rs, a.b_cs) : 0,
                      vec_ok<T>(a.out, a.G, 1)) == cudaSuccess
               ? MM_OK
               : MM_ERR_CUDA;
  });
}

}  // namespace

// A block takes 32 rows at least (a warp's kRows rows each), so that a few rows
// leave few partials to add.
int64_t balance_partial_blocks(int64_t rows) { return row_blocks(rows, kWarps * kRows, kPartialPerSm); }

size_t balance_workspace_bytes(int64_t rows, int64_t G) {
  return (size_t)balance_partial_blocks(rows) * (size_t)(2 * G + 2) * 4;
}

mm_status launch_balance(const BalanceArgs& a, void* ws, unsigned* status, cudaStream_t stream) {
  mm_status s = a.dtype == MM_F32    ? run_partial<float>(a, ws, status, stream)
                : a.dtype == MM_BF16 ? run_partial<__nv_bfloat16>(a, ws, status, stream)
                                     : run_partial<__half>(a, ws, status, stream);
  if (s != MM_OK) return s;
  const int64_t nb = balance_partial_blocks(a.rows);
  const float* psum = static_cast<const float*>(ws);
  return launch_pdl(balance_final_kernel, dim3(kFinalBlocks), dim3(1024), 0, stream, (int)a.G, (int)nb, psum,
                    reinterpret_cast<const int32_t*>(psum + nb * a.G), a.loss, a.counts, a.mean) == cudaSuccess
             ? MM_OK
             : MM_ERR_CUDA;
}

mm_status launch_balance_grad(const BalanceGradArgs& a, cudaStream_t stream) {
  switch (a.dtype) {
    case MM_F32: return run_grad<float>(a, stream);
    case MM_BF16: return run_grad<__nv_bfloat16>(a, stream);
    default: return run_grad<__half>(a, stream);
  }
}

}  // namespace qg
