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
// Both directions read the logits once.  A row belongs to LPR neighbouring lanes,
// which hold its 16-byte pieces in turn (piece q of lane i is the row's piece
// q * LPR + i), so that a warp reads 32 / LPR rows at once, each in whole
// sectors, and a sum over a row takes log2(LPR) shuffles for all of them.  A lane
// keeps the same columns for every row, so the column sums (forward) and the
// shares c / C (gradient) stay in its registers.  Each lane copies the pieces of
// rows to come into its own places in shared memory (cp.async, kAhead rows).  65536
// rows of 256 bf16 logits, forward and backward (101 MB, 15 us of memory): 95 us with
// a row over all 32 lanes and a branch per logit (276 instructions a row), 43 with
// two rows loaded into registers at a time, 37 so; what is left is latency (issue slots
// are half busy, with 107 instructions a row forward) and the second launch.  Column sums leave a block
// through shared memory, one partial per block, and a second launch, one cluster,
// adds the partials in a fixed order; picks are integers, counted with shared-memory
// atomics, whose order does not matter.
#include <type_traits>

#include "kernels.h"
#include "tc_ptx.cuh"

namespace qg {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kFinalBlocks = 8;      // the cluster of the second launch

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }

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

// A 16-byte piece as pairs of floats, NaN turned into -inf (the maximum with -inf
// drops NaN), and back with one rounding.
template <typename T> struct Pairs;
template <> struct Pairs<float> {
  static constexpr int kElems = 4;
  static __device__ __forceinline__ uint4 clean(uint4 u) {
    const auto f = [](uint32_t w) { return __float_as_uint(fmaxf(__uint_as_float(w), -INFINITY)); };
    return make_uint4(f(u.x), f(u.y), f(u.z), f(u.w));
  }
  static __device__ __forceinline__ float max(uint4 u) {
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
  static __device__ __forceinline__ void split(uint4 u, float2 (&x)[2]) {
    x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 join(const float2 (&x)[2]) {
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x), __float_as_uint(x[1].y));
  }
};
template <typename H2>
struct Pairs16 {
  static constexpr int kElems = 8;
  static __device__ __forceinline__ H2 as(uint32_t w) { return *reinterpret_cast<const H2*>(&w); }
  static __device__ __forceinline__ uint32_t bits(H2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
};
template <> struct Pairs<__nv_bfloat16> : Pairs16<__nv_bfloat162> {
  static __device__ __forceinline__ uint4 clean(uint4 u) {
    const __nv_bfloat162 low = as(0xFF80FF80u);
    return make_uint4(bits(__hmax2(as(u.x), low)), bits(__hmax2(as(u.y), low)), bits(__hmax2(as(u.z), low)),
                      bits(__hmax2(as(u.w), low)));
  }
  static __device__ __forceinline__ float max(uint4 u) {
    const __nv_bfloat162 m = __hmax2(__hmax2(as(u.x), as(u.y)), __hmax2(as(u.z), as(u.w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ void split(uint4 u, float2 (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint4 join(const float2 (&x)[4]) {
    return make_uint4(bits(__float22bfloat162_rn(x[0])), bits(__float22bfloat162_rn(x[1])),
                      bits(__float22bfloat162_rn(x[2])), bits(__float22bfloat162_rn(x[3])));
  }
};
template <> struct Pairs<__half> : Pairs16<__half2> {
  static __device__ __forceinline__ uint4 clean(uint4 u) {
    const __half2 low = as(0xFC00FC00u);
    return make_uint4(bits(__hmax2(as(u.x), low)), bits(__hmax2(as(u.y), low)), bits(__hmax2(as(u.z), low)),
                      bits(__hmax2(as(u.w), low)));
  }
  static __device__ __forceinline__ float max(uint4 u) {
    const __half2 m = __hmax2(__hmax2(as(u.x), as(u.y)), __hmax2(as(u.z), as(u.w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ void split(uint4 u, float2 (&x)[4]) {
    x[0] = __half22float2(as(u.x)); x[1] = __half22float2(as(u.y));
    x[2] = __half22float2(as(u.z)); x[3] = __half22float2(as(u.w));
  }
  static __device__ __forceinline__ uint4 join(const float2 (&x)[4]) {
    return make_uint4(bits(__float22half2_rn(x[0])), bits(__float22half2_rn(x[1])), bits(__float22half2_rn(x[2])),
                      bits(__float22half2_rn(x[3])));
  }
};

// A lane's NP pieces of a row, and their load element by element; past G they are `fill`.
template <typename T, int LPR, int NP>
struct Row {
  static constexpr int E = Pairs<T>::kElems;
  uint4 u[NP];
  __device__ __forceinline__ void load(const T* row, int64_t cs, int lane, int G, float fill) {
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      const int c0 = (q * LPR + lane) * E;
      __align__(16) T e[E];
#pragma unroll
      for (int j = 0; j < E; ++j) e[j] = c0 + j < G ? row[(c0 + j) * cs] : from_f32<T>(fill);
      u[q] = *reinterpret_cast<const uint4*>(e);
    }
  }
};

// e = exp(l - max) of a row's logits, in pairs; returns 1 / sum, or 0 for a row
// without an expert that can be picked.  The difference is rounded once and the
// function is off by 2 ulp and by |l - max| 2^-23.  A maximum of +inf takes the
// limit: 1 for the logits that reach it.
template <typename T, int LPR, int NP>
__device__ __forceinline__ float softmax_row(const Row<T, LPR, NP>& r, float2 (&e)[NP][Pairs<T>::kElems / 2]) {
  constexpr int H = Pairs<T>::kElems / 2;
  float top = -INFINITY;
  uint4 c[NP];
#pragma unroll
  for (int q = 0; q < NP; ++q) {
    c[q] = Pairs<T>::clean(r.u[q]);
    top = fmaxf(top, Pairs<T>::max(c[q]));
  }
  top = lanes_max<LPR>(top);
  const float base = top > -INFINITY ? top : 0.f;      // nothing to pick: exp(-inf - 0) = 0
  float2 sum = twice(0.f);
#pragma unroll
  for (int q = 0; q < NP; ++q) {
    float2 x[H];
    Pairs<T>::split(c[q], x);
#pragma unroll
    for (int j = 0; j < H; ++j) {
      const float2 d = mul2(add2(x[j], twice(-base)), twice(1.44269504f));
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[q][j].x) : "f"(d.x));
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[q][j].y) : "f"(d.y));
      sum = add2(sum, e[q][j]);
    }
  }
  if (base == INFINITY) {                              // rare: inf - inf above
    sum = twice(0.f);
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      float2 x[H];
      Pairs<T>::split(c[q], x);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        e[q][j] = make_float2(x[j].x == INFINITY ? 1.f : 0.f, x[j].y == INFINITY ? 1.f : 0.f);
        sum = add2(sum, e[q][j]);
      }
    }
  }
  const float s = lanes_sum<LPR>(sum.x + sum.y);
  return s > 0.f ? __fdividef(1.f, s) : 0.f;           // 1 <= s <= G
}

// A lane's queue of row pieces: kAhead rows are on their way while one is worked on.
// ASYNC (rows of whole aligned pieces): through the lane's own places in shared
// memory; otherwise each row is loaded when its turn comes.
template <int NP> constexpr int kAhead = NP <= 2 ? 6 : NP <= 4 ? 3 : 2;     // 48 to 64 KB a block
template <typename T, int LPR, int NP, bool ASYNC>
struct Queue {
  const T* base;
  int64_t rs, cs, rows;
  int lane, G;
  float fill;
  uint32_t place;                                // this lane's first place
  static constexpr int kBytes = kThreads * NP * 16 * kAhead<NP>;     // of a block
  __device__ __forceinline__ Queue(const void* p, int64_t rs_, int64_t cs_, int64_t rows_, int lane_, int G_, float fill_, uint8_t* sm)
      : base(static_cast<const T*>(p)), rs(rs_), cs(cs_), rows(rows_), lane(lane_), G(G_), fill(fill_),
        place(ptx::smem_u32(sm) + threadIdx.x * 16) {}
  __device__ __forceinline__ uint32_t at(int slot, int q) const { return place + (uint32_t)((slot * NP + q) * kThreads * 16); }
  __device__ __forceinline__ void issue(int64_t r, int slot) const {
    if (ASYNC) {
      if (r < rows) {
#pragma unroll
        for (int q = 0; q < NP; ++q) {
          const int c0 = (q * LPR + lane) * Pairs<T>::kElems;
          if (c0 < G)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at(slot, q)), "l"(base + r * rs + c0) : "memory");
        }
      }
    }
  }
  __device__ __forceinline__ void take(int64_t r, int slot, Row<T, LPR, NP>& row) const {
    if (ASYNC) {
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        const int c0 = (q * LPR + lane) * Pairs<T>::kElems;
        __align__(16) T e[Pairs<T>::kElems];
#pragma unroll
        for (int j = 0; j < Pairs<T>::kElems; ++j) e[j] = from_f32<T>(fill);
        row.u[q] = c0 < G && r < rows ? ptx::lds128(at(slot, q)) : *reinterpret_cast<const uint4*>(e);
      }
    } else {
      row.load(base + (r < rows ? r : 0) * rs, cs, lane, G, fill);
    }
  }
};
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int NP>
__device__ __forceinline__ void async_wait_oldest() { asm volatile("cp.async.wait_group %0;" ::"n"(kAhead<NP> - 1) : "memory"); }

// Partials of a block: psum [G] f32, then picks [G] i32, then rows that take
// part and picks in all.
template <typename T, int LPR, int NP, bool ASYNC>
__global__ void __launch_bounds__(kThreads, 2) balance_partial_kernel(const BalanceArgs a, float* psum, int32_t* cnt,
                                                                      unsigned* status) {
  pdl_begin();
  extern __shared__ __align__(16) uint8_t raw[];               // the queue, then [kWarps][G] column sums, [G + 2] counts
  using Q = Queue<T, LPR, NP, ASYNC>;
  float* sh = reinterpret_cast<float*>(raw + (ASYNC ? Q::kBytes : 0));
  int32_t* hist = reinterpret_cast<int32_t*>(sh + kWarps * a.G);
  constexpr int E = Pairs<T>::kElems, H = E / 2;
  const int G = (int)a.G, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < G + 2; i += kThreads) hist[i] = 0;
  __syncthreads();
  constexpr int kPerWarp = 32 / LPR;
  const int sub = lane / LPR, l = lane % LPR;
  const int64_t step = (int64_t)gridDim.x * kWarps * kPerWarp;
  int64_t r = ((int64_t)blockIdx.x * kWarps + warp) * kPerWarp + sub;
  const Q queue(a.logits, a.l_rs, a.l_cs, a.rows, l, G, -INFINITY, raw);
#pragma unroll
  for (int k = 0; k < kAhead<NP>; ++k) {                           // the first rows arrive while the picks are counted
    queue.issue(r + k * step, k);
    async_commit();
  }
  int mine = 0;
  bool bad = false;
  const int64_t picks = a.rows * a.k;
#pragma unroll 4
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
  float2 acc[NP][H];
#pragma unroll
  for (int q = 0; q < NP; ++q)
#pragma unroll
    for (int j = 0; j < H; ++j) acc[q][j] = twice(0.f);
  int alive = 0;
  int slot = 0;
  for (; r - sub < a.rows; r += step) {
    Row<T, LPR, NP> row;
    async_wait_oldest<NP>();
    queue.take(r, slot, row);
    float2 e[NP][H];
    const bool live = r < a.rows;
    const float inv = softmax_row<T, LPR, NP>(row, e);
    const float2 w = twice(live ? inv : 0.f);
    alive += live && inv > 0.f && l == 0;
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int j = 0; j < H; ++j) acc[p][j] = ptx::fma2_rn(e[p][j], w, acc[p][j]);
    queue.issue(r + kAhead<NP> * step, slot);                      // the place has been read
    async_commit();
    if (++slot == kAhead<NP>) slot = 0;
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
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int j = 0; j < H; ++j) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {                     // the warp's row groups
        acc[p][j].x += __shfl_xor_sync(0xffffffffu, acc[p][j].x, o);
        acc[p][j].y += __shfl_xor_sync(0xffffffffu, acc[p][j].y, o);
      }
      const int c = (p * LPR + l) * E + 2 * j;
      if (sub == 0 && c < G) sh[warp * G + c] = acc[p][j].x;
      if (sub == 0 && c + 1 < G) sh[warp * G + c + 1] = acc[p][j].y;
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
  pdl_begin();
  __shared__ float part[32];
  __shared__ int tot[2][32];
  __shared__ float mine;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = (int)ptx::cluster_ctarank();
  // 32 neighbouring columns at a time: lane = column for the reads, warps share the blocks.
  __shared__ float ps[32][33];
  __shared__ int cs[32][33];
  float s;
  int n;
  const auto add_up = [&](int c0) {
    s = 0.f;
    n = 0;
    if (c0 + lane < G) {
#pragma unroll 10
      for (int b = warp; b < nb; b += 32) {
        s += __ldg(psum + (int64_t)b * G + c0 + lane);
        n += __ldg(cnt + (int64_t)b * (G + 2) + c0 + lane);
      }
    }
  };
  // Rows and picks in all: every block adds them for itself.
  int rows = 0, picks = 0;
  for (int b = threadIdx.x; b < nb; b += 1024) {
    rows += __ldg(cnt + (int64_t)b * (G + 2) + G);
    picks += __ldg(cnt + (int64_t)b * (G + 2) + G + 1);
  }
  add_up(rank * 32);
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
  float lsum = 0.f;
  for (int c0 = rank * 32; c0 < G; c0 += kFinalBlocks * 32) {
    if (c0 != rank * 32) add_up(c0);
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

template <typename T, int LPR, int NP, bool BASE, bool ASYNC>
__global__ void __launch_bounds__(kThreads, 2) balance_grad_kernel(const BalanceGradArgs a, const int ovec) {
  pdl_begin();
  extern __shared__ __align__(16) uint8_t raw[];               // the queues
  constexpr int E = Pairs<T>::kElems, H = E / 2;
  constexpr int kPerWarp = 32 / LPR;
  const int G = (int)a.G, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / LPR, l = lane % LPR;
  T* out = static_cast<T*>(a.out);
  const int64_t step = (int64_t)gridDim.x * kWarps * kPerWarp;
  int64_t r = ((int64_t)blockIdx.x * kWarps + warp) * kPerWarp + sub;
  using Q = Queue<T, LPR, NP, ASYNC>;
  const Q queue(a.logits, a.l_rs, a.l_cs, a.rows, l, G, -INFINITY, raw);
  const Q add(a.base, a.b_rs, a.b_cs, a.rows, l, G, 0.f, raw + (ASYNC ? Q::kBytes : 0));
#pragma unroll
  for (int k = 0; k < kAhead<NP>; ++k) {
    queue.issue(r + k * step, k);
    if (BASE) add.issue(r + k * step, k);
    async_commit();
  }
  // The shares c / C of this lane's columns; a row's lanes hold all of them.
  float2 share[NP][H];
  int total = 0;
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int j = 0; j < H; ++j) {
      const int c = (p * LPR + l) * E + 2 * j;
      const int n0 = c < G ? __ldg(a.counts + c * a.counts_s) : 0, n1 = c + 1 < G ? __ldg(a.counts + (c + 1) * a.counts_s) : 0;
      total += n0 + n1;
      share[p][j] = make_float2((float)n0, (float)n1);
    }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int rows_in = __ldg(a.counts + G * a.counts_s);
  const float scale = total > 0 ? 1.f / (float)total : 0.f;
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int j = 0; j < H; ++j) share[p][j] = mul2(share[p][j], twice(scale));
  const float coef = rows_in > 0 ? __ldg(a.dloss) * ((float)G / (float)rows_in) : 0.f;
  int slot = 0;
  for (; r - sub < a.rows; r += step) {
    Row<T, LPR, NP> row, other;
    async_wait_oldest<NP>();
    queue.take(r, slot, row);
    if (BASE) add.take(r, slot, other);
    float2 e[NP][H];
    const float inv = softmax_row<T, LPR, NP>(row, e);
    float2 dots = twice(0.f);
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int j = 0; j < H; ++j) dots = ptx::fma2_rn(share[p][j], e[p][j], dots);
    const float dot = lanes_sum<LPR>(dots.x + dots.y) * inv;
    const float2 w = twice(inv * coef), nd = twice(-dot);
    T* dst = out + r * (int64_t)G;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      float2 v[H];
      if (BASE) Pairs<T>::split(other.u[p], v);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        const float2 k = mul2(e[p][j], w), d = add2(share[p][j], nd);
        v[j] = BASE ? ptx::fma2_rn(k, d, v[j]) : mul2(k, d);
      }
      const uint4 o = Pairs<T>::join(v);
      const int c0 = (p * LPR + l) * E;
      if (r < a.rows) {
        if (ovec && c0 + E <= G) {
          *reinterpret_cast<uint4*>(dst + c0) = o;
        } else {
#pragma unroll
          for (int j = 0; j < E; ++j)
            if (c0 + j < G) dst[c0 + j] = reinterpret_cast<const T*>(&o)[j];
        }
      }
    }
    queue.issue(r + kAhead<NP> * step, slot);                      // the places have been read
    if (BASE) add.issue(r + kAhead<NP> * step, slot);
    async_commit();
    if (++slot == kAhead<NP>) slot = 0;
  }
}

template <typename T>
int vec_ok(const void* p, int64_t rs, int64_t cs) {
  return cs == 1 && (rs * sizeof(T)) % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

// Lanes per row and 16-byte pieces per lane for G experts: 8 lanes with up to 16
// columns each, then more lanes; 32 columns a lane (from 513 experts on) leave
// registers for one row at a time.
template <typename T, typename F>
mm_status by_width(int64_t G, F&& f) {
  constexpr int kSixteen = 16 / Pairs<T>::kElems;      // pieces of 16 columns
#define QG_WIDTH(LPR, NP) \
  if (G <= LPR * NP * Pairs<T>::kElems) return f(std::integral_constant<int, LPR>(), std::integral_constant<int, NP>())
  QG_WIDTH(8, kSixteen / 2);
  QG_WIDTH(8, kSixteen);
  QG_WIDTH(16, kSixteen);
  QG_WIDTH(32, kSixteen);
  QG_WIDTH(32, 2 * kSixteen);
#undef QG_WIDTH
  return MM_ERR_UNSUPPORTED;
}

// Blocks for `rows` rows: enough for one round of kRows rows a warp, at most `per_sm` per SM.
int64_t row_blocks(int64_t rows, int rows_per_block, int per_sm) {
  const int64_t want = (rows + rows_per_block - 1) / rows_per_block, most = (int64_t)sm_count_public() * per_sm;
  return want < 1 ? 1 : want < most ? want : most;
}

constexpr int kPartialPerSm = 2, kGradPerSm = 2;

template <typename T, typename K, typename... A>
mm_status launch_queued(K kernel, int64_t blocks, size_t smem, cudaStream_t stream, A... args) {
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return MM_ERR_CUDA;
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), smem, stream, args...) == cudaSuccess ? MM_OK : MM_ERR_CUDA;
}

template <typename T>
mm_status run_partial(const BalanceArgs& a, void* ws, unsigned* status, cudaStream_t stream) {
  const int64_t nb = balance_partial_blocks(a.rows);
  float* psum = static_cast<float*>(ws);
  int32_t* cnt = reinterpret_cast<int32_t*>(psum + nb * a.G);
  const size_t sums = (size_t)(kWarps * a.G + a.G + 2) * 4;
  const bool async = vec_ok<T>(a.logits, a.l_rs, a.l_cs) && a.G % Pairs<T>::kElems == 0;
  return by_width<T>(a.G, [&](auto lpr, auto v) {
    constexpr int L = decltype(lpr)::value, P = decltype(v)::value;
    return async ? launch_queued<T>(balance_partial_kernel<T, L, P, true>, nb, sums + Queue<T, L, P, true>::kBytes, stream, a,
                                    psum, cnt, status)
                 : launch_queued<T>(balance_partial_kernel<T, L, P, false>, nb, sums, stream, a, psum, cnt, status);
  });
}

template <typename T>
mm_status run_grad(const BalanceGradArgs& a, cudaStream_t stream) {
  const int ov = vec_ok<T>(a.out, a.G, 1);
  const bool async = vec_ok<T>(a.logits, a.l_rs, a.l_cs) && a.G % Pairs<T>::kElems == 0 &&
                     (!a.base || vec_ok<T>(a.base, a.b_rs, a.b_cs));
  return by_width<T>(a.G, [&](auto lpr, auto v) {
    constexpr int L = decltype(lpr)::value, P = decltype(v)::value;
    const int64_t nb = row_blocks(a.rows, kWarps * (32 / L), kGradPerSm);
    const size_t q = async ? Queue<T, L, P, true>::kBytes : 0;
    if (a.base)
      return async ? launch_queued<T>(balance_grad_kernel<T, L, P, true, true>, nb, 2 * q, stream, a, ov)
                   : launch_queued<T>(balance_grad_kernel<T, L, P, true, false>, nb, 0, stream, a, ov);
    return async ? launch_queued<T>(balance_grad_kernel<T, L, P, false, true>, nb, q, stream, a, ov)
                 : launch_queued<T>(balance_grad_kernel<T, L, P, false, false>, nb, 0, stream, a, ov);
  });
}

}  // namespace

// A block takes 32 rows at least, so that a few rows leave few partials to add.
int64_t balance_partial_blocks(int64_t rows) { return row_blocks(rows, 32, kPartialPerSm); }

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
