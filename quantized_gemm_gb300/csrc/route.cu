// Top-k routing of tokens to experts (mm_route_topk) and its gradient.
//
// For a row of logits l over G experts, p_i = exp(l_i - max) / sum_j exp(l_j -
// max); the k largest logits are picked (ties to the lowest index) with weight
// p_i, or p_i over the picked p's sum.  A NaN or -inf logit is an expert that
// cannot be picked; it takes no part in the sums.  A +inf maximum takes the
// limit: equal shares among the +inf logits.
//
// A row belongs to LPR neighbouring lanes of a warp, lane i holding logits
// [i*V, (i+1)*V) in registers, so a row is read once.  Logits become unsigned
// keys in the same order (0: cannot be picked); each of the k rounds takes the
// group's largest key, and among the lanes holding it the lowest lane and
// within it the lowest position, which is the lowest index.
#include "kernels.h"

namespace qg {

namespace {

constexpr int kRouteThreads = 128;

// Unsigned keys in the order of the floats, 0 for NaN and -inf.  Adding +0
// makes -0 a +0, so that the two tie.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.f));
  if (!(x > -INFINITY)) return 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
// exp(l - top) for l <= top, with the limit for an infinite top.
__device__ __forceinline__ float share(float l, float top) { return l == top ? 1.f : expf(l - top); }

template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LPR>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Logits [lane*V, lane*V + V) of a row as floats (-inf past the end).
template <typename T, int V>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t row, int lane, int vec, float (&l)[V]) {
  const T* src = static_cast<const T*>(a.logits) + row * a.l_rs;
  constexpr int kPer = 16 / sizeof(T);
  if constexpr (V % kPer == 0) {
    if (vec && (int64_t)(lane + 1) * V <= a.G) {
#pragma unroll
      for (int q = 0; q < V / kPer; ++q) {
        const uint4 u = *reinterpret_cast<const uint4*>(src + lane * V + q * kPer);
        const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int j = 0; j < kPer; ++j) l[q * kPer + j] = to_f32(e[j]);
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t i = (int64_t)lane * V + j;
    l[j] = i < a.G ? to_f32(src[i * a.l_cs]) : -INFINITY;
  }
}

template <typename T, int LPR, int V>
__global__ void __launch_bounds__(kRouteThreads) route_topk_kernel(const RouteArgs a, const int vec) {
  pdl_begin();
  constexpr int kRows = kRouteThreads / LPR;
  const int lane = threadIdx.x % LPR, shift = (threadIdx.x & 31) / LPR * LPR;
  const unsigned gmask = (LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u)) << shift;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / LPR;
  const bool live = row < a.rows;
  float l[V];
  uint32_t key[V];
  load_logits<T, V>(a, live ? row : 0, lane, vec, l);
#pragma unroll
  for (int j = 0; j < V; ++j) key[j] = order_key(l[j]);
  float top = 0.f, sum = 0.f, mine = 0.f;
  int pick = -1;
#pragma unroll 1
  for (int r = 0; r < (int)a.k; ++r) {
    uint32_t best = key[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < V; ++j)
      if (key[j] > best) { best = key[j]; at = j; }
    const uint32_t m = group_max<LPR>(best);
    const int win = __ffs(__ballot_sync(0xffffffffu, best == m) & gmask) - 1 - shift;   // lowest lane of the group
    const int wat = __shfl_sync(0xffffffffu, at, win, LPR);
    if (r == 0) {
      top = m ? key_value(m) : 0.f;
      if (!a.normalize) {
#pragma unroll
        for (int j = 0; j < V; ++j) sum += key[j] ? share(l[j], top) : 0.f;
        sum = group_sum<LPR>(sum);
      }
    }
    if (lane == win) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j == wat) key[j] = 0u;
    }
    const float e = m ? share(key_value(m), top) : 0.f;
    if (a.normalize) sum += e;
    if (lane == r) {
      pick = m ? win * V + wat : -1;
      mine = e;
    }
  }
  if (live && lane < a.k) {
    static_cast<int32_t*>(a.indices)[row * a.k + lane] = pick;
    static_cast<float*>(a.weights)[row * a.k + lane] = pick >= 0 ? mine / sum : 0.f;
  }
}

// 16-bit logits: the key (16 bits) and the index fit one unsigned word, key
// above 0xFFFF - index, so that plain integer maxima order by logit and then by
// lowest index.  Each lane sorts its V words once (descending, by a merging
// network of min / max pairs); a round is then one maximum over the row's
// lanes, and the lane that holds it moves its list up.  65536 rows of 256
// bf16 logits, 8 picks: 22 us against 54 us for the form above, which searches
// all V keys of a lane in every round; bound by the integer compare and select
// instructions (issue slots 72 % busy, the integer pipe the limit), not by the
// 38 MB (5.6 us) it moves.
template <typename T> struct Bits16;
template <> struct Bits16<__nv_bfloat16> {
  using Pair = __nv_bfloat162;
  static constexpr uint32_t kInf = 0x7F80u;
};
template <> struct Bits16<__half> {
  using Pair = __half2;
  static constexpr uint32_t kInf = 0x7C00u;
};

// Descending order by Batcher's odd-even merging (V a power of two).
template <int V>
__device__ __forceinline__ void sort_descending(uint32_t (&w)[V]) {
#pragma unroll
  for (int p = 1; p < V; p <<= 1)
#pragma unroll
    for (int k = p; k >= 1; k >>= 1)
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t hi = max(w[i + j], w[i + j + k]), lo = min(w[i + j], w[i + j + k]);
            w[i + j] = hi;
            w[i + j + k] = lo;
          }
}

template <typename T, int V>
__device__ __forceinline__ void load_raw(const RouteArgs& a, int64_t row, int lane, int vec, uint32_t (&raw)[V / 2]) {
  const uint16_t* src = static_cast<const uint16_t*>(a.logits) + row * a.l_rs;
  if (vec && (int64_t)(lane + 1) * V <= a.G) {
#pragma unroll
    for (int q = 0; q < V / 8; ++q) {
      const uint4 u = *reinterpret_cast<const uint4*>(src + lane * V + q * 8);
      raw[4 * q] = u.x; raw[4 * q + 1] = u.y; raw[4 * q + 2] = u.z; raw[4 * q + 3] = u.w;
    }
  } else {
    constexpr uint32_t kMinusInf = 0x8000u | Bits16<T>::kInf;
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      const int64_t i = (int64_t)lane * V + 2 * j;
      const uint32_t lo = i < a.G ? src[i * a.l_cs] : kMinusInf, hi = i + 1 < a.G ? src[(i + 1) * a.l_cs] : kMinusInf;
      raw[j] = lo | hi << 16;
    }
  }
}

// Persistent: a block walks groups of kRows rows, the next one's logits read
// while it picks from the current one's.
// UNROLL: at most 8 picks; the rounds are unrolled and round r moves up only
// the places that later rounds can still reach.
template <typename T, int LPR, int V, bool UNROLL>
__global__ void __launch_bounds__(kRouteThreads) route_topk16_kernel(const RouteArgs a, const int vec) {
  pdl_begin();
  using Pair = typename Bits16<T>::Pair;
  constexpr uint32_t kNone = ((~(0x8000u | Bits16<T>::kInf)) & 0xFFFFu) << 16 | 0xFFFFu;   // -inf's key and below
  constexpr int kRows = kRouteThreads / LPR;
  const int lane = threadIdx.x % LPR;
  const int64_t step = (int64_t)gridDim.x * kRows;
  uint32_t next[V / 2];
  int64_t first = (int64_t)blockIdx.x * kRows;
  load_raw<T, V>(a, min(first + threadIdx.x / LPR, a.rows - 1), lane, vec, next);
  for (; first < a.rows; first += step) {
    const int64_t row = first + threadIdx.x / LPR;
    const bool live = row < a.rows;
    uint32_t raw[V / 2];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) raw[j] = next[j];
    if (first + step < a.rows) load_raw<T, V>(a, min(row + step, a.rows - 1), lane, vec, next);
    uint32_t w[V];
    const uint32_t low = 0xFFFFu - (uint32_t)(lane * V);   // no borrow below: the row's indices are < 2^16
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      // -0 + 0 is +0; the maximum of a NaN and -inf is -inf
      Pair x = *reinterpret_cast<const Pair*>(&raw[j]);
      const uint32_t ninf2 = (0x8000u | Bits16<T>::kInf) * 0x10001u, zero2 = 0u;
      x = __hmax2(__hadd2_rn(x, *reinterpret_cast<const Pair*>(&zero2)), *reinterpret_cast<const Pair*>(&ninf2));
      raw[j] = *reinterpret_cast<const uint32_t*>(&x);
      // both keys of the pair: all bits of a negative value flipped, the sign of a positive one
      const uint32_t key = raw[j] ^ (((raw[j] >> 15) & 0x00010001u) * 0x7FFFu | 0x80008000u);
      w[2 * j] = __byte_perm(key, low, 0x1054) - 2 * j;
      w[2 * j + 1] = __byte_perm(key, low, 0x3254) - (2 * j + 1);
    }
    sort_descending<V>(w);
    uint32_t mine = 0u, top = 0u;
    auto best = [&]() { return LPR == 32 ? __reduce_max_sync(0xffffffffu, w[0]) : group_max<LPR>(w[0]); };
    if constexpr (UNROLL) {
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (r >= (int)a.k) break;
        const uint32_t m = best();
        if (r == 0) top = m;
        if (lane == r) mine = m;
        const bool pop = w[0] == m;
#pragma unroll
        for (int j = 0; j < V && j < 7 - r; ++j) w[j] = pop ? (j + 1 < V ? w[j + 1] : 0u) : w[j];
      }
    } else {
#pragma unroll 1
      for (int r = 0; r < (int)a.k; ++r) {
        const uint32_t m = best();
        if (r == 0) top = m;
        if (lane == r) mine = m;
        const bool pop = w[0] == m;
#pragma unroll
        for (int j = 0; j + 1 < V; ++j) w[j] = pop ? w[j + 1] : w[j];
        w[V - 1] = pop ? 0u : w[V - 1];
      }
    }
    auto value = [](uint32_t word) {                        // the logit behind a word
      const uint32_t k = word & 0xFFFF0000u;
      const uint16_t b = (uint16_t)(((k & 0x80000000u) ? k ^ 0x80000000u : ~k) >> 16);
      return to_f32(*reinterpret_cast<const T*>(&b));
    };
    const bool some = top > kNone, ok = mine > kNone;
    const float tv = some ? value(top) : 0.f;
    const float e = ok ? share(value(mine), tv) : 0.f;
    float sum;
    if (a.normalize) {
      sum = group_sum<LPR>(e);
    } else {
      sum = 0.f;
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const T* x = reinterpret_cast<const T*>(&raw[j]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float l = to_f32(x[h]);
          sum += some && l > -INFINITY ? share(l, tv) : 0.f;
        }
      }
      sum = group_sum<LPR>(sum);
    }
    if (live && lane < a.k) {
      static_cast<int32_t*>(a.indices)[row * a.k + lane] = ok ? (int32_t)(0xFFFFu - (mine & 0xFFFFu)) : -1;
      static_cast<float*>(a.weights)[row * a.k + lane] = ok ? e / sum : 0.f;
    }
  }
}

// Gradient of the weights with respect to the logits, the weights recomputed
// from the logits.  With q the weights scattered over the experts (normalised)
// or the softmax (not), d the given gradient scattered likewise:
// dl_i = q_i (d_i - sum_j q_j d_j), for the normalised form only on the picks
// (q is 0 elsewhere).
template <typename T, int LPR, int V>
__global__ void __launch_bounds__(kRouteThreads)
    route_topk_grad_kernel(const RouteArgs a, const int vec, const int ovec, unsigned* status) {
  pdl_begin();
  constexpr int kRows = kRouteThreads / LPR;
  const int lane = threadIdx.x % LPR;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / LPR;
  const bool live = row < a.rows;
  const int64_t rr = live ? row : 0;
  float l[V], d[V];
  load_logits<T, V>(a, rr, lane, vec, l);
  int64_t my_i = -1;
  float my_d = 0.f;
  if (lane < a.k) {
    my_i = load_index(a.indices, rr * a.i_rs + lane * a.i_cs, a.ind64);
    if (my_i < -1 || my_i >= a.G) {
      if (live) atomicOr(status, kStatusIndexRange);
      my_i = -1;
    }
    if (my_i >= 0) my_d = static_cast<const float*>(a.gw)[rr * a.gw_rs + lane * a.gw_cs];
  }
  uint32_t best = 0u, picked = 0u;
#pragma unroll
  for (int j = 0; j < V; ++j) d[j] = 0.f;
  static_assert(V <= 32, "one bit per logit of a lane");
#pragma unroll 1
  for (int r = 0; r < (int)a.k; ++r) {
    const int i = __shfl_sync(0xffffffffu, (int)my_i, r, LPR);
    const float g = __shfl_sync(0xffffffffu, my_d, r, LPR);
    const int at = i - lane * V;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (i >= 0 && j == at) { d[j] += g; picked |= 1u << j; }
  }
  // The maximum of the logits that take part in the sum: the picks' own for the
  // normalised form, since a larger logit need not be among the picks given.
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (!a.normalize || ((picked >> j) & 1u)) best = max(best, order_key(l[j]));
  const uint32_t m = group_max<LPR>(best);
  const float top = m ? key_value(m) : 0.f;
  float sum = 0.f, dot = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const bool in = order_key(l[j]) != 0u && (!a.normalize || ((picked >> j) & 1u));
    l[j] = in ? share(l[j], top) : 0.f;
    sum += l[j];
  }
  sum = group_sum<LPR>(sum);
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    l[j] *= inv;
    dot += l[j] > 0.f ? l[j] * d[j] : 0.f;
  }
  dot = group_sum<LPR>(dot);
#pragma unroll
  for (int j = 0; j < V; ++j) l[j] = l[j] > 0.f ? l[j] * (d[j] - dot) : 0.f;
  if (!live) return;
  T* dst = static_cast<T*>(a.out) + row * a.G;
  constexpr int kPer = 16 / sizeof(T);
  if constexpr (V % kPer == 0) {
    if (ovec && (int64_t)(lane + 1) * V <= a.G) {
#pragma unroll
      for (int q = 0; q < V / kPer; ++q) {
        uint4 u;
        T* e = reinterpret_cast<T*>(&u);
#pragma unroll
        for (int j = 0; j < kPer; ++j) e[j] = from_f32<T>(l[q * kPer + j]);
        *reinterpret_cast<uint4*>(dst + lane * V + q * kPer) = u;
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
    if ((int64_t)lane * V + j < a.G) dst[(int64_t)lane * V + j] = from_f32<T>(l[j]);
}

template <typename T, int LPR, int V>
mm_status launch_one(const RouteArgs& a, bool grad, unsigned* status, cudaStream_t stream) {
  const int64_t rows_per_block = kRouteThreads / LPR, blocks = (a.rows + rows_per_block - 1) / rows_per_block;
  if (blocks > 0x7fffffffLL) return MM_ERR_UNSUPPORTED;
  const int per = 16 / (int)sizeof(T);
  const int vec = a.l_cs == 1 && a.l_rs % per == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
  if (!grad) {
    cudaError_t e;
    const int64_t resident = (int64_t)sm_count_public() * (2048 / kRouteThreads);   // blocks that fit the SMs at once
    if constexpr (sizeof(T) == 2)
      e = launch_pdl(a.k <= 8 ? route_topk16_kernel<T, LPR, V, true> : route_topk16_kernel<T, LPR, V, false>,
                     dim3((unsigned)(blocks < resident ? blocks : resident)), dim3(kRouteThreads), 0, stream, a, vec);
    else
      e = launch_pdl(route_topk_kernel<T, LPR, V>, dim3((unsigned)blocks), dim3(kRouteThreads), 0, stream, a, vec);
    return e == cudaSuccess ? MM_OK : MM_ERR_CUDA;
  }
  const int ovec = a.G % per == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
  return launch_pdl(route_topk_grad_kernel<T, LPR, V>, dim3((unsigned)blocks), dim3(kRouteThreads), 0, stream, a, vec,
                    ovec, status) == cudaSuccess ? MM_OK : MM_ERR_CUDA;
}

// Lanes per row and logits per lane: the fewest lanes that keep a row within
// 8 logits a lane (fewer lanes per row mean fewer shuffle steps per round),
// at least one lane per pick.
template <typename T>
mm_status launch_typed(const RouteArgs& a, bool grad, unsigned* status, cudaStream_t stream) {
  if (a.G <= 64 && a.k <= 8) return launch_one<T, 8, 8>(a, grad, status, stream);
  if (a.G <= 128 && a.k <= 16) return launch_one<T, 16, 8>(a, grad, status, stream);
  if (a.G <= 256) return launch_one<T, 32, 8>(a, grad, status, stream);
  if (a.G <= 512) return launch_one<T, 32, 16>(a, grad, status, stream);
  return launch_one<T, 32, 32>(a, grad, status, stream);
}

mm_status launch_any(const RouteArgs& a, bool grad, unsigned* status, cudaStream_t stream) {
  switch (a.dtype) {
    case MM_BF16: return launch_typed<__nv_bfloat16>(a, grad, status, stream);
    case MM_F16: return launch_typed<__half>(a, grad, status, stream);
    default: return launch_typed<float>(a, grad, status, stream);
  }
}

}  // namespace

mm_status launch_route_topk(const RouteArgs& a, cudaStream_t stream) { return launch_any(a, false, nullptr, stream); }

mm_status launch_route_topk_grad(const RouteArgs& a, unsigned* status, cudaStream_t stream) {
  return launch_any(a, true, status, stream);
}

}  // namespace qg
