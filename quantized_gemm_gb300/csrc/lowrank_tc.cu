// Per-row low-rank adapters for many rows (16-bit types): the narrow products
// on mma.sync tensor instructions.
//
// These products are N = R wide (a rank, 4 to 128 or so) and read one large
// matrix once: their bound is memory, at 2 R operations per 2 bytes read, so
// the warp-level instructions are enough and their register operands take any
// row pattern.
//
//   shrink   z[m, r]      = s_g sum_c x[m, c] a[g, c, r]
//   outer    out[g, c, r] = sum over the rows m of adapter g of x[m, c] z[m, r]
//
// and the preparation of the fused product Y[m] = X[m] W + z[m] b[g], in which
// the tcgen05 kernel (tc_gemm.cu, kLowRank) lets each row tile go on, after
// the k-blocks of X W, with one set of k-blocks per adapter that the tile's
// rows name: the rows' z, in two parts (lowrank_two_parts), zeros for the other
// adapters' rows, times that adapter.  The low-rank part then costs ceil(R / 32)
// k-blocks per adapter and tile (one part: ceil(R / 64)) on top of K / 64, and Y
// is written once.  A zero times an infinity or
// a NaN is not zero, so the adapters that the kernel reads are copies with
// their non-finite values set to 0.  What those values add to their own rows,
// and the whole low-rank part of the rows of any adapter past a tile's list
// (per_tile) or past kSlots in all, is written to Y before (lowrank_fix),
// rounded once, and added by the product.
//
// 8192 x 4096 x 14336 with 12 adapters of rank 16 in runs: the product takes
// 540 us (1.79 PFLOP/s; 40 to 50 adapters over its 32 row tiles of 64 k-blocks
// make 2 % more of them) and the call 0.57 to 0.60 ms, against 1.99 ms with the
// low-rank part expanded first and added through C.
#include <cstring>

#include "lowrank.cuh"
#include "tc_ptx.cuh"

namespace qg {

namespace {

// ------------------------------------------------------------------ building blocks

__device__ __forceinline__ uint32_t shared_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x2(uint32_t (&r)[2], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x2_t(uint32_t (&r)[2], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// Asynchronous copy of 16, 8 or 4 bytes, of which the first `valid` come from
// src and the rest are zeros.
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, int valid) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(valid) : "memory");
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  const __half2 c = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&c);
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// One warp's copy of `rows` rows of `len` elements into shared memory with
// `pitch` bytes a row, `per` elements a copy (8, 4 or 2; 1: plain loads);
// zeros past rows_ok rows and len_ok elements (which may end inside a copy).
// A row takes 2^lpr lanes.
template <typename T>
__device__ __forceinline__ void load_block(uint32_t dst, int pitch, const T* src, int64_t ld, int rows, int rows_ok,
                                           int len, int len_ok, int per, int lpr, int lane) {
  const int step = 32 >> lpr, width = 1 << lpr;
  for (int c = (lane & (width - 1)) * per; c < len; c += width * per)
    for (int r = lane >> lpr; r < rows; r += step) {
      const int ok = r < rows_ok ? max(0, min(per, len_ok - c)) : 0;
      const T* s = ok ? src + (int64_t)r * ld + c : src;
      const uint32_t d = dst + (uint32_t)(r * pitch + c * 2);
      if (per == 8) cp_async<16>(d, s, ok * 2);
      else if (per == 4) cp_async<8>(d, s, ok * 2);
      else if (per == 2) cp_async<4>(d, s, ok * 2);
      else {
        const uint16_t v = ok ? *reinterpret_cast<const uint16_t*>(s) : (uint16_t)0;
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(d), "h"(v) : "memory");
      }
    }
}

// ------------------------------------------------------------------ shrink

// A block takes 32 rows x 64 ranks; its 4 warps split c, 64 at a time in
// turn, each with its own ring (no block barrier until the warps' sums meet in
// shared memory): one lane streams 32 x 64 tiles of x by TMA (128-byte
// swizzle), the adapter arrives by asynchronous copies of whatever width its
// alignment allows.  Two blocks per SM (up to 16 ranks) keep 64 KB of x in
// flight.  The tile is multiplied once per adapter that its rows name (rows of
// a request are neighbours, so one or two); each pass keeps its own adapter's
// rows.  Their z goes out in fp32 (the fused product's operands are made of it)
// and, for the adapters' gradients, as two T values (zt).
//
// 8192 rows of 4096, rank 16: 18 us for one factor (67 MB, 3.7 TB/s), 32 us for
// a gradient's two (134 MB, 4.2 TB/s); bound by latency: 256 or 512 blocks of
// some 12 us on 304 places, and half as many bytes again of adapters out of the
// L2.  With one block for both adapters of a tile 27 and 41 us; x staged
// behind block barriers 43 us for one, x straight into the MMA's registers 43
// to 54 us (one block per SM for want of registers).
constexpr int kShRows = 32, kShK = 64, kShWarps = 4, kShThreads = 32 * kShWarps;
constexpr int kShXBytes = kShRows * kShK * 2;
constexpr int kShKPitch = kShK * 2 + 16;
constexpr int kShCtrl = 256;                   // barriers, abort flag

__host__ __device__ constexpr int shrink_a_bytes(bool ck, int rc) {
  return ck ? (rc + 7) / 8 * 8 * kShKPitch : kShK * ((rc + 7) / 8 * 16 + 16);
}
constexpr int kShStages = 3;
// The adapters of a tile's rows are dealt out to 2 to kShParts blocks, so that
// about kShBlocks start: rows in random order name up to 32 adapters a tile,
// and blocks past the tile's adapters end at once.  1024 rows of 4096 x 4096,
// rank 16, 32 adapters, the whole call: random order 89 us against 300 with
// one block a tile, runs 50 against 69 us.
constexpr int kShParts = 16, kShBlocks = 608;
__host__ __device__ constexpr int shrink_red_pitch(int rc) { return (rc + 7) / 8 * 8 + 4; }
// [x rings][control][adapter rings][sums]
__host__ __device__ constexpr int shrink_smem(bool ck, int rc) {
  return 1024 + kShWarps * kShStages * (kShXBytes + shrink_a_bytes(ck, rc)) + kShCtrl +
         kShWarps * kShRows * shrink_red_pitch(rc) * 4;
}

struct ShrinkArgs {
  int ck;                                      // c is a's unit-stride dimension
  int64_t C;
  const void* a; int64_t a_gs, a_ld;
  int per;                                     // elements per copy of the adapter
  float* z; int64_t z_ld;
  uint8_t* wide;
  void* zt; int32_t* zt_exp;
  unsigned long long timeout_ns, teardown_ns;
};

// v as two T values.
template <typename T>
__device__ __forceinline__ void split(float v, float lo_scale, T& hi, T& lo) {
  hi = from_f32<T>(v);
  const float back = to_f32(hi);
  lo = from_f32<T>(fabsf(back) < INFINITY ? (v - back) * lo_scale : 0.f);
}

// 2^k, |k| <= 126; v 2^k, |k| <= 250, by two factors.
__device__ __forceinline__ float pow2(int k) { return __int_as_float((127 + k) << 23); }
__device__ __forceinline__ float times_pow2(float v, int k) { return v * pow2(k / 2) * pow2(k - k / 2); }

// Exponents of f16 rows whose values are all 0 (they scale nothing), or all 0
// or not finite (they must not be scaled to 0).
constexpr int kExpZero = -1000, kExpAny = 1000;

// NT: 8-rank tiles that the accumulators hold.
template <typename T, bool CK, int NT>
__device__ void shrink_tile(const CUtensorMap* tmX, const LowRankArgs& l, const ShrinkArgs& p, int tile, int part, int parts,
                            uint8_t* sm_raw) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t m0 = (int64_t)tile * kShRows, C = p.C;
  const int r0 = blockIdx.y * 64, rc = (int)min((int64_t)64, l.R - r0), nt = (rc + 7) / 8;
  const int rows = (int)min((int64_t)kShRows, l.M - m0);
  constexpr int stages = kShStages;
  const int a_bytes = shrink_a_bytes(CK, rc);
  const int a_pitch = CK ? kShKPitch : nt * 16 + 16;
  const uint32_t raw = shared_u32(sm_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = sm_raw + (base - raw);
  const uint32_t xring = base + (uint32_t)(warp * stages * kShXBytes);
  const uint32_t ctrl = base + (uint32_t)(kShWarps * stages * kShXBytes);
  const uint32_t bar0 = ctrl + (uint32_t)(warp * 32);
  const uint32_t aring = ctrl + kShCtrl + (uint32_t)(warp * stages * a_bytes);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + (ctrl - base) + 240);
  float* red = reinterpret_cast<float*>(sm + (ctrl - base) + kShCtrl + kShWarps * stages * a_bytes);
  const int red_pitch = shrink_red_pitch(rc);
  const int nk = (int)((C + kShK - 1) / kShK);
  const int mine = nk > warp ? (nk - warp + kShWarps - 1) / kShWarps : 0;   // this warp's k-blocks
  int lpr = 0;                                            // 2^lpr lanes per adapter row
  while (lpr < 5 && (p.per << lpr) < (CK ? kShK : rc)) ++lpr;

  if (lane == 0)
    for (int i = 0; i < stages; ++i) ptx::mbar_init(bar0 + 8 * i, 1);
  if (tid == 0) *abort = 0;
  ptx::fence_mbar_init();
  __syncthreads();

  int g_lane = -1;
  if (lane < rows) {
    const int64_t g = load_index(l.idx, (m0 + lane) * l.idx_s, l.ind64);
    if (g >= 0 && g < l.G) g_lane = (int)g;
    else if (g != -1) atomicOr(l.status, kStatusIndexRange);
  }
  unsigned left = __ballot_sync(0xffffffffu, g_lane >= 0);
  T* zt = static_cast<T*>(p.zt);
  __shared__ unsigned row_max[kShRows];                   // largest finite |z| of a row, as bits
  __shared__ int row_wide[kShRows];
  uint32_t done = 0, issued = 0;       // this warp's k-blocks over all passes: stage = count % stages
  uint32_t istage = 0, dstage = 0, dphase = 0;
  bool ok = true;
  for (int pass = 0; left && ok; ++pass) {
    const int g = __shfl_sync(0xffffffffu, g_lane, __ffs(left) - 1);
    const unsigned sel = __ballot_sync(0xffffffffu, g_lane == g);
    left &= ~sel;
    if (pass % parts != part) continue;
    const T* ag = static_cast<const T*>(p.a) + (int64_t)g * p.a_gs;
    auto load = [&](int i) {
      const int64_t c0 = ((int64_t)i * kShWarps + warp) * kShK;
      if (lane == 0) {
        const uint32_t bar = bar0 + 8 * istage;
        ptx::mbar_arrive_expect_tx(bar, kShXBytes);
        ptx::tma_load_3d(xring + istage * kShXBytes, tmX, (int32_t)c0, (int32_t)m0, 0, bar);
      }
      const int cn = (int)min((int64_t)kShK, C - c0);
      const uint32_t s = aring + istage * (uint32_t)a_bytes;
      const T* src = CK ? ag + (int64_t)r0 * p.a_ld + c0 : ag + c0 * p.a_ld + r0;
      const int arows = CK ? rc : kShK, alen = CK ? kShK : rc;
      if (p.per == 8 && cn == kShK && (alen & 7) == 0) {     // whole 16-byte copies
        const int r = lane >> lpr, c = (lane & ((1 << lpr) - 1)) * 8, step = 32 >> lpr;
        const T* q = src + (int64_t)r * p.a_ld + c;
        uint32_t d = s + (uint32_t)(r * a_pitch + c * 2);
        if (c < alen)
          for (int e = r; e < arows; e += step, q += (int64_t)step * p.a_ld, d += (uint32_t)(step * a_pitch))
            cp_async<16>(d, q, 16);
      } else if constexpr (CK) {
        load_block<T>(s, a_pitch, src, p.a_ld, rc, rc, kShK, cn, p.per, lpr, lane);
      } else {
        load_block<T>(s, a_pitch, src, p.a_ld, kShK, cn, rc, rc, p.per, lpr, lane);
      }
      ++issued;
      if (++istage == (uint32_t)stages) istage = 0;
    };
    float acc[2][NT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[h][j][e] = 0.f;
    // stages - 1 blocks ahead: one group of copies per block, empty past the end
    for (int i = 0; i < stages - 1; ++i) {
      if (i < mine) load(i);
      cp_commit();
    }
    for (int i = 0; i < mine; ++i) {
      cp_wait<kShStages - 2>();
      ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar0 + 8 * dstage, dphase, abort, l.status, p.timeout_ns));
      if (!ok) break;
      __syncwarp();                      // block i has landed for every lane, and block i - 1 has been used
      if (i + stages - 1 < mine) load(i + stages - 1);
      cp_commit();
      const uint32_t xs = xring + dstage * kShXBytes, as = aring + dstage * (uint32_t)a_bytes;
#pragma unroll
      for (int k = 0; k < kShK / 16; ++k) {
        uint32_t fa[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = h * 16 + (lane & 15);
          ldsm_x4(fa[h], xs + (uint32_t)(row * 128 + (((k * 2 + (lane >> 4)) ^ (row & 7)) << 4)));
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (j >= nt) break;
          uint32_t fb[2];
          if constexpr (CK)
            ldsm_x2(fb, as + (uint32_t)((j * 8 + (lane & 7)) * a_pitch + k * 32 + ((lane >> 3) & 1) * 16));
          else
            ldsm_x2_t(fb, as + (uint32_t)((k * 16 + (lane & 15)) * a_pitch + j * 16));
#pragma unroll
          for (int h = 0; h < 2; ++h) mma16816<T>(acc[h][j], fa[h], fb);
        }
      }
      ++done;
      if (++dstage == (uint32_t)stages) { dstage = 0; dphase ^= 1; }
    }
    cp_wait<0>();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (j >= nt) break;
        float* q = red + (warp * kShRows + h * 16 + (lane >> 2)) * red_pitch + j * 8 + (lane & 3) * 2;
        q[0] = acc[h][j][0]; q[1] = acc[h][j][1];
        q[8 * red_pitch] = acc[h][j][2]; q[8 * red_pitch + 1] = acc[h][j][3];
      }
    if (tid < kShRows) {
      row_max[tid] = 0u;
      row_wide[tid] = 0;
    }
    ok = __syncthreads_and(ok);
    const float scale = l.scales ? l.scales[g * l.scales_s] : 1.f;
    constexpr bool kScaled = std::is_same<T, __half>::value;
    auto value = [&](int r, int c) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kShWarps; ++w) v += red[(w * kShRows + r) * red_pitch + c];
      return c < rc ? v * scale : 0.f;
    };
    auto put = [&](int r, int c, float v) {
      T hi, lo;
      split<T>(v, 1.f, hi, lo);
      T* q = zt + (m0 + r) * 2 * p.z_ld + r0 + c;
      q[0] = hi;
      q[p.z_ld] = lo;
    };
    for (int i = tid; i < rows * nt * 8; i += kShThreads) {
      const int r = i / (nt * 8), c = i - r * (nt * 8);
      if (!((sel >> r) & 1u)) continue;
      const float v = value(r, c);
      if (p.z) p.z[(m0 + r) * p.z_ld + r0 + c] = v;
      if (!(fabsf(to_f32(from_f32<T>(v))) < INFINITY)) row_wide[r] = 1;
      if (!zt) continue;
      if constexpr (!kScaled) put(r, c, v);
      else if (fabsf(v) < INFINITY) atomicMax(row_max + r, __float_as_uint(fabsf(v)));
    }
    __syncthreads();
    if (kScaled && zt) {
      auto exponent = [&](int r) {                        // -141 to 113
        return row_max[r] ? (int)(row_max[r] >> 23) - (127 + 14) : row_wide[r] ? kExpAny : kExpZero;
      };
      for (int i = tid; i < rows * nt * 8; i += kShThreads) {
        const int r = i / (nt * 8), c = i - r * (nt * 8);
        if ((sel >> r) & 1u) put(r, c, times_pow2(value(r, c), max(-150, min(150, -exponent(r)))));
      }
      if (tid < rows && ((sel >> tid) & 1u)) p.zt_exp[(int64_t)blockIdx.y * l.M + m0 + tid] = exponent(tid);
      __syncthreads();
    }
    if (p.wide && tid < rows && ((sel >> tid) & 1u)) p.wide[(int64_t)blockIdx.y * l.M + m0 + tid] = (uint8_t)row_wide[tid];
  }
  // After a wait that ran out: let the copies still in flight land.
  for (; done != issued; ++done) {
    if (lane == 0) ptx::mbar_wait_teardown(bar0 + 8 * dstage, dphase, p.teardown_ns);
    if (++dstage == (uint32_t)stages) { dstage = 0; dphase ^= 1; }
  }
}

// ------------------------------------------------------------------ rows in adapter order

// Rows in adapter order, a block per adapter: it reads all the indices, marks
// its own rows in a bitmap (a word per 32 rows, in shared memory) and counts
// them and those of lower adapters; then it writes its rows, ascending, at
// their place.  Sums over an adapter's rows therefore have a fixed order.
__device__ void adapter_sort(const LowRankArgs& l, const AdapterRows& t, int g, uint8_t* sm) {
  uint32_t* bits = reinterpret_cast<uint32_t*>(sm);
  __shared__ int own[kShWarps], low[kShWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int words = (int)((l.M + 31) / 32), per = (words + kShWarps - 1) / kShWarps;
  const int w0 = min(words, warp * per), w1 = min(words, w0 + per);
  constexpr int kAhead = 16;                        // index reads in flight
  int n = 0, below = 0;
  for (int w = w0; w < w1; w += kAhead) {
    int64_t v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t m = (int64_t)(w + i) * 32 + lane;
      v[i] = w + i < w1 && m < l.M ? load_index(l.idx, m * l.idx_s, l.ind64) : -1;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const unsigned eq = __ballot_sync(0xffffffffu, v[i] == g);
      below += __popc(__ballot_sync(0xffffffffu, v[i] >= 0 && v[i] < g));
      n += __popc(eq);
      if (lane == 0 && w + i < w1) bits[w + i] = eq;
    }
  }
  if (lane == 0) { own[warp] = n; low[warp] = below; }
  __syncthreads();
  int first = 0, at = 0, all = 0;
  for (int w = 0; w < kShWarps; ++w) {
    first += low[w];
    all += own[w];
    if (w < warp) at += own[w];
  }
  at += first;
  if (tid == 0) {
    t.offset[g] = first;
    if (g == l.G - 1) t.offset[g + 1] = first + all;
  }
  for (int w = w0; w < w1; ++w) {
    const uint32_t b = bits[w];
    if ((b >> lane) & 1u) t.row[at + __popc(b & ((1u << lane) - 1u))] = w * 32 + lane;
    at += __popc(b);
  }
}

// ------------------------------------------------------------------ adapters in use

// One block: the adapters in use, ascending, get slots 0, 1, .. (-1 past kSlots).
__device__ void adapter_slots(const LowRankArgs& l, const FusedTables& t, uint8_t* sm) {
  uint32_t* used = reinterpret_cast<uint32_t*>(sm);      // one bit per adapter
  __shared__ int wsum[kShWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, words = (int)((l.G + 31) / 32);
  for (int i = tid; i < words; i += kShThreads) used[i] = 0u;
  __syncthreads();
#pragma unroll 8
  for (int64_t m = tid; m < l.M; m += kShThreads) {
    const int64_t g = load_index(l.idx, m * l.idx_s, l.ind64);
    if (g >= 0 && g < l.G) atomicOr(used + (g >> 5), 1u << (g & 31));
  }
  __syncthreads();
  const int per = (words + kShThreads - 1) / kShThreads, lo = min(words, tid * per), hi = min(words, lo + per);
  int n = 0;
  for (int i = lo; i < hi; ++i) n += __popc(used[i]);
  int s = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) wsum[warp] = s;
  __syncthreads();
  s -= n;
  for (int w = 0; w < warp; ++w) s += wsum[w];
  for (int i = lo; i < hi; ++i)
    for (uint32_t b = used[i]; b; b &= b - 1, ++s) {
      const int g = i * 32 + __ffs(b) - 1;
      t.slot_of[g] = s < kSlots ? s : -1;
      if (s < kSlots) t.adapter_of[s] = g;
    }
  if (tid == kShThreads - 1) {
    t.head[0] = min(s, kSlots);
    t.head[1] = 0;                                  // rows or adapters left for the fix
  }
  if (tid < kSlots) t.bad[tid] = 0;
}

// The first blocks make the tables that later launches want (they depend on
// the indices alone): slots, then the sorted rows; the others shrink one tile
// each, of the first or the second problem (a gradient's V and U).
template <typename T, int NT>
__global__ void __launch_bounds__(kShThreads, NT <= 4 ? 2 : 1)
    shrink_tiles_kernel(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1,
                        const LowRankArgs l, const __grid_constant__ ShrinkArgs p0,
                        const __grid_constant__ ShrinkArgs p1, const int tiles,
                        const int problems, const int parts, const FusedTables slots, const AdapterRows sort) {
  pdl_begin();
  extern __shared__ __align__(16) uint8_t sm[];
  int tile = (int)blockIdx.x - ((int)gridDim.x - tiles * problems * parts);
  if (tile >= 0) {
    const int part = tile / (tiles * problems);
    tile -= part * tiles * problems;
    const bool second = tile >= tiles;
    const ShrinkArgs& p = second ? p1 : p0;
    const CUtensorMap* tm = second ? &tm1 : &tm0;
    const int t = second ? tile - tiles : tile;
    if (p.ck) shrink_tile<T, true, NT>(tm, l, p, t, part, parts, sm);
    else shrink_tile<T, false, NT>(tm, l, p, t, part, parts, sm);
  } else if (blockIdx.y == 0) {
    const int b = (int)blockIdx.x - (slots.head ? 1 : 0);
    if (b < 0) adapter_slots(l, slots, sm);
    else adapter_sort(l, sort, b, sm);
  }
}

// ------------------------------------------------------------------ outer

// A block sums one chunk (kChunkRows rows of one adapter) for 128 columns of x
// and 64 ranks: out[c, r] += x[m, c] z[m, r], 32 rows a step in a 3-stage
// ring.  An adapter of one chunk is written at once; the others' chunks are
// added, in order, by outer_sum.
//
// z comes in two parts, which meet the same fragments of x in one accumulator.
//
// dA and dB of 8192 rows, 4096 + 4096 columns, rank 16 (134 MB): bf16 36 to 39 us
// (3.7 TB/s), f16 39 us (its rows' scales), 31 us with z rounded once; the row
// gathering and the fragments' loads per 8 KB of x cost more than its four MMAs
// a warp.  A row's 256 bytes as one bulk copy took 85 us.
constexpr int kOutC = 128, kOutRows = 32, kOutStages = 3, kOutThreads = 256;
constexpr int kOutXPitch = kOutC * 2 + 16, kOutZPitch = 2 * 64 * 2 + 16;    // z: 64 ranks' hi, then their lo
constexpr int kOutStage = kOutRows * (kOutXPitch + kOutZPitch);

template <typename T>
struct OuterProblem {
  const T* x; int64_t x_rs, C;
  const T* zt; const int32_t* zt_exp;
  T* out; int64_t o_cs, o_rs;      // out [G, C, R] in the order of these strides
  float* part;
};

// Block bx: 128 columns of the first problem's x (below blocks0) or the second's;
// chunk number `number`, ranks from 64 `group`.
template <typename T>
__device__ void outer_tile(const LowRankArgs& l, const AdapterRows& t, const OuterProblem<T>& p0, const OuterProblem<T>& p1,
                           const int blocks0, const int64_t z_ld, const int bx, const int number, const int group, uint8_t* sm) {
  __shared__ int32_t rows[kChunkRows];
  __shared__ __align__(4) __half factor[kChunkRows];   // f16: what brings a row's z to the chunk's scale
  __shared__ int chunk_exp;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = (int)l.G;
  const OuterProblem<T>& p = bx < blocks0 ? p0 : p1;
  const int64_t C = p.C;
  if (tid == 0) chunk_exp = 2 * kExpZero;
  __shared__ int found;                             // the adapter with first_chunk(g) <= chunk < first_chunk(g + 1)
  for (int h = tid; h < G; h += kOutThreads)
    if (first_chunk(__ldcg(t.offset + h), h) <= number && number < first_chunk(__ldcg(t.offset + h + 1), h + 1))
      found = h;
  __syncthreads();
  if (number >= first_chunk(__ldcg(t.offset + G), G)) return;
  const int g = found, begin = __ldcg(t.offset + g), end = __ldcg(t.offset + g + 1);
  const int chunk = number - first_chunk(begin, g);          // of this adapter
  const int first = begin + chunk * kChunkRows;
  const int n = min(kChunkRows, end - first);
  if (n <= 0) return;
  // f16: row i's z is held divided by 2^e; the sum is taken divided by 2^E, E the
  // chunk's largest e, so a row's z comes in times 2^(e - E), exactly but for the
  // bits that leave f16 at the low end (2^-40 of the largest).  A row whose
  // largest z is less than 2^-24 of the chunk's adds nothing.
  constexpr bool kScaled = std::is_same<T, __half>::value;
  static_assert(kChunkRows == 2 * kOutThreads, "two rows a thread");
  int e[2] = {kExpZero, kExpZero};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = tid + q * kOutThreads;
    if (i >= n) continue;
    const int m = __ldcg(t.row + first + i);
    rows[i] = m;
    if constexpr (kScaled) e[q] = __ldcg(p.zt_exp + (int64_t)group * l.M + m);
  }
  __syncthreads();
  const int64_t c0 = (int64_t)(bx < blocks0 ? bx : bx - blocks0) * kOutC;
  const int cn = (int)min((int64_t)kOutC, C - c0);
  const int r0 = group * 64, rc = (int)min((int64_t)64, l.R - r0), nt = (rc + 7) / 8;
  const uint32_t ring = shared_u32(sm);
  const int steps = (n + kOutRows - 1) / kOutRows;
  // A thread's pieces: 16 bytes of x and of z (lanes 8 to 15 of 16: its lo) in rows tid / 16 and 16 more.
  const int xr = tid >> 4;
  const int x_ok = max(0, min(8, cn - (tid & 15) * 8)) * 2;
  const bool z_in = (tid & 7) < nt;
  const T* xc = p.x + c0 + (x_ok ? (tid & 15) * 8 : 0);
  const T* zc = p.zt + r0 + (z_in ? ((tid >> 3) & 1) * z_ld + (tid & 7) * 8 : 0);
  const uint32_t xd = ring + (uint32_t)(xr * kOutXPitch + (tid & 15) * 16);
  const uint32_t zd = ring + (uint32_t)(kOutRows * kOutXPitch + xr * kOutZPitch + (tid & 15) * 16);
  auto load = [&](int i, uint32_t st) {
    const int at = i * kOutRows;
    const bool all = at + kOutRows <= n;            // rows past the end: zeros
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
      const int i = at + xr + h;
      const bool in = all || i < n;
      const int64_t m = rows[all ? i : min(i, n - 1)];
      cp_async<16>(xd + st + h * kOutXPitch, xc + m * p.x_rs, in ? x_ok : 0);
      if (z_in) cp_async<16>(zd + st + h * kOutZPitch, zc + m * 2 * z_ld, in ? 16 : 0);
    }
  };
  float acc[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
#pragma unroll
  for (int i = 0; i < kOutStages - 1; ++i) {
    if (i < steps) load(i, (uint32_t)(i * kOutStage));
    cp_commit();
  }
  int E = 0;
  if constexpr (kScaled) {                          // here the first copies are under way
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (e[q] != kExpAny && e[q] != kExpZero) atomicMax(&chunk_exp, e[q]);
    __syncthreads();
    E = chunk_exp > kExpZero ? chunk_exp : 0;
#pragma unroll
    for (int q = 0; q < 2; ++q)
      factor[tid + q * kOutThreads] = __float2half_rn(e[q] == kExpAny ? 1.f : pow2(max(e[q] - E, -30)));
  }
  uint32_t cur = 0, nxt = (kOutStages - 1) * kOutStage;      // byte offsets of stages i and i + kOutStages - 1
  for (int i = 0; i < steps; ++i) {
    cp_wait<kOutStages - 2>();
    __syncthreads();
    if (i + kOutStages - 1 < steps) load(i + kOutStages - 1, nxt);
    cp_commit();
    const uint32_t s = ring + cur;
    cur = cur == (kOutStages - 1) * kOutStage ? 0u : cur + kOutStage;
    nxt = nxt == (kOutStages - 1) * kOutStage ? 0u : nxt + kOutStage;
#pragma unroll
    for (int k = 0; k < kOutRows / 16; ++k) {
      uint32_t fa[4];
      ldsm_x4_t(fa, s + (uint32_t)((k * 16 + (lane & 7) + ((lane >> 4) & 1) * 8) * kOutXPitch + warp * 32 +
                                   ((lane >> 3) & 1) * 16));
      uint32_t f0 = 0, f1 = 0;                      // of this lane's rows of z: 2 (lane % 4), the next, and 8 more
      if constexpr (kScaled) {
        const uint32_t* f = reinterpret_cast<const uint32_t*>(factor + i * kOutRows + k * 16) + (lane & 3);
        f0 = f[0];
        f1 = f[4];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j >= nt) break;
        uint32_t fb[4];                             // hi's fragment, then lo's
        ldsm_x4_t(fb, s + (uint32_t)(kOutRows * kOutXPitch + (k * 16 + (lane & 15)) * kOutZPitch + j * 16 + (lane >> 4) * 128));
        if constexpr (kScaled) {
#pragma unroll
          for (int h = 0; h < 4; ++h) fb[h] = mul_half2(fb[h], h & 1 ? f1 : f0);
        }
        const uint32_t hi[2] = {fb[0], fb[1]}, lo[2] = {fb[2], fb[3]};
        mma16816<T>(acc[j], fa, hi);
        mma16816<T>(acc[j], fa, lo);
      }
    }
  }
  const bool whole = end - begin <= kChunkRows;
  static_assert(kOutC == 128 && kOutThreads == 256, "a thread's 8 x 4 values are bits of `again`");
  uint32_t again = 0u;
  float* mine = p.part + (int64_t)(first_part(begin) + chunk) * C * l.R;
  T* out = p.out + (int64_t)g * C * l.R;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= nt) break;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t c = c0 + warp * 16 + (lane >> 2) + (e >> 1) * 8;
      const int r = r0 + j * 8 + (lane & 3) * 2 + (e & 1);
      if (c >= C || r >= l.R) continue;
      const float v = kScaled ? times_pow2(acc[j][e], E) : acc[j][e];
      if (isnan(v)) again |= 1u << (j * 4 + e);
      if (whole) out[c * p.o_cs + r * p.o_rs] = from_f32<T>(v);
      else mine[c * p.o_cs + r * p.o_rs] = v;
    }
  }
  // An infinite x makes hi's product infinite and lo's infinite of either sign
  // or, where lo is 0, NaN: such a value once more, from the sum of the parts.
  // Only NaN results come here.
#pragma unroll 1
  for (; again; again &= again - 1) {
    const int at = __ffs(again) - 1, j = at >> 2, e = at & 3;
    const int64_t c = c0 + warp * 16 + (lane >> 2) + (e >> 1) * 8;
    const int r = r0 + j * 8 + (lane & 3) * 2 + (e & 1);
    float v = 0.f;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int64_t m = rows[i];
      const T* zr = p.zt + m * 2 * z_ld + r;
      float z = to_f32(zr[0]) + to_f32(zr[z_ld]);
      if constexpr (kScaled) {
        const int k = __ldcg(p.zt_exp + (int64_t)group * l.M + m);
        if (k != kExpAny && k != kExpZero) z = times_pow2(z, k);
      }
      v = __fmaf_rn(to_f32(p.x[m * p.x_rs + c]), z, v);
    }
    if (whole) out[c * p.o_cs + r * p.o_rs] = from_f32<T>(v);
    else mine[c * p.o_cs + r * p.o_rs] = v;
  }
}

// The adapters with several chunks (their sum) or none (zeros); element e of
// an adapter's [C, R] in the output's own order; block bx of nbx.
template <typename T>
__device__ void outer_sum(const LowRankArgs& l, const AdapterRows& t, const OuterProblem<T>& p, const int g, const int bx,
                          const int nbx) {
  const int64_t n = p.C * l.R;
  const int begin = __ldcg(t.offset + g);
  const int k = (__ldcg(t.offset + g + 1) - begin + kChunkRows - 1) / kChunkRows;
  if (k == 1) return;
  const float* src = p.part + (int64_t)first_part(begin) * n;
  if (n % 4 == 0) {
    for (int64_t e = ((int64_t)bx * 256 + threadIdx.x) * 4; e < n; e += (int64_t)nbx * 1024) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int c = 0; c < k; ++c) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(src + (int64_t)c * n + e));
        v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
      }
      T o[4] = {from_f32<T>(v.x), from_f32<T>(v.y), from_f32<T>(v.z), from_f32<T>(v.w)};
#pragma unroll
      for (int j = 0; j < 4; ++j) p.out[(int64_t)g * n + e + j] = o[j];
    }
  } else {
    for (int64_t e = (int64_t)bx * 256 + threadIdx.x; e < n; e += (int64_t)nbx * 256) {
      float v = 0.f;
      for (int c = 0; c < k; ++c) v += __ldcg(src + (int64_t)c * n + e);
      p.out[(int64_t)g * n + e] = from_f32<T>(v);
    }
  }
}

// ------------------------------------------------------------------ the fused product's operands

// Blocks [0, parts * tiles): a row tile's adapters (the first per_tile, by
// slot) and a part of its blocks of factor rows.  The others: the adapters'
// copies, 1024 columns of one slot a block.
template <typename T>
struct PlaceArgs {
  int blocks;                    // 0: nothing to place
  int tile_rows, tiles, per_tile, parts;
  const float* z; int64_t z_ld;
  int two;                       // lowrank_two_parts: hi in columns [0, z_ld), lo in the next z_ld
  T* factors; int64_t f_ld;
  const T* b; int64_t b_gs, b_rs, b_ns, N;
  T* copy; int64_t c_ld, k_rows;
  int pieces, vec;
};

template <typename T>
__device__ void lowrank_place(const LowRankArgs& l, const FusedTables& t, const PlaceArgs<T>& p, const int bx) {
  const int tile_rows = p.tile_rows, tiles = p.tiles, per_tile = p.per_tile, parts = p.parts, pieces = p.pieces, vec = p.vec;
  const T* b = p.b;
  T *factors = p.factors, *copy = p.copy;
  const int64_t z_ld = p.z_ld, f_ld = p.f_ld, b_gs = p.b_gs, b_rs = p.b_rs, b_ns = p.b_ns, N = p.N, c_ld = p.c_ld;
  const int tid = threadIdx.x;
  constexpr bool kF16 = std::is_same<T, __half>::value;
  constexpr float kLoScale = kF16 ? kF16LoScale : 1.f;
  if (bx < tiles * parts) {
    __shared__ uint32_t named[kSlots / 32];
    __shared__ signed char entry[256];
    const int tile = bx / parts, part = bx % parts;
    const int64_t m = (int64_t)tile * tile_rows + tid;
    int slot = -1;
    bool has = false;
    if (tid < tile_rows && m < l.M) {
      const int64_t g = load_index(l.idx, m * l.idx_s, l.ind64);
      has = g >= 0 && g < l.G;
      if (has) {
        slot = __ldcg(t.slot_of + g);
        // a factor with values that T cannot hold: the fix takes the row in fp32
        for (int64_t q = 0; q < (l.R + 63) / 64; ++q)
          if (__ldcg(t.wide + q * l.M + m)) slot = -1;
      }
    }
    if (tid < kSlots / 32) named[tid] = 0u;
    __syncthreads();
    if (slot >= 0) atomicOr(named + (slot >> 5), 1u << (slot & 31));
    __syncthreads();
    // An adapter's place in the list: the named slots below its own.
    auto place_of = [&](int s) {
      int n = __popc(named[s >> 5] & ((1u << (s & 31)) - 1u));
      for (int w = 0; w < s >> 5; ++w) n += __popc(named[w]);
      return n;
    };
    int mine = slot >= 0 ? place_of(slot) : -1, n = 0;
    if (mine >= per_tile) mine = -1;
    for (int w = 0; w < kSlots / 32; ++w) n += __popc(named[w]);
    n = min(n, per_tile);
    entry[tid] = (signed char)mine;
    if (part == 0 && tid < kSlots && ((named[tid >> 5] >> (tid & 31)) & 1u)) {
      const int at = place_of(tid);
      if (at < per_tile) t.ext_slot[(int64_t)tile * per_tile + at] = tid;
    }
    if (part == 0 && tid == 0) t.ext_count[tile] = n;
    if (part == 0 && tid < tile_rows && m < l.M) {
      t.row_entry[m] = mine;
      if (has && mine < 0) atomicOr(t.head + 1, 1);
    }
    __syncthreads();
    const int pieces_row = (int)(f_ld / 8), total = n * tile_rows * pieces_row, part_cols = (int)z_ld;
    constexpr int kAhead = 4;                             // reads in flight before the first write
    const float* z0 = p.z + (int64_t)tile * tile_rows * z_ld;
    for (int i0 = part * 256 + tid; i0 < total; i0 += 256 * parts * kAhead) {
      float4 v[kAhead][2];
      int from[kAhead];                                   // 0: zeros, 1: hi, 2: lo
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int i = i0 + q * 256 * parts;
        const int row = i / pieces_row, r = row % tile_rows, j = row / tile_rows;     // row of the tile's n blocks
        int c = (i - row * pieces_row) * 8;
        from[q] = 1;
        if (p.two && c >= part_cols) {
          c -= part_cols;
          from[q] = 2;
        }
        if (i >= total || entry[r] != j || c >= part_cols) {
          from[q] = 0;
          continue;
        }
        const float4* src = reinterpret_cast<const float4*>(z0 + (int64_t)r * z_ld + c);
        v[q][0] = __ldcg(src);
        v[q][1] = __ldcg(src + 1);
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int i = i0 + q * 256 * parts;
        if (i >= total) break;
        uint4 o = make_uint4(0u, 0u, 0u, 0u);
        if (from[q]) {
          const float* s = reinterpret_cast<const float*>(v[q]);
          T* e = reinterpret_cast<T*>(&o);
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            T hi, lo;
            split<T>(s[h], kLoScale, hi, lo);
            e[h] = from[q] == 2 ? lo : hi;
          }
        }
        *reinterpret_cast<uint4*>(factors + (int64_t)tile * per_tile * tile_rows * f_ld + (int64_t)i * 8) = o;
      }
    }
    return;
  }
  const int rest = bx - tiles * parts;
  const int piece = rest % pieces, slot = rest / pieces;
  if (slot >= __ldcg(t.head)) return;
  constexpr uint16_t kExp = kF16 ? 0x7C00 : 0x7F80;
  const uint16_t* src = reinterpret_cast<const uint16_t*>(b) + (int64_t)__ldcg(t.adapter_of + slot) * b_gs;
  uint16_t* dst = reinterpret_cast<uint16_t*>(copy) + (int64_t)slot * p.k_rows * c_ld;
  const int64_t ranks = p.two ? z_ld : l.R;                // rows of a part: zeros past R
  auto second = [&](uint16_t v) {                          // what lo's columns multiply
    return kF16 ? __half_as_ushort(__float2half_rn(__half2float(__ushort_as_half(v)) * (1.f / kLoScale))) : v;
  };
  bool bad = false;
  auto finite = [&](uint16_t v) {
    const bool f = (v & kExp) != kExp;
    bad |= !f;
    return f ? v : (uint16_t)0;
  };
  constexpr int kAhead = 8;
  if (vec == 1) {                                          // n contiguous: 8 columns of every other rank
    const int64_t n = ((int64_t)piece * 128 + (tid & 127)) * 8;
    const int R = (int)l.R, last = (int)ranks;
    src += n;
    dst += n;
    for (int r0 = tid >> 7; n < N && r0 < last; r0 += 2 * kAhead) {
      uint4 u[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) u[q] = *reinterpret_cast<const uint4*>(src + min(r0 + 2 * q, R - 1) * b_rs);
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int r = r0 + 2 * q;
        if (r >= last) break;
        uint16_t* e = reinterpret_cast<uint16_t*>(&u[q]);
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = r < R ? finite(e[j]) : (uint16_t)0;
        uint16_t* to = dst + r * c_ld;
        *reinterpret_cast<uint4*>(to) = u[q];
        if (p.two) {
#pragma unroll
          for (int j = 0; j < 8; ++j) e[j] = second(e[j]);
          *reinterpret_cast<uint4*>(to + z_ld * c_ld) = u[q];
        }
      }
    }
  } else {                                                 // 4 columns, 8 ranks of each at a time
    for (int64_t r0 = 0; r0 < l.R; r0 += 8) {
      uint4 u[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t n = (int64_t)piece * 1024 + q * 256 + tid;
        u[q] = make_uint4(0u, 0u, 0u, 0u);
        if (n >= N) continue;
        const uint16_t* col = src + n * b_ns + r0 * b_rs;
        if (vec == 2) {
          u[q] = *reinterpret_cast<const uint4*>(col);
        } else {
          uint16_t* e = reinterpret_cast<uint16_t*>(&u[q]);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (r0 + j < l.R) e[j] = col[j * b_rs];
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t n = (int64_t)piece * 1024 + q * 256 + tid;
        const uint16_t* e = reinterpret_cast<const uint16_t*>(&u[q]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (n < c_ld && r0 + j < ranks) {
            const uint16_t v = finite(e[j]);
            dst[(r0 + j) * c_ld + n] = v;
            if (p.two) dst[(z_ld + r0 + j) * c_ld + n] = second(v);
          }
      }
    }
  }
  if (bad) {
    atomicOr(t.bad + slot, 1);
    atomicOr(t.head + 1, 1);
  }
}

// What the fused product's extra blocks leave out: Y[m] = z[m] b[g] for rows
// outside their tile's list, or the terms of non-finite adapter values alone;
// the product adds Y for these rows.  Usually nothing.
constexpr int kFixColumns = 8, kFixRows = 152;   // its blocks: 256 columns at a time, rows in turn

template <typename T>
struct FixArgs {
  int blocks;                    // 0: nothing to fix
  const float* z; int64_t z_ld;
  const T* b; int64_t b_gs, b_rs, b_ns, N;
  T* y;
};

template <typename T>
__device__ void lowrank_fix(const LowRankArgs& l, const FusedTables& t, const FixArgs<T>& p, const int bx) {
  if (__ldcg(t.head + 1) == 0) return;
  constexpr uint16_t kExp = std::is_same<T, __half>::value ? 0x7C00 : 0x7F80;
  for (int64_t m = bx / kFixColumns; m < l.M; m += kFixRows) {
    const int64_t g = load_index(l.idx, m * l.idx_s, l.ind64);
    const bool in = g >= 0 && g < l.G;
    const bool all = in && __ldcg(t.row_entry + m) < 0;
    const bool add = all || (in && __ldcg(t.bad + __ldcg(t.slot_of + g)));
    if (bx % kFixColumns == 0 && threadIdx.x == 0) t.row_c[m] = add;
    if (!add) continue;
    for (int64_t n = (int64_t)(bx % kFixColumns) * 256 + threadIdx.x; n < p.N; n += kFixColumns * 256) {
      const T* bn = p.b + g * p.b_gs + n * p.b_ns;
      float v = 0.f;
#pragma unroll 8
      for (int64_t r = 0; r < l.R; ++r) {
        const T q = bn[r * p.b_rs];
        const bool bad = (*reinterpret_cast<const uint16_t*>(&q) & kExp) == kExp;
        if (all || bad) v = __fmaf_rn(p.z[m * p.z_ld + r], to_f32(q), v);
      }
      p.y[m * p.N + n] = from_f32<T>(v);
    }
  }
}

// ------------------------------------------------------------------ kernels of several steps

// After the factors: the fused product's operands (9 us alone) and the adapters'
// gradients (columns, then chunks, then groups of ranks), which do not depend on
// each other.  Where the SMs hold every block at once the gradients' go first,
// being the longer ones (1027 x 2048 x 1000, rank 12, the call: 42.7 us, with the
// operands' first 45.2); where they do not, last, so that they fill the end
// (8192 x 4096 x 4096, rank 16: 229.6, with theirs first 233.0).
template <typename T>
__global__ void __launch_bounds__(256, 3)
    lowrank_middle_kernel(const LowRankArgs l, const FusedTables f, const __grid_constant__ PlaceArgs<T> place,
                          const AdapterRows t, const __grid_constant__ OuterProblem<T> p0,
                          const __grid_constant__ OuterProblem<T> p1, const int blocks0, const int columns,
                          const int chunks, const int place_at, const int64_t z_ld) {
  pdl_begin();
  extern __shared__ __align__(16) uint8_t sm[];
  const int at = (int)blockIdx.x - place_at;                // place_at: 0, or the number of the others
  if (at >= 0 && at < place.blocks) {
    lowrank_place<T>(l, f, place, at);
  } else {
    const int b = at < 0 ? (int)blockIdx.x : at - place.blocks, rest = b / columns;
    outer_tile<T>(l, t, p0, p1, blocks0, z_ld, b % columns, rest % chunks, rest / chunks, sm);
  }
}

// After those, and before the fused product: the fix (first blocks; 4 us, its
// launch, when there is nothing to fix) and the chunks' sums (8 us).
template <typename T>
__global__ void __launch_bounds__(256)
    lowrank_sums_kernel(const LowRankArgs l, const FusedTables f, const __grid_constant__ FixArgs<T> fix,
                        const AdapterRows t, const __grid_constant__ OuterProblem<T> p0,
                        const __grid_constant__ OuterProblem<T> p1, const int sum_blocks) {
  pdl_begin();
  int bx = (int)blockIdx.x;
  if (bx < fix.blocks) return lowrank_fix<T>(l, f, fix, bx);
  bx -= fix.blocks;
  const int per = (int)l.G * sum_blocks;
  outer_sum<T>(l, t, bx < per ? p0 : p1, bx % per / sum_blocks, bx % sum_blocks, sum_blocks);
}

// ------------------------------------------------------------------ host side

bool rows16(const void* x, int64_t rs, int64_t cs, int64_t rows) {
  return cs == 1 && reinterpret_cast<uintptr_t>(x) % 16 == 0 && (rs % 8 == 0 || rows == 1);
}

// x [M, C] as a tensor map of 32-row, 64-column tiles.
bool shrink_map(const LowRankArgs& l, const void* x, int64_t x_rs, int64_t C, OperandPlan* out) {
  BatchMap one;
  memset(&one, 0, sizeof(one));
  one.count = 1;
  for (int d = 0; d < kMaxBatchDims; ++d) one.shape[d] = 1;
  const int64_t none[kMaxBatchDims] = {};
  const int64_t rs = l.M == 1 ? (C + 7) / 8 * 8 : x_rs;     // one row: its stride is never used
  return plan_operand(x, l.dtype, l.M, C, rs, 1, one, none, kShRows, out) && !out->mn_major;
}

template <typename T>
mm_status shrink_launch(const LowRankArgs& l, const LowRankShrink* q, int problems, int64_t z_ld,
                        const FusedTables* slots, const AdapterRows* sort, cudaStream_t stream) {
  TcParams limits;                      // the pipelines' wait limits
  init_params(&limits);
  ShrinkArgs p[2];
  const int rc = (int)(l.R < 64 ? l.R : 64);
  int smem = 0;
  for (int i = 0; i < 2; ++i) {
    const LowRankShrink& s = q[i < problems ? i : 0];
    ShrinkArgs& a = p[i];
    memset(&a, 0, sizeof(a));
    a.ck = s.a_rs != 1;
    a.C = s.C;
    a.a = s.a; a.a_gs = s.a_gs; a.a_ld = a.ck ? s.a_rs : s.a_cs;
    a.per = 8;
    while (a.per > 1 && (reinterpret_cast<uintptr_t>(a.a) % (a.per * 2) || (l.G > 1 && a.a_gs % a.per) || a.a_ld % a.per))
      a.per >>= 1;
    a.z = s.z; a.z_ld = z_ld; a.wide = s.wide; a.zt = s.zt; a.zt_exp = s.zt_exp;
    a.timeout_ns = limits.timeout_ns; a.teardown_ns = limits.teardown_ns;
    const int need = shrink_smem(a.ck, rc);
    if (smem < need) smem = need;
  }
  const int tables = (int)(sort ? (l.M + 31) / 32 * 4 : 0), bits = (int)(slots ? (l.G + 31) / 32 * 4 : 0);
  for (int need : {tables, bits})
    if (smem < need) smem = need;
  const int64_t tiles = (l.M + kShRows - 1) / kShRows;
  const int64_t ranks = (l.R + 63) / 64;
  int64_t parts = kShBlocks / (tiles * problems * ranks);
  parts = parts < 2 ? 2 : parts > kShParts ? kShParts : parts;
  const int64_t blocks = tiles * problems * parts + (slots ? 1 : 0) + (sort ? l.G : 0);
  if (blocks > 0x7fffffffLL) return MM_ERR_UNSUPPORTED;
  const auto kernel = rc <= 16 ? shrink_tiles_kernel<T, 2> : rc <= 32 ? shrink_tiles_kernel<T, 4> : shrink_tiles_kernel<T, 8>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024) != cudaSuccess)
    return MM_ERR_CUDA;
  return launch_pdl(kernel, dim3((unsigned)blocks, (unsigned)ranks), dim3(kShThreads), (size_t)smem, stream,
                    q[0].map->map, q[problems - 1].map->map, l, p[0], p[1], (int)tiles, problems, (int)parts, slots ? *slots : FusedTables{},
                    sort ? *sort : AdapterRows{}) == cudaSuccess ? MM_OK : MM_ERR_CUDA;
}

}  // namespace

bool lowrank_shrink_tiles_supported(const LowRankArgs& l, const void* x, int64_t x_rs, int64_t x_cs, int64_t C,
                                    int64_t a_cs, int64_t a_rs, OperandPlan* map) {
  return (l.dtype == MM_BF16 || l.dtype == MM_F16) && l.M >= 1 && l.R >= 1 && l.G >= 1 && l.G <= 0x7fffffffLL && C >= 1 &&
         l.M <= 0x7fffffffLL && l.R <= 64 * 65535LL && rows16(x, x_rs, x_cs, l.M) && (a_rs == 1 || a_cs == 1) &&
         shrink_map(l, x, x_rs, C, map);
}

mm_status launch_lowrank_shrink_tiles(const LowRankArgs& l, const LowRankShrink* p, int problems, int64_t z_ld,
                                      const FusedTables* slots, const AdapterRows* sort, cudaStream_t stream) {
  return l.dtype == MM_F16 ? shrink_launch<__half>(l, p, problems, z_ld, slots, sort, stream)
                           : shrink_launch<__nv_bfloat16>(l, p, problems, z_ld, slots, sort, stream);
}

namespace {

int64_t factor_columns(const LowRankArgs& l) {
  const int64_t z_ld = (l.R + 7) / 8 * 8;
  return ((lowrank_two_parts(l) ? 2 * z_ld : l.R) + 63) / 64 * 64;
}
// Adapters that a row tile can list: all of them up to kExtPerTile, fewer
// (16 at least) where the factors' blocks would take more than 256 MB.
int64_t per_tile(const LowRankArgs& l) {
  const int64_t bytes = (l.M + 255) / 256 * 256 * factor_columns(l) * 2;
  int64_t n = kExtPerTile;
  while (n > 16 && n * bytes > (256ll << 20)) n /= 2;
  const int64_t most = l.G < l.M ? l.G : l.M;
  return n < most ? n : most;
}

}  // namespace

FusedLayout lowrank_fused_layout(const LowRankArgs& l, int64_t N) {
  FusedLayout w;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o = (o + bytes + 255) & ~(size_t)255; return at; };
  const int64_t rows = (l.M + 255) / 256 * 256, tiles = rows / 128;
  w.slots = l.G < l.M ? l.G : l.M;
  if (w.slots > kSlots) w.slots = kSlots;
  w.two = lowrank_two_parts(l);
  w.z_ld = (l.R + 7) / 8 * 8;
  w.k_rows = w.two ? 2 * w.z_ld : l.R;
  w.f_ld = factor_columns(l);
  w.per_tile = per_tile(l);
  w.c_ld = (N + 7) / 8 * 8;
  w.z = take((size_t)l.M * (size_t)w.z_ld * 4);
  w.head = take(8);
  w.slot_of = take((size_t)l.G * 4);
  w.adapter_of = take(kSlots * 4);
  w.bad = take(kSlots * 4);
  w.row_entry = take((size_t)l.M * 4);
  w.ext_count = take((size_t)tiles * 4);
  w.ext_slot = take((size_t)tiles * (size_t)w.per_tile * 4);
  w.row_c = take((size_t)l.M * 4);
  w.wide = take((size_t)l.M * (size_t)((l.R + 63) / 64));
  w.factors = take((size_t)rows * (size_t)w.per_tile * (size_t)w.f_ld * 2);
  w.copy = take((size_t)w.slots * (size_t)w.k_rows * (size_t)w.c_ld * 2);
  w.total = o;
  return w;
}

bool lowrank_fused_supported(const LowRankArgs& l, const GemmArgs& g, LowRankProduct* plan) {
  return (l.dtype == MM_BF16 || l.dtype == MM_F16) && l.M >= 1 && l.R >= 1 && l.R <= 4096 && l.G >= 1 && l.G <= 65536 &&
         l.M * per_tile(l) < (1ll << 30) && tc_lowrank_plan(g, plan);
}

FusedTables lowrank_fused_tables(const FusedLayout& w, char* ws) {
  FusedTables t;
  t.head = reinterpret_cast<int32_t*>(ws + w.head);
  t.slot_of = reinterpret_cast<int32_t*>(ws + w.slot_of);
  t.adapter_of = reinterpret_cast<int32_t*>(ws + w.adapter_of);
  t.bad = reinterpret_cast<int32_t*>(ws + w.bad);
  t.row_entry = reinterpret_cast<int32_t*>(ws + w.row_entry);
  t.ext_count = reinterpret_cast<int32_t*>(ws + w.ext_count);
  t.ext_slot = reinterpret_cast<int32_t*>(ws + w.ext_slot);
  t.row_c = reinterpret_cast<int32_t*>(ws + w.row_c);
  t.wide = reinterpret_cast<uint8_t*>(ws + w.wide);
  return t;
}

namespace {

template <typename T>
mm_status finish_typed(const LowRankArgs& l, const LowRankFused* u, const AdapterRows* t, const LowRankOuter* o,
                       int problems, int64_t z_ld, cudaStream_t stream) {
  FusedTables f = {};
  PlaceArgs<T> place = {};
  FixArgs<T> fix = {};
  LowRankExt e = {};
  if (u) {
    const FusedLayout& w = *u->layout;
    f = lowrank_fused_tables(w, u->ws);
    const int tile_rows = u->plan->tile_rows;
    e.factors = u->ws + w.factors; e.factor_ld = w.f_ld; e.per_tile = w.per_tile;
    e.adapters = u->ws + w.copy; e.slots = w.slots; e.k_rows = w.k_rows; e.adapter_ld = w.c_ld;
    e.count = f.ext_count; e.slot = f.ext_slot;
    e.head = f.head; e.row_c = f.row_c;
    const int64_t N = u->product.N, tiles = (l.M + tile_rows - 1) / tile_rows, pieces = (w.c_ld + 1023) / 1024;
    int64_t parts = 152 / tiles;      // blocks that write one tile's factors: about one per SM in all
    parts = parts < 4 ? 4 : parts > 32 ? 32 : parts;
    const int64_t blocks = tiles * parts + w.slots * pieces;
    if (blocks > (1 << 30)) return MM_ERR_UNSUPPORTED;
    // 16-byte reads of b along n (1) or along the ranks (2)
    const bool base = (l.G == 1 || u->b_gs % 8 == 0) && reinterpret_cast<uintptr_t>(u->b) % 16 == 0;
    place.blocks = (int)blocks;
    place.tile_rows = tile_rows; place.tiles = (int)tiles; place.per_tile = (int)w.per_tile; place.parts = (int)parts;
    place.z = u->z; place.z_ld = w.z_ld; place.two = w.two; place.k_rows = w.k_rows;
    place.factors = reinterpret_cast<T*>(u->ws + w.factors); place.f_ld = w.f_ld;
    place.b = static_cast<const T*>(u->b);
    place.b_gs = u->b_gs; place.b_rs = u->b_rs; place.b_ns = u->b_ns; place.N = N;
    place.copy = reinterpret_cast<T*>(u->ws + w.copy); place.c_ld = w.c_ld;
    place.pieces = (int)pieces;
    place.vec = base && u->b_ns == 1 && u->b_rs % 8 == 0 && N % 8 == 0     ? 1
                : base && u->b_rs == 1 && u->b_ns % 8 == 0 && l.R % 8 == 0 ? 2 : 0;
    fix.blocks = kFixColumns * kFixRows;
    fix.z = u->z; fix.z_ld = w.z_ld;
    fix.b = place.b; fix.b_gs = u->b_gs; fix.b_rs = u->b_rs; fix.b_ns = u->b_ns; fix.N = N;
    fix.y = static_cast<T*>(const_cast<void*>(u->product.y.ptr));
  }
  OuterProblem<T> p[2] = {};
  int64_t blocks[2] = {0, 0}, most = 0;
  for (int i = 0; i < problems; ++i) {
    p[i] = {static_cast<const T*>(o[i].x), o[i].x_rs, o[i].C, static_cast<const T*>(o[i].zt), o[i].zt_exp,
            static_cast<T*>(o[i].out), o[i].o_cs, o[i].o_rs, o[i].part};
    blocks[i] = (o[i].C + kOutC - 1) / kOutC;
    if (o[i].C > most) most = o[i].C;
  }
  const AdapterRows rows = t ? *t : AdapterRows{};
  const int64_t columns = blocks[0] + blocks[1], chunks = lowrank_max_chunks(l);
  const int64_t outers = columns * chunks * ((l.R + 63) / 64), middle = place.blocks + outers;
  const int64_t place_at = middle <= 3 * (int64_t)sm_count_public() ? outers : 0;
  if (middle > 0x7fffffffLL) return MM_ERR_UNSUPPORTED;     // the operands would not fit the memory
  if (cudaFuncSetAttribute(lowrank_middle_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOutStages * kOutStage) !=
      cudaSuccess)
    return MM_ERR_CUDA;
  if (launch_pdl(lowrank_middle_kernel<T>, dim3((unsigned)middle), dim3(256), problems ? (size_t)(kOutStages * kOutStage) : 0, stream, l, f,
                 place, rows, p[0], p[1], (int)blocks[0], (int)(columns > 0 ? columns : 1), (int)chunks, (int)place_at,
                 z_ld) !=
      cudaSuccess)
    return MM_ERR_CUDA;
  const int64_t per = (most * l.R + 1023) / 1024, sum_blocks = per < 64 ? per : 64;
  const int64_t last = fix.blocks + problems * l.G * sum_blocks;
  if (launch_pdl(lowrank_sums_kernel<T>, dim3((unsigned)last), dim3(256), 0, stream, l, f, fix, rows, p[0], p[1],
                 (int)(sum_blocks > 0 ? sum_blocks : 1)) != cudaSuccess)
    return MM_ERR_CUDA;
  return u ? launch_tc_lowrank(u->product, *u->plan, e, l.status, stream) : MM_OK;
}

}  // namespace

mm_status launch_lowrank_finish(const LowRankArgs& l, const LowRankFused* fused, const AdapterRows* rows,
                                const LowRankOuter* outer, int problems, int64_t z_ld, cudaStream_t stream) {
  return l.dtype == MM_F16 ? finish_typed<__half>(l, fused, rows, outer, problems, z_ld, stream)
                           : finish_typed<__nv_bfloat16>(l, fused, rows, outer, problems, z_ld, stream);
}

}  // namespace qg
