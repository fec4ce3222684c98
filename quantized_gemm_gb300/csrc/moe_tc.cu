// Mixture-of-experts layer for a few tokens (mm_moe_layer) on the tensor
// cores: three launches, the last two of which do all the work.
//
//   plan    one block: which experts are picked, by which tokens
//   hidden  h[row] = act(x Wg[e]) * (x Wu[e])    one row per (expert, token) pick
//   down    out[t] = sum over t's rows of weight * (h[row] Wd[e])
//
// A few tokens make the layer a stream of the picked experts' weights, each
// read once: the bound is memory.  So the weights take the MMA's 128-row side
// (a tile of 128 output columns, whatever the number of tokens) and the tokens
// its narrow side (N = 16 .. 128): D[column, token] += W[k, column] x[token, k].
// Every expert's tile multiplies all tokens at once; a column of D belongs to
// one token, and only the columns of tokens that picked the expert are used,
// so no token sees another's values or an unpicked expert's.
//
// h is held as the sum of two T values (16 bits of it for bf16, 22 for f16:
// store_h), which the second product takes as separate tokens side by side (N
// doubled) and adds in its epilogue: no rounding of h worth speaking of next to
// the output's, for 2 KB more per 16 KB of weights out of the L2.  (As
// two MMAs per step instead, one token's layer took 134 us against 125: an MMA
// this narrow takes as long as a wider one.)
//
// The work is one sequence of k-blocks of 64 (all tiles of all picked experts
// for `hidden`; for `down` each output tile's experts in turn), cut into equal
// contiguous shares, one per SM: every SM streams the same number of bytes
// however many experts are picked.  A tile whose blocks fall into several
// shares is finished by the last of its CTAs to arrive, which adds the shares'
// partial sums (fp32, in the workspace) in share order, so results do not
// depend on timing.
//
// One token, two experts of 4096 x 14336 (705 MB): 126 us.  plan 2, tables and
// first tile 4, weights 65 at 7.2 TB/s with 8 us between the first and the last
// SM done, 6 until `down` has h, 32 at 7.35 TB/s, 7 to the end.  64 tokens, 39
// experts (13.7 GB): 2.00 ms, 6.9 TB/s.  The last shares handed out dynamically
// in small pieces were slower (161 -> 238 us on 29 tokens over 128 experts):
// in `down` they fall into the same few tiles, whose partial sums pile up.
//
// A CTA has 6 warps: warp 0 streams weight and token tiles by TMA into a ring,
// warp 1 issues the MMAs into one of two TMEM accumulators, warps 2-5 (one
// TMEM lane quadrant each) run the epilogue.
#include <cuda.h>

#include <cstring>

#include "moe.cuh"
#include "tc.h"
#include "tc_internal.h"
#include "tc_ptx.cuh"

namespace qg {

using namespace ptx;

namespace {

constexpr int kTok = 128;                    // tokens per launch: one bit each in an expert's mask
constexpr int kMaskWords = kTok / 32;
constexpr int kTileBytes = 128 * 64 * 2;     // a weight tile: 128 columns x 64 k
constexpr int kMaxStages = 12;
constexpr int kThreads = 192;
constexpr int kCtrl = 512;                   // barriers, TMEM slot, flags
constexpr int kPlanThreads = 512;
constexpr int kPlanExperts = 2048;           // experts the plan's tables hold (shared memory)
// A share of fewer k-blocks than kMinShare is not worth its partial sums (three
// tokens, 12 picks of K = 1000, F = 712: 32 us with 4, 27 us with 16, 35 us
// with 24).  Where a tile (hidden) or an expert's part of one (down) has fewer
// blocks, whole ones are shares, in `down` from kMinDown blocks on.
constexpr uint32_t kMinShare = 12, kMinDown = 4;
constexpr int kSmemMax = 227 * 1024;

// Tables written by the plan, in the workspace (read through L2: the kernels
// that read them may have started before they were written).
struct MoeTables {
  int32_t* head;          // [0] picked experts, [1] rows
  int32_t* expert;        // [picked] expert id, ascending
  int32_t* offset;        // [picked + 1] first row
  uint32_t* mask;         // [picked][kMaskWords] tokens that picked it
  int32_t* row_token;     // [rows]
  float* row_weight;      // [rows]
  int32_t* count;         // [hidden tiles + down tiles] arrivals, zeroed
  int64_t count_n;
};

struct MoeTcParams {
  MoeTables tb;
  int64_t F, N;
  int tokens, nt;         // tokens of this launch; rounded up to 16
  int col_tiles;          // tiles of 128 columns (of F, of N)
  int kblocks;            // k-blocks of 64 (of K, of F)
  int gated, act, f16;
  int a_mn;               // the weights are MN-major (unit stride along the columns)
  int64_t g_bc, u_bc;     // TMA batch coordinate per expert
  int stages, stage_bytes;
  int max_picked, table_bytes;
  uint32_t tmem_cols, up_off, buf_off;   // TMEM columns: allocated, of the up product, of the second buffer
  uint32_t idesc0;        // instruction descriptor without N
  void* out;              // hidden: h, hi rows then lo rows [2 * h_rows, ld]; down: out [tokens, N]
  int64_t ld;
  int h_rows;
  float* part;            // partial sums, two slots per CTA
  int32_t* count;         // this phase's arrival counters
  unsigned* status;
  unsigned long long timeout_ns, teardown_ns;
};

// ------------------------------------------------------------------ plan

// T <= kTok tokens.  A token that names an expert twice is one row with the
// sum of the two weights.  An expert's tokens are bits of its mask, so a row's
// place (offset + number of lower tokens) needs no order of arrival.
__global__ void __launch_bounds__(kPlanThreads) moe_plan_kernel(const MoeArgs a, const int64_t t0, const int T,
                                                                const MoeTables tb, unsigned* status) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ uint32_t sm[];
  uint32_t* mask = sm;                                     // [G][kMaskWords]
  int* base = reinterpret_cast<int*>(sm + a.G * kMaskWords);   // [G] first row
  __shared__ int wsum[kPlanThreads / 32][2];
  const int G = (int)a.G, S = (int)a.S, n = T * S, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < G * kMaskWords; i += kPlanThreads) mask[i] = 0u;
  for (int64_t i = tid; i < tb.count_n; i += kPlanThreads) tb.count[i] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kPlanThreads) {
    const int t = i / S, s = i - t * S;
    const int64_t e = load_index(a.gi, (t0 + t) * a.gi_ts + s * a.gi_ss, a.ind64);
    if (e >= 0 && e < G) atomicOr(mask + e * kMaskWords + (t >> 5), 1u << (t & 31));
    else if (e != -1) atomicOr(status, kStatusIndexRange);
  }
  __syncthreads();
  // Exclusive sums, in expert order, of (picked, rows): a contiguous range per thread.
  const int per = (G + kPlanThreads - 1) / kPlanThreads, lo = min(G, tid * per), hi = min(G, lo + per);
  int act = 0, rows = 0;
  for (int g = lo; g < hi; ++g) {
    int c = 0;
#pragma unroll
    for (int w = 0; w < kMaskWords; ++w) c += __popc(mask[g * kMaskWords + w]);
    act += c > 0;
    rows += c;
  }
  int ia = act, ir = rows;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int ua = __shfl_up_sync(0xffffffffu, ia, o), ur = __shfl_up_sync(0xffffffffu, ir, o);
    if (lane >= o) { ia += ua; ir += ur; }
  }
  if (lane == 31) { wsum[warp][0] = ia; wsum[warp][1] = ir; }
  __syncthreads();
  int pa = ia - act, pr = ir - rows;
  for (int w = 0; w < warp; ++w) { pa += wsum[w][0]; pr += wsum[w][1]; }
  for (int g = lo; g < hi; ++g) {
    int c = 0;
#pragma unroll
    for (int w = 0; w < kMaskWords; ++w) c += __popc(mask[g * kMaskWords + w]);
    base[g] = pr;
    if (c > 0) {
      tb.expert[pa] = g;
      tb.offset[pa] = pr;
#pragma unroll
      for (int w = 0; w < kMaskWords; ++w) tb.mask[pa * kMaskWords + w] = mask[g * kMaskWords + w];
      ++pa;
      pr += c;
    }
  }
  if (tid == kPlanThreads - 1) {
    tb.head[0] = pa;
    tb.head[1] = pr;
    tb.offset[pa] = pr;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kPlanThreads) {
    const int t = i / S, s = i - t * S;
    const int64_t row0 = (t0 + t) * a.gi_ts;
    const int64_t e = load_index(a.gi, row0 + s * a.gi_ss, a.ind64);
    if (e < 0 || e >= G) continue;
    bool first = true;
    float w = 0.f;
    for (int q = 0; q < S; ++q) {
      if (load_index(a.gi, row0 + q * a.gi_ss, a.ind64) != e) continue;
      if (q < s) { first = false; break; }
      w += a.ew ? static_cast<const float*>(a.ew)[(t0 + t) * a.ew_ts + q * a.ew_ss] : 1.f;
    }
    if (!first) continue;
    int r = base[e];
    for (int v = 0; v < (t >> 5); ++v) r += __popc(mask[e * kMaskWords + v]);
    r += __popc(mask[e * kMaskWords + (t >> 5)] & ((1u << (t & 31)) - 1u));
    tb.row_token[r] = t;
    tb.row_weight[r] = w;
  }
}

// ------------------------------------------------------------------ shares

// CTA c of P owns k-blocks [U c / P, U (c + 1) / P).
struct Share {
  uint32_t U, P;
  __device__ __forceinline__ uint32_t begin(uint32_t c) const { return (uint32_t)((uint64_t)U * c / P); }
  __device__ __forceinline__ uint32_t owner(uint32_t u) const { return (uint32_t)(((uint64_t)(u + 1) * P - 1) / U); }
};

// A run of k-blocks of one tile and one expert within a share.
struct Seg {
  uint32_t item;          // tile (hidden: expert-major; down: column tile), indexes the counters
  uint32_t a, col;        // picked expert, column tile
  uint32_t kb0, kb1;
};

// The segment that begins at block u of a share that ends at `end`.
template <bool DOWN>
__device__ __forceinline__ Seg seg_at(const MoeTcParams& p, uint32_t picked, uint32_t u, uint32_t end) {
  Seg s;
  const uint32_t kb = (uint32_t)p.kblocks;
  const uint32_t q = u / kb;               // (tile, expert) pair
  s.kb0 = u - q * kb;
  s.kb1 = min(kb, s.kb0 + (end - u));
  if (DOWN) {
    s.item = s.col = q / picked;
    s.a = q - s.col * picked;
  } else {
    s.item = q;
    s.a = q / (uint32_t)p.col_tiles;
    s.col = q - s.a * (uint32_t)p.col_tiles;
  }
  return s;
}

// ------------------------------------------------------------------ kernel

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 2, 128;" ::: "memory"); }
// One decision for the four epilogue warps, which meet at barriers later on.
__device__ __forceinline__ bool epi_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

// Arrival of this CTA's share of a tile; true in every epilogue thread of the
// CTA that arrives last, which then sees all the shares' partial sums.
__device__ __forceinline__ bool last_to_arrive(int32_t* counter, int expected, volatile int* flag) {
  epi_sync();
  if (threadIdx.x == 64) {
    __threadfence();        // releases what the other threads wrote before the barrier, too
    const int last = atomicAdd(counter, 1) == expected - 1;
    __threadfence();
    *flag = last;
  }
  epi_sync();
  return *flag != 0;
}

// The partial sums of shares c0..c1 of the tile that starts at block t0, added
// in share order, for n <= N places `step` floats apart (the others read the
// last one's); slots are `stride` floats apart.  Only the first share can have
// begun before the tile; it then holds the tile in its second slot.
template <int N>
__device__ __forceinline__ void sum_shares(const float* at, int step, int n, int64_t stride, const Share& sh, uint32_t c0,
                                           uint32_t c1, uint32_t t0, float4 (&s)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (uint32_t c = c0; c <= c1; ++c) {
    const float* q = at + (int64_t)(2 * c + (c == c0 && sh.begin(c) < t0)) * stride;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(q + min(i, n - 1) * step));
      s[i].x += v.x; s[i].y += v.y; s[i].z += v.z; s[i].w += v.w;
    }
  }
}

__device__ __forceinline__ void store16(void* dst, int64_t i, float v, int f16) {
  if (f16) static_cast<__half*>(dst)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(dst)[i] = __float2bfloat16_rn(v);
}

// h[row, f] as its two parts, h = hi kHi + lo kLo.  bf16 has fp32's range and
// takes them as they are.  f16 does not: hi is scaled down, so that h may reach
// 2^20 (an infinite or NaN h is hi alone), and lo up, so that what hi leaves is
// a normal number of T however small h is: together 22 bits of h, and where
// that would be less 2^-32.  hi is never 0 where h is not: its product then has
// the infinity of an infinite weight.
constexpr float kF16Hi = 16.f, kF16Lo = 1.f / 128.f;    // bf16: 1 and 1
__device__ __forceinline__ uint16_t bits16(float v, int f16) {
  return f16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
__device__ __forceinline__ float value16(uint16_t b, int f16) {
  return f16 ? __half2float(__ushort_as_half(b)) : __bfloat162float(__ushort_as_bfloat16(b));
}
__device__ __forceinline__ void store_h(const MoeTcParams& p, int row, int64_t f, float h) {
  const float k_hi = p.f16 ? kF16Hi : 1.f, r_hi = p.f16 ? 1.f / kF16Hi : 1.f, r_lo = p.f16 ? 1.f / kF16Lo : 1.f;
  uint16_t hi = bits16(h * r_hi, p.f16);
  hi |= (hi & 0x7FFF) == 0 && h != 0.f;                     // the smallest number of h's sign
  const float back = value16(hi, p.f16) * k_hi;
  uint16_t* dst = static_cast<uint16_t*>(p.out) + (int64_t)row * p.ld + f;
  dst[0] = hi;
  dst[p.h_rows * p.ld] = bits16(fabsf(back) < INFINITY ? (h - back) * r_lo : 0.f, p.f16);
}

// The product of h from those of its parts.  An infinite weight makes hi's
// product infinite and lo's infinite of either sign or, where lo is 0, NaN: lo
// only corrects a finite product (hi is 0 only where h is).
__device__ __forceinline__ float join(float hi, float lo, float s_hi, float s_lo) {
  return fabsf(hi) == INFINITY ? hi : __fmaf_rn(lo, s_lo, hi * s_hi);
}

template <bool DOWN>
__global__ void __launch_bounds__(kThreads, 1)
    moe_tc_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmU,
                  const __grid_constant__ CUtensorMap tmX, const MoeTcParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  uint8_t* ctrl = smem_raw + (ring - raw) + p.stages * p.stage_bytes;
  const uint32_t cbase = ring + (uint32_t)(p.stages * p.stage_bytes);
  const uint32_t full0 = cbase, empty0 = cbase + 8 * kMaxStages, accf0 = empty0 + 8 * kMaxStages;
  const uint32_t acce0 = accf0 + 16, drain = acce0 + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 16 * kMaxStages + 40);
  volatile int* abort = reinterpret_cast<volatile int*>(ctrl + 16 * kMaxStages + 44);
  volatile int* flag = reinterpret_cast<volatile int*>(ctrl + 16 * kMaxStages + 48);
  int32_t* t_expert = reinterpret_cast<int32_t*>(ctrl + kCtrl);        // the plan's tables: a copy, [picked] and
  int32_t* t_offset = t_expert + p.max_picked;                         // [picked + 1]
  float* acc = reinterpret_cast<float*>(ctrl + kCtrl + p.table_bytes);   // down: [tokens][128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf0 + 8 * b, 1);
      mbar_init(acce0 + 8 * b, 4);
    }
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // `hidden` lets `down` be scheduled as its CTAs leave the SMs.  By then every
  // CTA of `hidden` has passed its wait, so the plan (and all work before it)
  // is complete: `down` streams weights before `hidden` has finished and waits
  // for it only before it touches h, the partial sums or the output.
  if (!DOWN) pdl_begin();
  else pdl_trigger();       // the next launch waits for this one before it touches anything

  // Places past the picked experts are read too, and not used: one latency.
  const uint32_t picked = (uint32_t)__ldcg(p.tb.head);
  for (int i = threadIdx.x; i < p.max_picked; i += kThreads) t_expert[i] = __ldcg(p.tb.expert + i);
  for (int i = threadIdx.x; i <= p.max_picked; i += kThreads) t_offset[i] = __ldcg(p.tb.offset + i);
  __syncthreads();
  auto seg_rows = [&](uint32_t a) { return t_offset[a + 1] - t_offset[a]; };
  Share sh;
  sh.U = picked * (uint32_t)p.col_tiles * (uint32_t)p.kblocks;
  sh.P = max(1u, min(gridDim.x, sh.U / max(min(kMinShare, (uint32_t)p.kblocks), DOWN ? kMinDown : 1u)));
  const uint32_t cta = blockIdx.x;
  const uint32_t ub = cta < sh.P ? sh.begin(cta) : 0u, ue = cta < sh.P ? sh.begin(cta + 1) : 0u;
  constexpr int kW = DOWN ? 1 : 2;                // weight tiles per k-block
  const int wtiles = DOWN ? 1 : (p.gated ? 2 : 1);

  if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&tmW);
      if (!DOWN && p.gated) prefetch_tmap(&tmU);
      prefetch_tmap(&tmX);
      uint32_t stage = 0, phase = 0, issued = 0, iparity = 0;
      uint32_t early_a[kMaxStages], early_kb[kMaxStages];     // down: stages whose h tile waits for `hidden`
      int early = DOWN ? p.stages : 0, nearly = 0;
      auto load_weights = [&](uint32_t dst, const CUtensorMap* tm, uint32_t col, uint32_t kb, int32_t b, uint32_t bar) {
        const int32_t c0 = (int32_t)col * 128, k0 = (int32_t)kb * 64;
        if (p.a_mn) {
          tma_load_3d(dst, tm, c0, k0, b, bar);
          tma_load_3d(dst + 8192, tm, c0 + 64, k0, b, bar);
        } else {
          tma_load_3d(dst, tm, k0, c0, b, bar);
        }
      };
      auto load_tokens = [&](uint32_t st, uint32_t a, uint32_t kb) {
        const uint32_t dst = ring + st * p.stage_bytes + kW * kTileBytes, bar = full0 + 8 * st;
        if (DOWN) {
          const int rows = seg_rows(a), r0 = t_offset[a];
          for (int r = 0; r < rows; r += 16)      // 16 rows' hi, then their lo
            tma_load_3d(dst + 2 * r * 128, &tmX, (int32_t)kb * 64, r0 + r, 0, bar);
        } else {
          tma_load_3d(dst, &tmX, (int32_t)kb * 64, 0, 0, bar);
        }
      };
      auto release_early = [&]() {
        pdl_wait();
        asm volatile("fence.proxy.async;" ::: "memory");      // h was written through the generic proxy
        for (int i = 0; i < nearly; ++i) load_tokens((uint32_t)i, early_a[i], early_kb[i]);
        early = 0;
      };
      bool ok = true;
      for (uint32_t u = ub; u < ue && ok;) {
        const Seg s = seg_at<DOWN>(p, picked, u, ue);
        const int32_t e = t_expert[s.a];
        const uint32_t tok_bytes = DOWN ? (uint32_t)((seg_rows(s.a) + 15) & ~15) * 256u : (uint32_t)p.nt * 128u;
        for (uint32_t kb = s.kb0; kb < s.kb1; ++kb) {
          if (DOWN && early && nearly == early) release_early();
          if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, abort, p.status, p.timeout_ns)) { ok = false; break; }
          const uint32_t full = full0 + 8 * stage, dst = ring + stage * p.stage_bytes;
          mbar_arrive_expect_tx(full, (uint32_t)wtiles * kTileBytes + tok_bytes);
          load_weights(dst, &tmW, s.col, kb, (int32_t)(e * p.g_bc), full);
          if (!DOWN && p.gated) load_weights(dst + kTileBytes, &tmU, s.col, kb, (int32_t)(e * p.u_bc), full);
          if (DOWN && early) {
            early_a[nearly] = s.a;
            early_kb[nearly++] = kb;
          } else {
            load_tokens(stage, s.a, kb);
          }
          issued |= 1u << stage;
          iparity = (iparity & ~(1u << stage)) | (phase << stage);
          if (++stage == (uint32_t)p.stages) { stage = 0; phase ^= 1; }
        }
        u += s.kb1 - s.kb0;
      }
      if (DOWN && early) release_early();
      // Let every issued copy land before the CTA can exit.
      for (int s = 0; s < p.stages; ++s)
        if (issued & (1u << s)) mbar_wait_teardown(full0 + 8 * s, (iparity >> s) & 1u, p.teardown_ns);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, seg = 0;
      bool ok = true;
      for (uint32_t u = ub; u < ue && ok; ++seg) {
        const Seg s = seg_at<DOWN>(p, picked, u, ue);
        const uint32_t buf = seg & 1, aph = (seg >> 1) & 1;
        if (!mbar_wait(acce0 + 8 * buf, aph ^ 1, abort, p.status, p.timeout_ns)) break;
        tc_fence_after();
        const uint32_t n = DOWN ? (uint32_t)((seg_rows(s.a) + 15) & ~15) * 2u : (uint32_t)p.nt;
        const uint32_t idesc = p.idesc0 | ((n >> 3) << 17), d = tmem + buf * p.buf_off;
        for (uint32_t kb = s.kb0; kb < s.kb1; ++kb) {
          if (!mbar_wait(full0 + 8 * stage, phase, abort, p.status, p.timeout_ns)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sw = ring + stage * p.stage_bytes, sx = sw + kW * kTileBytes;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t bd = smem_desc_sw128(sx + k * 32, 16, 1024);
            const uint32_t accum = (kb > s.kb0 || k > 0) ? 1u : 0u;
            const uint64_t ad = p.a_mn ? smem_desc_sw128(sw + k * 2048, 8192, 1024) : smem_desc_sw128(sw + k * 32, 16, 1024);
            tc_mma_f16(d, ad, bd, idesc, accum);
            if (!DOWN && p.gated) {
              const uint32_t su = sw + kTileBytes;
              const uint64_t ud = p.a_mn ? smem_desc_sw128(su + k * 2048, 8192, 1024) : smem_desc_sw128(su + k * 32, 16, 1024);
              tc_mma_f16(d + p.up_off, ud, bd, idesc, accum);
            }
          }
          tc_commit(empty0 + 8 * stage);
          if (++stage == (uint32_t)p.stages) { stage = 0; phase ^= 1; }
        }
        if (ok) tc_commit(accf0 + 8 * buf);
        u += s.kb1 - s.kb0;
      }
      tc_commit(drain);
      mbar_wait_teardown(drain, 0, p.teardown_ns);
    }
  } else {
    const int quad = warp & 3, l = quad * 32 + lane;          // column of the tile
    const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
    if (DOWN) pdl_wait();
    uint32_t seg = 0;
    auto release = [&](uint32_t buf) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acce0 + 8 * buf);
    };
    if (!DOWN) {
      for (uint32_t u = ub; u < ue; ++seg) {
        const Seg s = seg_at<false>(p, picked, u, ue);
        const uint32_t buf = seg & 1, aph = (seg >> 1) & 1;
        const int64_t f = (int64_t)s.col * 128 + l;
        const int r0 = t_offset[s.a], rows = seg_rows(s.a);
        const uint4 mk = __ldcg(reinterpret_cast<const uint4*>(p.tb.mask) + s.a);
        const bool whole = s.kb0 == 0 && s.kb1 == (uint32_t)p.kblocks;
        // the share's first tile unless the share begins before the tile
        const uint32_t slot = 2 * cta + (u == ub ? 0u : 1u);
        float* part = p.part + (int64_t)slot * p.tokens * 256 + l;
        if (!epi_all(mbar_wait(accf0 + 8 * buf, aph, abort, p.status, p.timeout_ns))) break;
        tc_fence_after();
        int r = 0;
        for (int g = 0; g < p.nt / 16; ++g) {
          const uint32_t word = g < 2 ? mk.x : g < 4 ? mk.y : g < 6 ? mk.z : mk.w;
          const uint32_t bits = (word >> (16 * (g & 1))) & 0xffffu;
          if (!bits) continue;
          uint32_t vg[16], vu[16];
          tmem_ld16(tl + buf * p.buf_off + g * 16, vg);
          if (p.gated) tmem_ld16(tl + buf * p.buf_off + p.up_off + g * 16, vu);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (!((bits >> j) & 1u)) continue;
            const float gv = __uint_as_float(vg[j]), uv = p.gated ? __uint_as_float(vu[j]) : 1.f;
            if (whole) {
              const float h = p.gated ? activate(gv, p.act) * uv : activate(gv, p.act);
              if (f < p.F) store_h(p, r0 + r, f, h);
            } else {
              part[(int64_t)r * 256] = gv;
              part[(int64_t)r * 256 + 128] = uv;
            }
            ++r;
          }
        }
        release(buf);
        if (!whole) {
          const uint32_t t0 = s.item * (uint32_t)p.kblocks;
          const uint32_t c0 = sh.owner(t0), c1 = sh.owner(t0 + (uint32_t)p.kblocks - 1);
          if (last_to_arrive(p.count + s.item, (int)(c1 - c0 + 1), flag)) {
            const int64_t f4 = (int64_t)s.col * 128 + lane * 4;
            for (int j = quad; j < rows; j += 4) {
              float4 o[2];
              sum_shares<2>(p.part + j * 256 + lane * 4, 128, 2, (int64_t)p.tokens * 256, sh, c0, c1, t0, o);
              const float4 gv = o[0], uv = o[1];
              const float g[4] = {gv.x, gv.y, gv.z, gv.w}, v[4] = {uv.x, uv.y, uv.z, uv.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (f4 + e < p.F) store_h(p, r0 + j, f4 + e, p.gated ? activate(g[e], p.act) * v[e] : activate(g[e], p.act));
            }
          }
        }
        u += s.kb1 - s.kb0;
      }
    } else {
      const uint32_t per_tile = picked * (uint32_t)p.kblocks;
      const float s_hi = p.f16 ? kF16Hi : 1.f, s_lo = p.f16 ? kF16Lo : 1.f;
      if (picked == 0)                                         // no pick at all: zeros
        for (uint32_t col = cta; col < (uint32_t)p.col_tiles; col += gridDim.x) {
          const int64_t n = (int64_t)col * 128 + l;
          for (int t = 0; t < p.tokens && n < p.N; ++t) store16(p.out, t * p.ld + n, 0.f, p.f16);
        }
      for (uint32_t u = ub; u < ue; ++seg) {
        const Seg s = seg_at<true>(p, picked, u, ue);
        const uint32_t buf = seg & 1, aph = (seg >> 1) & 1;
        const uint32_t t0 = s.item * per_tile, t1 = t0 + per_tile;
        if (u == ub || u == t0)
          for (int t = 0; t < p.tokens; ++t) acc[t * 128 + l] = 0.f;
        const int r0 = t_offset[s.a], rows = seg_rows(s.a);
        int tok_n;                                             // lane j: token and weight of row j0 + j % 16
        float wt_n;
        auto load_rows = [&](int j0) {
          const int mine = r0 + min(j0 + (lane & 15), rows - 1);
          tok_n = __ldcg(p.tb.row_token + mine);
          wt_n = __ldcg(p.tb.row_weight + mine);
        };
        load_rows(0);
        if (!epi_all(mbar_wait(accf0 + 8 * buf, aph, abort, p.status, p.timeout_ns))) break;
        tc_fence_after();
        for (int j0 = 0; j0 < rows; j0 += 16) {
          const int tok = tok_n;
          const float wt = wt_n;
          if (j0 + 16 < rows) load_rows(j0 + 16);
          uint32_t v[16], lo[16];
          tmem_ld16(tl + buf * p.buf_off + 2 * j0, v);
          tmem_ld16(tl + buf * p.buf_off + 2 * j0 + 16, lo);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int t = __shfl_sync(0xffffffffu, tok, j);
            const float w = __shfl_sync(0xffffffffu, wt, j);
            if (j0 + j < rows)
              acc[t * 128 + l] = __fmaf_rn(w, join(__uint_as_float(v[j]), __uint_as_float(lo[j]), s_hi, s_lo), acc[t * 128 + l]);
          }
        }
        release(buf);
        const uint32_t next = u + (s.kb1 - s.kb0);
        if (next == ue || next == t1) {                        // the share's last block of this tile
          const int64_t n = (int64_t)s.col * 128 + l;
          if (ub <= t0 && ue >= t1) {
            for (int t = 0; t < p.tokens && n < p.N; ++t) store16(p.out, t * p.ld + n, acc[t * 128 + l], p.f16);
          } else {
            const uint32_t slot = 2 * cta + (ub < t0 ? 1u : 0u);
            float* part = p.part + (int64_t)slot * p.tokens * 128 + l;
            for (int t = 0; t < p.tokens; ++t) part[t * 128] = acc[t * 128 + l];
            const uint32_t c0 = sh.owner(t0), c1 = sh.owner(t1 - 1);
            if (last_to_arrive(p.count + s.item, (int)(c1 - c0 + 1), flag)) {
              const int64_t n4 = (int64_t)s.col * 128 + lane * 4;
              for (int t = quad; t < p.tokens; t += 16) {
                float4 o[4];
                sum_shares<4>(p.part + t * 128 + lane * 4, 4 * 128, (p.tokens - t + 3) / 4, (int64_t)p.tokens * 128, sh, c0, c1,
                              t0, o);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float v[4] = {o[i].x, o[i].y, o[i].z, o[i].w};
                  if (t + 4 * i < p.tokens)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                      if (n4 + e < p.N) store16(p.out, (t + 4 * i) * p.ld + n4 + e, v[e], p.f16);
                }
              }
            }
          }
        }
        u = next;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

// ------------------------------------------------------------------ host side

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

struct MoeLayout {
  int64_t tok, rows, picked, f_tiles, n_tiles, h_ld;
  size_t off_head, off_expert, off_offset, off_mask, off_token, off_weight, off_count, off_h, off_part, total;
};

MoeLayout moe_layout(const MoeArgs& a) {
  MoeLayout l;
  l.tok = a.tokens < kTok ? a.tokens : kTok;
  l.rows = l.tok * a.S;
  l.picked = a.G < l.rows ? a.G : l.rows;
  l.f_tiles = (a.F + 127) / 128;
  l.n_tiles = (a.N + 127) / 128;
  l.h_ld = (a.F + 7) / 8 * 8;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o = round256(o + bytes); return at; };
  l.off_head = take(8);
  l.off_expert = take((size_t)l.picked * 4);
  l.off_offset = take((size_t)(l.picked + 1) * 4);
  l.off_mask = take((size_t)l.picked * kMaskWords * 4);
  l.off_token = take((size_t)l.rows * 4);
  l.off_weight = take((size_t)l.rows * 4);
  l.off_count = take((size_t)(l.picked * l.f_tiles + l.n_tiles) * 4);
  l.off_h = take((size_t)2 * (size_t)l.rows * (size_t)l.h_ld * 2);
  l.off_part = take((size_t)2 * (size_t)sm_count_public() * (size_t)l.tok * 256 * 4);
  l.total = o;
  return l;
}

bool plan_weights(const void* w, int dtype, int64_t G, int64_t cols, int64_t k, int64_t gs, int64_t cs, int64_t ks,
                  OperandPlan* out) {
  BatchMap bm;
  memset(&bm, 0, sizeof(bm));
  bm.nb = 1;
  bm.shape[0] = bm.count = G;
  for (int d = 1; d < kMaxBatchDims; ++d) bm.shape[d] = 1;
  int64_t bs[kMaxBatchDims] = {gs, 0, 0, 0, 0, 0};
  return plan_operand(w, dtype, cols, k, cs, ks, bm, bs, 128, out);
}

bool plan_rows(const void* x, int dtype, int64_t rows, int64_t k, int64_t rs, int64_t cs, int box, OperandPlan* out) {
  BatchMap bm;
  memset(&bm, 0, sizeof(bm));
  bm.count = 1;
  for (int d = 0; d < kMaxBatchDims; ++d) bm.shape[d] = 1;
  int64_t bs[kMaxBatchDims] = {};
  if (cs != 1 && k > 1) return false;
  if (rows == 1) rs = (k + 7) / 8 * 8;      // one row: its stride is never used
  return plan_operand(x, dtype, rows, k, rs, 1, bm, bs, box, out) && !out->mn_major;
}

}  // namespace

bool tc_moe_supported(const MoeArgs& a, MoeMaps* maps) {
  if (a.dtype != MM_BF16 && a.dtype != MM_F16) return false;
  if (a.tokens < 1 || a.S < 1 || a.G < 1 || a.K < 1 || a.F < 1 || a.N < 1) return false;
  if (a.G > kPlanExperts || a.S > 64) return false;
  const MoeLayout l = moe_layout(a);
  // block indices are 32-bit, with room for the shares' products
  const double blocks = (double)l.picked * (double)l.f_tiles * (double)((a.K + 63) / 64);
  const double blocks2 = (double)l.picked * (double)l.n_tiles * (double)((a.F + 63) / 64);
  if (blocks >= 2147483648.0 || blocks2 >= 2147483648.0) return false;
  OperandPlan x;
  if (!plan_weights(a.wg, a.dtype, a.G, a.F, a.K, a.wg_gs, a.wg_fs, a.wg_ks, &maps->gate)) return false;
  if (a.wu && (!plan_weights(a.wu, a.dtype, a.G, a.F, a.K, a.wu_gs, a.wu_fs, a.wu_ks, &maps->up) ||
               maps->up.mn_major != maps->gate.mn_major))
    return false;
  if (!plan_weights(a.wd, a.dtype, a.G, a.N, a.F, a.wd_gs, a.wd_ns, a.wd_fs, &maps->down)) return false;
  // The rows of x that later launches start at are 16-byte aligned too (more
  // than one row: the stride is a multiple of 8).
  return plan_rows(a.x, a.dtype, l.tok, a.K, a.x_rs, a.x_cs, 16, &x);
}

size_t tc_moe_workspace_bytes(const MoeArgs& a) { return moe_layout(a).total; }

mm_status launch_tc_moe(const MoeArgs& a, const MoeMaps& maps, void* workspace, unsigned* status, cudaStream_t stream) {
  const MoeLayout l = moe_layout(a);
  char* ws = static_cast<char*>(workspace);
  TcParams limits;                        // the pipelines' wait limits
  init_params(&limits);
  MoeTcParams p;
  memset(&p, 0, sizeof(p));
  p.tb.head = reinterpret_cast<int32_t*>(ws + l.off_head);
  p.tb.expert = reinterpret_cast<int32_t*>(ws + l.off_expert);
  p.tb.offset = reinterpret_cast<int32_t*>(ws + l.off_offset);
  p.tb.mask = reinterpret_cast<uint32_t*>(ws + l.off_mask);
  p.tb.row_token = reinterpret_cast<int32_t*>(ws + l.off_token);
  p.tb.row_weight = reinterpret_cast<float*>(ws + l.off_weight);
  p.tb.count = reinterpret_cast<int32_t*>(ws + l.off_count);
  p.tb.count_n = l.picked * l.f_tiles + l.n_tiles;
  p.F = a.F; p.N = a.N;
  p.h_rows = (int)l.rows;
  p.gated = a.wu != nullptr; p.act = a.act; p.f16 = a.dtype == MM_F16;
  p.part = reinterpret_cast<float*>(ws + l.off_part);
  p.status = status;
  p.timeout_ns = limits.timeout_ns; p.teardown_ns = limits.teardown_ns;

  const OperandPlan &wg = maps.gate, &wu = maps.up, &wd = maps.down;
  OperandPlan h, x;
  BatchMap parts;                          // h's hi and lo rows, 16 of each in one box
  memset(&parts, 0, sizeof(parts));
  parts.nb = 1;
  parts.shape[0] = parts.count = 2;
  const int64_t part_stride[kMaxBatchDims] = {l.rows * l.h_ld, 0, 0, 0, 0, 0};
  if (!plan_operand(ws + l.off_h, a.dtype, l.rows, a.F, l.h_ld, 1, parts, part_stride, 16, &h, 2) || h.mn_major)
    return MM_ERR_UNSUPPORTED;
  const int plan_smem = (int)(a.G * (kMaskWords + 1) * 4);
  const int sms = sm_count_public();
  for (int64_t t0 = 0; t0 < a.tokens; t0 += kTok) {
    const int T = (int)(a.tokens - t0 < kTok ? a.tokens - t0 : kTok);
    p.tokens = T;
    p.nt = (T + 15) / 16 * 16;
    if (launch_pdl(moe_plan_kernel, dim3(1), dim3(kPlanThreads), (size_t)plan_smem, stream, a, t0, T, p.tb, status) !=
        cudaSuccess)
      return MM_ERR_CUDA;
    for (int down = 0; down < 2; ++down) {
      MoeTcParams q = p;
      const OperandPlan& w = down ? wd : wg;
      if (!down && !plan_rows(static_cast<const uint16_t*>(a.x) + t0 * a.x_rs, a.dtype, T, a.K, a.x_rs, a.x_cs, p.nt, &x))
        return MM_ERR_UNSUPPORTED;
      q.col_tiles = (int)(down ? l.n_tiles : l.f_tiles);
      q.kblocks = (int)(((down ? a.F : a.K) + 63) / 64);
      q.a_mn = w.mn_major;
      q.g_bc = w.bc[0];
      q.u_bc = !down && a.wu ? wu.bc[0] : 0;
      q.idesc0 = make_idesc_mn(q.f16, q.a_mn, 0, 128, 0);
      q.out = down ? a.out : ws + l.off_h;
      if (down) q.out = static_cast<uint16_t*>(a.out) + t0 * a.N;
      q.ld = down ? a.N : l.h_ld;
      q.count = p.tb.count + (down ? l.picked * l.f_tiles : 0);
      q.stage_bytes = (down ? 1 : 2) * kTileBytes + (down ? 2 : 1) * p.nt * 128;
      q.max_picked = (int)l.picked;
      q.table_bytes = (int)((2 * l.picked + 1) * 4 + 15) / 16 * 16;
      const int acc_bytes = q.table_bytes + (down ? T * 128 * 4 : 0);
      const uint32_t ntp = p.nt <= 32 ? 32u : p.nt <= 64 ? 64u : 128u;
      q.up_off = ntp;
      q.buf_off = down || a.wu ? 2 * ntp : ntp;
      q.tmem_cols = 2 * q.buf_off;
      // The whole SM's shared memory: halving the rings, so that the CTAs of
      // both kernels fit an SM side by side, was slower (29 tokens over 128
      // experts: 161 -> 166 us).
      q.stages = (kSmemMax - 1024 - kCtrl - acc_bytes) / q.stage_bytes;
      if (q.stages > kMaxStages) q.stages = kMaxStages;
      const int smem = 1024 + q.stages * q.stage_bytes + kCtrl + acc_bytes;
      const auto kernel = down ? moe_tc_kernel<true> : moe_tc_kernel<false>;
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess)
        return MM_ERR_CUDA;
      if (launch_pdl(kernel, dim3((unsigned)sms), dim3(kThreads), (size_t)smem, stream, w.map,
                     !down && a.wu ? wu.map : w.map, down ? h.map : x.map, q) != cudaSuccess)
        return MM_ERR_CUDA;
    }
  }
  return MM_OK;
}

}  // namespace qg
