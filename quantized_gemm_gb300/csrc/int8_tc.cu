// The 8-bit product for a few tokens up to a few hundred (mm_int8_matmul): the
// weights stream once, as int8, and are the MMA's 128-row operand.
//
// There is no 8-bit integer tensor instruction on sm_103a, so int8 values are
// multiplied as f16, which holds them exactly.  A CTA owns `rows` output channels
// (64 to 128, chosen so that the CTAs fill the SMs) and NT tokens (16 to 256):
//   warp 0       streams [rows channels x 128 k] tiles of int8 weights by TMA into a
//                ring, before the launch in front of this one has ended (that one
//                only copies the tokens to f16);
//   warp 2       streams the tokens' f16 tiles [NT x 128 k] once it has;
//   warps 4-19   turn weight bytes into f16 pairs (flip the sign bit, put the byte
//                into the mantissa of 1024, subtract 1152: 1.25 instructions a value)
//                and store them to tensor memory, where the MMA takes its first
//                operand from (a thread owns a channel, that is a lane): the weights
//                pass through shared memory once, as bytes, which leaves its
//                bandwidth to the stream; two groups of 8 warps take turns;
//   warp 1       issues the MMAs, D[channel, token] in fp32.
// K is split over the CTAs of a cluster where that fills the SMs better; the
// partial sums meet in a fixed order through distributed shared memory, a token's
// channels in neighbouring lanes, and the epilogue scales and stores them in
// rows.  Bound: memory (one byte per weight) up to about 100 tokens, then the MMAs.
// 61 tokens by 4096 x 14336 (59 MB): 17.7 us with the tokens' copy; what is left
// above the stream's 9 are that launch, the hand-over of the first tiles and the
// split's last sums.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstring>

#include "int8.cuh"
#include "tc.h"
#include "tc_internal.h"
#include "tc_ptx.cuh"

namespace qg {

using namespace ptx;

namespace {

constexpr int kRows = 128;                       // channels of a CTA at most: the MMA's rows
constexpr int kDepth = 128;                      // k of a stage
constexpr int kWBytes = kRows * kDepth;
constexpr int kAStages = 4, kACols = kDepth / 2; // operand stages in tensor memory, columns each
constexpr int kConvWarp0 = 4, kConvWarps = 16;
constexpr int kThreads = (kConvWarp0 + kConvWarps) * 32;
constexpr int kCtrl = 512;

template <int NT>
struct Cfg {
  static constexpr int kXBytes = NT * kDepth * 2;
  static constexpr int kAccs = NT <= 64 ? 4 : NT <= 128 ? 2 : 1;   // accumulators that take the k steps in turn
  static constexpr int kXStages = NT <= 64 ? 4 : NT <= 128 ? 3 : 2;
  static constexpr int kWStages = NT <= 128 ? 7 : 5;
  static constexpr int kXOff = kWStages * kWBytes;
  static constexpr int kRing = kXOff + kXStages * kXBytes;
  static constexpr int kParam = (2 * kRows + NT) * 4;              // scales and bias of the channels, scales of the tokens
  static constexpr int kSmem = kRing + kCtrl + kParam + 1024;
  static_assert(kSmem <= 232448, "shared memory per block");
  static_assert(NT * kRows * 4 <= kRing, "the partial sums take the ring's place");
  static_assert(NT * kAccs + kAStages * kACols <= 512, "tensor memory");
};

struct StreamArgs {
  Int8Args q;
  int num_kb, split, mtiles, rows;
  int w_late;                                    // the launch in front of this one writes the weights
  int y_vec;                                     // rows of Y allow stores of four values
  uint32_t idesc;
  unsigned* status;
  unsigned long long timeout_ns, teardown_ns;
};

// D[tmem] (+)= A[tmem] * B[smem], f16 operands, fp32 accumulator.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <typename O>
__device__ __forceinline__ uint32_t pair_bits(O a, O b) {
  uint16_t x, y;
  memcpy(&x, &a, 2);
  memcpy(&y, &b, 2);
  return (uint32_t)x | (uint32_t)y << 16;
}
template <typename O, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    int8_stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                       const StreamArgs p) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  const uint32_t ctrl = sbase + C::kRing;
  const uint32_t wfull = ctrl, wempty = wfull + 8 * C::kWStages, xfull = wempty + 8 * C::kWStages,
                 xempty = xfull + 8 * C::kXStages, afull = xempty + 8 * C::kXStages, aempty = afull + 8 * kAStages,
                 accf = aempty + 8 * kAStages;
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + C::kRing + kCtrl - 16);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kRing + kCtrl - 8);
  static_assert(16 * C::kWStages + 16 * C::kXStages + 16 * kAStages + 8 <= kCtrl - 16, "control block");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kWStages; ++s) {
      mbar_init(wfull + 8 * s, 1);
      mbar_init(wempty + 8 * s, kConvWarps / 2);
    }
    for (int s = 0; s < C::kXStages; ++s) {
      mbar_init(xfull + 8 * s, 1);
      mbar_init(xempty + 8 * s, 1);
    }
    for (int s = 0; s < kAStages; ++s) {
      mbar_init(afull + 8 * s, kConvWarps / 2);
      mbar_init(aempty + 8 * s, 1);
    }
    mbar_init(accf, 1);
    *abort = 0;
    fence_mbar_init();
  }
  const int rank = (int)(blockIdx.x % (unsigned)p.split), tile = (int)(blockIdx.x / (unsigned)p.split);
  const int64_t n0 = (int64_t)(tile / p.mtiles) * p.rows, m0 = (int64_t)(tile % p.mtiles) * NT;
  const int kb0 = (int)((int64_t)rank * p.num_kb / p.split), kb1 = (int)((int64_t)(rank + 1) * p.num_kb / p.split);
  const int nkb = kb1 - kb0;
  // Unless they are a copy too, the weights were complete before the launch in
  // front of this one (the copy of the tokens, which lets this grid start only
  // after its own wait): the ring is filled at once.
  const auto load_weights = [&](int i) {
    const int s = i % C::kWStages;
    mbar_arrive_expect_tx(wfull + 8 * s, p.rows * kDepth);
    tma_load_3d(sbase + s * kWBytes, &tmW, (kb0 + i) * kDepth, (int32_t)n0, 0, wfull + 8 * s);
  };
  if (threadIdx.x == 0) {
    if (p.w_late) pdl_wait();
    for (int i = 0; i < nkb && i < C::kWStages; ++i) load_weights(i);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot, tmem_a = tmem + NT * C::kAccs;

  const int per = NT / p.split, cw = warp - kConvWarp0;
  constexpr int kMine = (NT + kConvWarps - 1) / kConvWarps;      // tokens of a warp at most
  float* param = reinterpret_cast<float*>(smem + C::kRing + kCtrl);
  if (warp == 0) {
    if (elect_one()) {
      int i = min(nkb, C::kWStages);
      for (; i < nkb; ++i) {
        if (!mbar_wait(wempty + 8 * (i % C::kWStages), ((i / C::kWStages) & 1) ^ 1, abort, p.status, p.timeout_ns)) break;
        load_weights(i);
      }
      for (int j = i > C::kWStages ? i - C::kWStages : 0; j < i; ++j)      // every copy lands before the CTA can end
        mbar_wait_teardown(wfull + 8 * (j % C::kWStages), (j / C::kWStages) & 1, p.teardown_ns);
    }
  } else if (warp == 2) {
    if (elect_one()) {
      prefetch_tmap(&tmX);
      pdl_wait();
      int i = 0;
      for (; i < nkb; ++i) {
        const int s = i % C::kXStages, ph = (i / C::kXStages) & 1;
        if (!mbar_wait(xempty + 8 * s, ph ^ 1, abort, p.status, p.timeout_ns)) break;
        mbar_arrive_expect_tx(xfull + 8 * s, C::kXBytes);
        const uint32_t dst = sbase + C::kXOff + s * C::kXBytes;
        tma_load_3d(dst, &tmX, (kb0 + i) * kDepth, (int32_t)m0, 0, xfull + 8 * s);
        tma_load_3d(dst + C::kXBytes / 2, &tmX, (kb0 + i) * kDepth + 64, (int32_t)m0, 0, xfull + 8 * s);
      }
      for (int j = i > C::kXStages ? i - C::kXStages : 0; j < i; ++j)
        mbar_wait_teardown(xfull + 8 * (j % C::kXStages), (j / C::kXStages) & 1, p.teardown_ns);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      for (int i = 0; i < nkb; ++i) {
        const int xs = i % C::kXStages, as = i % kAStages;
        if (!mbar_wait(xfull + 8 * xs, (i / C::kXStages) & 1, abort, p.status, p.timeout_ns)) break;
        if (!mbar_wait(afull + 8 * as, (i / kAStages) & 1, abort, p.status, p.timeout_ns)) break;
        tc_fence_after();
        const uint32_t x = sbase + C::kXOff + xs * C::kXBytes;
#pragma unroll
        for (int k = 0; k < kDepth / 16; ++k)
          mma_ts(tmem + k % C::kAccs * NT, tmem_a + as * kACols + k * 8,
                 smem_desc_sw128(x + (k >> 2) * (C::kXBytes / 2) + (k & 3) * 32, 16, 1024), p.idesc,
                 i > 0 || k >= C::kAccs);
        tc_commit(aempty + 8 * as);
        tc_commit(xempty + 8 * xs);
      }
      tc_commit(accf);
      mbar_wait_teardown(accf, 0, p.teardown_ns);
    }
  } else if (warp == 3) {
    // For the epilogue (inputs, complete like the weights).
    for (int j = lane; j < kRows; j += 32) {
      const bool in = j < p.rows && n0 + j < p.q.N;
      param[j] = in ? __ldg(p.q.sb + (n0 + j) * p.q.sb_s) : 0.f;
      param[kRows + j] = in ? bias_at<O>(p.q, n0 + j) : 0.f;
    }
    for (int j = lane; j < NT; j += 32) param[2 * kRows + j] = m0 + j < p.q.M ? __ldg(p.q.sa + (m0 + j) * p.q.sa_s) : 0.f;
  } else if (warp >= kConvWarp0) {
    const int quad = warp & 3, half = (cw >> 2) & 1, group = cw >> 3;
    const int row = quad * 32 + lane;
    for (int i = group; i < nkb; i += 2) {
      const int ws = i % C::kWStages, as = i % kAStages;
      if (!__all_sync(0xffffffffu, mbar_wait(wfull + 8 * ws, (i / C::kWStages) & 1, abort, p.status, p.timeout_ns))) break;
      uint4 u[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        u[c] = lds128(sbase + ws * kWBytes + row * kDepth + (((half * 4 + c) ^ (row & 7)) << 4));
      uint32_t r[32];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        halves(u[c].x, r[8 * c], r[8 * c + 1]);
        halves(u[c].y, r[8 * c + 2], r[8 * c + 3]);
        halves(u[c].z, r[8 * c + 4], r[8 * c + 5]);
        halves(u[c].w, r[8 * c + 6], r[8 * c + 7]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(wempty + 8 * ws);
      if (!__all_sync(0xffffffffu, mbar_wait(aempty + 8 * as, ((i / kAStages) & 1) ^ 1, abort, p.status, p.timeout_ns))) break;
      tc_fence_after();
      tmem_st32(tmem_a + as * kACols + half * 32 + ((uint32_t)(quad * 32) << 16), r);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(afull + 8 * as);
    }
    // This CTA's sums, [token][channel], into the drained ring.
    if (__all_sync(0xffffffffu, mbar_wait(accf, 0, abort, p.status, p.timeout_ns))) {
      tc_fence_after();
      float* part = reinterpret_cast<float*>(smem);
#pragma unroll 1
      for (int c = (cw >> 2) * 16; c < NT; c += 64) {
        uint32_t r[C::kAccs][16];
#pragma unroll
        for (int a = 0; a < C::kAccs; ++a) tmem_ld16(tmem + a * NT + c + ((uint32_t)(quad * 32) << 16), r[a]);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float v = __uint_as_float(r[0][j]);
#pragma unroll
          for (int a = 1; a < C::kAccs; ++a) v += __uint_as_float(r[a][j]);
          part[(c + j) * kRows + row] = v;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (p.split > 1) cluster_sync();
  pdl_wait();
  if (warp >= kConvWarp0 && !*abort) {
    // Tokens [rank * NT / split, ...), a warp per token, four channels a lane.
    const int64_t nl = n0 + lane * 4;
    const float4 s4 = *reinterpret_cast<const float4*>(param + lane * 4);
    const float4 b4 = *reinterpret_cast<const float4*>(param + kRows + lane * 4);
    const float sb[4] = {s4.x, s4.y, s4.z, s4.w}, bias[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll 4
    for (int t = 0; t < kMine; ++t) {
      const int tok = rank * per + cw + t * kConvWarps;
      const int64_t m = m0 + tok;
      if (cw + t * kConvWarps >= per || m >= p.q.M) break;
      const uint32_t src = sbase + (uint32_t)(tok * kRows + lane * 4) * 4;
      const float sa = param[2 * kRows + tok];
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      for (int rk = 0; rk < p.split; ++rk) {
        const float4 f = p.split > 1 ? lds128_cluster(mapa_shared(src, (uint32_t)rk))
                                     : *reinterpret_cast<const float4*>(smem + (src - sbase));
        v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
      }
      O o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = finish8<O>(v[j], sa, sb[j], bias[j]);
      O* y = static_cast<O*>(p.q.y) + m * p.q.N + nl;
      if (lane * 4 >= p.rows) continue;                // rows is a multiple of 4
      if (p.y_vec && nl + 4 <= p.q.N) {
        if constexpr (sizeof(O) == 4) *reinterpret_cast<float4*>(y) = make_float4(o[0], o[1], o[2], o[3]);
        else *reinterpret_cast<uint2*>(y) = make_uint2(pair_bits(o[0], o[1]), pair_bits(o[2], o[3]));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (nl + j < p.q.N) y[j] = o[j];
      }
    }
  }
  if (p.split > 1) cluster_sync();               // no CTA leaves while its sums are read
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The weights [N, K] int8 as [rows channels x 128 k] tiles, 128-byte swizzled.
bool weight_map(const Int8Args& q, int rows, CUtensorMap* map) {
  const auto encode = encode_fn();
  if (!encode) return false;
  const int64_t pitch = q.N == 1 ? (q.K + 15) / 16 * 16 : q.b_ns;
  const cuuint64_t dims[3] = {(cuuint64_t)q.K, (cuuint64_t)q.N, 1};
  const cuuint64_t strides[2] = {(cuuint64_t)pitch, (cuuint64_t)pitch * (cuuint64_t)q.N};
  if (strides[0] >= (1ull << 40) || strides[1] >= (1ull << 40)) return false;
  const cuuint32_t box[3] = {kDepth, (cuuint32_t)rows, 1}, estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t*>(q.b), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of `split` CTAs, one CTA an SM, that are resident at once (the SMs of a
// GPC that a cluster does not fill stay idle): 36 of 4 on 152 SMs.
int resident_clusters(int split) {
  static std::atomic<int> cache[128][4];         // value + 1 once known
  int dev = 0, at = 0;
  cudaGetDevice(&dev);
  if (split == 1 || dev < 0 || dev >= 128) return sm_count_public() / split;
  while ((1 << at) < split) ++at;
  const int known = cache[dev][at].load(std::memory_order_relaxed);
  if (known > 0) return known - 1;
  const auto kernel = int8_stream_kernel<float, 256>;      // any: all leave room for one CTA an SM
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(sm_count_public() / split * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<256>::kSmem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<256>::kSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  cache[dev][at].store(n + 1, std::memory_order_relaxed);
  return n;
}

// Tokens and channels per CTA and CTAs per cluster.  A CTA's stage takes the
// longer of its bytes (about 25 a cycle and SM, all SMs streaming) and its 8 MMAs
// (NT / 2 cycles each); starting, handing over the sums and storing take about 6000
// cycles more, for every round of resident clusters.  The least cycles win, the
// larger tile among equals: N = 14336 has 112 tiles of 128 channels but 150 of 96,
// which keep 150 of 152 SMs at work; 1027 tokens are 5 tiles of 256 or 9 of 128.
struct TilePlan {
  int nt, rows, split;
  int64_t rounds;
};
TilePlan plan_tiles(const Int8Args& q) {
  const int num_kb = (int)((q.K + kDepth - 1) / kDepth);
  int first = 16;
  while (first < 256 && first < q.M) first *= 2;
  TilePlan best = {first, kRows, 1, 1};
  double least = 0.;
  for (int nt = first; nt >= 128 || nt == first; nt /= 2) {
    const int64_t mtiles = (q.M + nt - 1) / nt;
    for (int s = 1; s <= 8 && (s == 1 || num_kb >= 2 * s); s *= 2) {
      const int64_t room = resident_clusters(s);
      if (room < 1) continue;
      for (int r = kRows; r >= 64; r -= 8) {
        const int64_t rounds = ((q.N + r - 1) / r * mtiles + room - 1) / room;
        const double bytes = r * kDepth / 25., mma = 4. * nt;
        const double cycles = (double)rounds * (((num_kb + s - 1) / s) * (bytes > mma ? bytes : mma) + 6000.);
        if (least == 0. || cycles < least) {
          least = cycles;
          best = {nt, r, s, rounds};
        }
      }
    }
  }
  return best;
}

template <typename O, int NT>
mm_status launch(const StreamArgs& p_in, const CUtensorMap& x, cudaStream_t stream) {
  StreamArgs p = p_in;
  p.mtiles = (int)((p.q.M + NT - 1) / NT);
  if (cudaFuncSetAttribute(int8_stream_kernel<O, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<NT>::kSmem) !=
      cudaSuccess)
    return MM_ERR_CUDA;
  const int split = p.split;
  const int64_t tiles = (p.q.N + p.rows - 1) / p.rows * p.mtiles;
  if (tiles * split > 0x7fffffffLL) return MM_ERR_UNSUPPORTED;
  CUtensorMap w;
  if (!weight_map(p.q, p.rows, &w)) return MM_ERR_UNSUPPORTED;
  p.idesc = make_idesc_mn(1, 0, 0, kRows, NT);
  const auto kernel = int8_stream_kernel<O, NT>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(tiles * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<NT>::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, w, x, p) == cudaSuccess ? MM_OK : MM_ERR_CUDA;
}

template <typename O>
mm_status launch_typed(const StreamArgs& p, int nt, const CUtensorMap& x, cudaStream_t stream) {
  switch (nt) {
    case 16: return launch<O, 16>(p, x, stream);
    case 32: return launch<O, 32>(p, x, stream);
    case 64: return launch<O, 64>(p, x, stream);
    case 128: return launch<O, 128>(p, x, stream);
    default: return launch<O, 256>(p, x, stream);
  }
}

}  // namespace

// B's columns contiguous along k, 16-byte aligned, none inside another (others are copied).
bool int8_stream_supported(const Int8Args& q) {
  return q.K >= 1 && q.b_ks == 1 && (q.N == 1 || (q.b_ns % 16 == 0 && q.b_ns >= q.K)) &&
         (reinterpret_cast<uintptr_t>(q.b) & 15) == 0;
}

// One round of CTAs, or so few rows that the f16 copies of the weights (3 bytes
// moved for each) and a last round of half-empty tiles cost the dense product more.
// us here and there, M = 300, 1024, 2048:
//   4096 x 14336   60  81    94 100   181 159
//   4096 x  4096   22  34    33  37    64  59
//   2048 x  2048   12  19    17  20    22  22
//   1024 x  1024   10  12    11  13    13  15
//   8192 x  1024   22  49    25  52    40  56     (K = 8192)
//    512 x  8192   11  12    22  16    41  23     (K = 512)
bool int8_stream_pays(const Int8Args& q) {
  return q.M <= 256 || (q.M <= 1024 && q.K >= 2048) || (q.M <= 2048 && plan_tiles(q).rounds == 1);
}

mm_status launch_int8_stream(const Int8Args& q, const void* x, int64_t ldx, int w_late, unsigned* status,
                             cudaStream_t stream) {
  if (!status) return MM_ERR_CUDA;
  StreamArgs p;
  memset(&p, 0, sizeof(p));
  p.q = q;
  p.w_late = w_late;
  const TilePlan t = plan_tiles(q);
  const int nt = t.nt;
  p.rows = t.rows;
  p.split = t.split;
  p.num_kb = (int)((q.K + kDepth - 1) / kDepth);
  const int size = q.out_dtype == MM_F32 ? 4 : 2;
  p.y_vec = q.N % 4 == 0 && (reinterpret_cast<uintptr_t>(q.y) & (size * 4 - 1)) == 0;
  p.status = status;
  TcParams limits;
  init_params(&limits);
  p.timeout_ns = limits.timeout_ns;
  p.teardown_ns = limits.teardown_ns;
  OperandPlan xp;
  BatchMap one;
  memset(&one, 0, sizeof(one));
  one.count = 1;
  for (int d = 0; d < kMaxBatchDims; ++d) one.shape[d] = 1;
  const int64_t none[kMaxBatchDims] = {};
  if (!plan_operand(x, MM_F16, q.M, q.K, ldx, 1, one, none, nt, &xp)) return MM_ERR_UNSUPPORTED;
  switch (q.out_dtype) {
    case MM_F32: return launch_typed<float>(p, nt, xp.map, stream);
    case MM_BF16: return launch_typed<__nv_bfloat16>(p, nt, xp.map, stream);
    default: return launch_typed<__half>(p, nt, xp.map, stream);
  }
}

}  // namespace qg
