// Launchers implemented by the kernel translation units and called by the
// C-ABI layer (api.cu).  Every launcher enqueues work on `stream` and returns
// MM_OK or MM_ERR_CUDA; arguments have been validated by the caller.
#pragma once

#include "common.cuh"

namespace qg {

// MatMul and Gemm: Y[b] = alpha * A[b] @ B[b] + beta * C (C broadcast view).
struct GemmArgs {
  int dtype;                 // mm_dtype shared by A, B, C, Y
  int64_t M, N, K;
  BatchMap bm;
  MatView a;                 // rows M, cols K
  MatView b;                 // rows K, cols N
  MatView c;                 // rows M, cols N (strides 0 where broadcast); ptr null = absent
  MatView y;                 // rows M, cols N, dense
  float alpha, beta;         // float types
  double alpha_d, beta_d;    // f64
  uint64_t alpha_i, beta_i;  // integer types: two's complement of the integral values
  // C and Y are touched by the previous launch on the stream, while A and B
  // were complete before that launch began: a few-row kernel may then read A
  // and B at once and wait for the previous launch only before its epilogue.
  int c_late;
  // 16-bit types: C holds fp32 values (c.rs, c.cs and the batch strides count
  // 16-bit units all the same).  Not every kernel takes it (dense_path).
  int c_f32;
  // Integer types with a non-integral alpha or beta: y = trunc(alpha*acc + beta*c)
  // evaluated in fp64 (each product, then the sum, rounded once), saturated to T.
  int int_float;
};

// QLinearMatMul.
struct QLinearArgs {
  int64_t M, N, K;
  BatchMap bm;
  MatView a, b, y;           // a: rows M cols K; b: rows K cols N; y dense
  int64_t a_bshape[kMaxBatchDims], b_bshape[kMaxBatchDims];  // operands' own batch sizes (1 = broadcast)
  VecView sa, za;            // indexed by row m (vs = 0 for per-tensor)
  VecView sb, zb;            // indexed by column n
  const void* ys;            // y_scale (one element)
  const void* yz;            // y_zero_point (one element)
  int a_signed, b_signed, y_signed;
  int sa_f16, sb_f16, ys_f16;
};

// GroupedMatMul.
struct GroupedArgs {
  int dtype;                 // T
  int ind64;                 // Tind is int64
  int64_t M, K, N, G, S;
  const void* x;   int64_t x_rs, x_cs;
  const void* w;   int64_t w_gs, w_ks, w_ns;
  const void* gi;  int64_t gi_ms, gi_ss;
  const void* bias; int64_t bias_gs, bias_ns;   // bias null = absent
  void* out;                 // dense [M, S, N]
  // Weight-only quantized experts: w holds int8 (wq == 1), uint8 (2), int4
  // (3) or uint4 (4) values and the weights are W = T((w - zero_point) *
  // scale), scale and zero point [G, Kb, N] indexed by (g, k / qblock, n).
  // 4-bit values are packed two per byte (element offset e: the low nibble
  // of byte e / 2 when e is even, else its high nibble; strides in elements).
  // wq == 0: w is T.
  int wq;
  const void* wsc; int64_t wsc_gs, wsc_bs, wsc_ns;   // scale, type T
  const void* wzp; int64_t wzp_gs, wzp_bs, wzp_ns;   // zero point (null = 0), type of w
  int64_t qblock;
};

// Top-k routing (mm_route_topk) and its gradient.
struct RouteArgs {
  int dtype;                 // T of logits (and grad_logits)
  int64_t rows, G, k;
  int normalize;
  const void* logits; int64_t l_rs, l_cs;
  void* indices; int64_t i_rs, i_cs;           // forward: out, dense int32; gradient: in, int32 or int64
  int ind64;
  void* weights;                               // forward: out, dense f32
  const void* gw; int64_t gw_rs, gw_cs;        // gradient: of the weights, f32
  void* out;                                   // gradient: of the logits, dense T
};
constexpr int64_t kRouteMaxExperts = 1024, kRouteMaxPicks = 32;

// The router's balance loss (mm_route_balance) and its gradient.
struct BalanceArgs {
  int dtype;                 // T of logits
  int ind64;
  int64_t rows, G, k;
  const void* logits;  int64_t l_rs, l_cs;
  const void* indices; int64_t i_rs, i_cs;
  float* loss;               // [1]
  int32_t* counts;           // [G + 1]: picks per expert, rows that take part
  float* mean;               // [G]
};
struct BalanceGradArgs {
  int dtype;
  int64_t rows, G;
  const void* logits; int64_t l_rs, l_cs;
  const int32_t* counts; int64_t counts_s;
  const float* dloss;        // [1]
  const void* base; int64_t b_rs, b_cs;        // T, null = none
  void* out;                 // dense T
};

// Rows to int8 with a scale each (mm_quantize_rows).
struct QuantizeArgs {
  int dtype;                 // of x
  int64_t M, K;
  const void* x; int64_t x_rs, x_cs;
  int8_t* q;                 // dense [M, K]
  float* scales;             // [M]
};

// 8-bit product with scales (mm_int8_matmul).
struct Int8Args {
  int out_dtype;             // of y and bias
  int64_t M, N, K;
  const int8_t* a; int64_t a_rs, a_cs;
  const int8_t* b; int64_t b_ks, b_ns;
  const float* sa; int64_t sa_s;
  const float* sb; int64_t sb_s;
  const void* bias; int64_t bias_s;            // null = none
  void* y;                   // dense [M, N]
};
constexpr int kInt8FewRows = 8, kInt8LooseRows = 4, kInt8FewCols = 2;
constexpr int64_t kInt8FewDepth = 8191 * 32 * 16;      // K: a lane's share of int32 sums
// An operand's copy, f16 or (bytes) int8: dst[r, c] = src[r * rs + c * cs], rows of
// `ld` values.
struct Int8Copy {
  const int8_t* src; int64_t rs, cs, rows, cols, ld;
  void* dst;
  int bytes;
};

// Orthogonalised update (mm_orthogonalize).
struct OrthoArgs {
  int dtype;
  int64_t M, N;
  BatchMap bm;
  MatView x;                 // any strides
  void* out;                 // dense
  int steps;
  const float* coef;         // host, [steps][3]
  float eps, scale;
};

// Mixture-of-experts layer (mm_moe_layer).
struct MoeArgs {
  int dtype;                 // T
  int ind64, act;
  int64_t tokens, S, G, K, F, N;
  const void* x;    int64_t x_rs, x_cs;
  const void* wg;   int64_t wg_gs, wg_ks, wg_fs;
  const void* wu;   int64_t wu_gs, wu_ks, wu_fs;   // null = no up projection
  const void* wd;   int64_t wd_gs, wd_fs, wd_ns;
  const void* gi;   int64_t gi_ts, gi_ss;
  const void* ew;   int64_t ew_ts, ew_ss;          // f32 (null = 1)
  void* out;                 // dense [tokens, N]
};

// Per-row low-rank adapters (mm_lowrank_matmul and its gradient).
struct LowRankArgs {
  int dtype;                 // T
  int ind64;
  int64_t M, G, R;
  const void* idx;  int64_t idx_s;
  const float* scales; int64_t scales_s;           // null = 1
  unsigned* status;
};

mm_status launch_route_topk(const RouteArgs& args, cudaStream_t stream);
mm_status launch_route_topk_grad(const RouteArgs& args, unsigned* status, cudaStream_t stream);

// Partial sums of every block, then one cluster that adds them.
int64_t balance_partial_blocks(int64_t rows);
size_t balance_workspace_bytes(int64_t rows, int64_t G);
mm_status launch_balance(const BalanceArgs& args, void* workspace, unsigned* status, cudaStream_t stream);
mm_status launch_balance_grad(const BalanceGradArgs& args, cudaStream_t stream);

mm_status launch_quantize_rows(const QuantizeArgs& args, cudaStream_t stream);
// Few rows against columns of B contiguous along k (16-byte aligned); every
// stride; the operands' copies for the tensor cores (A f16, B either).
bool int8_few_aligned(const Int8Args& args);
mm_status launch_int8_few_aligned(const Int8Args& args, cudaStream_t stream);
bool int8_few_supported(const Int8Args& args);         // aligned or not
mm_status launch_int8_few(const Int8Args& args, cudaStream_t stream);
mm_status launch_int8_any(const Int8Args& args, cudaStream_t stream);
mm_status launch_int8_copies(const Int8Copy& A, const Int8Copy& B, cudaStream_t stream);

// The norm, the division and the chain of products; or one launch, for matrices that
// fit a cluster's shared memory: with m the smaller side, any stack of m <= 64, of
// which a tile of the chain would use a quarter at most, and up to kOrthoSmallWork =
// m m n matrices above.  us in one launch and in the chain:
//   64 x 1000        62 177      300 of 64 x 64     110 209    128 x 1000       183 237
//   64 x 4000       163 300      300 of 64 x 256    209 295    8 of 128 x 512   135 189
//   200 of 32 x 32   25 137      1000 of 64 x 64    379 590    30 of 128 x 256  139 180
//   500 of 32 x 512 200 640      256 of 64 x 512    344 437    100 of 128 x 128 267 189
constexpr double kOrthoSmallWork = 1.5e8;
size_t ortho_workspace_bytes(const OrthoArgs& args);
mm_status launch_ortho(const OrthoArgs& args, void* workspace, cudaStream_t stream);

// h[t * S + s, f] (f32) and then the weighted sum over s, on the CUDA cores.
mm_status launch_simt_moe(const MoeArgs& args, float* h, unsigned* status, cudaStream_t stream);

// z[m, r] = scale_g * sum_c x[m, c] a[g, c, r], g the adapter of row m (0 without one).
mm_status launch_lowrank_shrink(const LowRankArgs& l, const void* x, int64_t x_rs, int64_t x_cs, int64_t C,
                                const void* a, int64_t a_gs, int64_t a_cs, int64_t a_rs, float* z,
                                cudaStream_t stream);
// y[m, n] = sum_r z[m, r] b[g, r, n] (dense rows of N; rows of z z_ld apart), rounded to T or fp32 (y_f32).
mm_status launch_lowrank_expand(const LowRankArgs& l, const float* z, int64_t z_ld, const void* b, int64_t b_gs,
                                int64_t b_rs, int64_t b_ns, int64_t N, void* y, int y_f32, cudaStream_t stream);
// out[g, c, r] = sum over the rows m of adapter g of x[m, c] z[m, r] (element strides of out given).
mm_status launch_lowrank_outer(const LowRankArgs& l, const void* x, int64_t x_rs, int64_t x_cs, int64_t C,
                               const float* z, void* out, int64_t o_gs, int64_t o_cs, int64_t o_rs,
                               cudaStream_t stream);

// Few rows of 16-bit types: both steps with vector reads, z's shares in zp.
// The host does not know whether rows of one adapter are neighbours, nor how
// many of the G adapters are in use.  The many-row kernels (lowrank_tc.cu) make
// one pass per adapter and row tile; these read each row's own adapter and do
// not care.  us for rows in random order and in runs, N = K = 4096, rank 16:
//      M     G    many-row         here
//    256     8    48   47         40   40
//    512     8    49   46         52   52
//    512    32    76   54         52   52
//   1024    16    73   48         73   73
//   1024    64   124   57         74   75
//   2048   128   267   91        142  147
//   4096   256   566  254        314  310
//  16384  1000  1996 1041       1304 1248
// so these take up to kFewPerAdapter rows per adapter, or kFewRows in all.
constexpr int64_t kFewRows = 256, kFewPerAdapter = 16, kFewMost = 16384;
inline bool lowrank_few_rows(int64_t M, int64_t G) {
  return M <= kFewRows || (M <= kFewMost && (M + kFewPerAdapter - 1) / kFewPerAdapter <= G);
}
struct LowRankFew {
  const void* x; int64_t x_rs, x_cs, C;
  const void* a; int64_t a_gs, a_cs, a_rs;     // [G, C, R]
  const void* b; int64_t b_gs, b_rs, b_ns;     // [G, R, N]
  int64_t N;
  void* y;                                     // dense [M, N]: T, or fp32
  int y_f32;
};
// Up to kFloatPartRows rows (those of the few-row products, which take C in
// fp32) the low-rank part joins the projection unrounded, from an fp32 [M, N]
// array; above, that array would outweigh the adapters, and the part is rounded
// to T in Y.  Rounded and not: one row of 4096 x 4096, rank 16, 11.2 and 11.5 us;
// 61 rows of 4096 x 14336, rank 32, 42.9 and 42.4 us.
constexpr int64_t kFloatPartRows = 64;
bool lowrank_few_supported(const LowRankArgs& l, const LowRankFew& f);
size_t lowrank_few_bytes(const LowRankArgs& l);
mm_status launch_lowrank_few(const LowRankArgs& l, const LowRankFew& f, float* zp, cudaStream_t stream);

mm_status launch_simt_gemm(const GemmArgs& args, cudaStream_t stream);
// Multiprocessors of the current device (cached per device).
int sm_count_public();
// Products with at most kVecMaxRows rows of A' (bf16, f16, f32): one pass over
// B' on the CUDA cores, for K-major B' (k contiguous in A' and B', 16-byte
// aligned rows of A' and columns of B') and for MN-major B' (n contiguous,
// 16-byte aligned rows of B'; A' any strides).  vec_gemm_supported says
// whether launch_vec_gemm takes the call, vec_gemm_preferred whether the
// planner should send it there.
constexpr int kVecMaxRows = 4;
bool vec_gemm_supported(const GemmArgs& args);
bool vec_gemm_preferred(const GemmArgs& args);
mm_status launch_vec_gemm(const GemmArgs& args, cudaStream_t stream);
mm_status launch_simt_qlinear(const QLinearArgs& args, cudaStream_t stream);
mm_status launch_simt_grouped(const GroupedArgs& args, unsigned* status, cudaStream_t stream);

// Streaming measurement kernels (stream.cu): bytes is a multiple of 16 and the
// buffers are 16-byte aligned (checked by the caller).
enum { kStreamWrite = 0, kStreamCopy = 1, kStreamWriteBulk = 2 };
// Arithmetic-rate probe: dependent multiply-add chains of one instruction.
enum { kAluImad = 0, kAluDfma = 1, kAluFfma = 2 };
constexpr int kAluChains = 16;     // independent chains per thread
constexpr int kAluThreads = 256;   // threads per block
constexpr int kAluBlocksPerSm = 4;
mm_status launch_alu_probe(int op, void* out, int64_t iters, int* threads_out, cudaStream_t stream);
mm_status launch_stream_probe(void* dst, const void* src, int64_t bytes, int mode, cudaStream_t stream);

}  // namespace qg
