// Tensor-core (tcgen05 / TMEM / TMA) paths for sm_103a.  Each *_supported()
// says whether the operands' types and layouts fit the kernels; the launchers
// enqueue the work on `stream`.
#pragma once

#include "kernels.h"

namespace qg {

// Limit of each pipeline wait in the tensor-core kernels (0 = the 2 s default).
void tc_set_wait_limit_ns(unsigned long long ns);

bool tc_gemm_supported(const GemmArgs& g);
// Whether launch_tc_gemm takes the few-row configuration (which takes a c_f32 call).
bool tc_gemm_few_rows(const GemmArgs& g);
mm_status launch_tc_gemm(const GemmArgs& g, unsigned* status, cudaStream_t stream);

bool tc_qlinear_supported(const QLinearArgs& q);
size_t tc_qlinear_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t a_count, int64_t b_count);
mm_status launch_tc_qlinear(const QLinearArgs& q, void* workspace, unsigned* status, cudaStream_t stream);

// Y = (A B) scaled per row and per column plus a bias, of f16 copies a (rows
// lda apart, K-major) and b (K-major [N, ldb], or with b_mn [K, ldb]).
mm_status launch_tc_int8(const Int8Args& q, const void* a, int64_t lda, const void* b, int64_t ldb, int b_mn,
                         unsigned* status, cudaStream_t stream);

// The same for fewer rows, of a's f16 copy (rows ldx apart) and int8 weights whose
// columns are contiguous along k and 16-byte aligned, as they lie or as a copy that
// the launch before makes (w_late).
bool int8_stream_supported(const Int8Args& q);
bool int8_stream_pays(const Int8Args& q);
mm_status launch_int8_stream(const Int8Args& q, const void* x, int64_t ldx, int w_late, unsigned* status,
                             cudaStream_t stream);

// A product of the orthogonalised update's chain, over `count` matrices of f16
// operands: sym != 0, Y = f16(alpha A B + beta C), symmetric (C optional); else
// the state's step S = alpha A B + beta S in fp32, in place, with Y = f16(up S);
// the last step rounds its result to y_dtype instead and leaves S as it was.
struct OrthoProduct {
  int sym, last, y_dtype;
  int64_t M, N, K, count;
  const void* a; int64_t a_rs, a_cs, a_step;
  const void* b; int64_t b_rs, b_cs, b_step;
  const void* c; int64_t c_rs, c_step;
  void* y; int64_t y_rs, y_step;
  float alpha, beta;
  float* s32; int64_t s_rs, s_step;
  float up;
  // split: operands, C and f16 results are pairs, their rests count matrices further.
  // Sums of `segment` products along K (a multiple of 64) are added up in fp32.
  int split, segment;
};
mm_status launch_tc_ortho(const OrthoProduct& g, unsigned* status, cudaStream_t stream);

bool tc_grouped_supported(const GroupedArgs& g);
size_t tc_grouped_workspace_bytes(const GroupedArgs& g);
// GroupedArgs with wq != 0 take the fused-dequantisation kernel (CTA pairs):
// the weights stay int8/uint8 in memory and are dequantised in shared memory.
mm_status launch_tc_grouped(const GroupedArgs& g, void* workspace, unsigned* status, cudaStream_t stream);

// Y = A B (16-bit, no batch) plus, per row tile, the products of the rows'
// factors with their adapters (device tables as TcParams describes them).
struct LowRankExt {
  const void* factors;           // [row tiles * per_tile * tile_rows, factor_ld], factor_ld a multiple of 64
  int64_t factor_ld, per_tile;   // per_tile: adapters that a tile can list
  const void* adapters;          // [slots, k_rows, adapter_ld], finite, adapter_ld a multiple of 8
  int64_t slots, k_rows, adapter_ld;
  const int32_t* count;
  const int32_t* slot;
  const int32_t* head;           // [1]: whether any row's Y holds a part to add
  const int32_t* row_c;          // [M] (read when it does): rows whose Y does
};
// The product's row tiles (256 rows: CTA pairs, 128: single CTAs) and operands,
// planned once per call; false where it does not fit the kernel.
struct LowRankProduct;
bool tc_lowrank_plan(const GemmArgs& g, LowRankProduct* plan);
mm_status launch_tc_lowrank(const GemmArgs& g, const LowRankProduct& plan, const LowRankExt& e, unsigned* status,
                            cudaStream_t stream);

// The mixture-of-experts layer for a few tokens (moe_tc.cu): every matrix with
// 16-byte aligned rows along a unit-stride matrix dimension, w_gate and w_up
// with the same one.  `maps` receives the weights' tensor maps for the launch.
struct MoeMaps;
bool tc_moe_supported(const MoeArgs& a, MoeMaps* maps);
size_t tc_moe_workspace_bytes(const MoeArgs& a);
mm_status launch_tc_moe(const MoeArgs& a, const MoeMaps& maps, void* workspace, unsigned* status, cudaStream_t stream);

}  // namespace qg
