// C-ABI entry points of the operators whose products select their weights per
// row: top-k routing, the mixture-of-experts layer and the low-rank adapters
// (include/mm.h).  Validation, workspace layout and dispatch only.
#include <cstring>

#include "api_internal.h"
#include "kernels.h"
#include "lowrank.cuh"
#include "moe.cuh"
#include "tc.h"

using namespace qg;

namespace {

bool is_float16_32(int dt) { return dt == MM_BF16 || dt == MM_F16 || dt == MM_F32; }
bool is_index(int dt) { return dt == MM_I32 || dt == MM_I64; }

bool has_shape(const mm_tensor* t, std::initializer_list<int64_t> shape) {
  if (t->ndim != (int)shape.size()) return false;
  int d = 0;
  for (int64_t n : shape)
    if (t->shape[d++] != n) return false;
  return true;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws && have >= need && (reinterpret_cast<uintptr_t>(ws) & 255) == 0);
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ top-k routing

mm_status mm_route_topk(const mm_tensor* logits, int32_t normalize, const mm_tensor* indices,
                        const mm_tensor* weights, void* stream) {
  mm_status s;
  if ((s = check_tensor(logits)) != MM_OK || (s = check_tensor(indices)) != MM_OK ||
      (s = check_tensor(weights)) != MM_OK)
    return s;
  if (!is_float16_32(logits->dtype)) return MM_ERR_DTYPE;
  if (logits->ndim != 2 || indices->ndim != 2) return MM_ERR_SHAPE;
  RouteArgs a;
  memset(&a, 0, sizeof(a));
  a.dtype = logits->dtype;
  a.rows = logits->shape[0]; a.G = logits->shape[1]; a.k = indices->shape[1];
  const int64_t oshape[2] = {a.rows, a.k};
  if ((s = check_output(indices, MM_I32, 2, oshape)) != MM_OK || (s = check_output(weights, MM_F32, 2, oshape)) != MM_OK)
    return s;
  if (a.k < 1 || a.k > a.G || a.k > kRouteMaxPicks) return MM_ERR_SHAPE;
  if (a.G > kRouteMaxExperts) return MM_ERR_UNSUPPORTED;
  if (a.rows == 0) return finish(MM_OK, MM_PATH_NONE);
  a.normalize = normalize != 0;
  a.logits = logits->data; a.l_rs = logits->strides[0]; a.l_cs = logits->strides[1];
  a.indices = indices->data;
  a.weights = weights->data;
  return finish(launch_route_topk(a, static_cast<cudaStream_t>(stream)), MM_PATH_SIMT);
}

mm_status mm_route_topk_grad(const mm_tensor* logits, const mm_tensor* indices, const mm_tensor* grad_weights,
                             int32_t normalize, const mm_tensor* grad_logits, void* stream) {
  mm_status s;
  if ((s = check_tensor(logits)) != MM_OK || (s = check_tensor(indices)) != MM_OK ||
      (s = check_tensor(grad_weights)) != MM_OK)
    return s;
  if (!is_float16_32(logits->dtype) || !is_index(indices->dtype) || grad_weights->dtype != MM_F32) return MM_ERR_DTYPE;
  if (logits->ndim != 2 || indices->ndim != 2) return MM_ERR_SHAPE;
  RouteArgs a;
  memset(&a, 0, sizeof(a));
  a.dtype = logits->dtype;
  a.rows = logits->shape[0]; a.G = logits->shape[1]; a.k = indices->shape[1];
  if (indices->shape[0] != a.rows || !has_shape(grad_weights, {a.rows, a.k})) return MM_ERR_SHAPE;
  if ((s = check_output(grad_logits, a.dtype, 2, logits->shape)) != MM_OK) return s;
  if (a.k < 1 || a.k > a.G || a.k > kRouteMaxPicks) return MM_ERR_SHAPE;
  if (a.G > kRouteMaxExperts) return MM_ERR_UNSUPPORTED;
  if (a.rows == 0) return finish(MM_OK, MM_PATH_NONE);
  a.normalize = normalize != 0;
  a.logits = logits->data; a.l_rs = logits->strides[0]; a.l_cs = logits->strides[1];
  a.indices = indices->data; a.ind64 = indices->dtype == MM_I64;
  a.i_rs = indices->strides[0]; a.i_cs = indices->strides[1];
  a.gw = grad_weights->data; a.gw_rs = grad_weights->strides[0]; a.gw_cs = grad_weights->strides[1];
  a.out = grad_logits->data;
  unsigned* status = device_status_ptr();
  if (!status) return MM_ERR_CUDA;
  return finish(launch_route_topk_grad(a, status, static_cast<cudaStream_t>(stream)), MM_PATH_SIMT);
}

}  // extern "C"

// ------------------------------------------------------------------ mixture-of-experts layer

namespace {

mm_status plan_moe(const mm_tensor* x, const mm_tensor* w_gate, const mm_tensor* w_up, const mm_tensor* w_down,
                   const mm_tensor* gi, MoeArgs* a) {
  mm_status s;
  if ((s = check_tensor(x)) != MM_OK || (s = check_tensor(w_gate)) != MM_OK || (s = check_tensor(w_down)) != MM_OK ||
      (s = check_tensor(gi)) != MM_OK)
    return s;
  if (w_up && (s = check_tensor(w_up)) != MM_OK) return s;
  if (!is_float16_32(x->dtype) || w_gate->dtype != x->dtype || w_down->dtype != x->dtype ||
      (w_up && w_up->dtype != x->dtype) || !is_index(gi->dtype))
    return MM_ERR_DTYPE;
  if (x->ndim != 2 || w_gate->ndim != 3 || w_down->ndim != 3 || gi->ndim != 2) return MM_ERR_SHAPE;
  memset(a, 0, sizeof(*a));
  a->dtype = x->dtype;
  a->ind64 = gi->dtype == MM_I64;
  a->tokens = x->shape[0]; a->K = x->shape[1];
  a->G = w_gate->shape[0]; a->F = w_gate->shape[2];
  a->N = w_down->shape[2]; a->S = gi->shape[1];
  if (w_gate->shape[1] != a->K || gi->shape[0] != a->tokens || w_down->shape[0] != a->G || w_down->shape[1] != a->F ||
      (w_up && !has_shape(w_up, {a->G, a->K, a->F})))
    return MM_ERR_SHAPE;
  a->x = x->data; a->x_rs = x->strides[0]; a->x_cs = x->strides[1];
  a->wg = w_gate->data; a->wg_gs = w_gate->strides[0]; a->wg_ks = w_gate->strides[1]; a->wg_fs = w_gate->strides[2];
  if (w_up) {
    a->wu = w_up->data; a->wu_gs = w_up->strides[0]; a->wu_ks = w_up->strides[1]; a->wu_fs = w_up->strides[2];
  }
  a->wd = w_down->data; a->wd_gs = w_down->strides[0]; a->wd_fs = w_down->strides[1]; a->wd_ns = w_down->strides[2];
  a->gi = gi->data; a->gi_ts = gi->strides[0]; a->gi_ss = gi->strides[1];
  return MM_OK;
}

// A CUDA-core thread walks K and then F, whatever the number of tokens; the
// tensor-core form's time is mostly its three launches.  One token, one pick,
// K = F = 64: 12 us each; 128: 21 against 13 us; 256: 38 against 16 us.
int moe_path(const MoeArgs& a, MoeMaps* maps) {
  return choose(tc_moe_supported(a, maps), a.K + a.F >= 256);
}

size_t moe_simt_bytes(const MoeArgs& a) { return align256((size_t)(a.tokens * a.S) * (size_t)a.F * sizeof(float)); }

}  // namespace

extern "C" {

mm_status mm_moe_layer_workspace_size(const mm_tensor* x, const mm_tensor* w_gate, const mm_tensor* w_up,
                                      const mm_tensor* w_down, const mm_tensor* expert_indices, size_t* bytes) {
  if (!bytes) return MM_ERR_INVALID_ARG;
  MoeArgs a;
  const mm_status s = plan_moe(x, w_gate, w_up, w_down, expert_indices, &a);
  if (s != MM_OK) return s;
  MoeMaps maps;
  *bytes = moe_path(a, &maps) == MM_PATH_TENSOR ? tc_moe_workspace_bytes(a) : moe_simt_bytes(a);
  return MM_OK;
}

mm_status mm_moe_layer(const mm_tensor* x, const mm_tensor* w_gate, const mm_tensor* w_up, const mm_tensor* w_down,
                       const mm_tensor* expert_indices, const mm_tensor* expert_weights, int32_t activation,
                       const mm_tensor* out, void* workspace, size_t workspace_bytes, void* stream) {
  MoeArgs a;
  mm_status s = plan_moe(x, w_gate, w_up, w_down, expert_indices, &a);
  if (s != MM_OK) return s;
  if (activation != MM_ACT_SILU && activation != MM_ACT_GELU && activation != MM_ACT_RELU) return MM_ERR_INVALID_ARG;
  if (expert_weights) {
    if ((s = check_tensor(expert_weights)) != MM_OK) return s;
    if (expert_weights->dtype != MM_F32) return MM_ERR_DTYPE;
    if (!has_shape(expert_weights, {a.tokens, a.S})) return MM_ERR_SHAPE;
    a.ew = expert_weights->data; a.ew_ts = expert_weights->strides[0]; a.ew_ss = expert_weights->strides[1];
  }
  const int64_t oshape[2] = {a.tokens, a.N};
  if ((s = check_output(out, a.dtype, 2, oshape)) != MM_OK) return s;
  a.act = activation;
  a.out = out->data;
  if (a.tokens == 0 || a.N == 0) return finish(MM_OK, MM_PATH_NONE);
  unsigned* status = device_status_ptr();
  if (!status) return MM_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  MoeMaps maps;
  const int path = moe_path(a, &maps);
  if (path < 0) return MM_ERR_UNSUPPORTED;
  if (path == MM_PATH_TENSOR) {
    if (!workspace_ok(workspace, workspace_bytes, tc_moe_workspace_bytes(a))) return MM_ERR_WORKSPACE;
    return finish(launch_tc_moe(a, maps, workspace, status, st), MM_PATH_TENSOR);
  }
  if (!workspace_ok(workspace, workspace_bytes, moe_simt_bytes(a))) return MM_ERR_WORKSPACE;
  return finish(launch_simt_moe(a, static_cast<float*>(workspace), status, st), MM_PATH_SIMT);
}

}  // extern "C"

// ------------------------------------------------------------------ low-rank adapters

namespace {

struct LowRankPlan {
  LowRankArgs l;
  int64_t K, N;
};

// idx may be NULL (workspace queries).
mm_status plan_lowrank(const mm_tensor* X, const mm_tensor* W, const mm_tensor* A, const mm_tensor* B,
                       const mm_tensor* idx, const mm_tensor* scales, LowRankPlan* p) {
  mm_status s;
  for (const mm_tensor* t : {X, W, A, B})
    if ((s = check_tensor(t)) != MM_OK) return s;
  if (!is_float16_32(X->dtype) || W->dtype != X->dtype || A->dtype != X->dtype || B->dtype != X->dtype)
    return MM_ERR_DTYPE;
  if (X->ndim != 2 || W->ndim != 2 || A->ndim != 3 || B->ndim != 3) return MM_ERR_SHAPE;
  memset(p, 0, sizeof(*p));
  p->K = X->shape[1];
  p->N = W->shape[1];
  LowRankArgs& l = p->l;
  l.dtype = X->dtype;
  l.M = X->shape[0]; l.G = A->shape[0]; l.R = A->shape[2];
  if (W->shape[0] != p->K || A->shape[1] != p->K || !has_shape(B, {l.G, l.R, p->N})) return MM_ERR_SHAPE;
  if (l.R > 65535 * 16) return MM_ERR_UNSUPPORTED;
  if (idx) {
    if ((s = check_tensor(idx)) != MM_OK) return s;
    if (!is_index(idx->dtype)) return MM_ERR_DTYPE;
    if (!has_shape(idx, {l.M})) return MM_ERR_SHAPE;
    l.idx = idx->data; l.idx_s = idx->strides[0]; l.ind64 = idx->dtype == MM_I64;
  }
  if (scales) {
    if ((s = check_tensor(scales)) != MM_OK) return s;
    if (scales->dtype != MM_F32) return MM_ERR_DTYPE;
    if (!has_shape(scales, {l.G})) return MM_ERR_SHAPE;
    l.scales = static_cast<const float*>(scales->data); l.scales_s = scales->strides[0];
  }
  return MM_OK;
}

// One factor's z [M, R] (or its shares, for few rows).
size_t factor_bytes(const LowRankArgs& l) {
  const size_t z = (size_t)l.M * (size_t)l.R * sizeof(float);
  return align256(lowrank_few_rows(l.M, l.G) && l.dtype != MM_F32 ? lowrank_few_bytes(l) : z);
}

// Workspace of the many-row gradient kernels.
struct GradLayout {
  FusedLayout fused;     // dX's product; its z is V's
  size_t vt, vt_exp, ut, ut_exp, row, offset, sums_a, sums_b, total;
};
GradLayout grad_layout(const LowRankPlan& p) {
  const LowRankArgs& l = p.l;
  GradLayout w;
  w.fused = lowrank_fused_layout(l, p.K);
  size_t o = w.fused.total;
  auto take = [&](size_t bytes) { const size_t at = o; o = align256(o + bytes); return at; };
  const size_t part = (size_t)l.M * (size_t)w.fused.z_ld * 2, groups = (size_t)((l.R + 63) / 64);
  const size_t exps = l.dtype == MM_F16 ? groups * (size_t)l.M * 4 : 0;
  w.vt = take(2 * part);
  w.vt_exp = take(exps);
  w.ut = take(2 * part);
  w.ut_exp = take(exps);
  w.row = take((size_t)l.M * 4);
  w.offset = take((size_t)(l.G + 1) * 4);
  w.sums_a = take((size_t)lowrank_max_parts(l) * (size_t)p.K * (size_t)l.R * 4);
  w.sums_b = take((size_t)lowrank_max_parts(l) * (size_t)p.N * (size_t)l.R * 4);
  w.total = o;
  return w;
}
// Independent of the operands' layout, so that the workspace query needs none of it.
bool many_rows(const LowRankArgs& l) {
  return path_policy() != MM_PATH_SIMT && (l.dtype == MM_BF16 || l.dtype == MM_F16) && l.M >= 1 && l.R >= 1 &&
         lowrank_sort_supported(l);
}

// What a call asks for, whichever of its kernels then runs: the factors and what
// belongs to them, then (few rows) the low-rank part in fp32.
size_t lowrank_base_bytes(const LowRankPlan& p) {
  const size_t few = factor_bytes(p.l), many = many_rows(p.l) ? lowrank_fused_layout(p.l, p.N).total : 0;
  return few > many ? few : many;
}
size_t lowrank_grad_base_bytes(const LowRankPlan& p) {
  const size_t few = 2 * factor_bytes(p.l), many = many_rows(p.l) ? grad_layout(p).total : 0;
  return few > many ? few : many;
}
bool float_part(const LowRankArgs& l) { return l.dtype != MM_F32 && l.M <= kFloatPartRows; }
size_t part_bytes(const LowRankArgs& l, int64_t N) {
  return float_part(l) ? align256((size_t)l.M * (size_t)N * sizeof(float)) : 0;
}
size_t lowrank_bytes(const LowRankPlan& p) { return lowrank_base_bytes(p) + part_bytes(p.l, p.N); }
size_t lowrank_grad_bytes(const LowRankPlan& p) { return lowrank_grad_base_bytes(p) + part_bytes(p.l, p.K); }

// Y = x w for dense Y [M, N].
GemmArgs projection(const LowRankArgs& l, const void* x, int64_t x_rs, int64_t x_cs, int64_t K, const void* w,
                    int64_t w_rs, int64_t w_cs, int64_t N, void* y) {
  GemmArgs g;
  memset(&g, 0, sizeof(g));
  g.dtype = l.dtype; g.M = l.M; g.N = N; g.K = K;
  g.bm.nb = 0; g.bm.count = 1;
  for (int d = 0; d < kMaxBatchDims; ++d) g.bm.shape[d] = 1;
  g.a.ptr = x; g.a.rs = x_rs; g.a.cs = x_cs;
  g.b.ptr = w; g.b.rs = w_rs; g.b.cs = w_cs;
  g.y.ptr = y; g.y.rs = N; g.y.cs = 1;
  g.alpha = 1.f; g.beta = 1.f; g.alpha_d = 1.0; g.beta_d = 1.0; g.alpha_i = 1; g.beta_i = 1;
  return g;
}

// Y = x w plus the low-rank part, which an expansion puts at part() before: an
// fp32 array of the workspace (few rows) or Y itself.
struct Projection {
  GemmArgs g;
  int path;
  bool f32;
  void* part() const { return const_cast<void*>(g.c.ptr); }
  mm_status run(cudaStream_t st) const { return run_dense_on(path, g, st); }
};
Projection plan_projection(const LowRankArgs& l, const GemmArgs& g, char* float_array) {
  Projection p;
  // A long sum over k leaves the CUDA-core tiles waiting even where the work is
  // small: 4 rows of 512 x 512 take 17 us there and 8 us on the tensor cores.
  const bool long_k = g.dtype != MM_F32 && g.K >= 256;
  p.g = g;
  // Every kernel of the dense product reads an element of C in the thread
  // that then writes that element of Y (or before its tile's store).
  p.g.c = g.y;
  p.f32 = false;
  p.path = dense_path(p.g, long_k || tensor_pays_dense(g.dtype, g.M, g.N, g.K, 1), float_part(l) ? &p.f32 : nullptr);
  if (p.f32) {
    p.g.c.ptr = float_array;
    p.g.c.rs = 2 * g.N;
    p.g.c.cs = 2;
    p.g.c_f32 = 1;
  }
  return p;
}

// Whether a 16-bit product may take the fused kernel (the dense products' rules).
bool fused_pays(const LowRankArgs& l, const GemmArgs& g, LowRankProduct* plan) {
  return choose(true, tensor_pays_dense(g.dtype, g.M, g.N, g.K, 1)) == MM_PATH_TENSOR && lowrank_fused_supported(l, g, plan);
}

}  // namespace

extern "C" {

mm_status mm_lowrank_matmul_workspace_size(const mm_tensor* X, const mm_tensor* W, const mm_tensor* A,
                                           const mm_tensor* B, size_t* bytes) {
  if (!bytes) return MM_ERR_INVALID_ARG;
  LowRankPlan p;
  const mm_status s = plan_lowrank(X, W, A, B, nullptr, nullptr, &p);
  if (s != MM_OK) return s;
  *bytes = lowrank_bytes(p);
  return MM_OK;
}

mm_status mm_lowrank_matmul(const mm_tensor* X, const mm_tensor* W, const mm_tensor* A, const mm_tensor* B,
                            const mm_tensor* adapter_indices, const mm_tensor* scales, const mm_tensor* Y,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (!adapter_indices) return MM_ERR_INVALID_ARG;
  LowRankPlan p;
  mm_status s = plan_lowrank(X, W, A, B, adapter_indices, scales, &p);
  if (s != MM_OK) return s;
  LowRankArgs& l = p.l;
  const int64_t yshape[2] = {l.M, p.N};
  if ((s = check_output(Y, l.dtype, 2, yshape)) != MM_OK) return s;
  if (l.M == 0 || p.N == 0) return finish(MM_OK, MM_PATH_NONE);
  if (!workspace_ok(workspace, workspace_bytes, lowrank_bytes(p))) return MM_ERR_WORKSPACE;
  if (!(l.status = device_status_ptr())) return MM_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* z = static_cast<float*>(workspace);
  const GemmArgs g = projection(l, X->data, X->strides[0], X->strides[1], p.K, W->data, W->strides[0], W->strides[1], p.N,
                                Y->data);
  char* float_array = static_cast<char*>(workspace) + lowrank_base_bytes(p);
  LowRankFew f = {X->data, X->strides[0], X->strides[1], p.K, A->data, A->strides[0], A->strides[1], A->strides[2],
                  B->data, B->strides[0], B->strides[1], B->strides[2], p.N, nullptr, 0};
  if (path_policy() != MM_PATH_SIMT && lowrank_few_supported(l, f)) {
    Projection late = plan_projection(l, g, float_array);
    if (late.path < 0) return MM_ERR_UNSUPPORTED;
    f.y = late.part();
    f.y_f32 = late.f32;
    if ((s = launch_lowrank_few(l, f, z, st)) != MM_OK) return s;
    // The expansion lets the product start while it runs; the first of the two
    // launches waited for all earlier work, X and W included.
    late.g.c_late = 1;
    return late.run(st);
  }
  OperandPlan x_map;
  LowRankProduct product;
  if (many_rows(l) && p.K >= 1 &&
      lowrank_shrink_tiles_supported(l, X->data, X->strides[0], X->strides[1], p.K, A->strides[1], A->strides[2], &x_map) &&
      fused_pays(l, g, &product)) {
    const FusedLayout w = lowrank_fused_layout(l, p.N);
    char* ws = static_cast<char*>(workspace);
    z = reinterpret_cast<float*>(ws + w.z);
    const FusedTables slots = lowrank_fused_tables(w, ws);
    const LowRankShrink q = {&x_map, p.K, A->data, A->strides[0], A->strides[1], A->strides[2], z,
                             slots.wide, nullptr, nullptr};
    s = launch_lowrank_shrink_tiles(l, &q, 1, w.z_ld, &slots, nullptr, st);
    const LowRankFused u = {g, &product, &w, ws, z, B->data, B->strides[0], B->strides[1], B->strides[2]};
    if (s == MM_OK) s = launch_lowrank_finish(l, &u, nullptr, nullptr, 0, w.z_ld, st);
    return finish(s, MM_PATH_TENSOR);
  }
  if ((s = launch_lowrank_shrink(l, X->data, X->strides[0], X->strides[1], p.K, A->data, A->strides[0], A->strides[1],
                                 A->strides[2], z, st)) != MM_OK)
    return s;
  const Projection rest = plan_projection(l, g, float_array);
  if ((s = launch_lowrank_expand(l, z, l.R, B->data, B->strides[0], B->strides[1], B->strides[2], p.N, rest.part(),
                                 rest.f32, st)) != MM_OK)
    return s;
  return rest.run(st);
}

mm_status mm_lowrank_matmul_grad_workspace_size(const mm_tensor* X, const mm_tensor* W, const mm_tensor* A,
                                                const mm_tensor* B, size_t* bytes) {
  if (!bytes) return MM_ERR_INVALID_ARG;
  LowRankPlan p;
  const mm_status s = plan_lowrank(X, W, A, B, nullptr, nullptr, &p);
  if (s != MM_OK) return s;
  *bytes = lowrank_grad_bytes(p);
  return MM_OK;
}

mm_status mm_lowrank_matmul_grad(const mm_tensor* dY, const mm_tensor* X, const mm_tensor* W, const mm_tensor* A,
                                 const mm_tensor* B, const mm_tensor* adapter_indices, const mm_tensor* scales,
                                 const mm_tensor* dX, const mm_tensor* dA, const mm_tensor* dB, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (!adapter_indices) return MM_ERR_INVALID_ARG;
  LowRankPlan p;
  mm_status s = plan_lowrank(X, W, A, B, adapter_indices, scales, &p);
  if (s != MM_OK) return s;
  LowRankArgs& l = p.l;
  const int64_t K = p.K, N = p.N;
  if ((s = check_tensor(dY)) != MM_OK) return s;
  if (dY->dtype != l.dtype) return MM_ERR_DTYPE;
  if (!has_shape(dY, {l.M, N})) return MM_ERR_SHAPE;
  const int64_t xshape[2] = {l.M, K}, ashape[3] = {l.G, K, l.R}, bshape[3] = {l.G, l.R, N};
  if (dX && (s = check_output(dX, l.dtype, 2, xshape)) != MM_OK) return s;
  if (dA && (s = check_output(dA, l.dtype, 3, ashape)) != MM_OK) return s;
  if (dB && (s = check_output(dB, l.dtype, 3, bshape)) != MM_OK) return s;
  if (!workspace_ok(workspace, workspace_bytes, lowrank_grad_bytes(p))) return MM_ERR_WORKSPACE;
  if (!(l.status = device_status_ptr())) return MM_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* v = static_cast<float*>(workspace);
  float* u = reinterpret_cast<float*>(static_cast<char*>(workspace) + factor_bytes(l));
  char* float_array = static_cast<char*>(workspace) + lowrank_grad_base_bytes(p);
  s = finish(MM_OK, MM_PATH_NONE);
  OperandPlan dy_map, x_map;
  if (many_rows(l) && K >= 1 && N >= 1 &&
      lowrank_shrink_tiles_supported(l, dY->data, dY->strides[0], dY->strides[1], N, B->strides[2], B->strides[1],
                                     &dy_map) &&
      lowrank_shrink_tiles_supported(l, X->data, X->strides[0], X->strides[1], K, A->strides[1], A->strides[2], &x_map)) {
    const GradLayout w = grad_layout(p);
    char* ws = static_cast<char*>(workspace);
    float* zv = reinterpret_cast<float*>(ws + w.fused.z);
    int32_t* v_exp = reinterpret_cast<int32_t*>(ws + w.vt_exp);
    int32_t* u_exp = reinterpret_cast<int32_t*>(ws + w.ut_exp);
    const int64_t z_ld = w.fused.z_ld;
    const AdapterRows t = {reinterpret_cast<int32_t*>(ws + w.row), reinterpret_cast<int32_t*>(ws + w.offset)};
    const FusedTables slots = lowrank_fused_tables(w.fused, ws);
    LowRankShrink q[2];
    int factors = 0;
    if (dX || dA)
      q[factors++] = {&dy_map, N, B->data, B->strides[0], B->strides[2], B->strides[1],
                      dX ? zv : nullptr, dX ? slots.wide : nullptr, dA ? ws + w.vt : nullptr, v_exp};
    if (dB)
      q[factors++] = {&x_map, K, A->data, A->strides[0], A->strides[1], A->strides[2], nullptr, nullptr,
                      ws + w.ut, u_exp};
    if (factors) s = launch_lowrank_shrink_tiles(l, q, factors, z_ld, dX ? &slots : nullptr, dA || dB ? &t : nullptr, st);
    LowRankOuter o[2];
    int problems = 0;
    if (dA)
      o[problems++] = {X->data, X->strides[0], K, ws + w.vt, v_exp, dA->data, l.R, 1, reinterpret_cast<float*>(ws + w.sums_a)};
    if (dB)
      o[problems++] = {dY->data, dY->strides[0], N, ws + w.ut, u_exp, dB->data, 1, N, reinterpret_cast<float*>(ws + w.sums_b)};
    const GemmArgs g = projection(l, dY->data, dY->strides[0], dY->strides[1], N, W->data, W->strides[1], W->strides[0], K,
                                  dX ? dX->data : nullptr);
    LowRankProduct product;
    const bool fuse = dX && fused_pays(l, g, &product);
    const LowRankFused u = {g, &product, &w.fused, ws, zv, A->data, A->strides[0], A->strides[2], A->strides[1]};
    if (s == MM_OK && (problems || fuse))
      s = finish(launch_lowrank_finish(l, fuse ? &u : nullptr, &t, o, problems, z_ld, st),
                 fuse ? MM_PATH_TENSOR : MM_PATH_SIMT);
    if (s == MM_OK && dX && !fuse) {
      const Projection rest = plan_projection(l, g, float_array);
      s = launch_lowrank_expand(l, zv, z_ld, A->data, A->strides[0], A->strides[2], A->strides[1], K, rest.part(), rest.f32,
                                st);
      if (s == MM_OK) s = rest.run(st);
    }
    return s;
  }
  if (dX || dA)
    s = launch_lowrank_shrink(l, dY->data, dY->strides[0], dY->strides[1], N, B->data, B->strides[0], B->strides[2],
                              B->strides[1], v, st);
  if (s == MM_OK && dB)
    s = launch_lowrank_shrink(l, X->data, X->strides[0], X->strides[1], K, A->data, A->strides[0], A->strides[1],
                              A->strides[2], u, st);
  if (s == MM_OK && dA)
    s = launch_lowrank_outer(l, X->data, X->strides[0], X->strides[1], K, v, dA->data, K * l.R, l.R, 1, st);
  if (s == MM_OK && dB)
    s = launch_lowrank_outer(l, dY->data, dY->strides[0], dY->strides[1], N, u, dB->data, l.R * N, 1, N, st);
  if (s == MM_OK && dX && l.M > 0 && K > 0) {
    const Projection rest = plan_projection(l, projection(l, dY->data, dY->strides[0], dY->strides[1], N, W->data,
                                                          W->strides[1], W->strides[0], K, dX->data), float_array);
    s = launch_lowrank_expand(l, v, l.R, A->data, A->strides[0], A->strides[2], A->strides[1], K, rest.part(), rest.f32, st);
    if (s == MM_OK) s = rest.run(st);
  }
  return s;
}

}  // extern "C"
