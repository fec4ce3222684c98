// C-ABI entry points of the 8-bit product with its quantisation and of the
// orthogonalised update (include/mm.h).  Validation, workspace layout and
// dispatch only.
#include <cmath>
#include <cstring>

#include "api_internal.h"
#include "kernels.h"
#include "tc.h"

using namespace qg;

namespace {

bool is_vector(const mm_tensor* t, int64_t n) { return t->ndim == 1 && t->shape[0] == n; }

}  // namespace

extern "C" {

// ------------------------------------------------------------------ quantisation of rows

mm_status mm_quantize_rows(const mm_tensor* x, const mm_tensor* q, const mm_tensor* scales, void* stream) {
  mm_status s;
  if ((s = check_tensor(x)) != MM_OK) return s;
  if (!is_float16_32(x->dtype)) return MM_ERR_DTYPE;
  if (x->ndim != 2) return MM_ERR_SHAPE;
  if ((s = check_output(q, MM_I8, 2, x->shape)) != MM_OK || (s = check_output(scales, MM_F32, 1, x->shape)) != MM_OK)
    return s;
  QuantizeArgs a;
  memset(&a, 0, sizeof(a));
  a.dtype = x->dtype;
  a.M = x->shape[0]; a.K = x->shape[1];
  if (a.M >= (1ll << 31)) return MM_ERR_UNSUPPORTED;
  if (a.M == 0) return finish(MM_OK, MM_PATH_NONE);
  a.x = x->data; a.x_rs = x->strides[0]; a.x_cs = a.K == 1 ? 1 : x->strides[1];
  a.q = static_cast<int8_t*>(q->data);
  a.scales = static_cast<float*>(scales->data);
  return finish(launch_quantize_rows(a, static_cast<cudaStream_t>(stream)), MM_PATH_SIMT);
}

}  // extern "C"

// ------------------------------------------------------------------ 8-bit product

namespace {

mm_status plan_int8(const mm_tensor* A, const mm_tensor* B, int32_t out_dtype, Int8Args* a) {
  mm_status s;
  if ((s = check_tensor(A)) != MM_OK || (s = check_tensor(B)) != MM_OK) return s;
  if (A->dtype != MM_I8 || B->dtype != MM_I8 || !is_float16_32(out_dtype)) return MM_ERR_DTYPE;
  if (A->ndim != 2 || B->ndim != 2 || A->shape[1] != B->shape[0]) return MM_ERR_SHAPE;
  memset(a, 0, sizeof(*a));
  a->out_dtype = out_dtype;
  a->M = A->shape[0]; a->K = A->shape[1]; a->N = B->shape[1];
  if (a->M >= (1ll << 31) || a->N >= (1ll << 31) || a->K >= (1ll << 31)) return MM_ERR_UNSUPPORTED;
  a->a = static_cast<const int8_t*>(A->data);
  a->b = static_cast<const int8_t*>(B->data);
  a->a_rs = A->strides[0]; a->a_cs = A->strides[1];
  a->b_ks = B->strides[0]; a->b_ns = B->strides[1];
  return MM_OK;
}

// The tensor cores' f16 copies: A [M, lda]; B as it lies, [N, ldb] or (columns
// contiguous) [K, ldb].
struct Int8Plan {
  int path, stream, as_is;   // stream: B in bytes, K-major, as it lies or as a copy [N, ldb]
  int64_t lda, ldb;
  int b_mn;
  size_t a, b, bytes;
};
Int8Plan int8_path(const Int8Args& a) {
  Int8Plan p;
  memset(&p, 0, sizeof(p));
  const int pol = path_policy();
  if ((pol == MM_PATH_AUTO || pol == MM_PATH_VECTOR) && int8_few_supported(a)) {
    p.path = MM_PATH_VECTOR;
    return p;
  }
  p.path = choose(a.K > 0, tensor_pays(a.M, a.N, a.K, 1));
  if (p.path != MM_PATH_TENSOR) return p;
  p.lda = (a.K + 7) / 8 * 8;
  if (int8_stream_pays(a)) {
    p.stream = 1;
    p.as_is = int8_stream_supported(a);
    p.ldb = (a.K + 15) / 16 * 16;
    p.b = align256((size_t)a.M * (size_t)p.lda * 2);
    p.bytes = p.b + (p.as_is ? 0 : align256((size_t)a.N * (size_t)p.ldb));
    return p;
  }
  p.b_mn = a.b_ns == 1 && a.b_ks != 1;      // (only the dense product's copy keeps that order)
  p.ldb = ((p.b_mn ? a.N : a.K) + 7) / 8 * 8;
  p.a = 0;
  p.b = align256((size_t)a.M * (size_t)p.lda * 2);
  p.bytes = p.b + align256((size_t)(p.b_mn ? a.K : a.N) * (size_t)p.ldb * 2);
  return p;
}

}  // namespace

extern "C" {

mm_status mm_int8_matmul_workspace_size(const mm_tensor* A, const mm_tensor* B, int32_t out_dtype, size_t* bytes) {
  if (!bytes) return MM_ERR_INVALID_ARG;
  Int8Args a;
  const mm_status s = plan_int8(A, B, out_dtype, &a);
  if (s != MM_OK) return s;
  *bytes = a.M == 0 || a.N == 0 ? 0 : int8_path(a).bytes;
  return MM_OK;
}

mm_status mm_int8_matmul(const mm_tensor* A, const mm_tensor* B, const mm_tensor* a_scale, const mm_tensor* b_scale,
                         const mm_tensor* bias, const mm_tensor* Y, void* workspace, size_t workspace_bytes,
                         void* stream) {
  mm_status s;
  if ((s = check_tensor(Y)) != MM_OK) return s;
  Int8Args a;
  if ((s = plan_int8(A, B, Y->dtype, &a)) != MM_OK) return s;
  if ((s = check_tensor(a_scale)) != MM_OK || (s = check_tensor(b_scale)) != MM_OK) return s;
  if (bias && (s = check_tensor(bias)) != MM_OK) return s;
  if (a_scale->dtype != MM_F32 || b_scale->dtype != MM_F32 || (bias && bias->dtype != Y->dtype)) return MM_ERR_DTYPE;
  if (!is_vector(a_scale, a.M) || !is_vector(b_scale, a.N) || (bias && !is_vector(bias, a.N))) return MM_ERR_SHAPE;
  const int64_t shape[2] = {a.M, a.N};
  if ((s = check_output(Y, Y->dtype, 2, shape)) != MM_OK) return s;
  if (a.M == 0 || a.N == 0) return finish(MM_OK, MM_PATH_NONE);
  a.sa = static_cast<const float*>(a_scale->data); a.sa_s = a_scale->strides[0];
  a.sb = static_cast<const float*>(b_scale->data); a.sb_s = b_scale->strides[0];
  if (bias) { a.bias = bias->data; a.bias_s = bias->strides[0]; }
  a.y = Y->data;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Int8Plan p = int8_path(a);
  if (p.path < 0) return MM_ERR_UNSUPPORTED;
  if (p.path == MM_PATH_VECTOR) return finish(launch_int8_few(a, st), MM_PATH_VECTOR);
  if (p.path == MM_PATH_SIMT) return finish(launch_int8_any(a, st), MM_PATH_SIMT);
  if (!workspace_ok(workspace, workspace_bytes, p.bytes)) return MM_ERR_WORKSPACE;
  unsigned* status = device_status_ptr();
  if (!status) return MM_ERR_CUDA;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  Int8Copy ca, cb;
  memset(&ca, 0, sizeof(ca));
  memset(&cb, 0, sizeof(cb));
  ca.src = a.a; ca.rs = a.a_rs; ca.cs = a.a_cs; ca.rows = a.M; ca.cols = a.K; ca.ld = p.lda;
  ca.dst = w + p.a;
  if (!p.as_is) {
    cb.src = a.b; cb.ld = p.ldb;
    cb.rs = p.b_mn ? a.b_ks : a.b_ns; cb.cs = p.b_mn ? a.b_ns : a.b_ks;
    cb.rows = p.b_mn ? a.K : a.N; cb.cols = p.b_mn ? a.N : a.K;
    cb.dst = w + p.b;
    cb.bytes = p.stream;
  }
  if ((s = launch_int8_copies(ca, cb, st)) != MM_OK) return s;
  if (p.stream) {
    if (!p.as_is) {
      a.b = static_cast<const int8_t*>(cb.dst);
      a.b_ks = 1;
      a.b_ns = p.ldb;
    }
    return finish(launch_int8_stream(a, ca.dst, p.lda, !p.as_is, status, st), MM_PATH_TENSOR);
  }
  return finish(launch_tc_int8(a, ca.dst, p.lda, cb.dst, p.ldb, p.b_mn, status, st), MM_PATH_TENSOR);
}

}  // extern "C"

// ------------------------------------------------------------------ orthogonalised update

namespace {

mm_status plan_ortho(const mm_tensor* X, OrthoArgs* o) {
  const mm_status s = check_tensor(X);
  if (s != MM_OK) return s;
  if (!is_float16_32(X->dtype)) return MM_ERR_DTYPE;
  if (X->ndim < 2) return MM_ERR_SHAPE;
  memset(o, 0, sizeof(*o));
  o->dtype = X->dtype;
  o->bm.nb = X->ndim - 2;
  o->bm.count = 1;
  for (int d = 0; d < kMaxBatchDims; ++d) o->bm.shape[d] = 1;
  for (int d = 0; d < o->bm.nb; ++d) {
    o->bm.shape[d] = X->shape[d];
    o->bm.count *= X->shape[d];
    o->x.bstride[d] = X->strides[d];
  }
  o->M = X->shape[X->ndim - 2]; o->N = X->shape[X->ndim - 1];
  if (o->M >= (1ll << 31) || o->N >= (1ll << 31)) return MM_ERR_UNSUPPORTED;
  o->x.ptr = X->data;
  o->x.rs = X->strides[X->ndim - 2];
  o->x.cs = o->N == 1 ? 1 : X->strides[X->ndim - 1];
  return MM_OK;
}
bool empty(const OrthoArgs& o) { return o.M == 0 || o.N == 0 || o.bm.count == 0; }

}  // namespace

extern "C" {

mm_status mm_orthogonalize_workspace_size(const mm_tensor* X, size_t* bytes) {
  if (!bytes) return MM_ERR_INVALID_ARG;
  OrthoArgs o;
  const mm_status s = plan_ortho(X, &o);
  if (s != MM_OK) return s;
  *bytes = empty(o) ? 0 : ortho_workspace_bytes(o);
  return MM_OK;
}

mm_status mm_orthogonalize(const mm_tensor* X, int32_t steps, const float* coefficients, float eps, float scale,
                           const mm_tensor* Y, void* workspace, size_t workspace_bytes, void* stream) {
  mm_status s;
  OrthoArgs o;
  if ((s = plan_ortho(X, &o)) != MM_OK) return s;
  if (steps < 0 || steps > MM_ORTHO_MAX_STEPS || (steps > 0 && !coefficients)) return MM_ERR_INVALID_ARG;
  for (int i = 0; i < 3 * steps; ++i)
    if (!std::isfinite(coefficients[i])) return MM_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(scale)) return MM_ERR_INVALID_ARG;
  if ((s = check_output(Y, X->dtype, X->ndim, X->shape)) != MM_OK) return s;
  if (empty(o)) return finish(MM_OK, MM_PATH_NONE);
  o.out = Y->data;
  o.steps = steps;
  o.coef = coefficients;
  o.eps = eps;
  o.scale = scale;
  if (!workspace_ok(workspace, workspace_bytes, ortho_workspace_bytes(o))) return MM_ERR_WORKSPACE;
  return launch_ortho(o, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
