// Host-side helpers of the C-ABI layer (defined in api.cu) shared by its
// translation units: argument checks, path choice and the dense product.
#pragma once

#include "kernels.h"

namespace qg {

// Device-side status word of the current device (NULL on failure).
unsigned* device_status_ptr();

int elem_size(int dt);
bool is_int_type(int dt);
bool is_matmul_type(int dt);
bool is_q8(int dt);
bool is_q4(int dt);
int64_t numel(const mm_tensor* t);
mm_status check_tensor(const mm_tensor* t);
bool is_dense(const mm_tensor* t);
mm_status check_output(const mm_tensor* y, int dtype, int ndim, const int64_t* shape);

// The process-wide planner policy (an mm_path value).
int path_policy();
// MM_PATH_TENSOR or MM_PATH_SIMT for a call, honouring the policy; -1 when a
// forced tensor-core path cannot run it.
int choose(bool tensor_ok, bool tensor_pays);
bool tensor_pays(int64_t M, int64_t N, int64_t K, int64_t batch);
bool tensor_pays_dense(int dtype, int64_t M, int64_t N, int64_t K, int64_t batch);
// Records the path of a successful call.
mm_status finish(mm_status s, int path);
// MatMul and Gemm after validation: the path that a product takes (an mm_path
// value, -1: none) and, where asked for, whether its kernel takes C in fp32
// (GemmArgs::c_f32); the product on that path; both.
int dense_path(const GemmArgs& g, bool pays, bool* c_f32);
mm_status run_dense_on(int path, const GemmArgs& g, cudaStream_t st);
mm_status run_dense(const GemmArgs& g, bool pays, cudaStream_t st);

}  // namespace qg
