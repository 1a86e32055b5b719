// Internal launcher interface of the mixture-of-experts operators (include/mxq_moe.h). Arguments
// are validated by the C ABI layer (moe_api.cu) before any of these is called.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mxq_moe.h"

namespace mxq {

struct AddRmsnormLaunch {
  const void* x;
  int64_t ldx;
  const void* residual;
  bool fp32_stream;
  int64_t ldr;
  const void* gamma;
  float eps;
  int64_t T, H;
  void* residual_out;
  int64_t ldro;
  void* y;   // may be null
  void* yq;  // may be null
  void* sf_packed;
  void* sf_rowmajor;
  void* sf_tiled;
};
cudaError_t launch_add_rmsnorm(const AddRmsnormLaunch& a, cudaStream_t stream);

struct RouteLaunch {
  const void* logits;
  bool bf16_logits;
  int64_t ldl;
  const float* bias;
  int64_t T;
  int32_t E, k;
  bool softmax;
  int32_t groups, topk_groups, group_top;
  bool renormalize;
  float scale;
  int32_t* ids;
  float* weights;
};
cudaError_t launch_route(const RouteLaunch& a, cudaStream_t stream);

struct ExpertsLaunch {
  const mxq_mx_tensor* x;
  const int32_t* ids;
  const float* weights;
  int64_t T;
  int32_t k;
  const mxq_mx_tensor* w13;
  const mxq_mx_tensor* w2;
  int32_t E;
  int64_t H, I;
  void* out;
  int64_t ldo;
  void* workspace;
  int32_t* status;
};
cudaError_t launch_experts(const ExpertsLaunch& a, cudaStream_t stream);
int64_t experts_workspace_bytes(int64_t T, int32_t k, int32_t E, int64_t H, int64_t I);

}  // namespace mxq
