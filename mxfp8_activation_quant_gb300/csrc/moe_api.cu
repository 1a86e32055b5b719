// C ABI of the mixture-of-experts operators: argument checks on the host, then the launches of
// mxq_moe_internal.h. The operators are documented in include/mxq_moe.h.
#include <cuda_runtime.h>

#include <cstdint>

#include "mxq_internal.h"
#include "mxq_moe_internal.h"
#include "mxq_overlap.h"

namespace {

constexpr int64_t kMaxStride = int64_t(1) << 40;  // a tensor map's

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

mxq_status check_weights(const mxq_mx_tensor* t, int64_t rows, int64_t cols) {
  if (t == nullptr || t->data == nullptr || t->sf == nullptr) return MXQ_ERR_INVALID_ARG;
  if (t->sf_layout != MXQ_SF_TILED_128X4) return MXQ_ERR_LAYOUT;
  if (t->rows != rows || t->cols != cols || t->ld < cols) return MXQ_ERR_UNSUPPORTED_SHAPE;
  if (!al16(t->data) || !al16(t->sf) || t->ld % 16 != 0) return MXQ_ERR_MISALIGNED;
  if (t->ld >= kMaxStride || rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31))
    return MXQ_ERR_UNSUPPORTED_SHAPE;
  return MXQ_OK;
}

bool experts_shape_ok(int64_t T, int32_t k, int32_t E, int64_t H, int64_t I) {
  return T >= 1 && k >= 1 && k <= 64 && E >= 1 && E <= 1024 && H >= 128 && I >= 128 && H % 128 == 0 && I % 128 == 0 &&
         T <= (int64_t(1) << 24) && T * k <= (int64_t(1) << 24) && H <= 65536 && I <= 65536;
}

}  // namespace

extern "C" {

mxq_status add_rmsnorm_dual_out(const void* x_bf16, int64_t ldx, const void* residual, int32_t residual_type,
                                int64_t ldr, const void* gamma_bf16, float eps, int64_t T, int64_t H,
                                void* residual_out, int64_t ldro, void* y_bf16, void* y_q, void* y_sf_packed_i32,
                                void* y_sf_rowmajor, void* y_sf_128x4, void* stream) {
  if (x_bf16 == nullptr || residual == nullptr || gamma_bf16 == nullptr || residual_out == nullptr)
    return MXQ_ERR_INVALID_ARG;
  if (residual_type != MXQ_TYPE_BF16 && residual_type != MXQ_TYPE_FP32) return MXQ_ERR_INVALID_ARG;
  const bool any_sf = y_sf_packed_i32 != nullptr || y_sf_rowmajor != nullptr || y_sf_128x4 != nullptr;
  if ((y_q != nullptr) != any_sf || (y_q == nullptr && y_bf16 == nullptr)) return MXQ_ERR_INVALID_ARG;
  if (T <= 0 || H <= 0 || !(eps >= 0.0f)) return MXQ_ERR_INVALID_ARG;
  if (T == 1) ldx = ldr = ldro = H;  // a single row has no stride
  if (H % 32 != 0 || H > 16384 || ldx < H || ldr < H || ldro < H) return MXQ_ERR_UNSUPPORTED_SHAPE;
  if (y_sf_packed_i32 != nullptr && H % 128 != 0) return MXQ_ERR_UNSUPPORTED_SHAPE;
  if (T >= (int64_t(1) << 31) || ldx >= kMaxStride || ldr >= kMaxStride || ldro >= kMaxStride)
    return MXQ_ERR_UNSUPPORTED_SHAPE;
  const int64_t es = residual_type == MXQ_TYPE_FP32 ? 4 : 2;
  if (!al16(x_bf16) || !al16(residual) || !al16(gamma_bf16) || !al16(residual_out) || !al16(y_bf16) || !al16(y_q) ||
      !al16(y_sf_packed_i32) || !al16(y_sf_rowmajor) || !al16(y_sf_128x4))
    return MXQ_ERR_MISALIGNED;
  if ((ldx * 2) % 16 != 0 || (ldr * es) % 16 != 0 || (ldro * es) % 16 != 0) return MXQ_ERR_MISALIGNED;
  const bool in_place = residual_out == residual && ldro == ldr;
  if (!in_place && mxq::rows_overlap(residual, ldr * es, H * es, residual_out, ldro * es, H * es, T)) return MXQ_ERR_INVALID_ARG;
  if (mxq::rows_overlap(x_bf16, ldx * 2, H * 2, residual_out, ldro * es, H * es, T)) return MXQ_ERR_INVALID_ARG;
  mxq::AddRmsnormLaunch l{x_bf16, ldx, residual, residual_type == MXQ_TYPE_FP32, ldr, gamma_bf16, eps, T, H,
                          residual_out, ldro, y_bf16, y_q, y_sf_packed_i32, y_sf_rowmajor, y_sf_128x4};
  return mxq::from_cuda(mxq::launch_add_rmsnorm(l, static_cast<cudaStream_t>(stream)));
}

mxq_status moe_route(const void* logits, int32_t logits_type, int64_t ldl, const void* bias_f32, int64_t T, int32_t E,
                     int32_t k, int32_t scoring, int32_t groups, int32_t topk_groups, int32_t group_top,
                     int32_t renormalize, float scale, void* ids_i32, void* weights_f32, void* stream) {
  if (logits == nullptr || ids_i32 == nullptr || weights_f32 == nullptr) return MXQ_ERR_INVALID_ARG;
  if (logits_type != MXQ_TYPE_BF16 && logits_type != MXQ_TYPE_FP32) return MXQ_ERR_INVALID_ARG;
  if (scoring != MXQ_MOE_SIGMOID && scoring != MXQ_MOE_SOFTMAX) return MXQ_ERR_INVALID_ARG;
  if (T <= 0 || E <= 0 || k <= 0 || groups <= 0 || topk_groups <= 0 || topk_groups > groups) return MXQ_ERR_INVALID_ARG;
  if ((group_top != 1 && group_top != 2) || !(scale - scale == 0.0f)) return MXQ_ERR_INVALID_ARG;
  if (T == 1) ldl = E;  // a single row has no stride
  if (E > 1024 || k > 32 || groups > 32 || E % groups != 0 || k > topk_groups * (E / groups) || ldl < E)
    return MXQ_ERR_UNSUPPORTED_SHAPE;
  if (T >= (int64_t(1) << 31) || ldl >= kMaxStride) return MXQ_ERR_UNSUPPORTED_SHAPE;
  const uintptr_t es = logits_type == MXQ_TYPE_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % es != 0 || reinterpret_cast<uintptr_t>(bias_f32) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(ids_i32) % 4 != 0 || reinterpret_cast<uintptr_t>(weights_f32) % 4 != 0)
    return MXQ_ERR_MISALIGNED;
  mxq::RouteLaunch l{logits, logits_type == MXQ_TYPE_BF16, ldl, static_cast<const float*>(bias_f32), T, E, k,
                     scoring == MXQ_MOE_SOFTMAX, groups, topk_groups, group_top, renormalize != 0, scale,
                     static_cast<int32_t*>(ids_i32), static_cast<float*>(weights_f32)};
  return mxq::from_cuda(mxq::launch_route(l, static_cast<cudaStream_t>(stream)));
}

int64_t mxq_moe_workspace_bytes(int64_t T, int32_t k, int32_t E, int64_t H, int64_t I) {
  return experts_shape_ok(T, k, E, H, I) ? mxq::experts_workspace_bytes(T, k, E, H, I) : 0;
}

mxq_status moe_experts_mxfp8(const mxq_mx_tensor* x, const void* ids_i32, const void* weights_f32, int64_t T, int32_t k,
                             const mxq_mx_tensor* w13, const mxq_mx_tensor* w2, int32_t E, int64_t H, int64_t I,
                             void* out_bf16, int64_t ldo, void* workspace, int64_t workspace_bytes, void* status,
                             void* stream) {
  if (x == nullptr || x->data == nullptr || x->sf == nullptr || ids_i32 == nullptr || weights_f32 == nullptr ||
      out_bf16 == nullptr || workspace == nullptr)
    return MXQ_ERR_INVALID_ARG;
  if (T <= 0 || k <= 0 || E <= 0 || H <= 0 || I <= 0) return MXQ_ERR_INVALID_ARG;
  if (x->sf_layout != MXQ_SF_ROWMAJOR_U8 && x->sf_layout != MXQ_SF_TILED_128X4) return MXQ_ERR_LAYOUT;
  mxq_mx_tensor xt = *x;
  if (T == 1) xt.ld = ldo = H;  // a single row has no stride
  if (!experts_shape_ok(T, k, E, H, I) || xt.rows != T || xt.cols != H || xt.ld < H || xt.ld >= kMaxStride || ldo < H ||
      ldo >= kMaxStride)
    return MXQ_ERR_UNSUPPORTED_SHAPE;
  mxq_status st = check_weights(w13, static_cast<int64_t>(E) * 2 * I, H);
  if (st != MXQ_OK) return st;
  if ((st = check_weights(w2, static_cast<int64_t>(E) * H, I)) != MXQ_OK) return st;
  if (!al16(xt.data) || !al16(xt.sf) || xt.ld % 16 != 0 || !al16(out_bf16) || (ldo * 2) % 16 != 0 ||
      !al16(workspace) || !al16(status) || reinterpret_cast<uintptr_t>(ids_i32) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(weights_f32) % 4 != 0)
    return MXQ_ERR_MISALIGNED;
  if (workspace_bytes < mxq::experts_workspace_bytes(T, k, E, H, I)) return MXQ_ERR_INVALID_ARG;
  mxq::ExpertsLaunch l{&xt, static_cast<const int32_t*>(ids_i32), static_cast<const float*>(weights_f32), T, k, w13, w2,
                       E, H, I, out_bf16, ldo, workspace, static_cast<int32_t*>(status)};
  return mxq::from_cuda(mxq::launch_experts(l, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
