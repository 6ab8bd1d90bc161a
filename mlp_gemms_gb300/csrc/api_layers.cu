// C ABI of the layers around the expert MLP: host-side validation and launches
// of the layer norm (norm.cu).  Nothing here allocates device memory.
#include <cmath>

#include "api_checks.h"

using mx::aligned;
using mx::check_dim;
using mx::check_matrix;
using mx::check_ptr;
using mx::check_workspace;
using mx::cuda_result;

namespace {

mx_status_t check_type(int32_t t, const char* name) {
  MX_CHECK(t == MX_BF16 || t == MX_F32, MX_ERR_INVALID_ARG, "%s = %d is neither MX_BF16 nor MX_F32", name, t);
  return MX_OK;
}

mx_status_t check_norm(int64_t R, int64_t D, int32_t x_type, int32_t w_type, const void* weight, const void* bias,
                       int32_t rms) {
  mx_status_t st;
  if ((st = check_type(x_type, "x_type")) != MX_OK || (st = check_type(w_type, "w_type")) != MX_OK) return st;
  MX_CHECK(rms == 0 || rms == 1, MX_ERR_INVALID_ARG, "rms = %d", rms);
  MX_CHECK(R >= 0 && R < (1ll << 31), MX_ERR_SHAPE, "R = %lld is out of range", (long long)R);
  if ((st = check_dim(D, "D", 8)) != MX_OK) return st;
  MX_CHECK(D <= mx::MAX_NORM_D, MX_ERR_NOT_SUPPORTED, "D = %lld; rows of at most %lld columns", (long long)D,
           (long long)mx::MAX_NORM_D);
  if (weight && (st = check_ptr(weight, "weight")) != MX_OK) return st;
  return bias ? check_ptr(bias, "bias") : MX_OK;
}

// Per-row or per-column scalars.
mx_status_t check_floats(const float* p, const char* name) {
  MX_CHECK(aligned(p, 4), MX_ERR_ALIGNMENT, "%s must be 4-byte aligned", name);
  return MX_OK;
}

}  // namespace

extern "C" {

mx_status_t mx_layernorm_fwd(const void* x, int32_t x_type, int64_t R, int64_t D, int64_t ld_x, const void* res,
                             int64_t ld_res, void* sum, int64_t ld_sum, const void* weight, const void* bias,
                             int32_t w_type, float eps, int32_t rms, void* y_bf16, int64_t ld_y, float* mean,
                             float* rstd, mx_stream_t stream) {
  mx_status_t st;
  if ((st = check_norm(R, D, x_type, w_type, weight, bias, rms)) != MX_OK) return st;
  MX_CHECK(eps >= 0.f && std::isfinite(eps), MX_ERR_INVALID_ARG, "eps = %g", (double)eps);
  if ((st = check_matrix(x, "x", R, D, ld_x)) != MX_OK) return st;
  if ((st = check_matrix(y_bf16, "y", R, D, ld_y)) != MX_OK) return st;
  if (res) {
    if ((st = check_matrix(res, "res", R, D, ld_res)) != MX_OK) return st;
    if ((st = check_matrix(sum, "sum", R, D, ld_sum)) != MX_OK) return st;
    MX_CHECK((sum != x || ld_sum == ld_x) && (sum != res || ld_sum == ld_res), MX_ERR_ALIGNMENT,
             "sum is x or res with another row stride");
  }
  if ((st = check_floats(mean, "mean")) != MX_OK || (st = check_floats(rstd, "rstd")) != MX_OK) return st;
  if (R == 0) return MX_OK;
  int sms;
  if ((st = mx::device_sms(&sms)) != MX_OK) return st;
  mx::NormParams p{};
  p.R = R; p.D = D;
  p.x_f32 = x_type == MX_F32; p.w_f32 = w_type == MX_F32;
  p.rms = rms; p.eps = eps;
  p.x = x; p.ld_x = ld_x;
  p.res = res; p.ld_res = ld_res;
  p.sum = sum; p.ld_sum = ld_sum;
  p.weight = weight; p.bias = bias;
  p.y = static_cast<uint16_t*>(y_bf16); p.ld_y = ld_y;
  p.mean = mean; p.rstd = rstd;
  return cuda_result(mx::launch_norm_fwd(p, sms, reinterpret_cast<cudaStream_t>(stream)), "layer norm launch");
}

size_t mx_layernorm_workspace_bytes(int64_t R, int64_t D) {
  if (R <= 0 || D <= 0 || D > mx::MAX_NORM_D) return 0;
  return (size_t)mx::norm_bwd_blocks(R, D) * 2 * (size_t)D * sizeof(float);
}

mx_status_t mx_layernorm_bwd(const void* dy_bf16, int64_t ld_dy, const void* x, int32_t x_type, int64_t R, int64_t D,
                             int64_t ld_x, const float* mean, const float* rstd, const void* weight, int32_t w_type,
                             int32_t rms, const void* dres, int64_t ld_dres, void* dx, int64_t ld_dx, float* dweight,
                             float* dbias, int32_t accumulate, void* workspace, size_t workspace_bytes,
                             mx_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  mx_status_t st;
  if ((st = check_norm(R, D, x_type, w_type, weight, nullptr, rms)) != MX_OK) return st;
  MX_CHECK(accumulate == 0 || accumulate == 1, MX_ERR_INVALID_ARG, "accumulate = %d", accumulate);
  if ((st = check_matrix(dy_bf16, "dy", R, D, ld_dy)) != MX_OK) return st;
  if ((st = check_matrix(x, "x", R, D, ld_x)) != MX_OK) return st;
  if ((st = check_matrix(dx, "dx", R, D, ld_dx)) != MX_OK) return st;
  if (dres && (st = check_matrix(dres, "dres", R, D, ld_dres)) != MX_OK) return st;
  MX_CHECK(dres != dx || ld_dres == ld_dx || R == 0, MX_ERR_ALIGNMENT, "dx is dres with another row stride");
  MX_CHECK(R == 0 || (rstd != nullptr && (rms || mean != nullptr)), MX_ERR_INVALID_ARG, "mean or rstd is NULL");
  if ((st = check_floats(mean, "mean")) != MX_OK || (st = check_floats(rstd, "rstd")) != MX_OK) return st;
  if ((st = check_floats(dweight, "dweight")) != MX_OK || (st = check_floats(dbias, "dbias")) != MX_OK) return st;
  const size_t need = dweight || dbias ? mx_layernorm_workspace_bytes(R, D) : 0;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MX_OK) return st;
  if (R == 0 && (accumulate || (!dweight && !dbias))) return MX_OK;
  int sms;
  if ((st = mx::device_sms(&sms)) != MX_OK) return st;
  if (R == 0) {
    for (float* d : {dweight, dbias})
      if (d && (st = cuda_result(cudaMemsetAsync(d, 0, (size_t)D * sizeof(float), s), "clearing a gradient")) != MX_OK)
        return st;
    return MX_OK;
  }
  mx::NormParams p{};
  p.R = R; p.D = D;
  p.x_f32 = x_type == MX_F32; p.w_f32 = w_type == MX_F32;
  p.rms = rms;
  p.x = x; p.ld_x = ld_x;
  p.res = dres; p.ld_res = ld_dres;
  p.weight = weight;
  p.mean = const_cast<float*>(mean); p.rstd = const_cast<float*>(rstd);
  p.dy = static_cast<const uint16_t*>(dy_bf16); p.ld_dy = ld_dy;
  p.dx = dx; p.ld_dx = ld_dx;
  p.dweight = dweight; p.dbias = dbias;
  p.accumulate = accumulate;
  p.partials = static_cast<float*>(workspace);
  return cuda_result(mx::launch_norm_bwd(p, s), "layer norm backward launch");
}

}  // extern "C"
