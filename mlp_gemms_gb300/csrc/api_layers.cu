// C ABI of the layers around the expert MLP: host-side validation and launches
// of the layer norm (norm.cu), the expert routing (route.cu) and the combine's
// gradient (combine.cu).  Nothing here allocates device memory.
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
  int64_t blocks = mx::norm_bwd_blocks(R, D, false);
  if (mx::norm_bwd_blocks(R, D, true) > blocks) blocks = mx::norm_bwd_blocks(R, D, true);
  return (size_t)blocks * 2 * (size_t)D * sizeof(float);
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

namespace {

mx_status_t check_route(const void* logits, int32_t x_type, int64_t T, int32_t G, int64_t ld, int32_t k, int32_t score,
                        int32_t renorm, float scale) {
  mx_status_t st;
  if ((st = check_type(x_type, "x_type")) != MX_OK) return st;
  MX_CHECK(score == MX_SCORE_SOFTMAX || score == MX_SCORE_SIGMOID, MX_ERR_INVALID_ARG, "score = %d", score);
  MX_CHECK(renorm == 0 || renorm == 1, MX_ERR_INVALID_ARG, "renorm = %d", renorm);
  MX_CHECK(std::isfinite(scale), MX_ERR_INVALID_ARG, "scale = %g", (double)scale);
  MX_CHECK(G >= 1, MX_ERR_INVALID_ARG, "G = %d; at least one expert is required", G);
  MX_CHECK(G <= 1024, MX_ERR_NOT_SUPPORTED, "G = %d; at most 1024 experts", G);
  MX_CHECK(k >= 1 && k <= G, MX_ERR_INVALID_ARG, "k = %d of %d experts", k, G);
  MX_CHECK(k <= 32, MX_ERR_NOT_SUPPORTED, "k = %d; at most 32 choices", k);
  MX_CHECK(T >= 0 && T < (1ll << 31) && T * k < (1ll << 31), MX_ERR_SHAPE, "T = %lld is out of range", (long long)T);
  MX_CHECK(ld >= G && ld < (1ll << 38) && mx::fits(T, ld), MX_ERR_SHAPE, "ld = %lld of logits with %d experts",
           (long long)ld, G);
  return T == 0 ? MX_OK : check_ptr(logits, "logits");
}

}  // namespace

extern "C" {

size_t mx_moe_topk_workspace_bytes(int64_t T, int32_t G) {
  if (T <= 0 || G <= 0) return 0;
  return (size_t)mx::route_blocks(T) * (size_t)G * 8;
}

mx_status_t mx_moe_topk(const void* logits, int32_t x_type, int64_t T, int32_t G, int64_t ld, int32_t k, int32_t score,
                        const float* bias, int32_t groups, int32_t topk_groups, int32_t group_top, int32_t renorm,
                        float scale, float* weights, int32_t* ids, int32_t* load, float* score_sum, void* workspace,
                        size_t workspace_bytes, mx_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  mx_status_t st;
  if ((st = check_route(logits, x_type, T, G, ld, k, score, renorm, scale)) != MX_OK) return st;
  MX_CHECK(groups >= 1 && groups <= 32 && G % groups == 0, MX_ERR_INVALID_ARG, "groups = %d of %d experts", groups, G);
  MX_CHECK(topk_groups >= 1 && topk_groups <= groups, MX_ERR_INVALID_ARG, "topk_groups = %d of %d", topk_groups, groups);
  MX_CHECK(k <= topk_groups * (G / groups), MX_ERR_INVALID_ARG, "k = %d choices from %d experts", k,
           topk_groups * (G / groups));
  MX_CHECK(group_top == 1 || (group_top == 2 && (groups == 1 || G / groups >= 2)), MX_ERR_INVALID_ARG,
           "group_top = %d of %d", group_top, G / groups);
  MX_CHECK((load == nullptr) == (score_sum == nullptr), MX_ERR_INVALID_ARG, "load and score_sum come together");
  if ((st = check_floats(bias, "bias")) != MX_OK || (st = check_floats(score_sum, "score_sum")) != MX_OK) return st;
  MX_CHECK(aligned(load, 4), MX_ERR_ALIGNMENT, "load must be 4-byte aligned");
  if (T > 0 && ((st = check_ptr(weights, "weights")) != MX_OK || (st = check_ptr(ids, "ids")) != MX_OK)) return st;
  const size_t need = load ? mx_moe_topk_workspace_bytes(T, G) : 0;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MX_OK) return st;
  if (T == 0 && !load) return MX_OK;
  int sms;
  if ((st = mx::device_sms(&sms)) != MX_OK) return st;
  if (T == 0) {
    st = cuda_result(cudaMemsetAsync(load, 0, (size_t)G * 4, s), "clearing load");
    return st != MX_OK ? st : cuda_result(cudaMemsetAsync(score_sum, 0, (size_t)G * 4, s), "clearing score_sum");
  }
  mx::RouteParams p{};
  p.T = T; p.G = G; p.k = k;
  p.x_f32 = x_type == MX_F32; p.sigmoid = score == MX_SCORE_SIGMOID;
  p.renorm = renorm; p.scale = scale;
  p.groups = groups == topk_groups ? 1 : groups;  // all kept: none to choose
  p.topk_groups = topk_groups; p.group_top = group_top;
  p.logits = logits; p.ld = ld;
  p.bias = bias;
  p.weights = weights; p.ids = ids;
  p.load = load; p.score_sum = score_sum;
  if (load) {
    p.partial_load = static_cast<int32_t*>(workspace);
    p.partial_sum = reinterpret_cast<float*>(p.partial_load + mx::route_blocks(T) * G);
  }
  return cuda_result(mx::launch_route_fwd(p, s), "expert routing launch");
}

mx_status_t mx_moe_topk_bwd(const void* logits, int32_t x_type, int64_t T, int32_t G, int64_t ld, int32_t k,
                            int32_t score, int32_t renorm, float scale, const int32_t* ids, const float* dweights,
                            const float* dscore_sum, void* dlogits, int64_t ld_d, mx_stream_t stream) {
  mx_status_t st;
  if ((st = check_route(logits, x_type, T, G, ld, k, score, renorm, scale)) != MX_OK) return st;
  MX_CHECK(ld_d >= G && ld_d < (1ll << 38) && mx::fits(T, ld_d), MX_ERR_SHAPE, "ld of dlogits = %lld",
           (long long)ld_d);
  MX_CHECK(dlogits != logits || ld_d == ld || T == 0, MX_ERR_ALIGNMENT, "dlogits is logits with another row stride");
  if ((st = check_floats(dscore_sum, "dscore_sum")) != MX_OK) return st;
  if (T == 0) return MX_OK;
  if ((st = check_ptr(ids, "ids")) != MX_OK || (st = check_ptr(dweights, "dweights")) != MX_OK ||
      (st = check_ptr(dlogits, "dlogits")) != MX_OK)
    return st;
  int sms;
  if ((st = mx::device_sms(&sms)) != MX_OK) return st;
  mx::RouteParams p{};
  p.T = T; p.G = G; p.k = k;
  p.x_f32 = x_type == MX_F32; p.sigmoid = score == MX_SCORE_SIGMOID;
  p.renorm = renorm; p.scale = scale;
  p.groups = p.topk_groups = p.group_top = 1;
  p.logits = logits; p.ld = ld;
  p.ids = const_cast<int32_t*>(ids);
  p.dweights = dweights; p.dsum = dscore_sum;
  p.dlogits = dlogits; p.ld_d = ld_d;
  return cuda_result(mx::launch_route_bwd(p, reinterpret_cast<cudaStream_t>(stream)), "expert routing backward launch");
}

mx_status_t mx_moe_unpermute_bwd(const void* dout_bf16, int64_t T, int64_t D, const void* in_bf16, int64_t R,
                                 const int32_t* row_of_dev, int32_t k, const float* weights_dev, const int32_t* src_dev,
                                 void* din_bf16, float* dweights, mx_stream_t stream) {
  mx_status_t st;
  MX_CHECK(k >= 1, MX_ERR_INVALID_ARG, "k = %d", k);
  MX_CHECK(T >= 0 && T < (1ll << 31) && T * k < (1ll << 31), MX_ERR_SHAPE, "T = %lld is out of range", (long long)T);
  MX_CHECK(R >= 0, MX_ERR_SHAPE, "R = %lld is out of range", (long long)R);
  if ((st = check_dim(D, "D", 8)) != MX_OK) return st;
  if ((st = check_matrix(dout_bf16, "dout", T, D, D)) != MX_OK) return st;
  if (dweights && (st = check_matrix(in_bf16, "in", R, D, D)) != MX_OK) return st;
  if (din_bf16 && (st = check_matrix(din_bf16, "din", R, D, D)) != MX_OK) return st;
  MX_CHECK(din_bf16 == nullptr || din_bf16 != in_bf16, MX_ERR_INVALID_ARG, "din is in");
  if (T > 0 && (st = check_ptr(row_of_dev, "row_of")) != MX_OK) return st;
  if ((st = check_floats(weights_dev, "weights")) != MX_OK || (st = check_floats(dweights, "dweights")) != MX_OK)
    return st;
  MX_CHECK(aligned(src_dev, 4), MX_ERR_ALIGNMENT, "src must be 4-byte aligned");
  if (!din_bf16 && !dweights) return MX_OK;
  if (T == 0 && (R == 0 || !din_bf16 || !src_dev)) return MX_OK;
  int sms;
  if ((st = mx::device_sms(&sms)) != MX_OK) return st;
  mx::CombineBwdParams p{};
  p.T = T; p.R = R; p.D = D; p.k = k;
  p.dout = static_cast<const uint16_t*>(dout_bf16);
  p.in = static_cast<const uint16_t*>(in_bf16);
  p.row_of = row_of_dev; p.weights = weights_dev; p.src = src_dev;
  p.din = static_cast<uint16_t*>(din_bf16);
  p.dweights = dweights;
  return cuda_result(mx::launch_combine_bwd(p, sms, reinterpret_cast<cudaStream_t>(stream)), "combine backward launch");
}

}  // extern "C"
