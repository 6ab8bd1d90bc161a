// C ABI of the BF16 layers: host-side validation and launches of the ragged
// products (ragged.cu) and the 8-bit activation checkpoints (ckpt.cu).
// Nothing here allocates device memory.
#include <vector>

#include "api_checks.h"

using mx::aligned;
using mx::check_dim;
using mx::check_matrix;
using mx::check_ptr;
using mx::check_workspace;
using mx::cuda_result;

namespace {

mx_status_t check_segments(const int32_t* offsets, int32_t G, int64_t R, cudaStream_t s) {
  MX_CHECK(G >= 1, MX_ERR_INVALID_ARG, "G = %d; at least one expert is required", G);
  MX_CHECK(G <= mx::MAX_RAGGED_G, MX_ERR_NOT_SUPPORTED, "G = %d; at most %d experts", G, mx::MAX_RAGGED_G);
  MX_CHECK(R >= 0 && R < (1ll << 31), MX_ERR_SHAPE, "R = %lld is out of range", (long long)R);
  if (offsets == nullptr && G == 1) return MX_OK;
  MX_CHECK(offsets != nullptr, MX_ERR_INVALID_ARG, "offsets is NULL");
  MX_CHECK(aligned(offsets, 4), MX_ERR_ALIGNMENT, "offsets must be 4-byte aligned");
  if (!mx::validate_offsets_requested()) return MX_OK;
  std::vector<int32_t> h((size_t)G);
  cudaError_t e = cudaMemcpyAsync(h.data(), offsets, sizeof(int32_t) * (size_t)G, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_result(e, "reading offsets");
  int64_t prev = 0;
  for (int g = 0; g < G; g++) {
    MX_CHECK(h[g] >= prev, MX_ERR_OFFSETS, "offsets[%d] = %d decreases (previous %lld)", g, h[g], (long long)prev);
    prev = h[g];
  }
  MX_CHECK(prev <= R, MX_ERR_OFFSETS, "offsets[G-1] = %lld exceeds R = %lld", (long long)prev, (long long)R);
  return MX_OK;
}

// The weights [G, N, K]: G * N rows are TMA coordinates.
mx_status_t check_weights(const void* w, const char* name, int32_t G, int64_t N, int64_t K) {
  MX_CHECK(G * N < (1ll << 31) && G * K < (1ll << 31) && G * N < (1ll << 46) / K, MX_ERR_SHAPE, "%s is too large",
           name);
  return check_ptr(w, name);
}

mx_status_t check_ckpt(const mx_tensor_t* t, int64_t rows, int64_t cols) {
  MX_CHECK(t != nullptr, MX_ERR_INVALID_ARG, "ckpt is NULL");
  MX_CHECK(t->rows == rows && t->cols == cols, MX_ERR_SHAPE, "ckpt is [%lld, %lld], expected [%lld, %lld]",
           (long long)t->rows, (long long)t->cols, (long long)rows, (long long)cols);
  MX_CHECK(t->fmt == MX_E4M3, MX_ERR_INVALID_ARG, "ckpt has format %d, expected E4M3", t->fmt);
  MX_CHECK(t->hadamard == 0, MX_ERR_INVALID_ARG, "ckpt must not carry the rotation");
  if (rows == 0) return MX_OK;
  mx_status_t st = check_ptr(t->data, "ckpt data");
  return st != MX_OK ? st : check_ptr(t->scale, "ckpt scale");
}

}  // namespace

extern "C" {

mx_status_t mx_ragged_gemm(const void* a_bf16, int64_t R, int64_t K, int64_t ld_a, const void* w_bf16, int64_t N,
                           int32_t G, int32_t w_layout, const int32_t* offsets_dev, void* out_bf16, int64_t ld_out,
                           mx_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  mx_status_t st;
  MX_CHECK(w_layout == MX_W_NK || w_layout == MX_W_KN, MX_ERR_INVALID_ARG, "w_layout = %d", w_layout);
  if ((st = check_dim(K, "K", 8)) != MX_OK || (st = check_dim(N, "N", 8)) != MX_OK) return st;
  if ((st = check_segments(offsets_dev, G, R, s)) != MX_OK) return st;
  if ((st = check_matrix(a_bf16, "a", R, K, ld_a)) != MX_OK) return st;
  if ((st = check_matrix(out_bf16, "out", R, N, ld_out)) != MX_OK) return st;
  if ((st = check_weights(w_bf16, "w", G, N, K)) != MX_OK) return st;
  if (R == 0) return MX_OK;
  int sms;
  if ((st = mx::device_sms(&sms)) != MX_OK) return st;
  mx::RaggedParams p{};
  p.G = G; p.offsets = offsets_dev;
  p.R = R; p.K = K; p.N = N;
  p.a = static_cast<const uint16_t*>(a_bf16); p.ld_a = ld_a;
  p.w = static_cast<const uint16_t*>(w_bf16); p.w_kn = w_layout == MX_W_KN;
  p.out = static_cast<uint16_t*>(out_bf16); p.ld_out = ld_out;
  return cuda_result(mx::launch_ragged_gemm(p, sms, s), "ragged GEMM launch");
}

mx_status_t mx_linear_fwd(const void* x_bf16, int64_t M, int64_t K, int64_t ld_x, const void* w_bf16, int64_t N,
                          const void* bias_bf16, int32_t act, const void* res_bf16, int64_t ld_res, void* out_bf16,
                          int64_t ld_out, const mx_tensor_t* ckpt, mx_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  mx_status_t st;
  MX_CHECK(act >= MX_ACT_SWIGLU && act <= MX_ACT_RELU, MX_ERR_INVALID_ARG, "activation %d", act);
  MX_CHECK(act != MX_ACT_SWIGLU, MX_ERR_NOT_SUPPORTED, "SwiGLU needs two products: mx_ragged_gemm, mx_act_ckpt_fwd");
  if ((st = check_dim(K, "K", 8)) != MX_OK || (st = check_dim(N, "N", ckpt ? 32 : 8)) != MX_OK) return st;
  MX_CHECK(M >= 0 && M < (1ll << 31), MX_ERR_SHAPE, "M = %lld is out of range", (long long)M);
  if ((st = check_matrix(x_bf16, "x", M, K, ld_x)) != MX_OK) return st;
  if ((st = check_matrix(out_bf16, "out", M, N, ld_out)) != MX_OK) return st;
  if (res_bf16 && (st = check_matrix(res_bf16, "res", M, N, ld_res)) != MX_OK) return st;
  MX_CHECK(res_bf16 != out_bf16 || ld_res == ld_out || M == 0, MX_ERR_ALIGNMENT,
           "res is the output with another row stride (%lld, %lld)", (long long)ld_res, (long long)ld_out);
  if ((st = check_weights(w_bf16, "w", 1, N, K)) != MX_OK) return st;
  if (bias_bf16 && (st = check_ptr(bias_bf16, "bias")) != MX_OK) return st;
  if (ckpt && (st = check_ckpt(ckpt, M, N)) != MX_OK) return st;
  if (M == 0) return MX_OK;
  int sms;
  if ((st = mx::device_sms(&sms)) != MX_OK) return st;
  mx::RaggedParams p{};
  p.G = 1; p.offsets = nullptr;
  p.R = M; p.K = K; p.N = N;
  p.a = static_cast<const uint16_t*>(x_bf16); p.ld_a = ld_x;
  p.w = static_cast<const uint16_t*>(w_bf16);
  p.out = static_cast<uint16_t*>(out_bf16); p.ld_out = ld_out;
  p.epi.bias = static_cast<const uint16_t*>(bias_bf16);
  p.epi.act = act;
  p.epi.res = static_cast<const uint16_t*>(res_bf16); p.epi.ld_res = ld_res;
  if (ckpt) {
    p.epi.q = static_cast<uint8_t*>(ckpt->data);
    p.epi.q_scale = ckpt->scale;
  }
  return cuda_result(mx::launch_ragged_gemm(p, sms, s), "linear launch");
}

size_t mx_ragged_gemm_wgrad_workspace_bytes(int64_t N, int64_t K, int64_t R, int32_t G) {
  if (N <= 0 || K <= 0 || R <= 0 || G <= 0) return 0;
  return mx::ragged_wgrad_workspace(N, K, R, G);
}

}  // extern "C"

namespace {

mx_status_t wgrad(const void* dy, int64_t N, int64_t ld_dy, const void* x, int64_t K, int64_t ld_x, int64_t R,
                  int32_t G, const int32_t* offsets, void* grad, bool f32, int accumulate, void* workspace,
                  size_t workspace_bytes, cudaStream_t s) {
  mx_status_t st;
  if ((st = check_dim(K, "K", 8)) != MX_OK || (st = check_dim(N, "N", 8)) != MX_OK) return st;
  if ((st = check_segments(offsets, G, R, s)) != MX_OK) return st;
  if ((st = check_matrix(dy, "dy", R, N, ld_dy)) != MX_OK) return st;
  if ((st = check_matrix(x, "x", R, K, ld_x)) != MX_OK) return st;
  if ((st = check_weights(grad, "grad", G, N, K)) != MX_OK) return st;
  const size_t need = mx_ragged_gemm_wgrad_workspace_bytes(N, K, R, G);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MX_OK) return st;
  int sms;
  if ((st = mx::device_sms(&sms)) != MX_OK) return st;
  if (R == 0) {
    if (accumulate) return MX_OK;
    return cuda_result(cudaMemsetAsync(grad, 0, (size_t)G * N * K * (f32 ? 4 : 2), s), "clearing grad");
  }
  mx::RaggedWgradParams p{};
  p.G = G; p.offsets = offsets;
  p.R = R; p.N = N; p.K = K;
  p.dy = static_cast<const uint16_t*>(dy); p.ld_dy = ld_dy;
  p.x = static_cast<const uint16_t*>(x); p.ld_x = ld_x;
  p.grad = f32 ? nullptr : static_cast<uint16_t*>(grad);
  p.grad_f32 = f32 ? static_cast<float*>(grad) : nullptr;
  p.accumulate = accumulate;
  p.workspace = workspace;
  return cuda_result(mx::launch_ragged_wgrad(p, sms, s), "ragged weight-gradient launch");
}

}  // namespace

extern "C" {

mx_status_t mx_ragged_gemm_wgrad(const void* dy_bf16, int64_t N, int64_t ld_dy, const void* x_bf16, int64_t K,
                                 int64_t ld_x, int64_t R, int32_t G, const int32_t* offsets_dev, void* grad_bf16,
                                 void* workspace, size_t workspace_bytes, mx_stream_t stream) {
  return wgrad(dy_bf16, N, ld_dy, x_bf16, K, ld_x, R, G, offsets_dev, grad_bf16, false, 0, workspace,
               workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

mx_status_t mx_ragged_gemm_wgrad_f32(const void* dy_bf16, int64_t N, int64_t ld_dy, const void* x_bf16, int64_t K,
                                     int64_t ld_x, int64_t R, int32_t G, const int32_t* offsets_dev, float* grad_f32,
                                     int32_t accumulate, void* workspace, size_t workspace_bytes,
                                     mx_stream_t stream) {
  MX_CHECK(accumulate == 0 || accumulate == 1, MX_ERR_INVALID_ARG, "accumulate = %d", accumulate);
  return wgrad(dy_bf16, N, ld_dy, x_bf16, K, ld_x, R, G, offsets_dev, grad_f32, true, accumulate, workspace,
               workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

namespace {

mx_status_t check_act_cols(int32_t act, int64_t C) {
  MX_CHECK(act >= MX_ACT_SWIGLU && act <= MX_ACT_RELU, MX_ERR_INVALID_ARG, "activation %d", act);
  MX_CHECK(act != MX_ACT_NONE, MX_ERR_NOT_SUPPORTED, "a checkpoint of the identity: use mx_quantize");
  return check_dim(C, "C", act == MX_ACT_SWIGLU ? 64 : 32);
}

}  // namespace

extern "C" {

mx_status_t mx_act_ckpt_fwd(const void* z_bf16, int64_t R, int64_t C, int64_t ld_z, int32_t act, void* h_bf16,
                            int64_t ld_h, const mx_tensor_t* ckpt, mx_stream_t stream) {
  mx_status_t st;
  if ((st = check_act_cols(act, C)) != MX_OK) return st;
  MX_CHECK(R >= 0 && R < (1ll << 31), MX_ERR_SHAPE, "R = %lld is out of range", (long long)R);
  const int64_t H = act == MX_ACT_SWIGLU ? C / 2 : C;
  if ((st = check_matrix(z_bf16, "z", R, C, ld_z)) != MX_OK) return st;
  if ((st = check_matrix(h_bf16, "h", R, H, ld_h)) != MX_OK) return st;
  if ((st = check_ckpt(ckpt, R, C)) != MX_OK) return st;
  if (R == 0) return MX_OK;
  int sms;
  if ((st = mx::device_sms(&sms)) != MX_OK) return st;
  mx::CkptParams p{};
  p.R = R; p.C = C; p.act = act;
  p.q = static_cast<uint8_t*>(ckpt->data); p.q_scale = ckpt->scale;
  p.z = static_cast<const uint16_t*>(z_bf16); p.ld_z = ld_z;
  p.h = static_cast<uint16_t*>(h_bf16); p.ld_h = ld_h;
  return cuda_result(mx::launch_ckpt_fwd(p, reinterpret_cast<cudaStream_t>(stream)), "checkpoint launch");
}

size_t mx_act_ckpt_workspace_bytes(int64_t R, int64_t C) {
  if (R <= 0 || C <= 0) return 0;
  return (size_t)mx::ckpt_partials(R, C) * sizeof(float);
}

mx_status_t mx_act_ckpt_bwd(const mx_tensor_t* ckpt, int32_t act, const void* dh_bf16, int64_t ld_dh, void* dz_bf16,
                            int64_t ld_dz, void* h_bf16, int64_t ld_h, float* db, void* workspace,
                            size_t workspace_bytes, mx_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  mx_status_t st;
  MX_CHECK(ckpt != nullptr, MX_ERR_INVALID_ARG, "ckpt is NULL");
  const int64_t R = ckpt->rows, C = ckpt->cols;
  if ((st = check_act_cols(act, C)) != MX_OK) return st;
  MX_CHECK(R >= 0 && R < (1ll << 31), MX_ERR_SHAPE, "ckpt has %lld rows", (long long)R);
  if ((st = check_ckpt(ckpt, R, C)) != MX_OK) return st;
  const int64_t H = act == MX_ACT_SWIGLU ? C / 2 : C;
  if ((st = check_matrix(dh_bf16, "dh", R, H, ld_dh)) != MX_OK) return st;
  if ((st = check_matrix(dz_bf16, "dz", R, C, ld_dz)) != MX_OK) return st;
  if (h_bf16 && (st = check_matrix(h_bf16, "h", R, H, ld_h)) != MX_OK) return st;
  if (db && (st = check_ptr(db, "db")) != MX_OK) return st;
  const size_t need = db ? mx_act_ckpt_workspace_bytes(R, C) : 0;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MX_OK) return st;
  int sms;
  if ((st = mx::device_sms(&sms)) != MX_OK) return st;
  if (R == 0) {
    if (db == nullptr) return MX_OK;
    return cuda_result(cudaMemsetAsync(db, 0, (size_t)C * sizeof(float), s), "clearing db");
  }
  mx::CkptParams p{};
  p.R = R; p.C = C; p.act = act;
  p.q = static_cast<uint8_t*>(ckpt->data); p.q_scale = ckpt->scale;
  p.dh = static_cast<const uint16_t*>(dh_bf16); p.ld_dh = ld_dh;
  p.dz = static_cast<uint16_t*>(dz_bf16); p.ld_dz = ld_dz;
  p.h = static_cast<uint16_t*>(h_bf16); p.ld_h = ld_h;
  p.db = db;
  p.partials = need ? static_cast<float*>(workspace) : nullptr;
  return cuda_result(mx::launch_ckpt_bwd(p, s), "checkpoint backward launch");
}

}  // extern "C"
