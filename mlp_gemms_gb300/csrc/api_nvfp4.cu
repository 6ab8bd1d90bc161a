// C ABI of the 4-bit tensors with scales per 16: host-side validation and launches
// of the quantization (nvfp4.cu) and the product (gemm_pair.cu).
#include "api_checks.h"

using mx::aligned;
using mx::check_dim;
using mx::check_matrix;
using mx::check_ptr;
using mx::cuda_result;

namespace {

mx_status_t check_tensor(const mx_nvfp4_t* t, const char* name, bool operand) {
  mx_status_t st;
  MX_CHECK(t != nullptr, MX_ERR_INVALID_ARG, "%s is NULL", name);
  MX_CHECK(t->cols > 0 && t->cols % 32 == 0 && t->cols < (1ll << 31), MX_ERR_SHAPE,
           "%s has %lld columns, not a positive multiple of 32 below 2^31", name, (long long)t->cols);
  MX_CHECK(t->rows >= 0 && t->rows < (1ll << 31) - 256 && t->rows * t->cols < (1ll << 46), MX_ERR_SHAPE,
           "%s is too large (%lld rows of %lld)", name, (long long)t->rows, (long long)t->cols);
  if (t->rows == 0) return MX_OK;
  if ((st = check_ptr(t->data, name)) != MX_OK || (st = check_ptr(t->scale, name)) != MX_OK) return st;
  if (!operand || t->row_scale) return check_ptr(t->row_scale, name);
  return MX_OK;
}

}  // namespace

extern "C" {

size_t mx_nvfp4_scale_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows >= (1ll << 31) || cols >= (1ll << 31)) return 0;
  return mx::scale_bytes(rows, (cols + 15) / 16);
}

size_t mx_nvfp4_quantize_workspace_bytes(int64_t T, int64_t K, int64_t R) {
  if (T <= 0 || K <= 0 || R <= 0 || T >= (1ll << 31) || K > mx::MAX_NVFP4_K || R >= (1ll << 31)) return 0;
  return mx::nvfp4_workspace(T, K, R);
}

mx_status_t mx_nvfp4_quantize(const void* x_bf16, int64_t T, int64_t K, int64_t ld, const int32_t* src_dev,
                              const int32_t* offsets_dev, int32_t G, const mx_nvfp4_t* out, void* workspace,
                              size_t workspace_bytes, mx_stream_t stream) {
  mx_status_t st;
  if ((st = check_dim(K, "K", 32)) != MX_OK) return st;
  MX_CHECK(K <= mx::MAX_NVFP4_K, MX_ERR_NOT_SUPPORTED, "K = %lld; rows of at most %lld columns", (long long)K,
           (long long)mx::MAX_NVFP4_K);
  MX_CHECK(T >= 0 && T < (1ll << 31), MX_ERR_SHAPE, "T = %lld is out of range", (long long)T);
  if ((st = check_matrix(x_bf16, "x", T, K, ld)) != MX_OK || (st = check_tensor(out, "out", false)) != MX_OK) return st;
  MX_CHECK(out->cols == K && (src_dev != nullptr || out->rows == T), MX_ERR_SHAPE, "out is [%lld, %lld]",
           (long long)out->rows, (long long)out->cols);
  MX_CHECK(aligned(src_dev, 4) && aligned(offsets_dev, 4), MX_ERR_ALIGNMENT, "src and offsets must be 4-byte aligned");
  MX_CHECK(offsets_dev == nullptr || G >= 1, MX_ERR_INVALID_ARG, "G = %d; at least one expert is required", G);
  const size_t need = src_dev && workspace ? mx_nvfp4_quantize_workspace_bytes(T, K, out->rows) : 0;
  if ((st = mx::check_workspace(workspace, workspace_bytes, need)) != MX_OK) return st;
  if (out->rows == 0) return MX_OK;
  int sms;
  if ((st = mx::device_sms(&sms)) != MX_OK) return st;
  mx::Nvfp4Params p{};
  p.T = T; p.K = K; p.R = out->rows;
  p.x = static_cast<const uint16_t*>(x_bf16); p.ld = ld;
  p.src = src_dev; p.offsets = offsets_dev; p.G = G;
  p.data = static_cast<uint8_t*>(out->data); p.scale = out->scale; p.row_scale = out->row_scale;
  return cuda_result(mx::launch_nvfp4_quantize(p, need ? workspace : nullptr, sms,
                                               reinterpret_cast<cudaStream_t>(stream)), "quantization launch");
}

mx_status_t mx_nvfp4_gemm(const mx_nvfp4_t* a, const mx_nvfp4_t* b, int32_t G, const int32_t* offsets_dev,
                          void* out_bf16, int64_t ld_out, mx_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  mx_status_t st;
  if ((st = check_tensor(a, "a", true)) != MX_OK || (st = check_tensor(b, "b", true)) != MX_OK) return st;
  MX_CHECK(G >= 1, MX_ERR_INVALID_ARG, "G = %d; at least one expert is required", G);
  MX_CHECK(G <= mx::MAX_PAIR_G_HOST, MX_ERR_NOT_SUPPORTED, "G = %d; at most %d experts", G, mx::MAX_PAIR_G_HOST);
  MX_CHECK(a->cols == b->cols, MX_ERR_SHAPE, "a has K = %lld, b has K = %lld", (long long)a->cols, (long long)b->cols);
  MX_CHECK(b->rows % G == 0, MX_ERR_SHAPE, "b has %lld rows, not a multiple of G = %d", (long long)b->rows, G);
  const int64_t K = a->cols, R = a->rows, N = b->rows / G;
  if ((st = check_dim(N, "N", G > 1 ? 128 : 8)) != MX_OK) return st;
  if ((st = check_matrix(out_bf16, "out", R, N, ld_out)) != MX_OK) return st;
  MX_CHECK(offsets_dev == nullptr || R % 128 == 0, MX_ERR_SHAPE, "R = %lld is not a multiple of 128", (long long)R);
  if ((st = mx::check_padded_offsets(offsets_dev, G, R, s)) != MX_OK) return st;
  if (R == 0) return MX_OK;
  int sms;
  if ((st = mx::device_sms(&sms)) != MX_OK) return st;
  mx::PairParams p{};
  p.nv4 = 1;
  p.G = G; p.offsets = offsets_dev;
  p.rows = R; p.R = mx::round_up_i64(R, 128);
  p.K = K; p.Nb = N;
  p.a_scale = a->row_scale; p.b_scale = b->row_scale;
  p.n_tiles = (N + 255) / 256;
  // 256-row tiles per expert segment: at most R / 256 plus one half-filled
  // tile for every expert with an odd number of 128-row blocks
  p.num_tiles = ((p.R + 255) / 256 + (offsets_dev ? (G + 1) / 2 : 0)) * p.n_tiles;
  // Fewer than 128 rows in all: A's boxes end with them.  The MMA's rows past them
  // hold what the shared memory held, reach only their own outputs and are not
  // stored.  (Boxes of 128 rows of which 127 lie outside the tensor: 44 us for one
  // row, 4096 -> 16384; 14 like this.)
  const int a_rows = R < 128 ? (int)mx::round_up_i64(R, 8) : 128;
  // one CTA's stage: 128 bytes of A's and B's rows, four scale chunks of A's row block and of both of B's
  p.tx_bytes = 128u * (uint32_t)a_rows + 16384u + 12u * 512u;
  p.out = static_cast<uint16_t*>(out_bf16); p.ld_out = ld_out;
  p.wide = aligned(out_bf16, 32) && ld_out % 16 == 0;
  CUtensorMap ta, tb, tsa, tsb;
  if ((st = mx::encode_packed_map(&ta, a->data, R, K, a_rows)) != MX_OK ||
      (st = mx::encode_packed_map(&tb, b->data, b->rows, K, 128)) != MX_OK ||
      (st = mx::encode_scales_map(&tsa, a->scale, R, K / 16, 1, 4)) != MX_OK ||
      (st = mx::encode_scales_map(&tsb, b->scale, b->rows, K / 16, 2, 4)) != MX_OK)
    return st;
  return cuda_result(mx::launch_gemm_pair(p, ta, tb, tsa, tsb, ta, s, sms), "4-bit GEMM launch");
}

}  // extern "C"
