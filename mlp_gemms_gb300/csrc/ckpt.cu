// 8-bit activation checkpoints: the activation with an E4M3 / E8M0 copy of
// its input, and the backward pass that reads the copy.
#include "act.cuh"
#include "mx_internal.h"

namespace mx {

// A thread owns one 32-column block of one row (SWIGLU: the gate block and
// the up block of the same columns).
__device__ __forceinline__ void load32(const uint16_t* p, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
      v[8 * i + 2 * j] = bf16_bits_to_float(w[j] & 0xFFFFu);
      v[8 * i + 2 * j + 1] = bf16_bits_to_float(w[j] >> 16);
    }
  }
}
__device__ __forceinline__ void store32(uint16_t* p, const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; i++)
    reinterpret_cast<uint4*>(p)[i] =
        make_uint4(float2_to_bf16x2(v[8 * i], v[8 * i + 1]), float2_to_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                   float2_to_bf16x2(v[8 * i + 4], v[8 * i + 5]), float2_to_bf16x2(v[8 * i + 6], v[8 * i + 7]));
}
__device__ __forceinline__ void store_block(const CkptParams& p, int64_t r, int64_t c, float (&v)[32]) {
  const uint32_t b = rceil_scale_byte<E4M3>(amax_abs_bits<32>(v));
  uint32_t w[8];
  quantize_block_words<E4M3>(v, b, w);
  uint4* d = reinterpret_cast<uint4*>(p.q + r * p.C + c);
  d[0] = make_uint4(w[0], w[1], w[2], w[3]);
  d[1] = make_uint4(w[4], w[5], w[6], w[7]);
  p.q_scale[blocked_offset(r, c / 32, p.C / 32)] = (uint8_t)b;
}
// Two E4M3 codes -> two fp32 values, exact.
__device__ __forceinline__ void e4m3x2_to_f32(uint32_t two, float* lo, float* hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(*lo), "=f"(*hi) : "r"(h));
}
// The scale byte's power of two (0xFF: NaN).
__device__ __forceinline__ float scale_from_byte(uint32_t b) {
  return b == 0xFFu ? __uint_as_float(0x7FC00000u) : (b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23));
}
__device__ __forceinline__ void read_block(const CkptParams& p, int64_t r, int64_t c, float (&v)[32]) {
  const uint4* d = reinterpret_cast<const uint4*>(p.q + r * p.C + c);
  const float s = scale_from_byte(p.q_scale[blocked_offset(r, c / 32, p.C / 32)]);
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const uint4 q = __ldg(d + i);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
      e4m3x2_to_f32(w[j] & 0xFFFFu, &v[16 * i + 4 * j], &v[16 * i + 4 * j + 1]);
      e4m3x2_to_f32(w[j] >> 16, &v[16 * i + 4 * j + 2], &v[16 * i + 4 * j + 3]);
    }
  }
#pragma unroll
  for (int i = 0; i < 32; i++) v[i] *= s;
}

template <int ACT>
__global__ void __launch_bounds__(256) ckpt_fwd_simple(const CkptParams p) {
  const int64_t cols = ACT == MX_ACT_SWIGLU ? p.C / 2 : p.C, per = cols / 32;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.R * per; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per, c = i % per * 32;
    float z[32], h[32];
    load32(p.z + r * p.ld_z + c, z);
    if constexpr (ACT == MX_ACT_SWIGLU) {
      float u[32];
      load32(p.z + r * p.ld_z + cols + c, u);
#pragma unroll
      for (int j = 0; j < 32; j++) h[j] = act_f32<MX_ACT_SILU>(z[j]) * u[j];
      store_block(p, r, cols + c, u);
    } else {
#pragma unroll
      for (int j = 0; j < 32; j++) h[j] = act_f32<ACT>(z[j]);
    }
    store32(p.h + r * p.ld_h + c, h);
    store_block(p, r, c, z);
  }
}

constexpr int ROWS_PER_BLOCK = 64;
int64_t ckpt_row_blocks(int64_t R) { return (R + ROWS_PER_BLOCK - 1) / ROWS_PER_BLOCK; }

template <int ACT>
__global__ void __launch_bounds__(128) ckpt_bwd_simple(const CkptParams p) {
  const int64_t cols = ACT == MX_ACT_SWIGLU ? p.C / 2 : p.C;
  const int64_t c = ((int64_t)blockIdx.x * 128 + threadIdx.x) * 32;
  if (c >= cols) return;
  const int64_t r0 = (int64_t)blockIdx.y * ROWS_PER_BLOCK, r1 = r0 + ROWS_PER_BLOCK < p.R ? r0 + ROWS_PER_BLOCK : p.R;
  float sum[32] = {}, sum_u[32] = {};
  for (int64_t r = r0; r < r1; r++) {
    float z[32], dh[32], h[32];
    load32(p.dh + r * p.ld_dh + c, dh);
    read_block(p, r, c, z);
    if constexpr (ACT == MX_ACT_SWIGLU) {
      float u[32];
      read_block(p, r, cols + c, u);
#pragma unroll
      for (int j = 0; j < 32; j++) {
        float a, d;
        act_slope_f32<MX_ACT_SILU>(z[j], &a, &d);
        h[j] = a * u[j];
        z[j] = dh[j] * u[j] * d;
        u[j] = dh[j] * a;
        sum_u[j] += u[j];
      }
      store32(p.dz + r * p.ld_dz + cols + c, u);
    } else {
#pragma unroll
      for (int j = 0; j < 32; j++) {
        float d;
        act_slope_f32<ACT>(z[j], &h[j], &d);
        z[j] = dh[j] * d;
      }
    }
#pragma unroll
    for (int j = 0; j < 32; j++) sum[j] += z[j];
    store32(p.dz + r * p.ld_dz + c, z);
    if (p.h) store32(p.h + r * p.ld_h + c, h);
  }
  if (p.db) {
    float* d = p.partials + (int64_t)blockIdx.y * p.C + c;
#pragma unroll
    for (int j = 0; j < 32; j++) d[j] = sum[j];
    if constexpr (ACT == MX_ACT_SWIGLU) {
#pragma unroll
      for (int j = 0; j < 32; j++) d[cols + j] = sum_u[j];
    }
  }
}

cudaError_t launch_ckpt_fwd(const CkptParams& p, int num_sms, cudaStream_t s) {
  // padding scales are zero
  cudaError_t e = cudaMemsetAsync(p.q_scale, 0, scale_bytes(p.R, p.C / 32), s);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(num_sms * 8);
  switch (p.act) {
    case MX_ACT_SWIGLU: ckpt_fwd_simple<MX_ACT_SWIGLU><<<grid, 256, 0, s>>>(p); break;
    case MX_ACT_GELU_TANH: ckpt_fwd_simple<MX_ACT_GELU_TANH><<<grid, 256, 0, s>>>(p); break;
    case MX_ACT_SILU: ckpt_fwd_simple<MX_ACT_SILU><<<grid, 256, 0, s>>>(p); break;
    default: ckpt_fwd_simple<MX_ACT_RELU><<<grid, 256, 0, s>>>(p); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_ckpt_bwd(const CkptParams& p, int, cudaStream_t s) {
  const int64_t cols = p.act == MX_ACT_SWIGLU ? p.C / 2 : p.C;
  const dim3 grid((unsigned)((cols / 32 + 127) / 128), (unsigned)ckpt_row_blocks(p.R));
  switch (p.act) {
    case MX_ACT_SWIGLU: ckpt_bwd_simple<MX_ACT_SWIGLU><<<grid, 128, 0, s>>>(p); break;
    case MX_ACT_GELU_TANH: ckpt_bwd_simple<MX_ACT_GELU_TANH><<<grid, 128, 0, s>>>(p); break;
    case MX_ACT_SILU: ckpt_bwd_simple<MX_ACT_SILU><<<grid, 128, 0, s>>>(p); break;
    default: ckpt_bwd_simple<MX_ACT_RELU><<<grid, 128, 0, s>>>(p); break;
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.db == nullptr) return e;
  return launch_colsum_reduce(p.partials, ckpt_row_blocks(p.R), p.C, p.db, s);
}

}  // namespace mx
