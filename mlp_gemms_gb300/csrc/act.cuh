// Device helpers of the BF16 layers: activations and their slopes in fp32,
// programmatic launches.
#pragma once
#include "../../include/mx.h"
#include "mx_common.cuh"

namespace mx {

// Programmatic launches: everything the stream's earlier kernels wrote is
// visible after pdl_wait(); pdl_trigger() lets the stream's next kernel start
// as far as its own pdl_wait().
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// 1 / (1 + exp(-x)): exp by the hardware's 2^x and one approximate
// reciprocal (relative error a few 2^-23, against the 2^-9 of the BF16 the
// results are rounded to).  exp(-x) overflows to +Inf below -88: 0.
__device__ __forceinline__ float sigmoid_f32(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

constexpr float GELU_2A = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float GELU_B = 0.044715f;

// act(z).  The tanh GELU is z * sigmoid(2 sqrt(2/pi) (z + b z^3)), since
// (1 + tanh(u)) / 2 = sigmoid(2u): no cancellation for negative z.  ReLU
// keeps a NaN.
template <int ACT>
__device__ __forceinline__ float act_f32(float z) {
  if constexpr (ACT == MX_ACT_RELU) return z < 0.f ? 0.f : z;
  else if constexpr (ACT == MX_ACT_SILU) return z * sigmoid_f32(z);
  else if constexpr (ACT == MX_ACT_GELU_TANH) return z * sigmoid_f32(GELU_2A * fmaf(GELU_B * z * z, z, z));
  else return z;
}

// act(z) and act'(z) together.
template <int ACT>
__device__ __forceinline__ void act_slope_f32(float z, float* h, float* d) {
  if constexpr (ACT == MX_ACT_RELU) {
    *h = z < 0.f ? 0.f : z;
    *d = z > 0.f ? 1.f : 0.f;
  } else if constexpr (ACT == MX_ACT_SILU) {
    const float s = sigmoid_f32(z);
    *h = z * s;
    *d = fmaf(*h, 1.f - s, s);
  } else {
    const float z2 = z * z;
    const float s = sigmoid_f32(GELU_2A * fmaf(GELU_B * z2, z, z));
    *h = z * s;
    *d = fmaf(*h * (1.f - s), GELU_2A * fmaf(3.f * GELU_B, z2, 1.f), s);
  }
}

}  // namespace mx
