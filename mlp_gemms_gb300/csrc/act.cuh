// Device helpers of the BF16 layers: activations and their slopes in fp32,
// programmatic launches.
#pragma once
#include "../../include/mx.h"
#include "mx_common.cuh"

namespace mx {

// Programmatic launches: everything the stream's earlier kernels wrote is
// visible after pdl_wait(); pdl_trigger() lets the stream's next kernel start
// as far as its own pdl_wait().  Global memory is read by plain loads or by
// volatile asm after the wait, not by __ldg nor through const __restrict__
// pointers: the compiler may take what those read for constant and move the
// load up across the wait.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Two fp32 values that go through the packed instructions (each lane an
// ordinary round-to-nearest operation).
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float* lo, float* hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t both(float v) { return pack2(v, v); }

// 1 / (1 + 2^x) of both lanes: the hardware's 2^x and reciprocal (relative
// error a few 2^-23, against the 2^-9 of the BF16 the results are rounded
// to; a result below 2^-126, from x = 126 on, is 0).  2^x overflows to +Inf past
// 128: 0.
__device__ __forceinline__ uint64_t inv_1p_exp2(uint64_t x) {
  float a, b;
  unpack2(x, &a, &b);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
  unpack2(add2(pack2(a, b), both(1.f)), &a, &b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
  return pack2(a, b);
}

constexpr float LOG2E = 1.4426950408889634f;
constexpr float GELU_2A = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float GELU_B = 0.044715f;

// sigmoid(k z (1 + b z^2)) of both lanes: SiLU's gate (k = 1, b = 0) and the
// tanh GELU's, since (1 + tanh(u)) / 2 = sigmoid(2u): no cancellation for
// negative z.
template <int ACT>
__device__ __forceinline__ uint64_t gate2(uint64_t z, uint64_t z2) {
  if constexpr (ACT == MX_ACT_SILU) return inv_1p_exp2(mul2(z, both(-LOG2E)));
  else return inv_1p_exp2(mul2(z, fma2(z2, both(-LOG2E * GELU_2A * GELU_B), both(-LOG2E * GELU_2A))));
}

// act(z) of two values.  ReLU keeps a NaN.
template <int ACT>
__device__ __forceinline__ void act2(float* a, float* b) {
  if constexpr (ACT == MX_ACT_RELU) {
    *a = *a < 0.f ? 0.f : *a;
    *b = *b < 0.f ? 0.f : *b;
  } else if constexpr (ACT != MX_ACT_NONE) {
    const uint64_t z = pack2(*a, *b);
    unpack2(mul2(z, gate2<ACT>(z, mul2(z, z))), a, b);
  }
}

// act(z) and act'(z) of two values (SiLU, GELU).  GELU: the slope's z^2 ends
// at 2^20, far past where t has become exactly 0: unbounded it is Inf from
// |z| = 2^64 on, and 0 times that NaN.  (A NaN z stays one through t.)
template <int ACT>
__device__ __forceinline__ void act_slope2(uint64_t z, uint64_t* h, uint64_t* d) {
  const uint64_t z2 = mul2(z, z), s = gate2<ACT>(z, z2);
  *h = mul2(z, s);
  const uint64_t t = mul2(*h, fma2(s, both(-1.f), both(1.f)));
  if constexpr (ACT == MX_ACT_SILU) {
    *d = add2(t, s);
  } else {
    float a, b;
    unpack2(z2, &a, &b);
    *d = fma2(t, fma2(pack2(fminf(a, 1048576.f), fminf(b, 1048576.f)), both(3.f * GELU_B * GELU_2A), both(GELU_2A)), s);
  }
}

// act(z) and the gradient dh act'(z) of two values.  ReLU selects: an Inf or
// NaN behind a closed gate is not multiplied by zero.
template <int ACT>
__device__ __forceinline__ void act_bwd2(uint64_t z, uint64_t dh, uint64_t* h, uint64_t* dz) {
  if constexpr (ACT == MX_ACT_RELU) {
    float a, b, da, db;
    unpack2(z, &a, &b);
    unpack2(dh, &da, &db);
    *h = pack2(a < 0.f ? 0.f : a, b < 0.f ? 0.f : b);
    *dz = pack2(a > 0.f ? da : 0.f, b > 0.f ? db : 0.f);
  } else {
    uint64_t slope;
    act_slope2<ACT>(z, h, &slope);
    *dz = mul2(dh, slope);
  }
}

}  // namespace mx
