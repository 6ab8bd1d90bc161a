// Eight consecutive values of a row, BF16 (16 bytes) or fp32 (32), as raw
// words and as fp32 values.
#pragma once
#include "act.cuh"

namespace mx {

template <bool F32> struct Raw8 { uint4 q[F32 ? 2 : 1]; };

// Streaming load: nothing here is read twice.  (Volatile: stays behind the
// programmatic wait.  Not the read-only path: an output may be the input itself.)
__device__ __forceinline__ uint4 load_stream16(const void* p) {
  uint4 q;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "l"(p));
  return q;
}
template <bool F32>
__device__ __forceinline__ Raw8<F32> load_raw8(const void* base, int64_t at) {  // element index, a multiple of 8
  Raw8<F32> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + at * (F32 ? 4 : 2));
  r.q[0] = load_stream16(p);
  if constexpr (F32) r.q[1] = load_stream16(p + 1);
  return r;
}
template <bool F32>
__device__ __forceinline__ void unpack_raw8(const Raw8<F32>& r, float (&v)[8]) {
  if constexpr (F32) {
    const uint32_t w[8] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w, r.q[1].x, r.q[1].y, r.q[1].z, r.q[1].w};
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = __uint_as_float(w[i]);
  } else {
    const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = bf16_bits_to_float(w[i] & 0xFFFFu);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
template <bool F32>
__device__ __forceinline__ Raw8<F32> pack_raw8(const float (&v)[8]) {
  Raw8<F32> r;
  if constexpr (F32) {
    r.q[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    r.q[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  } else {
    r.q[0] = make_uint4(float2_to_bf16x2(v[0], v[1]), float2_to_bf16x2(v[2], v[3]), float2_to_bf16x2(v[4], v[5]),
                        float2_to_bf16x2(v[6], v[7]));
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ void store_raw8(void* base, int64_t at, const Raw8<F32>& r) {
  uint4* p = reinterpret_cast<uint4*>(static_cast<char*>(base) + at * (F32 ? 4 : 2));
  p[0] = r.q[0];
  if constexpr (F32) p[1] = r.q[1];
}
// Eight values as four fp32 pairs for the packed instructions.
template <bool F32>
__device__ __forceinline__ void unpack_pairs(const Raw8<F32>& r, uint64_t (&v)[4]) {
  float f[8];
  unpack_raw8<F32>(r, f);
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = pack2(f[2 * i], f[2 * i + 1]);
}
template <bool F32>
__device__ __forceinline__ Raw8<F32> pack_pairs(const uint64_t (&v)[4]) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; i++) unpack2(v[i], &f[2 * i], &f[2 * i + 1]);
  return pack_raw8<F32>(f);
}
__device__ __forceinline__ float sum_pairs(const uint64_t (&v)[4]) {
  float a, b;
  unpack2(add2(add2(v[0], v[1]), add2(v[2], v[3])), &a, &b);
  return a + b;
}

// Eight values of a vector that many rows share (kept in L1).
__device__ __forceinline__ void load_shared8(const void* base, bool f32, int64_t at, float (&v)[8]) {
  if (f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    Raw8<false> r;
    r.q[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    unpack_raw8<false>(r, v);
  }
}

// Rows copied ahead into shared memory, 16 bytes at a time, without registers held by
// what is in flight, by the thread that will read them (no barrier) or by its warp
// (__syncwarp() between the wait and the reads, and between the reads and the copies
// that take their place).  A ring of S stages: wait_ahead<S - 2>() leaves the newest S - 2
// rows in flight.
__device__ __forceinline__ void copy_ahead16(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void commit_ahead() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_ahead() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

}  // namespace mx
