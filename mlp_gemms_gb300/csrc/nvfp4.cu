// Quantization of BF16 rows to packed E2M1 with an E4M3 scale for every 16
// values and a power of two for every row.
#include "mx_internal.h"
#include "vec8.cuh"

namespace mx {

static __device__ unsigned g_nvfp4_status = 0;

// Largest |value| of BF16 pairs, NaN if any is one (as bit patterns: a NaN's
// magnitude is above Inf's).
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a & 0x7FFF7FFFu), "r"(b & 0x7FFF7FFFu));
  return d;
}
__device__ __forceinline__ uint32_t max_halves(uint32_t a) {
  const uint32_t lo = a & 0xFFFFu, hi = a >> 16;
  return lo > hi ? lo : hi;
}

// For every row: 2^e the smallest power of two with amax <= 6 * 448 * 2^e (e >=
// -100), for every 16 values the scale s = E4M3(block amax / 2^e / 6), for every
// value the E2M1 code nearest to x / (2^e s), of two equally near ones the even.
//
// The quotient's rounding must not decide: x has 8 significant bits, s 4, a
// midpoint m of two codes 3, so x / (2^e s) either is m or differs from it by at
// least 1 / 255 of its value, 2^-10 for the smallest (m = 1 / 4).  The product with
// the rounded reciprocal is off by 2^-22, and adding and taking away 6144 rounds
// it to a multiple of 2^-11: a quotient that is a midpoint becomes exactly that,
// and none crosses one.
//
// Bound by memory (2 bytes read, 9 / 16 written a value).  A group of W warps
// holds a row in its registers, 16 values a lane and piece, as the norm does.
template <int C>
__global__ void __launch_bounds__(512) nvfp4_quantize_kernel(const Nvfp4Params p, int W) {
  __shared__ uint32_t part[2][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / W, wr = warp - group * W, groups = (blockDim.x >> 5) / W;
  const int64_t c0 = ((int64_t)wr * 32 + lane) * 16, step = (int64_t)W * 512, sc = p.K >> 4;
  int flip = 0;
  pdl_trigger();
  pdl_wait();
  int64_t rows = p.R;
  if (p.offsets != nullptr) {
    const int64_t end = *(p.offsets + p.G - 1);
    rows = end < 0 ? 0 : end < rows ? end : rows;
  }
  for (int64_t r = (int64_t)blockIdx.x * groups + group; r < rows; r += (int64_t)gridDim.x * groups) {
    int64_t from = r;
    if (p.src != nullptr) {
      from = *(p.src + r);
      if (from >= p.T) {
        if (wr == 0 && lane == 0) atomicOr(&g_nvfp4_status, DEV_BAD_INDEX);
        from = -1;
      }
    }
    uint4 x[C][2];
    uint32_t amax[C], top = 0;
#pragma unroll
    for (int c = 0; c < C; c++) {
      const int64_t at = c0 + c * step;
      x[c][0] = x[c][1] = make_uint4(0, 0, 0, 0);
      if (from >= 0 && at < p.K) {
        x[c][0] = load_stream16(p.x + from * p.ld + at);
        x[c][1] = load_stream16(p.x + from * p.ld + at + 8);
      }
    }
#pragma unroll
    for (int c = 0; c < C; c++) {
      uint32_t a = max_abs_bf16x2(x[c][0].x, x[c][0].y);
      a = max_abs_bf16x2(a, max_abs_bf16x2(x[c][0].z, x[c][0].w));
      a = max_abs_bf16x2(a, max_abs_bf16x2(x[c][1].x, x[c][1].y));
      a = max_abs_bf16x2(a, max_abs_bf16x2(x[c][1].z, x[c][1].w));
      amax[c] = max_halves(a);
      top = amax[c] > top ? amax[c] : top;
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (W > 1) {
      if (lane == 0) part[flip][warp] = top;
      named_bar(1 + group, 32 * W);
      for (int w = 0; w < W; w++) {
        const uint32_t t = part[flip][group * W + w];
        top = t > top ? t : top;
      }
      flip ^= 1;
    }
    const bool finite = top < 0x7F80u;
    int e = (int)(top >> 7) - 127 - 11 + ((top & 0x7Fu) > 40u ? 1 : 0);  // 6 * 448 = 1.3125 * 2^11; 40 / 128 = 0.3125
    e = e < -100 ? -100 : e;
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e, e in [-100, 117]
    if (wr == 0 && lane == 0)
      p.row_scale[r] = finite ? __uint_as_float((uint32_t)(127 + e) << 23) : __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int c = 0; c < C; c++) {
      const int64_t at = c0 + c * step;
      const float want = __fdiv_rn(bf16_bits_to_float(amax[c]) * down, 6.f);
      const uint32_t s8 = finite ? cvt_e4m3x2(want, 0.f) & 0xFFu : 0u;
      uint32_t h;
      float s, unused;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)s8));
      asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
          : "=f"(s), "=f"(unused) : "r"(h));
      const float inv = s8 == 0 ? 0.f : __fdiv_rn(1.f, s) * down;
      const uint32_t w[8] = {x[c][0].x, x[c][0].y, x[c][0].z, x[c][0].w, x[c][1].x, x[c][1].y, x[c][1].z, x[c][1].w};
      uint32_t out[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; i++) {
        float lo, hi;
        const uint64_t v = pack2(bf16_bits_to_float(w[i] & 0xFFFFu), __uint_as_float(w[i] & 0xFFFF0000u));
        unpack2(add2(fma2(v, both(inv), both(6144.f)), both(-6144.f)), &lo, &hi);
        out[i >> 2] |= cvt_e2m1x2(lo, hi) << (8 * (i & 3));
      }
      if (at < p.K)
        *reinterpret_cast<uint2*>(p.data + r * (p.K >> 1) + (at >> 1)) = finite ? make_uint2(out[0], out[1]) : make_uint2(0, 0);
      // the scale bytes of four lanes make a word of the blocked layout; past the
      // row's last block they are the padding's zeros
      uint32_t word = at < p.K ? s8 : 0u;
      word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1) << 8;
      word = (word & 0xFFFFu) | __shfl_xor_sync(0xFFFFFFFFu, word, 2) << 16;
      if ((lane & 3) == 0 && at < p.K) *reinterpret_cast<uint32_t*>(p.scale + blocked_offset(r, at >> 4, sc)) = word;
    }
  }
  if (blockIdx.x == 0 && p.offsets == nullptr) {  // the layout's rows past the last
    const int64_t chunks = (sc + 3) / 4, top_row = (p.R + 127) / 128 * 128;
    for (int64_t i = threadIdx.x; i < (top_row - p.R) * chunks; i += blockDim.x)
      *reinterpret_cast<uint32_t*>(p.scale + blocked_offset(p.R + i / chunks, i % chunks * 4, sc)) = 0u;
  }
}

cudaError_t launch_nvfp4_quantize(const Nvfp4Params& p, int num_sms, cudaStream_t s) {
  const int64_t v = (p.K + 15) / 16;
  int W = 1;
  while ((int64_t)W * 32 * 4 < v && W < 16) W *= 2;
  const int C = (int)((v + 32 * W - 1) / (32 * W));
  const int threads = W * 32 > 256 ? W * 32 : 256, groups = threads / (32 * W);
  const int64_t want = (p.R + groups - 1) / groups, cap = (int64_t)num_sms * 16;
  const dim3 grid((unsigned)(want < cap ? want : cap));
  switch (C) {
    case 1: return launch_pdl(nvfp4_quantize_kernel<1>, grid, threads, 0, s, dim3(1), p, W);
    case 2: return launch_pdl(nvfp4_quantize_kernel<2>, grid, threads, 0, s, dim3(1), p, W);
    case 3: return launch_pdl(nvfp4_quantize_kernel<3>, grid, threads, 0, s, dim3(1), p, W);
    default: return launch_pdl(nvfp4_quantize_kernel<4>, grid, threads, 0, s, dim3(1), p, W);
  }
}

cudaError_t read_nvfp4_status(unsigned* out) { return cudaMemcpyFromSymbol(out, g_nvfp4_status, sizeof(unsigned)); }
cudaError_t reset_nvfp4_status() {
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_nvfp4_status, &zero, sizeof(unsigned));
}

}  // namespace mx
