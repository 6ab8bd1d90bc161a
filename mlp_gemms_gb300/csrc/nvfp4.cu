// Quantization of BF16 rows to packed E2M1 with an E4M3 scale for every 16
// values and a power of two for every row.
#include "mx_internal.h"
#include "vec8.cuh"

namespace mx {

static __device__ unsigned g_nvfp4_status = 0;

// Larger magnitude of BF16 pairs, a NaN if either is one (the sign bits are
// meaningless); as bit patterns a NaN's magnitude is above Inf's.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Eight fp32 values -> eight E2M1 codes, the first in the lowest nibble.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r) : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
__device__ __forceinline__ uint32_t max_halves(uint32_t a) {
  const uint32_t lo = a & 0x7FFFu, hi = a >> 16 & 0x7FFFu;
  return lo > hi ? lo : hi;
}

// Row r's first scale byte in the blocked layout.
__device__ __forceinline__ int64_t row_place(int64_t r, int64_t chunks) {
  return (r >> 7) * chunks * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4;
}
// Bytes of a row of scales kept row-major, in whole 16-byte pieces.
__host__ __device__ __forceinline__ int64_t scale_pitch(int64_t K) { return (K + 255) / 256 * 16; }
// The layout's rows past the last, zero: a warp takes a chunk of the last row
// block, a lane the four rows that share its 16 bytes.
__device__ __forceinline__ void pad_scales(const Nvfp4Params& p, int64_t chunks) {
  const int first = (int)(p.R & 127), warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  for (int64_t c = (int64_t)blockIdx.x * warps + warp; c < chunks; c += (int64_t)gridDim.x * warps) {
    uint32_t* const to = reinterpret_cast<uint32_t*>(p.scale + ((p.R >> 7) * chunks + c) * 512 + lane * 16);
#pragma unroll
    for (int q = 0; q < 4; q++)
      if (32 * q + lane >= first) to[q] = 0u;
  }
}

// For every row: 2^e the smallest power of two with amax <= 6 * 448 * 2^e (e >=
// -100), for every 16 values the scale s = E4M3(block amax / 2^e / 6), for every
// value the E2M1 code nearest to x / (2^e s), of two equally near ones the even.
//
// No rounding on the way may decide.  x has 8 significant bits, s 4, a midpoint m
// of two codes 3: so x / (2^e s) either is m or differs from it by at least 1 / 255
// of its value, 2^-10 for the smallest (m = 1 / 4).  The product with the
// approximate reciprocal is off by 2^-22, and adding and taking away 6144 rounds
// it to a multiple of 2^-11: a quotient that is a midpoint becomes exactly that,
// and none crosses one.  Likewise amax / 6 and the E4M3 midpoints (5 bits): the
// product with fl(1 / 6), off by 2^-25, rounds to a midpoint where the quotient is
// one (their significands are at most 1.9375, half a unit is then more than that).
//
// Reads 2 bytes and writes 9 / 16 a value, but about six instructions a value are
// the nearer limit.  A group of W warps holds a row in its registers, 16 values a
// lane and piece; the next row's loads (and the source after that) are issued
// before this row's maximum is exchanged.
template <int C>
__global__ void __launch_bounds__(512) nvfp4_quantize_kernel(const Nvfp4Params p, int W) {
  __shared__ uint32_t part[2][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / W, wr = warp - group * W, groups = (blockDim.x >> 5) / W;
  const int c0 = (wr * 32 + lane) * 16, step = W * 512, K = (int)p.K;
  const int64_t chunks = (p.K + 63) >> 6, chunk_bytes = p.linear ? 4 : 512, stride = (int64_t)gridDim.x * groups;
  int flip = 0;
  pdl_trigger();
  pdl_wait();
  int64_t rows = p.R;
  if (p.offsets != nullptr) {
    const int64_t end = *(p.offsets + p.G - 1);
    rows = end < 0 ? 0 : end < rows ? end : rows;
  }
  const auto source = [&](int64_t r) -> int64_t {
    if (r >= rows) return -1;
    if (p.src == nullptr) return r;
    const int64_t from = *(p.src + r);
    if (from < p.T) return from;
    if (wr == 0 && lane == 0) atomicOr(&g_nvfp4_status, DEV_BAD_INDEX);
    return -1;
  };
  uint4 next[C][2];
  const auto load_row = [&](int64_t from) {
#pragma unroll
    for (int c = 0; c < C; c++) {
      const int at = c0 + c * step;
      next[c][0] = next[c][1] = make_uint4(0, 0, 0, 0);
      if (from >= 0 && at < K) {
        next[c][0] = load_stream16(p.x + from * p.ld + at);
        next[c][1] = load_stream16(p.x + from * p.ld + at + 8);
      }
    }
  };
  int64_t r = (int64_t)blockIdx.x * groups + group;
  load_row(source(r));
  int64_t after = source(r + stride);
  for (; r < rows; r += stride) {
    uint32_t x[C][8], amax[C], top = 0;
#pragma unroll
    for (int c = 0; c < C; c++) {
      const uint4 a = next[c][0], b = next[c][1];
      x[c][0] = a.x; x[c][1] = a.y; x[c][2] = a.z; x[c][3] = a.w;
      x[c][4] = b.x; x[c][5] = b.y; x[c][6] = b.z; x[c][7] = b.w;
      const uint32_t m = max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(x[c][0], x[c][1]), max_abs_bf16x2(x[c][2], x[c][3])),
                                        max_abs_bf16x2(max_abs_bf16x2(x[c][4], x[c][5]), max_abs_bf16x2(x[c][6], x[c][7])));
      amax[c] = max_halves(m);
      top = amax[c] > top ? amax[c] : top;
    }
    load_row(after);
    after = source(r + 2 * stride);
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
    const float down = finite ? __uint_as_float((uint32_t)(127 - e) << 23) : 0.f;  // 2^-e, e in [-100, 117]
    if (wr == 0 && lane == 0)
      p.row_scale[r] = finite ? __uint_as_float((uint32_t)(127 + e) << 23) : __uint_as_float(0x7FC00000u);
    // scale (r, c) of the blocked layout: the row's place in a chunk, then a chunk every four columns
    uint8_t* const scales = p.scale + (p.linear ? r * scale_pitch(p.K) : row_place(r, chunks));
    uint8_t* const data = p.data + r * (p.K >> 1);
#pragma unroll
    for (int c = 0; c < C; c++) {
      const int at = c0 + c * step;
      const float want = finite ? bf16_bits_to_float(amax[c]) * down * (1.f / 6.f) : 0.f;
      const uint32_t s8 = cvt_e4m3x2(want, 0.f) & 0xFFu;
      uint32_t h;
      float s, inv;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)s8));
      asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(s) : "r"(h));
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
      inv = s8 == 0 ? 0.f : inv * down;
      uint32_t out[2];
#pragma unroll
      for (int o = 0; o < 2; o++) {
        float q[8];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const uint32_t w = x[c][4 * o + i];
          const uint64_t v = pack2(bf16_bits_to_float(w & 0xFFFFu), __uint_as_float(w & 0xFFFF0000u));
          unpack2(add2(fma2(v, both(inv), both(6144.f)), both(-6144.f)), &q[2 * i], &q[2 * i + 1]);
        }
        out[o] = cvt_e2m1x8(q);
        if (!finite) out[o] = 0;  // Inf * 0 is a NaN
      }
      // the scale bytes of four lanes make a word of the blocked layout; past the
      // row's last block they are the padding's zeros
      uint32_t word = at < K ? s8 : 0u;
      word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1) << 8;
      word = (word & 0xFFFFu) | __shfl_xor_sync(0xFFFFFFFFu, word, 2) << 16;
      if (at < K) {
        *reinterpret_cast<uint2*>(data + (at >> 1)) = make_uint2(out[0], out[1]);
        if ((lane & 3) == 0) *reinterpret_cast<uint32_t*>(scales + (at >> 6) * chunk_bytes) = word;
      }
    }
  }
  if ((p.R & 127) != 0 && p.offsets == nullptr && !p.linear) pad_scales(p, chunks);
}

// Gathered rows of tokens that are quantized already (each for itself, so all of
// a token's rows are the same bytes): codes, scales (row-major, 16-byte pieces) and
// row scales of T tokens, copied to every row that names one.  A block takes a row
// block of 128: a warp copies the codes of 16 rows, four at a time, and turns the
// scales of four chunks, where a lane holds the four rows that share 16 bytes of the
// layout (written row by row, as words: 36 us for 8192 tokens' quantization and
// 73700 rows; 28 this way).
__global__ void __launch_bounds__(256, 4) nvfp4_gather_kernel(const Nvfp4Params p, const uint8_t* data, const uint8_t* scale,
                                                              const float* row_scale) {
  __shared__ int from_s[128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t chunks = (p.K + 63) >> 6, bytes = p.K >> 1, pitch = scale_pitch(p.K);
  pdl_trigger();
  pdl_wait();
  int64_t rows = p.R;
  if (p.offsets != nullptr) {
    const int64_t end = *(p.offsets + p.G - 1);
    rows = end < 0 ? 0 : end < rows ? end : rows;
  }
  for (int64_t b0 = (int64_t)blockIdx.x * 128; b0 < rows; b0 += (int64_t)gridDim.x * 128) {
    __syncthreads();  // the block before has been copied
    if (threadIdx.x < 128) {
      const int64_t r = b0 + threadIdx.x;
      int from = r < rows ? *(p.src + r) : -1;
      if (from >= p.T) {
        atomicOr(&g_nvfp4_status, DEV_BAD_INDEX);
        from = -1;
      }
      from_s[threadIdx.x] = from;
      if (r < rows) p.row_scale[r] = from >= 0 ? *(row_scale + from) : __uint_as_float((uint32_t)(127 - 100) << 23);
    }
    __syncthreads();
    for (int i0 = warp * 16; i0 < warp * 16 + 16; i0 += 4) {
      for (int64_t at = lane * 16; at < bytes; at += 512) {
        uint4 q[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int64_t from = from_s[i0 + i];
          q[i] = from >= 0 ? *reinterpret_cast<const uint4*>(data + from * bytes + at) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (b0 + i0 + i < rows) *reinterpret_cast<uint4*>(p.data + (b0 + i0 + i) * bytes + at) = q[i];
      }
    }
    // rows past the last: the layout's padding, zero; with offsets not this call's
    const int64_t limit = p.offsets != nullptr ? rows - b0 : 128;
    for (int64_t c0 = warp * 4; c0 < chunks; c0 += 32) {
      uint4 v[4];
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int64_t from = from_s[lane + 32 * q];
        v[q] = from >= 0 ? *reinterpret_cast<const uint4*>(scale + from * pitch + c0 * 4) : make_uint4(0, 0, 0, 0);
      }
      const uint32_t w[4][4] = {{v[0].x, v[1].x, v[2].x, v[3].x}, {v[0].y, v[1].y, v[2].y, v[3].y},
                                {v[0].z, v[1].z, v[2].z, v[3].z}, {v[0].w, v[1].w, v[2].w, v[3].w}};
#pragma unroll
      for (int j = 0; j < 4; j++) {
        if (c0 + j >= chunks) break;
        uint32_t* const to = reinterpret_cast<uint32_t*>(p.scale + ((b0 >> 7) * chunks + c0 + j) * 512 + lane * 16);
        if (limit >= 128) {
          *reinterpret_cast<uint4*>(to) = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
        } else {
#pragma unroll
          for (int q = 0; q < 4; q++)
            if (lane + 32 * q < limit) to[q] = w[j][q];
        }
      }
    }
  }
}

// Where rows name tokens three times on average and there is enough to save for
// the second launch, they are copied from the tokens' quantization (us, each row
// quantized for itself in brackets): 8192 tokens of 2048 columns to 73700 rows 28
// (68), to 32768 rows 25 (31), to 16384 rows 17.3 (17.5); 64 tokens to 512 rows 5.4
// (2.8).
size_t nvfp4_workspace(int64_t T, int64_t K, int64_t R) {
  if (R < 3 * T || (R - T) * K < (1 << 24)) return 0;
  return (size_t)round_up_i64(T * (K >> 1), 16) + (size_t)(T * scale_pitch(K)) + (size_t)T * 4;
}

static cudaError_t launch_rows(const Nvfp4Params& p, int num_sms, cudaStream_t s) {
  const int64_t v = (p.K + 15) / 16;
  int W = 1;
  while ((int64_t)W * 32 * 2 < v && W < 16) W *= 2;
  const int C = (int)((v + 32 * W - 1) / (32 * W));
  const int threads = W * 32 > 256 ? W * 32 : 256, groups = threads / (32 * W);
  const int64_t want = (p.R + groups - 1) / groups, cap = (int64_t)num_sms * (threads > 256 ? 4 : 8);
  const dim3 grid((unsigned)(want < cap ? want : cap));
  if (C == 1) return launch_pdl(nvfp4_quantize_kernel<1>, grid, threads, 0, s, dim3(1), p, W);
  if (C == 2) return launch_pdl(nvfp4_quantize_kernel<2>, grid, threads, 0, s, dim3(1), p, W);
  return launch_pdl(nvfp4_quantize_kernel<4>, grid, threads, 0, s, dim3(1), p, W);
}

cudaError_t launch_nvfp4_quantize(const Nvfp4Params& p, void* workspace, int num_sms, cudaStream_t s) {
  if (workspace == nullptr) return launch_rows(p, num_sms, s);
  Nvfp4Params t = p;
  t.R = p.T;
  t.src = t.offsets = nullptr;
  t.linear = 1;
  t.data = static_cast<uint8_t*>(workspace);
  t.scale = t.data + round_up_i64(p.T * (p.K >> 1), 16);
  t.row_scale = reinterpret_cast<float*>(t.scale + p.T * scale_pitch(p.K));
  const cudaError_t e = launch_rows(t, num_sms, s);
  if (e != cudaSuccess) return e;
  const int64_t want = (p.R + 127) / 128, cap = (int64_t)num_sms * 4;
  return launch_pdl(nvfp4_gather_kernel, dim3((unsigned)(want < cap ? want : cap)), 256, 0, s, dim3(1), p, t.data, t.scale,
                    t.row_scale);
}

cudaError_t read_nvfp4_status(unsigned* out) { return cudaMemcpyFromSymbol(out, g_nvfp4_status, sizeof(unsigned)); }
cudaError_t reset_nvfp4_status() {
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_nvfp4_status, &zero, sizeof(unsigned));
}

}  // namespace mx
