// BF16 products over ragged expert segments (any length, no padding): the
// grouped product with W [G, N, K] or [G, K, N], the weight gradient, and the
// dense linear layer's epilogue.
#include "act.cuh"
#include "mx_internal.h"

namespace mx {

static __device__ unsigned g_ragged_status = 0;

// Segment g of the offsets as [begin, end); false (and the status bit) when
// it decreases or passes R.
__device__ __forceinline__ bool segment(const int32_t* offsets, int g, int64_t R, int64_t* begin, int64_t* end) {
  *begin = (offsets && g) ? (int64_t)__ldg(offsets + g - 1) : 0;
  *end = offsets ? (int64_t)__ldg(offsets + g) : R;
  if (*begin < 0 || *end < *begin || *end > R) {
    atomicOr(&g_ragged_status, DEV_BAD_OFFSETS);
    return false;
  }
  return true;
}

constexpr int TS = 64, TK = 16;

// acc[i][j] += sum_k A(m, k) B(n, k) for a 64 x 64 tile, both read through
// strides; 256 threads, 4 x 4 values each.
__device__ __forceinline__ void tile_product(const uint16_t* a, int64_t sam, int64_t sak, int64_t m, const uint16_t* b,
                                             int64_t sbn, int64_t sbk, int64_t n, int64_t k, float (&acc)[4][4]) {
  __shared__ float sa[TK][TS + 1], sb[TK][TS + 1];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int64_t k0 = 0; k0 < k; k0 += TK) {
    for (int i = threadIdx.x; i < TS * TK; i += 256) {
      const int r = i / TK, c = i % TK;
      sa[c][r] = (r < m && k0 + c < k) ? bf16_bits_to_float(a[r * sam + (k0 + c) * sak]) : 0.f;
      sb[c][r] = (r < n && k0 + c < k) ? bf16_bits_to_float(b[r * sbn + (k0 + c) * sbk]) : 0.f;
    }
    __syncthreads();
    for (int c = 0; c < TK; c++)
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i][j] = fmaf(sa[c][ty * 4 + i], sb[c][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
}

__device__ __forceinline__ float act_any(float z, int act) {
  return act == MX_ACT_RELU ? act_f32<MX_ACT_RELU>(z)
         : act == MX_ACT_SILU ? act_f32<MX_ACT_SILU>(z)
         : act == MX_ACT_GELU_TANH ? act_f32<MX_ACT_GELU_TANH>(z) : z;
}

__device__ __forceinline__ uint16_t bf16_of(float v) { return (uint16_t)float2_to_bf16x2(v, 0.f); }

__global__ void __launch_bounds__(256) ragged_gemm_simple(const RaggedParams p) {
  __shared__ int64_t s_m0, s_rows;
  __shared__ int s_g;
  if (threadIdx.x == 0) {
    int64_t t = blockIdx.y;
    s_g = -1;
    for (int g = 0; g < p.G; g++) {
      int64_t b, e;
      if (!segment(p.offsets, g, p.R, &b, &e)) continue;
      const int64_t n = (e - b + TS - 1) / TS;
      if (t < n) {
        s_g = g; s_m0 = b + t * TS; s_rows = e - s_m0 < TS ? e - s_m0 : TS;
        break;
      }
      t -= n;
    }
  }
  __syncthreads();
  if (s_g < 0) return;
  const int64_t m0 = s_m0, rows = s_rows, n0 = (int64_t)blockIdx.x * TS;
  const uint16_t* w = p.w + (int64_t)s_g * p.N * p.K;
  const int64_t sbn = p.w_kn ? 1 : p.K, sbk = p.w_kn ? p.N : 1;
  float acc[4][4] = {};
  tile_product(p.a + m0 * p.ld_a, p.ld_a, 1, rows, w + n0 * sbn, sbn, sbk, p.N - n0, p.K, acc);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  __shared__ float sz[TS][TS + 1];
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int64_t r = ty * 4 + i, n = n0 + tx * 4 + j;
      if (r >= rows || n >= p.N) continue;
      float z = acc[i][j];
      if (p.epi.bias) z += bf16_bits_to_float(p.epi.bias[n]);
      sz[ty * 4 + i][tx * 4 + j] = z;
      float v = act_any(z, p.epi.act);
      if (p.epi.res) v += bf16_bits_to_float(p.epi.res[(m0 + r) * p.epi.ld_res + n]);
      p.out[(m0 + r) * p.ld_out + n] = bf16_of(v);
    }
  if (p.epi.q == nullptr) return;
  __syncthreads();
  if (threadIdx.x < 2 * TS) {
    const int r = threadIdx.x >> 1, c = (threadIdx.x & 1) * 32;
    if (r < rows && n0 + c < p.N) {
      float v[32];
      for (int i = 0; i < 32; i++) v[i] = sz[r][c + i];
      const uint32_t b = rceil_scale_byte<E4M3>(amax_abs_bits<32>(v));
      uint32_t words[8];
      quantize_block_words<E4M3>(v, b, words);
      uint32_t* d = reinterpret_cast<uint32_t*>(p.epi.q + (m0 + r) * p.N + n0 + c);
      for (int i = 0; i < 8; i++) d[i] = words[i];
      p.epi.q_scale[blocked_offset(m0 + r, (n0 + c) / 32, p.N / 32)] = (uint8_t)b;
    }
  }
}

cudaError_t launch_ragged_gemm(const RaggedParams& p, int, cudaStream_t s) {
  if (p.epi.q) {
    const cudaError_t e = cudaMemsetAsync(p.epi.q_scale, 0, scale_bytes(p.R, p.N / 32), s);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((unsigned)((p.N + TS - 1) / TS), (unsigned)((p.R + TS - 1) / TS + (p.offsets ? p.G : 0)));
  ragged_gemm_simple<<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

__global__ void __launch_bounds__(256) ragged_wgrad_simple(const RaggedWgradParams p) {
  const int g = blockIdx.z;
  int64_t b, e;
  if (!segment(p.offsets, g, p.R, &b, &e)) e = b;
  const int64_t n0 = (int64_t)blockIdx.y * TS, k0 = (int64_t)blockIdx.x * TS;
  float acc[4][4] = {};
  if (e > b)
    tile_product(p.dy + b * p.ld_dy + n0, 1, p.ld_dy, p.N - n0, p.x + b * p.ld_x + k0, 1, p.ld_x, p.K - k0, e - b,
                 acc);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int64_t n = n0 + ty * 4 + i, k = k0 + tx * 4 + j;
      if (n >= p.N || k >= p.K) continue;
      const int64_t at = ((int64_t)g * p.N + n) * p.K + k;
      if (p.grad) p.grad[at] = bf16_of(acc[i][j]);
      else p.grad_f32[at] = p.accumulate ? p.grad_f32[at] + acc[i][j] : acc[i][j];
    }
}

cudaError_t launch_ragged_wgrad(const RaggedWgradParams& p, int, cudaStream_t s) {
  const dim3 grid((unsigned)((p.K + TS - 1) / TS), (unsigned)((p.N + TS - 1) / TS), (unsigned)p.G);
  ragged_wgrad_simple<<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t read_ragged_status(unsigned* out) { return cudaMemcpyFromSymbol(out, g_ragged_status, sizeof(unsigned)); }
cudaError_t reset_ragged_status() {
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_ragged_status, &zero, sizeof(unsigned));
}

}  // namespace mx
