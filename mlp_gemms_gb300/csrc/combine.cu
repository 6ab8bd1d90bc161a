// The gradient of the experts' weighted sum (mx_moe_unpermute): of the experts'
// outputs and of the weights.
#include "mx_internal.h"
#include "vec8.cuh"

namespace mx {

static __device__ unsigned g_combine_status = 0;

// din[row of (t, j)] = w[t, j] dout[t], dw[t, j] = sum over columns of
// dout[t] in[row].  Bound by memory: a token's gradient is read once for all its
// choices, every expert row read and written once.  A block takes a token, a
// thread 8 columns of it at a time for up to 8 choices, whose loads are all in
// flight together; the dot products' sums meet in shared memory, in a fixed
// order.
constexpr int JB = 8;
__global__ void __launch_bounds__(256) combine_bwd_kernel(const CombineBwdParams p) {
  __shared__ float part[2][8][JB];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  int flip = 0;
  pdl_trigger();
  pdl_wait();
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    for (int j0 = 0; j0 < p.k; j0 += JB) {
      const int n = p.k - j0 < JB ? p.k - j0 : JB;
      int64_t row[JB];
      float w[JB], dot[JB] = {};
#pragma unroll
      for (int j = 0; j < JB; j++) {
        row[j] = -1;
        w[j] = 1.f;
        if (j < n) {
          row[j] = *(p.row_of + t * p.k + j0 + j);
          if (p.weights != nullptr) w[j] = *(p.weights + t * p.k + j0 + j);
        }
        if (row[j] >= p.R) {
          if (tid == 0) atomicOr(&g_combine_status, DEV_BAD_INDEX);
          row[j] = -1;
        }
      }
      for (int64_t c = (int64_t)tid * 8; c < p.D; c += (int64_t)blockDim.x * 8) {
        const Raw8<false> dr = load_raw8<false>(p.dout, t * p.D + c);
        Raw8<false> xr[JB];
        if (p.dweights != nullptr) {
#pragma unroll
          for (int j = 0; j < JB; j++)
            if (row[j] >= 0) xr[j] = load_raw8<false>(p.in, row[j] * p.D + c);
        }
        float d[8];
        unpack_raw8<false>(dr, d);
#pragma unroll
        for (int j = 0; j < JB; j++) {
          if (row[j] < 0) continue;
          float v[8];
          if (p.dweights != nullptr) {
            unpack_raw8<false>(xr[j], v);
#pragma unroll
            for (int i = 0; i < 8; i++) dot[j] = fmaf(d[i], v[i], dot[j]);
          }
          if (p.din != nullptr) {
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = w[j] * d[i];
            store_raw8<false>(p.din, row[j] * p.D + c, pack_raw8<false>(v));
          }
        }
      }
      if (p.dweights == nullptr) continue;
#pragma unroll
      for (int j = 0; j < JB; j++) {
        const float s = warp_sum(dot[j]);
        if (lane == 0) part[flip][warp][j] = s;
      }
      __syncthreads();
      if (tid < n) {
        float s = 0.f;
        for (int i = 0; i < warps; i++) s += part[flip][i][tid];
        p.dweights[t * p.k + j0 + tid] = s;
      }
      flip ^= 1;  // the next sums go elsewhere while these are read
    }
  }
  if (p.src == nullptr || p.din == nullptr) return;
  // empty rows, 32 of a warp's at a time
  for (int64_t r0 = ((int64_t)blockIdx.x * warps + warp) * 32; r0 < p.R; r0 += (int64_t)gridDim.x * warps * 32) {
    unsigned empty = __ballot_sync(0xFFFFFFFFu, r0 + lane < p.R && *(p.src + (r0 + lane < p.R ? r0 + lane : r0)) < 0);
    while (empty != 0) {
      const int64_t r = r0 + __ffs(empty) - 1;
      empty &= empty - 1;
      for (int64_t c = lane * 8; c < p.D; c += 256) *reinterpret_cast<uint4*>(p.din + r * p.D + c) = make_uint4(0, 0, 0, 0);
    }
  }
}

cudaError_t launch_combine_bwd(const CombineBwdParams& p, int num_sms, cudaStream_t s) {
  const int threads = p.D >= 2048 ? 256 : (int)((p.D / 8 + 31) / 32 * 32);
  const int64_t cap = (int64_t)num_sms * 8, rows = p.src && p.din ? (p.R + 31) / 32 : 0;
  int64_t want = p.T > rows ? p.T : rows;
  want = want < 1 ? 1 : want < cap ? want : cap;
  return launch_pdl(combine_bwd_kernel, dim3((unsigned)want), threads, 0, s, dim3(1), p);
}

cudaError_t read_combine_status(unsigned* out) { return cudaMemcpyFromSymbol(out, g_combine_status, sizeof(unsigned)); }
cudaError_t reset_combine_status() {
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_combine_status, &zero, sizeof(unsigned));
}

}  // namespace mx
