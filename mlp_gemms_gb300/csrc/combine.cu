// The gradient of the experts' weighted sum (mx_moe_unpermute): of the experts'
// outputs and of the weights.
#include "mx_internal.h"
#include "vec8.cuh"

namespace mx {

static __device__ unsigned g_combine_status = 0;

// The sums over a warp of eight values a lane: after each exchange a lane keeps
// half of its values, so that lane l ends with the sum of value l / 4 (9 shuffles
// instead of 40).
__device__ __forceinline__ float warp_sum8(float (&v)[8], int lane) {
#pragma unroll
  for (int half = 4; half >= 1; half >>= 1) {
    const bool up = lane & (4 * half);
#pragma unroll
    for (int i = 0; i < half; i++) {
      const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, 4 * half);
    }
  }
  float s = v[0];
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
  return s + __shfl_xor_sync(0xFFFFFFFFu, s, 1);
}

// din[row of (t, j)] = w[t, j] dout[t], dw[t, j] = sum over columns of
// dout[t] in[row].  Bound by memory: a token's gradient is read once for all its
// choices, every expert row read and written once.  A block takes a token and up
// to 8 choices at a time, a thread 8 columns of them, whose loads are all in flight
// together; the next item's rows and weights are asked for before this one's
// columns.  The dot products' sums meet in shared memory, in a fixed order.
constexpr int JB = 8;
__global__ void __launch_bounds__(256, 3) combine_bwd_kernel(const CombineBwdParams p) {
  __shared__ float part[2][8][JB];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  const int per = (p.k + JB - 1) / JB;
  const int64_t items = p.T * per;
  int flip = 0, row_next = -1;
  float w_next = 1.f;
  pdl_trigger();
  pdl_wait();
  const auto ask = [&](int64_t item) {  // lane j: choice j of the item
    row_next = -1;
    if (item >= items) return;
    const int64_t t = per == 1 ? item : item / per;
    const int j = (int)(item - t * per) * JB + lane;
    if (lane >= JB || j >= p.k) return;
    row_next = *(p.row_of + t * p.k + j);
    if (p.weights != nullptr) w_next = *(p.weights + t * p.k + j);
  };
  ask(blockIdx.x);
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t t = per == 1 ? item : item / per;
    const int j0 = (int)(item - t * per) * JB;
    int row_mine = row_next;
    const float w_mine = w_next;
    if (row_mine >= p.R) {
      if (warp == 0) atomicOr(&g_combine_status, DEV_BAD_INDEX);
      row_mine = -1;
    }
    ask(item + gridDim.x);
    float dot[JB] = {};
    for (int64_t c0 = (int64_t)warp * 256; c0 < p.D; c0 += (int64_t)blockDim.x * 8) {  // the whole warp
      const int64_t c = c0 + lane * 8;
      const bool in = c < p.D;
      Raw8<false> dr = {}, xr[JB];
      if (in) dr = load_raw8<false>(p.dout, t * p.D + c);
#pragma unroll
      for (int j = 0; j < JB; j++) {
        const int row = __shfl_sync(0xFFFFFFFFu, row_mine, j);
        xr[j] = {};
        if (p.dweights != nullptr && in && row >= 0) xr[j] = load_raw8<false>(p.in, (int64_t)row * p.D + c);
      }
      uint64_t d[4];
      unpack_pairs<false>(dr, d);
#pragma unroll
      for (int j = 0; j < JB; j++) {
        const float w = __shfl_sync(0xFFFFFFFFu, w_mine, j);
        const int row = __shfl_sync(0xFFFFFFFFu, row_mine, j);
        if (row < 0) continue;  // the same for the whole warp
        uint64_t v[4];
        unpack_pairs<false>(xr[j], v);
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = mul2(d[i], v[i]);
        dot[j] += sum_pairs(v);
        if (p.din != nullptr && in) {
#pragma unroll
          for (int i = 0; i < 4; i++) v[i] = mul2(both(w), d[i]);
          store_raw8<false>(p.din, (int64_t)row * p.D + c, pack_pairs<false>(v));
        }
      }
    }
    if (p.dweights == nullptr) continue;
    const float s8 = warp_sum8(dot, lane);
    if ((lane & 3) == 0) part[flip][warp][lane >> 2] = s8;
    __syncthreads();
    if (tid < JB && j0 + tid < p.k) {
      float s = 0.f;
      for (int i = 0; i < warps; i++) s += part[flip][i][tid];
      p.dweights[t * p.k + j0 + tid] = s;
    }
    flip ^= 1;  // the next sums go elsewhere while these are read
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
  const int64_t cap = (int64_t)num_sms * 3 * (256 / threads), rows = p.src && p.din ? (p.R + 31) / 32 : 0;
  int64_t want = p.T * ((p.k + JB - 1) / JB);
  want = want > rows ? want : rows;
  want = want < 1 ? 1 : want < cap ? want : cap;
  return launch_pdl(combine_bwd_kernel, dim3((unsigned)want), threads, 0, s, dim3(1), p);
}

cudaError_t read_combine_status(unsigned* out) { return cudaMemcpyFromSymbol(out, g_combine_status, sizeof(unsigned)); }
cudaError_t reset_combine_status() {
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_combine_status, &zero, sizeof(unsigned));
}

}  // namespace mx
