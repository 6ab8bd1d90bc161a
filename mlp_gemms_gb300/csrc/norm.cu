// Layer norm (and its form without a mean): forward with the residual added in
// the same pass, and the backward pass with the weight's and the bias's
// gradients.
#include "mx_internal.h"
#include "vec8.cuh"

namespace mx {

// Both kernels are bound by memory: every value is read once and written once.
// A row is held in the registers of `W` warps (a power of two), 8 C columns a
// lane, so that its statistics, its centred squares and its result need no
// second read; a block's warps form groups of W, each with a row of its own.

// The group's barrier: its W warps, W > 1.
__device__ __forceinline__ void group_bar(int group, int W) { named_bar(1 + group, 32 * W); }

// Forward.  Mean and centred sum of squares without cancellation, with one
// exchange between the warps: each warp takes the mean of its own n_w values
// and the squares around that, and the parts join as
//   mean = sum n_w mean_w / D,  M2 = sum (M2_w + n_w (mean_w - mean)^2)
// (Chan, Golub and LeVeque's pairwise formula).
template <bool F32, int C, bool RES>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormParams p, int W) {
  __shared__ float2 part[2][16];
  __shared__ float count[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / W, wr = warp - group * W, groups = (blockDim.x >> 5) / W;
  const int64_t c0 = ((int64_t)wr * 32 + lane) * 8, step = (int64_t)W * 256;
  int n_lane = 0;
#pragma unroll
  for (int c = 0; c < C; c++) n_lane += c0 + c * step < p.D ? 8 : 0;
  const float n_w = warp_sum((float)n_lane), inv_nw = n_w > 0.f ? 1.f / n_w : 0.f, inv_d = 1.f / (float)p.D;
  if (lane == 0) count[warp] = n_w;
  int flip = 0;
  pdl_trigger();
  pdl_wait();
  for (int64_t r = (int64_t)blockIdx.x * groups + group; r < p.R; r += (int64_t)gridDim.x * groups) {
    float v[C][8];
#pragma unroll
    for (int c = 0; c < C; c++) {
      const int64_t at = c0 + c * step;
      if (at < p.D) {
        unpack_raw8<F32>(load_raw8<F32>(p.x, r * p.ld_x + at), v[c]);
        if constexpr (RES) {
          float a[8];
          unpack_raw8<F32>(load_raw8<F32>(p.res, r * p.ld_res + at), a);
#pragma unroll
          for (int i = 0; i < 8; i++) a[i] += v[c][i];
          const Raw8<F32> s = pack_raw8<F32>(a);  // the stream's own rounding: what the norm and its backward pass see
          store_raw8<F32>(p.sum, r * p.ld_sum + at, s);
          unpack_raw8<F32>(s, v[c]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; i++) v[c][i] = 0.f;
      }
    }
    float mean = 0.f;
    if (!p.rms) {
#pragma unroll
      for (int c = 0; c < C; c++)
#pragma unroll
        for (int i = 0; i < 8; i++) mean += v[c][i];
      mean = warp_sum(mean) * inv_nw;
    }
    float m2 = 0.f;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float d = v[c][i] - mean;
        m2 = c0 + c * step < p.D ? fmaf(d, d, m2) : m2;
      }
    m2 = warp_sum(m2);
    if (W > 1) {
      if (lane == 0) part[flip][warp] = make_float2(mean, m2);
      group_bar(group, W);
      const float2* q = &part[flip][group * W];
      float total = 0.f;
      m2 = 0.f;
      const float* n = &count[group * W];
      for (int w = 0; w < W; w++) total = fmaf(q[w].x, n[w], total);
      mean = total * inv_d;
      for (int w = 0; w < W; w++) {
        const float d = q[w].x - mean;
        m2 += fmaf(d * d, n[w], q[w].y);
      }
      flip ^= 1;  // the next row's parts go elsewhere: this row's are still being read
    }
    const float rstd = rsqrtf(fmaf(m2, inv_d, p.eps));
    if (wr == 0 && lane == 0) {
      if (p.mean != nullptr && !p.rms) p.mean[r] = mean;
      if (p.rstd != nullptr) p.rstd[r] = rstd;
    }
#pragma unroll
    for (int c = 0; c < C; c++) {
      const int64_t at = c0 + c * step;
      if (at >= p.D) continue;
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; i++) v[c][i] = (v[c][i] - mean) * rstd;
      if (p.weight != nullptr) {
        load_shared8(p.weight, p.w_f32, at, w);
#pragma unroll
        for (int i = 0; i < 8; i++) v[c][i] *= w[i];
      }
      if (p.bias != nullptr) {
        load_shared8(p.bias, p.w_f32, at, w);
#pragma unroll
        for (int i = 0; i < 8; i++) v[c][i] += w[i];
      }
      store_raw8<false>(p.y, r * p.ld_y + at, pack_raw8<false>(v[c]));
    }
  }
}

// Backward.  With g = dy w and xh = (x - mean) rstd:
//   dx = rstd (g - sum(g) / D - xh sum(g xh) / D) (+ dres),  dw = sum over rows dy xh,  db = sum over rows dy.
// A group takes every `stride`th row; its lanes keep the sums of dw and db of
// their own columns over all of them (in registers; SMEM: in shared memory,
// where a row's values fill the registers).  The block's groups then add theirs
// in order, and a second launch the blocks': no atomics, the same bits each time.
// The next row's loads are issued before this row's sums are exchanged.
template <bool F32, int C, bool DRES, bool WG, bool SMEM>
__global__ void __launch_bounds__(512, 1) norm_bwd_kernel(const NormParams p, int W) {
  extern __shared__ float acc_smem[];
  __shared__ float2 part[2][16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = warp / W, wr = warp - group * W, groups = (blockDim.x >> 5) / W;
  const int64_t c0 = ((int64_t)wr * 32 + lane) * 8, step = (int64_t)W * 256;
  const float inv_d = 1.f / (float)p.D;
  constexpr int A = WG && !SMEM ? C : 1;
  float dw[A][8] = {}, db[A][8] = {};
  if constexpr (WG && SMEM)
#pragma unroll 1
    for (int i = 0; i < 16 * C; i++) acc_smem[i * blockDim.x + tid] = 0.f;
  Raw8<F32> xr[C], sr[C];
  Raw8<false> dr[C];
  float mean = 0.f, rstd = 0.f;
  int flip = 0;
  const int64_t stride = (int64_t)gridDim.x * groups;
  int64_t r = (int64_t)blockIdx.x * groups + group;
  const auto load_row = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < C; c++) {
      const int64_t at = c0 + c * step;
      if (at < p.D) {
        xr[c] = load_raw8<F32>(p.x, row * p.ld_x + at);
        dr[c] = load_raw8<false>(p.dy, row * p.ld_dy + at);
        if constexpr (DRES) sr[c] = load_raw8<F32>(p.res, row * p.ld_res + at);
      }
    }
    if (!p.rms) mean = *(p.mean + row);
    rstd = *(p.rstd + row);
  };
  pdl_trigger();
  pdl_wait();
#pragma unroll
  for (int c = 0; c < C; c++) {  // columns past the row add nothing
    xr[c] = {};
    dr[c] = {};
    sr[c] = {};
  }
  if (r < p.R) load_row(r);
  for (; r < p.R; r += stride) {
    float xh[C][8], g[C][8], s1 = 0.f, s2 = 0.f;
    Raw8<F32> skip[C];
    const float inv = rstd;
#pragma unroll
    for (int c = 0; c < C; c++) {
      const int64_t at = c0 + c * step;
      unpack_raw8<F32>(xr[c], xh[c]);
      unpack_raw8<false>(dr[c], g[c]);
      if constexpr (DRES) skip[c] = sr[c];
      if (at >= p.D) continue;  // x = 0 there, but xh need not be
#pragma unroll
      for (int i = 0; i < 8; i++) {
        xh[c][i] = (xh[c][i] - mean) * rstd;
        if constexpr (WG && !SMEM) {
          dw[c][i] = fmaf(g[c][i], xh[c][i], dw[c][i]);
          db[c][i] += g[c][i];
        }
        if constexpr (WG && SMEM) {
          acc_smem[(c * 8 + i) * blockDim.x + tid] += g[c][i] * xh[c][i];
          acc_smem[((C + c) * 8 + i) * blockDim.x + tid] += g[c][i];
        }
      }
      if (p.weight != nullptr) {
        float w[8];
        load_shared8(p.weight, p.w_f32, at, w);
#pragma unroll
        for (int i = 0; i < 8; i++) g[c][i] *= w[i];
      }
#pragma unroll
      for (int i = 0; i < 8; i++) {
        s1 += g[c][i];
        s2 = fmaf(g[c][i], xh[c][i], s2);
      }
    }
    if (r + stride < p.R) load_row(r + stride);
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (W > 1) {
      if (lane == 0) part[flip][warp] = make_float2(s1, s2);
      group_bar(group, W);
      s1 = s2 = 0.f;
      for (int w = 0; w < W; w++) {
        const float2 q = part[flip][group * W + w];
        s1 += q.x;
        s2 += q.y;
      }
      flip ^= 1;
    }
    s1 = p.rms ? 0.f : s1 * inv_d;
    s2 *= inv_d;
#pragma unroll
    for (int c = 0; c < C; c++) {
      const int64_t at = c0 + c * step;
      if (at >= p.D) continue;
      float d[8] = {};
      if constexpr (DRES) unpack_raw8<F32>(skip[c], d);
#pragma unroll
      for (int i = 0; i < 8; i++) d[i] = fmaf(inv, fmaf(-xh[c][i], s2, g[c][i] - s1), d[i]);
      store_raw8<F32>(p.dx, r * p.ld_dx + at, pack_raw8<F32>(d));
    }
  }
  if constexpr (WG) {
    float* const out = p.partials + (int64_t)blockIdx.x * 2 * p.D;
#pragma unroll 1
    for (int which = 0; which < 2; which++) {
      if (!SMEM && groups > 1) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
          for (int i = 0; i < 8; i++)
            if constexpr (!SMEM) acc_smem[(c * 8 + i) * blockDim.x + tid] = which ? db[c][i] : dw[c][i];
        __syncthreads();
      }
      if (group != 0) continue;
#pragma unroll
      for (int c = 0; c < C; c++) {
        const int64_t at = c0 + c * step;
        if (at >= p.D) continue;
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
          if constexpr (SMEM) t[i] = acc_smem[((which * C + c) * 8 + i) * blockDim.x + tid];
          else t[i] = which ? db[c][i] : dw[c][i];
          for (int k = 1; k < groups; k++) t[i] += acc_smem[(c * 8 + i) * blockDim.x + k * W * 32 + tid];
        }
        store_raw8<true>(out, which * p.D + at, pack_raw8<true>(t));
      }
    }
  }
}

// The blocks' sums added in order, to what the gradients hold if `accumulate`: a
// block takes 32 columns of [dw | db], its 8 warps every eighth block.
__global__ void __launch_bounds__(256) norm_wgrad_kernel(const NormParams p, int64_t blocks) {
  __shared__ float s[8][32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t j = (int64_t)blockIdx.x * 32 + lane;
  float t = 0.f;
  pdl_trigger();
  pdl_wait();
  if (j < 2 * p.D) {
#pragma unroll 4
    for (int64_t b = w; b < blocks; b += 8) t += p.partials[b * 2 * p.D + j];
  }
  s[w][lane] = t;
  __syncthreads();
  if (w == 0 && j < 2 * p.D) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) a += s[i][lane];
    float* const out = j < p.D ? p.dweight : p.dbias;
    const int64_t c = j < p.D ? j : j - p.D;
    if (out != nullptr) out[c] = p.accumulate ? out[c] + a : a;
  }
}

// Warps of a row and 8-column pieces of a lane.  Forward: up to four pieces a
// lane; backward: one as long as 16 warps cover the row.
struct NormShape { int W, C; };
static NormShape norm_shape(int64_t D, int most) {
  const int64_t v = (D + 7) / 8;
  int W = 1;
  while ((int64_t)W * 32 * most < v && W < 16) W *= 2;
  return {W, (int)((v + 32 * W - 1) / (32 * W))};
}
static NormShape bwd_shape(int64_t D) {
  const NormShape s = norm_shape(D, 1);
  return {s.W, s.C > 2 ? 4 : s.C};
}

template <bool F32, bool RES>
static cudaError_t launch_fwd(const NormParams& p, int sms, cudaStream_t s) {
  const NormShape n = norm_shape(p.D, 4);
  const int threads = n.W * 32 > 256 ? n.W * 32 : 256, groups = threads / (32 * n.W);
  const int64_t want = (p.R + groups - 1) / groups, cap = (int64_t)sms * 16;
  const dim3 grid((unsigned)(want < cap ? want : cap));
  switch (n.C) {
    case 1: return launch_pdl(norm_fwd_kernel<F32, 1, RES>, grid, threads, 0, s, dim3(1), p, n.W);
    case 2: return launch_pdl(norm_fwd_kernel<F32, 2, RES>, grid, threads, 0, s, dim3(1), p, n.W);
    case 3: return launch_pdl(norm_fwd_kernel<F32, 3, RES>, grid, threads, 0, s, dim3(1), p, n.W);
    default: return launch_pdl(norm_fwd_kernel<F32, 4, RES>, grid, threads, 0, s, dim3(1), p, n.W);
  }
}

cudaError_t launch_norm_fwd(const NormParams& p, int sms, cudaStream_t s) {
  if (p.x_f32) return p.res ? launch_fwd<true, true>(p, sms, s) : launch_fwd<true, false>(p, sms, s);
  return p.res ? launch_fwd<false, true>(p, sms, s) : launch_fwd<false, false>(p, sms, s);
}

int64_t norm_bwd_blocks(int64_t R, int64_t D) {
  const int groups = 16 / bwd_shape(D).W;
  const int64_t want = (R + groups - 1) / groups;
  return want < 152 ? want : 152;  // one on every SM (GB300: 152)
}

template <bool F32, int C, bool DRES, bool WG>
static cudaError_t launch_bwd(const NormParams& p, int W, cudaStream_t s) {
  constexpr bool SMEM = WG && C == 4;
  const int64_t blocks = norm_bwd_blocks(p.R, p.D);
  const int smem = !WG ? 0 : (SMEM ? 2 : 1) * C * 8 * 512 * 4;
  const cudaError_t e = smem > 48 * 1024 ? ensure_smem_attr<norm_bwd_kernel<F32, C, DRES, WG, SMEM>>(smem) : cudaSuccess;
  if (e != cudaSuccess) return e;
  const cudaError_t l = launch_pdl(norm_bwd_kernel<F32, C, DRES, WG, SMEM>, dim3((unsigned)blocks), 512, smem, s, dim3(1), p, W);
  if (l != cudaSuccess || !WG) return l;
  return launch_pdl(norm_wgrad_kernel, dim3((unsigned)((2 * p.D + 31) / 32)), 256, 0, s, dim3(1), p, blocks);
}

template <bool F32, bool DRES, bool WG>
static cudaError_t launch_bwd_c(const NormParams& p, cudaStream_t s) {
  const NormShape n = bwd_shape(p.D);
  switch (n.C) {
    case 1: return launch_bwd<F32, 1, DRES, WG>(p, n.W, s);
    case 2: return launch_bwd<F32, 2, DRES, WG>(p, n.W, s);
    default: return launch_bwd<F32, 4, DRES, WG>(p, n.W, s);
  }
}

cudaError_t launch_norm_bwd(const NormParams& p, cudaStream_t s) {
  const bool wg = p.dweight != nullptr || p.dbias != nullptr;
  if (p.x_f32) {
    if (p.res) return wg ? launch_bwd_c<true, true, true>(p, s) : launch_bwd_c<true, true, false>(p, s);
    return wg ? launch_bwd_c<true, false, true>(p, s) : launch_bwd_c<true, false, false>(p, s);
  }
  if (p.res) return wg ? launch_bwd_c<false, true, true>(p, s) : launch_bwd_c<false, true, false>(p, s);
  return wg ? launch_bwd_c<false, false, true>(p, s) : launch_bwd_c<false, false, false>(p, s);
}

}  // namespace mx
