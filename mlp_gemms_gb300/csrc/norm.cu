// Layer norm (and its form without a mean): forward with the residual added in
// the same pass, and the backward pass with the weight's and the bias's
// gradients.
#include "mx_internal.h"
#include "pair_common.cuh"
#include "vec8.cuh"

namespace mx {

// Both kernels are bound by memory: every value is read once and written once.
// A row is held in the registers of `W` warps, 8 C columns a lane, so that its
// statistics, its centred squares and its result need no second read; a block's warps
// form groups of W, each with a row of its own.

// A vector [8 n8] of all rows in shared memory, as fp32: the first four values of
// each lane's eight, then the last four, so that neighbouring lanes read
// neighbouring 16 bytes.
__device__ __forceinline__ void keep_vector(const void* p, bool f32, int n8, float4* to) {
  if (p == nullptr) return;
  for (int i = threadIdx.x; i < n8; i += blockDim.x) {
    float v[8];
    load_shared8(p, f32, (int64_t)i * 8, v);
    to[i] = make_float4(v[0], v[1], v[2], v[3]);
    to[n8 + i] = make_float4(v[4], v[5], v[6], v[7]);
  }
}
__device__ __forceinline__ void kept_pairs(const float4* kept, int n8, int i, uint64_t (&v)[4]) {
  const float4 a = kept[i], b = kept[n8 + i];
  v[0] = pack2(a.x, a.y);
  v[1] = pack2(a.z, a.w);
  v[2] = pack2(b.x, b.y);
  v[3] = pack2(b.z, b.w);
}

// The group's barrier: its W warps, W > 1.
__device__ __forceinline__ void group_bar(int group, int W) { named_bar(1 + group, 32 * W); }

// Forward.  Mean and centred sum of squares without cancellation, with one
// exchange between the warps: each warp takes the mean of its own n_w values
// and the squares around that, and the parts join as
//   mean = sum n_w mean_w / D,  M2 = sum (M2_w + n_w (mean_w - mean)^2)
// (Chan, Golub and LeVeque's pairwise formula).
// Weight and bias wait in shared memory, as fp32, and the next row's loads are
// issued before this row's sums are exchanged.  FULL: the group's columns are the
// row's, with no lane past its end.
template <bool F32, int C, bool RES, bool FULL>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormParams p, int W) {
  extern __shared__ float4 vectors[];
  __shared__ float2 part[2][16];
  __shared__ float count[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / W, wr = warp - group * W, groups = (blockDim.x >> 5) / W;
  const int D = (int)p.D, c0 = (wr * 32 + lane) * 8, step = W * 256;
  const auto in = [&](int c) { return FULL || c0 + c * step < D; };
  int n_lane = 0;
#pragma unroll
  for (int c = 0; c < C; c++) n_lane += in(c) ? 8 : 0;
  const float n_w = FULL ? (float)(C * 256) : warp_sum((float)n_lane);
  const float inv_nw = n_w > 0.f ? 1.f / n_w : 0.f, inv_d = 1.f / (float)D;
  if (lane == 0) count[warp] = n_w;
  int flip = 0;
  Raw8<F32> next[C], next_res[RES ? C : 1];
  const auto load_row = [&](int64_t r) {
#pragma unroll
    for (int c = 0; c < C; c++) {
      if (!FULL) next[c] = {};
      if (!in(c)) continue;
      next[c] = load_raw8<F32>(p.x, r * p.ld_x + c0 + c * step);
      if constexpr (RES) next_res[c] = load_raw8<F32>(p.res, r * p.ld_res + c0 + c * step);
    }
  };
  const int64_t stride = (int64_t)gridDim.x * groups;
  int64_t r = (int64_t)blockIdx.x * groups + group;
  pdl_trigger();
  pdl_wait();
  if (r < p.R) load_row(r);
  const int n8 = D >> 3;
  keep_vector(p.weight, p.w_f32, n8, vectors);
  keep_vector(p.bias, p.w_f32, n8, vectors + 2 * n8);
  __syncthreads();
  for (; r < p.R; r += stride) {
    uint64_t v[C][4], total[4] = {}, squares[4] = {};  // four sums each: short chains
#pragma unroll
    for (int c = 0; c < C; c++) {
      unpack_pairs<F32>(next[c], v[c]);
      if constexpr (RES) {
        if (in(c)) {
          uint64_t a[4];
          unpack_pairs<F32>(next_res[c], a);
#pragma unroll
          for (int i = 0; i < 4; i++) a[i] = add2(a[i], v[c][i]);
          const Raw8<F32> s = pack_pairs<F32>(a);  // the stream's own rounding: what the norm and its backward pass see
          store_raw8<F32>(p.sum, r * p.ld_sum + c0 + c * step, s);
          unpack_pairs<F32>(s, v[c]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; i++) total[i] = add2(total[i], v[c][i]);
    }
    if (r + stride < p.R) load_row(r + stride);
    float mean = p.rms ? 0.f : warp_sum(sum_pairs(total)) * inv_nw;
#pragma unroll
    for (int c = 0; c < C; c++) {
      if (!in(c)) continue;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const uint64_t d = add2(v[c][i], both(-mean));
        squares[i] = fma2(d, d, squares[i]);
      }
    }
    float m2 = warp_sum(sum_pairs(squares));
    if (W > 1) {
      if (lane == 0) part[flip][warp] = make_float2(mean, m2);
      group_bar(group, W);
      const float2* q = &part[flip][group * W];
      const float* n = &count[group * W];
      float sum = 0.f;
      m2 = 0.f;
      for (int w = 0; w < W; w++) sum = fmaf(q[w].x, n[w], sum);
      mean = sum * inv_d;
      for (int w = 0; w < W; w++) {
        const float d = q[w].x - mean;
        m2 += fmaf(d * d, n[w], q[w].y);
      }
      flip ^= 1;  // the next row's parts go elsewhere: this row's are still being read
    }
    // Squares past fp32's range (an Inf in the row among them) are no statistics: NaN for
    // the whole row, where rsqrt(Inf) = 0 would pass for values of 0.
    const float rstd = m2 <= 3.4028235e38f ? rsqrtf(fmaf(m2, inv_d, p.eps)) : __uint_as_float(0x7FC00000u);
    if (wr == 0 && lane == 0) {
      if (p.mean != nullptr && !p.rms) p.mean[r] = mean;
      if (p.rstd != nullptr) p.rstd[r] = rstd;
    }
#pragma unroll
    for (int c = 0; c < C; c++) {
      if (!in(c)) continue;
      const int at = (c0 + c * step) >> 3;
#pragma unroll
      for (int i = 0; i < 4; i++) v[c][i] = mul2(add2(v[c][i], both(-mean)), both(rstd));
      uint64_t w[4];
      if (p.weight != nullptr) {
        kept_pairs(vectors, n8, at, w);
#pragma unroll
        for (int i = 0; i < 4; i++) v[c][i] = mul2(v[c][i], w[i]);
      }
      if (p.bias != nullptr) {
        kept_pairs(vectors + 2 * n8, n8, at, w);
#pragma unroll
        for (int i = 0; i < 4; i++) v[c][i] = add2(v[c][i], w[i]);
      }
      store_raw8<false>(p.y, r * p.ld_y + c0 + c * step, pack_pairs<false>(v[c]));
    }
  }
}

// Backward.  With g = dy w and xh = (x - mean) rstd:
//   dx = rstd (g - sum(g) / D - xh sum(g xh) / D) (+ dres),  dw = sum over rows dy xh,  db = sum over rows dy.
// A group takes every `stride`th row; its lanes keep the sums of dw and db of
// their own columns over all of them in registers.  The block's groups then add
// theirs in order, and a second launch the blocks': no atomics, the same bits each
// time.  The next one or two rows are on their way into shared memory: with one
// row ahead in registers, the sums left room for 32 KB of loads in flight an SM
// ([65536, 2048] BF16 152 us, 137 this way; [32768, 4096] fp32 with dres 310, 279 =
// 99 % of the copy rate; [16384, 8192] fp32 489, 275).
// PAIR: more than 8192 columns, half of them in each block of a cluster of two,
// which exchange their halves of a row's two sums ([10217, 13136] BF16 with dres in one
// block with the sums of dw and db in shared memory 638 us, 347 this way; [8192, 16384]
// without 219 and 264: two exchanges a row, 2.4 us).
__host__ __device__ constexpr int bwd_half(int D) { return ((D >> 3) + 1) / 2 * 8; }
constexpr int bwd_stages(bool f32, int C, bool res) {
  return ((f32 ? 32 : 16) * (res ? 2 : 1) + 16) * C * 512 * 3 <= 150 * 1024 ? 3 : 2;
}
template <bool F32, int C, bool DRES, bool WG, bool FULL, bool PAIR>
__global__ void __launch_bounds__(512, 1) norm_bwd_kernel(NormParams p, int W) {
  extern __shared__ float4 vectors[];  // the weight, the ring, the groups' sums
  __shared__ float2 part[2][16];
  __shared__ float2 other[2];  // PAIR: the other block's half of a row's sums
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = warp / W, wr = warp - group * W, groups = (blockDim.x >> 5) / W;
  const int c0 = (wr * 32 + lane) * 8, step = W * 256;
  const float inv_d = 1.f / (float)p.D;
  int D = (int)p.D, first = 0;  // this block's columns
  const uint32_t rank = PAIR ? cluster_rank() : 0;
  if constexpr (PAIR) {
    const int half = bwd_half(D);
    first = rank ? half : 0;
    D = rank ? D - half : half;
    p.x = static_cast<const char*>(p.x) + first * (F32 ? 4 : 2);
    p.dx = static_cast<char*>(p.dx) + first * (F32 ? 4 : 2);
    if (DRES) p.res = static_cast<const char*>(p.res) + first * (F32 ? 4 : 2);
    p.dy += first;
    if (p.weight != nullptr) p.weight = static_cast<const char*>(p.weight) + first * (p.w_f32 ? 4 : 2);
  }
  const int n8 = D >> 3;
  constexpr int S = bwd_stages(F32, C, DRES), Q = F32 ? 2 : 1;
  uint4* const ring = reinterpret_cast<uint4*>(vectors + 2 * n8) + threadIdx.x;
  const int stage_size = ((DRES ? 2 : 1) * Q + 1) * C * blockDim.x;
  float* const acc_smem = reinterpret_cast<float*>(vectors + 2 * n8 + S * stage_size);
  const auto in = [&](int c) { return FULL || c0 + c * step < D; };
  constexpr int A = WG ? C : 1;
  uint64_t dw[A][4] = {}, db[A][4] = {};
  float means[S - 1] = {}, rstds[S - 1] = {};  // of the rows ahead
  int flip = 0, stage = 0;
  const int64_t stride = (int64_t)(PAIR ? gridDim.x / 2 : gridDim.x) * groups;
  int64_t r = (int64_t)(PAIR ? blockIdx.x / 2 : blockIdx.x) * groups + group;
  // pieces of a stage: dy's, then x's, then dres's
  const auto slot = [&](int st, int c, int which) {
    return ring + st * stage_size + (which == 0 ? c : C + ((which - 1) * C + c) * Q) * blockDim.x;
  };
  // An fp32 piece is 1024 bytes of a warp, copied 512 at a time (32 bytes a lane
  // would take half of each sector with either copy) and read by other lanes.
  const auto copy_x = [&](int st, int c, int which, const void* base, int64_t row_at) {
    if constexpr (F32) {
      const int64_t at = row_at + (c0 - lane * 8) + c * step;  // the warp's first column
      uint4* const to = slot(st, c, which) - tid + warp * 64;
#pragma unroll
      for (int h = 0; h < 2; h++)
        if (FULL || (c0 - lane * 8) + c * step + h * 128 + lane * 4 < D)
          copy_ahead16(to + h * 32 + lane, static_cast<const float*>(base) + at + h * 128 + lane * 4);
    } else {
      copy_ahead16(slot(st, c, which), static_cast<const uint16_t*>(base) + row_at + c0 + c * step);
    }
  };
  const auto take_x = [&](int st, int c, int which) {
    Raw8<F32> v;
    const uint4* const from = F32 ? slot(st, c, which) - tid + warp * 64 + lane * 2 : slot(st, c, which);
    v.q[0] = from[0];
    if constexpr (F32) v.q[1] = from[1];
    return v;
  };
  const auto load_row = [&](int64_t row, int st, float* m, float* s) {
    if (row < p.R) {
#pragma unroll
      for (int c = 0; c < C; c++) {
        if (F32 || in(c)) {
          copy_x(st, c, 1, p.x, row * p.ld_x);
          if constexpr (DRES) copy_x(st, c, 2, p.res, row * p.ld_res);
        }
        if (in(c)) copy_ahead16(slot(st, c, 0), p.dy + row * p.ld_dy + c0 + c * step);
      }
      if (!p.rms) *m = *(p.mean + row);
      *s = *(p.rstd + row);
    }
    commit_ahead();
  };
  pdl_trigger();
  pdl_wait();
#pragma unroll
  for (int i = 0; i < S - 1; i++) load_row(r + i * stride, i, &means[i], &rstds[i]);
  keep_vector(p.weight, p.w_f32, n8, vectors);
  if constexpr (PAIR) cluster_sync_all();  // the other block runs: its memory may be stored to
  else __syncthreads();
  for (; r < p.R; r += stride) {
    uint64_t xh[C][4], g[C][4], t1[4] = {}, t2[4] = {};
    const float mean = means[0], rstd = rstds[0];
    wait_ahead<S - 2>();
    if constexpr (F32) __syncwarp();
#pragma unroll
    for (int c = 0; c < C; c++) {
      if (!in(c)) continue;
      Raw8<false> d;
      d.q[0] = *slot(stage, c, 0);
      unpack_pairs<F32>(take_x(stage, c, 1), xh[c]);
      unpack_pairs<false>(d, g[c]);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        xh[c][i] = mul2(add2(xh[c][i], both(-mean)), both(rstd));
        if constexpr (WG) {
          dw[c][i] = fma2(g[c][i], xh[c][i], dw[c][i]);
          db[c][i] = add2(db[c][i], g[c][i]);
        }
      }
      if (p.weight != nullptr) {
        uint64_t w[4];
        kept_pairs(vectors, n8, (c0 + c * step) >> 3, w);
#pragma unroll
        for (int i = 0; i < 4; i++) g[c][i] = mul2(g[c][i], w[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; i++) {
        t1[i] = add2(t1[i], g[c][i]);
        t2[i] = fma2(g[c][i], xh[c][i], t2[i]);
      }
    }
#pragma unroll
    for (int i = 0; i + 2 < S; i++) {
      means[i] = means[i + 1];
      rstds[i] = rstds[i + 1];
    }
    if constexpr (F32) __syncwarp();  // the row before, whose place is copied over, has been read by all lanes
    load_row(r + (S - 1) * stride, stage == 0 ? S - 1 : stage - 1, &means[S - 2], &rstds[S - 2]);
    float s1 = warp_sum(sum_pairs(t1)), s2 = warp_sum(sum_pairs(t2));
    if (W > 1) {
      if (lane == 0) part[flip][warp] = make_float2(s1, s2);
      group_bar(group, W);
      s1 = s2 = 0.f;
      for (int w = 0; w < W; w++) {
        const float2 q = part[flip][group * W + w];
        s1 += q.x;
        s2 += q.y;
      }
      if constexpr (PAIR) {  // both halves, the first block's first
        if (tid == 0) {
          const uint32_t to = rank ? leader_addr(&other[flip]) : peer_addr(&other[flip]);
          st_cluster_u32(to, __float_as_uint(s1));
          st_cluster_u32(to + 4, __float_as_uint(s2));
        }
        __syncwarp();
        cluster_sync_all();
        const float2 o = other[flip];
        s1 = rank ? o.x + s1 : s1 + o.x;
        s2 = rank ? o.y + s2 : s2 + o.y;
      }
      flip ^= 1;
    }
    s1 = p.rms ? 0.f : s1 * inv_d;
    s2 *= inv_d;
#pragma unroll
    for (int c = 0; c < C; c++) {
      if (!in(c)) continue;
      uint64_t d[4] = {};
      if constexpr (DRES) unpack_pairs<F32>(take_x(stage, c, 2), d);
#pragma unroll
      for (int i = 0; i < 4; i++)
        d[i] = fma2(both(rstd), fma2(xh[c][i], both(-s2), add2(g[c][i], both(-s1))), d[i]);
      store_raw8<F32>(p.dx, r * p.ld_dx + c0 + c * step, pack_pairs<F32>(d));
    }
    stage = stage == S - 1 ? 0 : stage + 1;
  }
  if constexpr (WG) {
    float* const out = p.partials + (int64_t)(PAIR ? blockIdx.x / 2 : blockIdx.x) * 2 * p.D + first;
#pragma unroll
    for (int which = 0; which < 2; which++) {
      if (groups > 1) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            float a, b;
            unpack2(which ? db[c][i] : dw[c][i], &a, &b);
            acc_smem[(c * 8 + 2 * i) * blockDim.x + tid] = a;
            acc_smem[(c * 8 + 2 * i + 1) * blockDim.x + tid] = b;
          }
        __syncthreads();
      }
      if (group != 0) continue;
#pragma unroll
      for (int c = 0; c < C; c++) {
        if (!in(c)) continue;
        float t[8];
#pragma unroll
        for (int i = 0; i < 4; i++) unpack2(which ? db[c][i] : dw[c][i], &t[2 * i], &t[2 * i + 1]);
#pragma unroll
        for (int i = 0; i < 8; i++)
          for (int k = 1; k < groups; k++) t[i] += acc_smem[(c * 8 + i) * blockDim.x + k * W * 32 + tid];
        store_raw8<true>(out, which * p.D + c0 + c * step, pack_raw8<true>(t));
      }
    }
  }
}

// The blocks' sums added in order, to what the gradients hold if `accumulate`: a
// block takes 32 columns of [dw | db], its 16 warps every 16th block each, all of
// them in flight at a time.
__global__ void __launch_bounds__(512) norm_wgrad_kernel(const NormParams p, int64_t blocks) {
  __shared__ float s[16][32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t j = (int64_t)blockIdx.x * 32 + lane;
  float t = 0.f;
  pdl_trigger();
  pdl_wait();
  if (j < 2 * p.D) {
#pragma unroll 10
    for (int64_t b = w; b < blocks; b += 16) t += p.partials[b * 2 * p.D + j];
  }
  s[w][lane] = t;
  __syncthreads();
  if (w == 0 && j < 2 * p.D) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i++) a += s[i][lane];
    float* const out = j < p.D ? p.dweight : p.dbias;
    const int64_t c = j < p.D ? j : j - p.D;
    if (out != nullptr) out[c] = p.accumulate ? out[c] + a : a;
  }
}

// Warps of a row and 8-column pieces of a lane: `most` pieces where the row is
// long enough, and a number of warps whose columns are the row's where there is one
// (warps need not be a power of two: 5120 columns are 5 x 4 pieces of 256, 7168 7 x
// 4).
constexpr int SMEM_MOST = 226 * 1024;  // dynamic, beside the kernels' own few hundred bytes
struct NormShape {
  int W, C;
  bool full;
};
static NormShape norm_shape(int64_t D, int most) {
  const int v = (int)((D + 7) / 8), least = (v + 32 * most - 1) / (32 * most);
  for (int W = least; W <= 16 && W <= least + 2; W++)
    if (D % 8 == 0 && v % (32 * W) == 0) return {W, v / (32 * W), true};
  return {least, (v + 32 * least - 1) / (32 * least), false};
}
static int norm_groups(int W, int warps) { return W >= warps ? 1 : warps / W; }

template <bool F32, bool RES, bool FULL, int C>
static cudaError_t launch_fwd(const NormParams& p, int W, dim3 grid, int threads, cudaStream_t s) {
  const int smem = (p.weight || p.bias ? 8 : 0) * (int)p.D;
  if (smem > 32 * 1024) {
    const cudaError_t e = ensure_smem_attr<norm_fwd_kernel<F32, C, RES, FULL>>(8 * (int)MAX_NORM_D);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(norm_fwd_kernel<F32, C, RES, FULL>, grid, threads, smem, s, dim3(1), p, W);
}
template <bool F32, bool RES, bool FULL>
static cudaError_t launch_fwd(const NormParams& p, const NormShape& n, int sms, cudaStream_t s) {
  const int groups = norm_groups(n.W, 8), threads = 32 * n.W * groups;
  const int64_t want = (p.R + groups - 1) / groups, cap = (int64_t)sms * ((n.C == 1 ? 1024 : 512) / threads);
  const dim3 grid((unsigned)(want < cap ? want : cap));
  switch (n.C) {
    case 1: return launch_fwd<F32, RES, FULL, 1>(p, n.W, grid, threads, s);
    case 2: return launch_fwd<F32, RES, FULL, 2>(p, n.W, grid, threads, s);
    case 3: return launch_fwd<F32, RES, FULL, 3>(p, n.W, grid, threads, s);
    default: return launch_fwd<F32, RES, FULL, 4>(p, n.W, grid, threads, s);
  }
}
template <bool F32, bool RES>
static cudaError_t launch_fwd(const NormParams& p, int sms, cudaStream_t s) {
  const NormShape n = norm_shape(p.D, F32 && RES && p.D <= 8192 ? 2 : 4);
  return n.full ? launch_fwd<F32, RES, true>(p, n, sms, s) : launch_fwd<F32, RES, false>(p, n, sms, s);
}

cudaError_t launch_norm_fwd(const NormParams& p, int sms, cudaStream_t s) {
  if (p.x_f32) return p.res ? launch_fwd<true, true>(p, sms, s) : launch_fwd<true, false>(p, sms, s);
  return p.res ? launch_fwd<false, true>(p, sms, s) : launch_fwd<false, false>(p, sms, s);
}

// Fewer warps a row, with more columns a lane, exchange less (us, one row ahead in
// registers: [65536, 2048] BF16 with two pieces a lane 152, with one 193; [20000,
// 2728] 89 and 120).  fp32 rows, twice as long in bytes, take two where one does not
// cover them.
struct BwdShape {
  NormShape n;  // of a block's columns
  bool pair;
};
static BwdShape bwd_shape(int64_t D, bool f32) {
  if (D > 8192) {
    const int64_t half = bwd_half((int)D);
    NormShape n = norm_shape(half, 2);
    n.full = n.full && 2 * half == D;
    return {n, true};
  }
  return {norm_shape(D, f32 && D <= 4096 ? 1 : 2), false};
}
int64_t norm_bwd_blocks(int64_t R, int64_t D, bool f32) {
  const BwdShape b = bwd_shape(D, f32);
  const int groups = norm_groups(b.n.W, 16), most = b.pair ? 76 : 152;  // a block on every SM (GB300: 152)
  const int64_t want = (R + groups - 1) / groups;
  return want < most ? want : most;
}

template <bool F32, int C, bool DRES, bool WG, bool FULL, bool PAIR>
static cudaError_t launch_bwd(const NormParams& p, int W, cudaStream_t s) {
  const int64_t blocks = norm_bwd_blocks(p.R, p.D, F32);  // PAIR: pairs
  const int threads = 32 * W * norm_groups(W, 16), D = PAIR ? bwd_half((int)p.D) : (int)p.D;
  constexpr int RING = bwd_stages(F32, C, DRES) * ((F32 ? 32 : 16) * (DRES ? 2 : 1) + 16) * C;  // bytes a thread
  const int smem = 4 * D + RING * threads + (WG ? C * 8 * threads * 4 : 0);
  const cudaError_t e =
      smem > 32 * 1024 ? ensure_smem_attr<norm_bwd_kernel<F32, C, DRES, WG, FULL, PAIR>>(SMEM_MOST) : cudaSuccess;
  if (e != cudaSuccess) return e;
  const cudaError_t l = launch_pdl(norm_bwd_kernel<F32, C, DRES, WG, FULL, PAIR>, dim3((unsigned)blocks * (PAIR ? 2 : 1)),
                                   threads, smem, s, dim3(PAIR ? 2 : 1), p, W);
  if (l != cudaSuccess || !WG) return l;
  return launch_pdl(norm_wgrad_kernel, dim3((unsigned)((2 * p.D + 31) / 32)), 512, 0, s, dim3(1), p, blocks);
}

template <bool F32, bool DRES, bool WG, bool FULL>
static cudaError_t launch_bwd_c(const NormParams& p, const BwdShape& b, cudaStream_t s) {
  if (b.pair) return launch_bwd<F32, 2, DRES, WG, FULL, true>(p, b.n.W, s);  // half of more than 8192: two pieces
  return b.n.C == 1 ? launch_bwd<F32, 1, DRES, WG, FULL, false>(p, b.n.W, s)
                    : launch_bwd<F32, 2, DRES, WG, FULL, false>(p, b.n.W, s);
}
template <bool F32, bool DRES, bool WG>
static cudaError_t launch_bwd_f(const NormParams& p, cudaStream_t s) {
  const BwdShape b = bwd_shape(p.D, F32);
  return b.n.full ? launch_bwd_c<F32, DRES, WG, true>(p, b, s) : launch_bwd_c<F32, DRES, WG, false>(p, b, s);
}

cudaError_t launch_norm_bwd(const NormParams& p, cudaStream_t s) {
  const bool wg = p.dweight != nullptr || p.dbias != nullptr;
  if (p.x_f32) {
    if (p.res) return wg ? launch_bwd_f<true, true, true>(p, s) : launch_bwd_f<true, true, false>(p, s);
    return wg ? launch_bwd_f<true, false, true>(p, s) : launch_bwd_f<true, false, false>(p, s);
  }
  if (p.res) return wg ? launch_bwd_f<false, true, true>(p, s) : launch_bwd_f<false, true, false>(p, s);
  return wg ? launch_bwd_f<false, false, true>(p, s) : launch_bwd_f<false, false, false>(p, s);
}

}  // namespace mx
