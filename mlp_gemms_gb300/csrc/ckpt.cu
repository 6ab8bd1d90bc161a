// 8-bit activation checkpoints: the activation with an E4M3 / E8M0 copy of
// its input, and the backward pass that reads the copy.
#include "act.cuh"
#include "mx_internal.h"
#include "pair_common.cuh"

namespace mx {

// Both kernels are bound by memory.  The backward pass gives a lane 8 columns
// (16 bytes of BF16, 8 of payload) of a row, so every access of a warp covers
// one contiguous piece of a row, and a block 256 columns (SWIGLU: of each
// half) and a run of rows, each warp every eighth of them: the column sums
// stay in registers.
constexpr int COLS = 256, WARPS = 8;

__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    v[2 * i] = bf16_bits_to_float(w[i] & 0xFFFFu);
    v[2 * i + 1] = bf16_bits_to_float(w[i] >> 16);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(float2_to_bf16x2(v[0], v[1]), float2_to_bf16x2(v[2], v[3]), float2_to_bf16x2(v[4], v[5]),
                    float2_to_bf16x2(v[6], v[7]));
}
// Streaming loads: nothing here is read twice.
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 q;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "l"(p));
  return q;
}
__device__ __forceinline__ uint2 load_once8(const void* p) {
  uint2 q;
  asm("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(q.x), "=r"(q.y) : "l"(p));
  return q;
}

// Two E4M3 codes -> two fp32 values, exact.
__device__ __forceinline__ void e4m3x2_to_f32(uint32_t two, float* lo, float* hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(*lo), "=f"(*hi) : "r"(h));
}
// The scale byte's power of two (0xFF: NaN).
__device__ __forceinline__ float scale_from_byte(uint32_t b) {
  return b == 0xFFu ? __uint_as_float(0x7FC00000u) : (b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23));
}
__device__ __forceinline__ void read8(const uint2& w, uint32_t b, float (&v)[8]) {
  e4m3x2_to_f32(w.x & 0xFFFFu, &v[0], &v[1]);
  e4m3x2_to_f32(w.x >> 16, &v[2], &v[3]);
  e4m3x2_to_f32(w.y & 0xFFFFu, &v[4], &v[5]);
  e4m3x2_to_f32(w.y >> 16, &v[6], &v[7]);
  scale_values<8>(v, scale_from_byte(b));
}

// Rows a warp has in flight at a time: its loads are issued before the first
// of them is used.
constexpr int BATCH = 4;

// Zero the scale layout's padding (rows R .. 128 * ceil(R / 128), column
// blocks C / 32 .. 4 * ceil(C / 128)), by one block.
__device__ __forceinline__ void zero_scale_padding(const CkptParams& p) {
  const int64_t sc = p.C >> 5, chunks = (sc + 3) / 4, top = (p.R + 127) / 128 * 128;
  for (int64_t i = threadIdx.x; i < (top - p.R) * chunks; i += blockDim.x)
    *reinterpret_cast<uint32_t*>(p.q_scale + blocked_offset(p.R + i / chunks, i % chunks * 4, sc)) = 0u;
}

// 32 BF16 columns of a row in one thread (four 16-byte accesses; the warp's
// four accesses cover 2 KB of consecutive lines between them).
__device__ __forceinline__ void load32(const uint16_t* p, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
      v[8 * i + 2 * j] = bf16_bits_to_float(w[j] & 0xFFFFu);
      v[8 * i + 2 * j + 1] = bf16_bits_to_float(w[j] >> 16);
    }
  }
}
__device__ __forceinline__ void store32(uint16_t* p, const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; i++)
    reinterpret_cast<uint4*>(p)[i] =
        make_uint4(float2_to_bf16x2(v[8 * i], v[8 * i + 1]), float2_to_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                   float2_to_bf16x2(v[8 * i + 4], v[8 * i + 5]), float2_to_bf16x2(v[8 * i + 6], v[8 * i + 7]));
}
__device__ __forceinline__ void save32(const CkptParams& p, int64_t r, int c, float (&v)[32]) {
  const uint32_t b = rceil_scale_byte_sel<E4M3>(amax_abs_bits<32>(v));
  uint32_t w[8];
  quantize_block_words<E4M3>(v, b, w);
  uint4* d = reinterpret_cast<uint4*>(p.q + r * p.C + c);
  d[0] = make_uint4(w[0], w[1], w[2], w[3]);
  d[1] = make_uint4(w[4], w[5], w[6], w[7]);
  p.q_scale[blocked_offset(r, c >> 5, p.C >> 5)] = (uint8_t)b;
}

// Forward: a thread owns one 32-column block of a row (SWIGLU: the gate's and
// the up half's), so the block's amax needs no exchange.  Measured against
// the backward kernel's mapping (8 columns a lane, four lanes a block,
// amax by shuffles): 69 against 96 us on [65536, 1536] SWIGLU, 5.8 TB/s; the
// exchange and its address arithmetic cost more issue slots than the
// coalescing saves.
template <int ACT>
__global__ void __launch_bounds__(256) ckpt_fwd_kernel(const CkptParams p, uint32_t per) {
  constexpr bool GLU = ACT == MX_ACT_SWIGLU;
  const int64_t F = GLU ? p.C / 2 : p.C;
  pdl_trigger();
  pdl_wait();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.R * per; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i < (1ll << 32) ? (uint32_t)i / per : i / per;
    const int c = (int)(i - r * per) * 32;
    float z[32], h[32];
    load32(p.z + r * p.ld_z + c, z);
    if constexpr (GLU) {
      float u[32];
      load32(p.z + r * p.ld_z + F + c, u);
#pragma unroll
      for (int j = 0; j < 32; j++) h[j] = act_f32<MX_ACT_SILU>(z[j]) * u[j];
      save32(p, r, (int)F + c, u);
    } else {
#pragma unroll
      for (int j = 0; j < 32; j++) h[j] = act_f32<ACT>(z[j]);
    }
    store32(p.h + r * p.ld_h + c, h);
    save32(p, r, c, z);
    if (c == 0)  // column padding behind the last block
      for (int64_t sc = p.C >> 5, k = sc; k & 3; k++) p.q_scale[blocked_offset(r, k, sc)] = 0;
  }
  if (blockIdx.x == 0) zero_scale_padding(p);
}

// Row blocks of the backward pass: one wave of two blocks on every SM (GB300:
// 152) where the columns alone do not give it, each with a row for each of its
// warps.  col_blocks counts SWIGLU's columns twice: its blocks do two halves'
// work.
static int64_t ckpt_row_blocks(int64_t R, int64_t C) {
  const int64_t col_blocks = (C + COLS - 1) / COLS;
  int64_t want = 152 * 4 / col_blocks;
  const int64_t most = (R + WARPS - 1) / WARPS;
  if (want > most) want = most;
  return want < 1 ? 1 : want;
}

// Column sums of up to CLUSTER_ROWS rows: a cluster of blocks holds all rows of
// its columns and adds its blocks' sums through shared memory, with no
// partials in memory and no second launch (measured on [333, 8192]: CLUSTER_FIG).
// More rows want more row blocks than a cluster has.
constexpr int CLUSTER = 8, CLUSTER_ROWS = 512;
int64_t ckpt_partials(int64_t R, int64_t C) { return R <= CLUSTER_ROWS ? 0 : ckpt_row_blocks(R, C) * C; }

// DB: 0 no column sums, 1 partials per row block, 2 summed in the cluster.
template <int ACT, bool H, int DB>
__global__ void __launch_bounds__(32 * WARPS, 2) ckpt_bwd_kernel(const CkptParams p, int64_t rows_per_block) {
  constexpr bool GLU = ACT == MX_ACT_SWIGLU;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t F = ACT == MX_ACT_SWIGLU ? p.C / 2 : p.C;
  const int64_t c = (int64_t)blockIdx.x * COLS + 8 * lane, sc = p.C >> 5;
  const bool in = c < F;
  const int64_t r0 = (int64_t)blockIdx.y * rows_per_block;
  const int64_t r1 = r0 + rows_per_block < p.R ? r0 + rows_per_block : p.R;
  float sum[8] = {}, sum_u[8] = {};
  pdl_trigger();
  pdl_wait();
  for (int64_t rb = r0 + warp; in && rb < r1; rb += WARPS * BATCH) {
    uint2 qz[BATCH], qu[BATCH];
    uint32_t bz[BATCH], bu[BATCH];
    uint4 qd[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; i++) {
      const int64_t r = rb + i * WARPS < r1 ? rb + i * WARPS : r1 - 1;
      qz[i] = load_once8(p.q + r * p.C + c);
      bz[i] = __ldg(p.q_scale + blocked_offset(r, c >> 5, sc));
      if (GLU) {
        qu[i] = load_once8(p.q + r * p.C + F + c);
        bu[i] = __ldg(p.q_scale + blocked_offset(r, (F + c) >> 5, sc));
      }
      qd[i] = load_once(p.dh + r * p.ld_dh + c);
    }
#pragma unroll
    for (int i = 0; i < BATCH; i++) {
      const int64_t r = rb + i * WARPS;
      if (r >= r1) break;
      float z[8], d[8], h[8];
      read8(qz[i], bz[i], z);
      unpack8(qd[i], d);
      if constexpr (GLU) {
        float u[8];
        read8(qu[i], bu[i], u);
#pragma unroll
        for (int j = 0; j < 8; j++) {
          float a, s;
          act_slope_f32<MX_ACT_SILU>(z[j], &a, &s);
          h[j] = a * u[j];
          z[j] = d[j] * u[j] * s;
          u[j] = d[j] * a;
          if (DB != 0) sum_u[j] += u[j];
        }
        *reinterpret_cast<uint4*>(p.dz + r * p.ld_dz + F + c) = pack8(u);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) {
          float s;
          act_slope_f32<ACT>(z[j], &h[j], &s);
          z[j] = d[j] * s;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (DB != 0) sum[j] += z[j];
      *reinterpret_cast<uint4*>(p.dz + r * p.ld_dz + c) = pack8(z);
      if (H) *reinterpret_cast<uint4*>(p.h + r * p.ld_h + c) = pack8(h);
    }
  }
  if constexpr (DB != 0) {  // the warps' sums in warp order, then the blocks'
    __shared__ float part[WARPS][COLS];
    __shared__ float block_sum[GLU ? 2 : 1][COLS];
#pragma unroll
    for (int half = 0; half < (GLU ? 2 : 1); half++) {
      if (half) __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; j++) part[warp][8 * lane + j] = half ? sum_u[j] : sum[j];
      __syncthreads();
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; w++) t += part[w][threadIdx.x];
      if constexpr (DB == 2) {
        block_sum[half][threadIdx.x] = t;
      } else {
        const int64_t col = (int64_t)blockIdx.x * COLS + threadIdx.x;
        if (col < F) p.partials[(int64_t)blockIdx.y * p.C + half * F + col] = t;
      }
    }
    if constexpr (DB == 2) {
      cluster_sync_all();
      const int64_t col = (int64_t)blockIdx.x * COLS + threadIdx.x;
      const unsigned rank = blockIdx.y, blocks = gridDim.y;  // the cluster is the grid's whole y extent
      if (threadIdx.x % blocks == rank && col < F) {
#pragma unroll
        for (int half = 0; half < (GLU ? 2 : 1); half++) {
          float t = 0.f;
          for (unsigned b = 0; b < blocks; b++) {
            uint32_t at;
            float v;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(&block_sum[half][threadIdx.x])), "r"(b));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
            t += v;
          }
          p.db[half * F + col] = t;
        }
      }
      cluster_sync_all();  // no block leaves while another reads its sums
    }
  }
}

// Column sums of the partials: a block takes 32 columns, its 8 warps every
// eighth row block, summed in a fixed order.
__global__ void __launch_bounds__(256) ckpt_colsum_kernel(const float* __restrict__ part, int64_t blocks, int64_t C,
                                                          float* __restrict__ db) {
  __shared__ float s[8][32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;  // C is a multiple of 32
  float t = 0.f;
  pdl_trigger();
  pdl_wait();
#pragma unroll 4
  for (int64_t b = w; b < blocks; b += 8) t += part[b * C + c];
  s[w][lane] = t;
  __syncthreads();
  if (w == 0) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) a += s[i][lane];
    db[c] = a;
  }
}

template <int ACT>
static cudaError_t launch_fwd(const CkptParams& p, cudaStream_t s) {
  const int64_t per = (ACT == MX_ACT_SWIGLU ? p.C / 2 : p.C) / 32, blocks = (p.R * per + 255) / 256;
  return launch_pdl(ckpt_fwd_kernel<ACT>, dim3((unsigned)(blocks < 152 * 8 ? blocks : 152 * 8)), 256, 0, s, 1, p,
                    (uint32_t)per);
}

cudaError_t launch_ckpt_fwd(const CkptParams& p, cudaStream_t s) {
  switch (p.act) {
    case MX_ACT_SWIGLU: return launch_fwd<MX_ACT_SWIGLU>(p, s);
    case MX_ACT_GELU_TANH: return launch_fwd<MX_ACT_GELU_TANH>(p, s);
    case MX_ACT_SILU: return launch_fwd<MX_ACT_SILU>(p, s);
    default: return launch_fwd<MX_ACT_RELU>(p, s);
  }
}

template <int ACT>
static cudaError_t launch_bwd(const CkptParams& p, cudaStream_t s) {
  constexpr unsigned T = 32 * WARPS;
  const int64_t F = ACT == MX_ACT_SWIGLU ? p.C / 2 : p.C;
  const bool cluster = p.db && p.partials == nullptr;
  const int64_t most = (p.R + WARPS - 1) / WARPS;
  const int64_t blocks = cluster ? (most < CLUSTER ? most : CLUSTER) : ckpt_row_blocks(p.R, p.C);
  const int64_t rows = (p.R + blocks - 1) / blocks;
  const dim3 grid((unsigned)((F + COLS - 1) / COLS), (unsigned)blocks);
  const unsigned cy = (unsigned)blocks;
  if (cluster)
    return p.h ? launch_pdl(ckpt_bwd_kernel<ACT, true, 2>, grid, T, 0, s, cy, p, rows)
               : launch_pdl(ckpt_bwd_kernel<ACT, false, 2>, grid, T, 0, s, cy, p, rows);
  if (p.db == nullptr)
    return p.h ? launch_pdl(ckpt_bwd_kernel<ACT, true, 0>, grid, T, 0, s, 1, p, rows)
               : launch_pdl(ckpt_bwd_kernel<ACT, false, 0>, grid, T, 0, s, 1, p, rows);
  const cudaError_t e = p.h ? launch_pdl(ckpt_bwd_kernel<ACT, true, 1>, grid, T, 0, s, 1, p, rows)
                            : launch_pdl(ckpt_bwd_kernel<ACT, false, 1>, grid, T, 0, s, 1, p, rows);
  if (e != cudaSuccess) return e;
  return launch_pdl(ckpt_colsum_kernel, dim3((unsigned)(p.C / 32)), 256, 0, s, 1, p.partials, blocks, p.C, p.db);
}

cudaError_t launch_ckpt_bwd(const CkptParams& p, cudaStream_t s) {
  switch (p.act) {
    case MX_ACT_SWIGLU: return launch_bwd<MX_ACT_SWIGLU>(p, s);
    case MX_ACT_GELU_TANH: return launch_bwd<MX_ACT_GELU_TANH>(p, s);
    case MX_ACT_SILU: return launch_bwd<MX_ACT_SILU>(p, s);
    default: return launch_bwd<MX_ACT_RELU>(p, s);
  }
}

}  // namespace mx
