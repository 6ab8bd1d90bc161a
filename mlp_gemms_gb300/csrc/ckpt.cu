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
// stay in registers.  [65536, 1536] SWIGLU with h: 82.1 us = 6.2 TB/s, 92 % of
// the copy rate (a thread per 32-column block, as in the forward pass: 137).
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
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "l"(p));
  return q;
}
__device__ __forceinline__ uint2 load_once8(const void* p) {
  uint2 q;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(q.x), "=r"(q.y) : "l"(p));
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

// Rows a backward warp has in flight at a time (its loads are issued before the
// first of them is used) and blocks of an SM.  What fits the registers: SWIGLU
// with h takes three rows (us with three and four: [65536, 1536] 82, 83.5; with
// db 86, 91), without h four (70, 67); the others six (with four: [16384, 8192]
// GELU with db 118, 124; [333, 8192] 6.4, 6.9) or, with neither h nor db, four in
// each of three blocks (108, two blocks 120).
constexpr int bwd_rows(bool glu, bool h, bool db) { return glu ? (h ? 3 : 4) : h || db ? 6 : 4; }
constexpr int bwd_blocks(bool glu, bool h, bool db) { return glu || h || db ? 2 : 3; }

// Zero the scale layout's padding (rows R .. 128 * ceil(R / 128), column
// blocks C / 32 .. 4 * ceil(C / 128)), by one block.
__device__ __forceinline__ void zero_scale_padding(const CkptParams& p) {
  const int64_t sc = p.C >> 5, chunks = (sc + 3) / 4, top = (p.R + 127) / 128 * 128;
  for (int64_t i = threadIdx.x; i < (top - p.R) * chunks; i += blockDim.x)
    *reinterpret_cast<uint32_t*>(p.q_scale + blocked_offset(p.R + i / chunks, i % chunks * 4, sc)) = 0u;
}

// 32 BF16 columns of a row in one thread.  WIDE: 32-byte accesses, so that a
// lane reads and writes whole sectors (needs rows that start on 32 bytes);
// otherwise 16-byte ones.
template <bool WIDE>
__device__ __forceinline__ void load32(const uint16_t* p, uint32_t (&w)[16]) {
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < 2; i++)
      asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
          : "=r"(w[8 * i]), "=r"(w[8 * i + 1]), "=r"(w[8 * i + 2]), "=r"(w[8 * i + 3]), "=r"(w[8 * i + 4]),
            "=r"(w[8 * i + 5]), "=r"(w[8 * i + 6]), "=r"(w[8 * i + 7]) : "l"(p + 16 * i));
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint4 q = *(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
    }
  }
}
template <bool WIDE>
__device__ __forceinline__ void store_words(void* p, const uint32_t* w) {  // 8 words
  if constexpr (WIDE) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ void unpack32(const uint32_t (&w)[16], float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 16; j++) {
    v[2 * j] = bf16_bits_to_float(w[j] & 0xFFFFu);
    v[2 * j + 1] = bf16_bits_to_float(w[j] >> 16);
  }
}
template <bool WIDE>
__device__ __forceinline__ void store32(uint16_t* p, const float (&v)[32]) {
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 16; j++) w[j] = float2_to_bf16x2(v[2 * j], v[2 * j + 1]);
  store_words<WIDE>(p, w);
  store_words<WIDE>(p + 16, w + 8);
}
template <bool WIDE>
__device__ __forceinline__ void save32(const CkptParams& p, int64_t r, int c, float (&v)[32]) {
  const uint32_t b = rceil_scale_byte_sel<E4M3>(amax_abs_bits<32>(v));
  uint32_t w[8];
  quantize_block_words<E4M3>(v, b, w);
  store_words<WIDE>(p.q + r * p.C + c, w);
  p.q_scale[blocked_offset(r, c >> 5, p.C >> 5)] = (uint8_t)b;
}

// Forward: a thread owns one 32-column block of a row (SWIGLU: the gate's and
// the up half's), so the block's amax needs no exchange.  [65536, 1536] SWIGLU:
// 61.2 us = 6.6 TB/s, 99 % of the copy rate (with 16-byte accesses, which
// touch each sector twice, 68.5; with 8 columns a lane and the amax by
// shuffles, 72.8: issue slots).  [16384, 8192]: GELU 104 to 105 us = 96 %, with
// three blocks an SM, which keep two to four registers of SiLU and GELU in local
// memory (two blocks 110; four spill in earnest: 142).  Eight to twelve waves of
// blocks, each with a few items a thread (two waves 63.3 and 110, as many blocks
// as items 62.8 and 104).
template <int ACT, bool WIDE>
__global__ void __launch_bounds__(256, ACT == MX_ACT_SWIGLU ? 2 : 3) ckpt_fwd_kernel(const CkptParams p, uint32_t per) {
  constexpr bool GLU = ACT == MX_ACT_SWIGLU;
  const int64_t F = GLU ? p.C / 2 : p.C;
  pdl_trigger();
  pdl_wait();
  const int64_t items = p.R * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i < (1ll << 32) ? (uint32_t)i / per : i / per;
    const int c = (int)(i - r * per) * 32;
    uint32_t wz[16], wu[16];
    load32<WIDE>(p.z + r * p.ld_z + c, wz);
    if constexpr (GLU) load32<WIDE>(p.z + r * p.ld_z + F + c, wu);
    float z[32], h[32];
    unpack32(wz, z);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      h[j] = z[j];
      h[j + 1] = z[j + 1];
      act2<GLU ? MX_ACT_SILU : ACT>(&h[j], &h[j + 1]);
    }
    save32<WIDE>(p, r, c, z);
    if constexpr (GLU) {
      float u[32];
      unpack32(wu, u);
#pragma unroll
      for (int j = 0; j < 32; j += 2)
        unpack2(mul2(pack2(h[j], h[j + 1]), pack2(u[j], u[j + 1])), &h[j], &h[j + 1]);
      store32<WIDE>(p.h + r * p.ld_h + c, h);
      save32<WIDE>(p, r, (int)F + c, u);
    } else {
      store32<WIDE>(p.h + r * p.ld_h + c, h);
    }
    if (c == 0)  // column padding behind the last block
      for (int64_t sc = p.C >> 5, k = sc; k & 3; k++) p.q_scale[blocked_offset(r, k, sc)] = 0;
  }
  if (blockIdx.x == 0) zero_scale_padding(p);
}

// Row blocks of the backward pass: one wave of blocks on every SM (GB300: 152),
// or two, where the columns alone do not give it, each with a row for each of its
// warps.  col_blocks counts SWIGLU's columns twice: its blocks do two halves'
// work.
static int64_t ckpt_row_blocks(int64_t R, int64_t C, int per_sm) {
  const int64_t col_blocks = (C + COLS - 1) / COLS;
  int64_t want = 152 * 2 * per_sm / col_blocks;
  const int64_t most = (R + WARPS - 1) / WARPS;
  if (want > most) want = most;
  return want < 1 ? 1 : want;
}

// Column sums of up to CLUSTER_ROWS rows: a cluster of blocks holds all rows of
// its columns and adds its blocks' sums through shared memory, with no
// partials in memory and no second launch (measured on [333, 8192] GELU: 6.4 us
// against 7.8, and no workspace to allocate).
// More rows want more row blocks than a cluster has.
constexpr int CLUSTER = 8, CLUSTER_ROWS = 512;
int64_t ckpt_partials(int64_t R, int64_t C) { return R <= CLUSTER_ROWS ? 0 : ckpt_row_blocks(R, C, 2) * C; }

// DB: 0 no column sums, 1 partials per row block, 2 summed in the cluster.
template <int ACT, bool H, int DB>
__global__ void __launch_bounds__(32 * WARPS, bwd_blocks(ACT == MX_ACT_SWIGLU, H, DB != 0))
ckpt_bwd_kernel(const CkptParams p, int64_t rows_per_block) {
  constexpr bool GLU = ACT == MX_ACT_SWIGLU;
  constexpr int BATCH = bwd_rows(GLU, H, DB != 0);
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
      bz[i] = *(p.q_scale + blocked_offset(r, c >> 5, sc));
      if (GLU) {
        qu[i] = load_once8(p.q + r * p.C + F + c);
        bu[i] = *(p.q_scale + blocked_offset(r, (F + c) >> 5, sc));
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
        for (int j = 0; j < 8; j += 2) {
          uint64_t a, s;
          act_slope2<MX_ACT_SILU>(pack2(z[j], z[j + 1]), &a, &s);
          const uint64_t uu = pack2(u[j], u[j + 1]), dd = pack2(d[j], d[j + 1]);
          unpack2(mul2(a, uu), &h[j], &h[j + 1]);
          unpack2(mul2(mul2(dd, uu), s), &z[j], &z[j + 1]);
          unpack2(mul2(dd, a), &u[j], &u[j + 1]);
          if (DB != 0) {
            sum_u[j] += u[j];
            sum_u[j + 1] += u[j + 1];
          }
        }
        *reinterpret_cast<uint4*>(p.dz + r * p.ld_dz + F + c) = pack8(u);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          uint64_t a, g;
          act_bwd2<ACT>(pack2(z[j], z[j + 1]), pack2(d[j], d[j + 1]), &a, &g);
          unpack2(a, &h[j], &h[j + 1]);
          unpack2(g, &z[j], &z[j + 1]);
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
__global__ void __launch_bounds__(256) ckpt_colsum_kernel(const float* part, int64_t blocks, int64_t C, float* db) {
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
  const dim3 grid((unsigned)(blocks < 152 * 24 ? blocks : 152 * 24));
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.z) | reinterpret_cast<uintptr_t>(p.h) |
                       reinterpret_cast<uintptr_t>(p.q) | (uintptr_t)(p.ld_z * 2) | (uintptr_t)(p.ld_h * 2);
  return (at & 31) == 0 ? launch_pdl(ckpt_fwd_kernel<ACT, true>, grid, 256, 0, s, dim3(1), p, (uint32_t)per)
                        : launch_pdl(ckpt_fwd_kernel<ACT, false>, grid, 256, 0, s, dim3(1), p, (uint32_t)per);
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
  const int per_sm = bwd_blocks(ACT == MX_ACT_SWIGLU, p.h != nullptr, p.db != nullptr);
  const int64_t blocks = cluster ? (most < CLUSTER ? most : CLUSTER) : ckpt_row_blocks(p.R, p.C, per_sm);
  const int64_t rows = (p.R + blocks - 1) / blocks;
  const dim3 grid((unsigned)((F + COLS - 1) / COLS), (unsigned)blocks);
  const unsigned cy = (unsigned)blocks;
  if (cluster)
    return p.h ? launch_pdl(ckpt_bwd_kernel<ACT, true, 2>, grid, T, 0, s, dim3(1, cy), p, rows)
               : launch_pdl(ckpt_bwd_kernel<ACT, false, 2>, grid, T, 0, s, dim3(1, cy), p, rows);
  if (p.db == nullptr)
    return p.h ? launch_pdl(ckpt_bwd_kernel<ACT, true, 0>, grid, T, 0, s, dim3(1), p, rows)
               : launch_pdl(ckpt_bwd_kernel<ACT, false, 0>, grid, T, 0, s, dim3(1), p, rows);
  const cudaError_t e = p.h ? launch_pdl(ckpt_bwd_kernel<ACT, true, 1>, grid, T, 0, s, dim3(1), p, rows)
                            : launch_pdl(ckpt_bwd_kernel<ACT, false, 1>, grid, T, 0, s, dim3(1), p, rows);
  if (e != cudaSuccess) return e;
  return launch_pdl(ckpt_colsum_kernel, dim3((unsigned)(p.C / 32)), 256, 0, s, dim3(1), p.partials, blocks, p.C, p.db);
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
