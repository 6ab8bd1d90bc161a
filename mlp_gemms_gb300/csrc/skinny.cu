// The ragged product and the linear layer for a few rows (decode steps): every
// weight is read once and meets at most a few tokens, so the time is the
// weights' way through HBM plus the launch.  A CTA takes 16 (32 with a
// checkpoint) features of one expert and all of K, split over its eight warps
// in turns of 32: 64 consecutive bytes of a row per warp, 512 per CTA.  The
// weights go from global memory straight into the registers of mma.sync's A
// operand: the sum over k may be taken in any order as long as both operands
// use the same one, so a lane's 16-byte load (8 consecutive k) serves as two
// fragments without a shuffle, and so does the tokens' load on the B side.
// No shared-memory ring, no barriers before the first load: a tcgen05 tile
// costs its prologue (tensor-memory allocation, cluster barrier, descriptor
// fetch) before any weight arrives.  Measured: 8 rows of 8 of 128 experts,
// 2048 -> 1536, 11.4 us (4.4 TB/s) against 14.5 on the tensor-core tiles; one
// row, 4096 -> 16384, 23.5 us (5.7 TB/s) against 25.7; 2048 -> 2048, 4.5 against
// 8.3.  Up to 32 rows meet a weight at once, eight to an MMA (16 rows, 2048 ->
// 2048: 4.9 us).  The rows staged in shared memory by bulk copies instead: 11.9
// and 23.7 us, and 28 for 8 rows, 4096 -> 16384, where the tokens' loads wait
// behind the barrier (here 27.3 to 27.9; with the checkpoint's 32 features a CTA
// 24.5).
#include "act.cuh"
#include "mx_internal.h"

namespace mx {

static __device__ unsigned g_skinny_status = 0;

constexpr int SK_WARPS = 8;

// 32-k chunks a warp loads before it uses the first, with MT x 16 features and
// NT x 8 tokens of a pass (more tokens go over the weights again, from L2).
constexpr int sk_batch(int mt, int nt) { return mt * nt <= 2 ? 4 : 2; }

__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) {
  uint4 q;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "l"(p));
  return q;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The want-th expert with rows, by one warp; false when there are fewer.
__device__ __forceinline__ bool find_expert(const RaggedParams& p, int want, int lane, int* g_out, int64_t* r0,
                                            int64_t* r1, bool report) {
  if (p.offsets == nullptr) {
    *g_out = 0; *r0 = 0; *r1 = p.R;
    return want == 0;
  }
  int32_t high = 0;
  int seen = 0;
  bool bad = false, found = false;
  for (int b0 = 0; b0 < p.G; b0 += 128) {
    int32_t end[4], start[4];  // 128 experts' loads in flight at a time
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int g = b0 + 32 * i + lane;
      end[i] = g < p.G ? *(p.offsets + g) : 0;
      start[i] = g < p.G && g ? *(p.offsets + g - 1) : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int g = b0 + 32 * i + lane;
      const int32_t s0 = start[i], s1 = end[i];
      int32_t top = s0;
      if (__any_sync(0xFFFFFFFFu, g < p.G && (s0 < high || s1 < s0))) {  // a decreasing end: the largest so far counts
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int32_t u = __shfl_up_sync(0xFFFFFFFFu, top, o);
          if (lane >= o && u > top) top = u;
        }
        if (high > top) top = high;
      }
      const bool ok = s0 >= top && s1 >= s0 && (int64_t)s1 <= p.R;
      high = max(high, __shfl_sync(0xFFFFFFFFu, top, 31));
      if (g < p.G && !ok) bad = true;
      const unsigned has = __ballot_sync(0xFFFFFFFFu, g < p.G && ok && s1 > s0);
      const int n = __popc(has);
      if (!found && want < seen + n) {
        const bool it = (has >> lane & 1u) && __popc(has & ((1u << lane) - 1u)) == want - seen;
        const int src = __ffs(__ballot_sync(0xFFFFFFFFu, it)) - 1;
        *g_out = b0 + 32 * i + src;
        *r0 = __shfl_sync(0xFFFFFFFFu, s0, src);
        *r1 = __shfl_sync(0xFFFFFFFFu, s1, src);
        found = true;
        if (!report) return true;
      }
      seen += n;
    }
  }
  if (report && __any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(&g_skinny_status, DEV_BAD_OFFSETS);
  return found;
}

// Three CTAs an SM with 4 chunks in flight (two with 32 features or more
// tokens): measured on one token of 4096 -> 16384 against 2 x 8, 4 x 4, 4 x 2 and
// 5 x 2 chunks 23.9 us against 24.0, 29.0, 24.4, 35.1, and on 8 experts' rows
// 12.8 against 14.0, 16.5, 13.9, 17.8 (more CTAs spill; measured with an earlier
// search for the expert, which cost the latter 1.1 us more).
template <int MT, int NT, bool EPI>
__global__ void __launch_bounds__(32 * SK_WARPS, MT * NT == 1 ? 3 : 2) skinny_kernel(const RaggedParams p) {
  constexpr int ROWS = 16 * MT, TOK = 8 * NT, SK_BATCH = sk_batch(MT, NT);
  __shared__ float red[SK_WARPS][TOK][ROWS + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g4 = lane >> 2, t4 = lane & 3;
  pdl_trigger();
  pdl_wait();
  int g = 0;
  int64_t r0, r1;
  if (!find_expert(p, (int)blockIdx.y, lane, &g, &r0, &r1, blockIdx.x == 0 && blockIdx.y == 0 && warp == 0)) return;
  const int64_t n0 = (int64_t)blockIdx.x * ROWS;
  const uint16_t* w[2 * MT];
  bool win[2 * MT];
#pragma unroll
  for (int i = 0; i < 2 * MT; i++) {
    win[i] = n0 + g4 + 8 * i < p.N;
    w[i] = p.w + ((int64_t)g * p.N + (win[i] ? n0 + g4 + 8 * i : 0)) * p.K + 8 * t4;
  }
  const int chunks = (int)((p.K + 31) / 32);
  for (int64_t m0 = r0; m0 < r1; m0 += TOK) {
    float acc[MT][NT][4] = {};
    bool xin[NT];
    const uint16_t* x[NT];
#pragma unroll
    for (int n = 0; n < NT; n++) {
      xin[n] = m0 + 8 * n + g4 < r1;
      x[n] = p.a + (xin[n] ? m0 + 8 * n + g4 : m0) * p.ld_a + 8 * t4;
    }
    for (int c0 = warp; c0 < chunks; c0 += SK_WARPS * SK_BATCH) {
      uint4 qw[SK_BATCH][2 * MT], qx[SK_BATCH][NT];
#pragma unroll
      for (int b = 0; b < SK_BATCH; b++) {
        const uint32_t k = (uint32_t)(c0 + b * SK_WARPS) * 32;  // ends up to 800 columns past K: beyond 2^31
        const bool kin = k + 8 * t4 < (uint32_t)p.K;
#pragma unroll
        for (int i = 0; i < 2 * MT; i++) qw[b][i] = kin && win[i] ? ld_stream(w[i] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int n = 0; n < NT; n++)
          qx[b][n] = kin && xin[n] ? *(reinterpret_cast<const uint4*>(x[n] + k)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int b = 0; b < SK_BATCH; b++)
#pragma unroll
        for (int m = 0; m < MT; m++) {
          const uint4 &u = qw[b][2 * m], &v = qw[b][2 * m + 1];
#pragma unroll
          for (int n = 0; n < NT; n++) {
            mma_16816(acc[m][n], u.x, v.x, u.y, v.y, qx[b][n].x, qx[b][n].y);
            mma_16816(acc[m][n], u.z, v.z, u.w, v.w, qx[b][n].z, qx[b][n].w);
          }
        }
    }
    if (m0 != r0) __syncthreads();  // the last group's sums have been read
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int i = 0; i < 4; i++)
          red[warp][8 * n + 2 * t4 + (i & 1)][16 * m + g4 + 8 * (i >> 1)] = acc[m][n][i];
    __syncthreads();
    // the warps' sums in warp order; consecutive threads hold consecutive features
    const int count = r1 - m0 < TOK ? (int)(r1 - m0) : TOK;
    for (int i = threadIdx.x; i < TOK * ROWS; i += 32 * SK_WARPS) {
      const int t = i / ROWS, f = i % ROWS;
      float z = 0.f;
#pragma unroll
      for (int s = 0; s < SK_WARPS; s++) z += red[s][t][f];
      const int64_t row = m0 + t, col = n0 + f;
      const bool in = t < count && col < p.N;
      float v = z;
      if constexpr (EPI) {
        if (p.epi.bias && in) z += bf16_bits_to_float(*(p.epi.bias + col));
        if (MT == 2 && p.epi.q) {  // a warp's 32 lanes are one scale block
          float m = z;
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) m = max_abs_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
          const uint32_t b = rceil_scale_byte_sel<E4M3>(__float_as_uint(m) & 0x7FFFFFFFu);
          const int64_t sc = p.N >> 5;
          if (in) {
            p.epi.q[row * p.N + col] =
                b == 0xFFu ? 0x7Fu : (uint8_t)cvt_e4m3x2(z * inv_scale_from_byte(b & 0xFFu), 0.f);
            if (f == 0) p.epi.q_scale[blocked_offset(row, col >> 5, sc)] = (uint8_t)b;
          }
        }
        float idle = 0.f;
        v = z;
        if (p.epi.act == MX_ACT_GELU_TANH) act2<MX_ACT_GELU_TANH>(&v, &idle);
        else if (p.epi.act == MX_ACT_SILU) act2<MX_ACT_SILU>(&v, &idle);
        else if (p.epi.act == MX_ACT_RELU) act2<MX_ACT_RELU>(&v, &idle);
        if (p.epi.res && in) v += bf16_bits_to_float(p.epi.res[row * p.epi.ld_res + col]);
      }
      if (in) p.out[row * p.ld_out + col] = (uint16_t)float2_to_bf16x2(v, 0.f);
    }
  }
  if constexpr (EPI && MT == 2) {  // zero padding of the scale layout: rows to 128, columns to 4
    if (p.epi.q && n0 < p.N) {
      const int64_t sc = p.N >> 5, top = (p.R + 127) / 128 * 128;
      for (int64_t c = n0 >> 5; c < ((n0 >> 5) + 1 == sc ? (sc + 3) / 4 * 4 : (n0 >> 5) + 1); c++)
        for (int64_t r = (c < sc ? p.R : 0) + threadIdx.x; r < top; r += blockDim.x)
          p.epi.q_scale[blocked_offset(r, c, sc)] = 0;
    }
  }
}

template <int MT, int NT, bool EPI>
static cudaError_t launch(const RaggedParams& p, cudaStream_t s) {
  const dim3 grid((unsigned)((p.N + 16 * MT - 1) / (16 * MT)), (unsigned)(p.offsets ? (p.G < p.R ? p.G : p.R) : 1));
  return launch_pdl(skinny_kernel<MT, NT, EPI>, grid, 32 * SK_WARPS, 0, s, dim3(1), p);
}

template <int NT>
static cudaError_t launch_tokens(const RaggedParams& p, cudaStream_t s) {
  if (p.epi.q) return launch<2, NT, true>(p, s);
  const bool epi = p.epi.bias || p.epi.act != MX_ACT_NONE || p.epi.res;
  return epi ? launch<1, NT, true>(p, s) : launch<1, NT, false>(p, s);
}

// Experts' segments are short here: 8 rows at a time.
cudaError_t launch_skinny(const RaggedParams& p, cudaStream_t s) {
  if (p.offsets != nullptr || p.R <= 8) return launch_tokens<1>(p, s);
  return p.R <= 16 ? launch_tokens<2>(p, s) : launch_tokens<4>(p, s);
}

cudaError_t read_skinny_status(unsigned* out) { return cudaMemcpyFromSymbol(out, g_skinny_status, sizeof(unsigned)); }
cudaError_t reset_skinny_status() {
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_skinny_status, &zero, sizeof(unsigned));
}

}  // namespace mx
