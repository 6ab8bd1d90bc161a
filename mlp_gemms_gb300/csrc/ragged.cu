// BF16 products over ragged expert segments (any length, no padding) on the
// 5th-generation tensor core: the grouped product with W [G, N, K] or
// [G, K, N], the weight gradient, and the dense linear layer's epilogue.
//
// One kernel computes out[t, f] = sum_k Q[t, k] P[f, k].  P is the side whose
// index runs along the output's rows in memory: the weights' features for the
// forward product and the input gradient, X's columns for the weight
// gradient.  P takes the MMA's M = 256 rows of a CTA pair (tcgen05
// .cta_group::2, 128 rows per CTA), Q the N side, whose width follows the
// segment: a tile holds up to 256 tokens and rounds them to 32.  Expert
// segments are short and ragged (tokens) while features are long and even, so
// the padding is at most 31 tokens per expert instead of up to 255, and a
// decode step's few tokens cost an N = 32 MMA under a weight stream that stays
// bound by memory.  Both operands may be K-major (rows of K) or MN-major
// (rows of the contraction index), so no operand is transposed in memory:
//
//            P (M side)                    Q (N side)
//   NK       W[g] [N, K]   K-major         A [R, K]   K-major
//   KN       W[g] [K, N]   MN-major        A [R, K]   K-major
//   WGRAD    X [R, K]      MN-major        dY [R, N]  MN-major
//
// Accumulators (128 lanes x 256 fp32 columns, two of them) live in tensor
// memory; while the eight epilogue warps drain one, the MMA thread fills the
// other.  A lane of the accumulator is a feature, a column a token, so the
// epilogue reads it in 8x8 fragments (tcgen05.ld 16x256b) and turns it with
// stmatrix.trans; two warps with neighbouring features share a staging buffer
// and store whole 128-byte lines.
//
// What bounds it (us at 8192 tokens x 8 choices, 128 experts, skewed, K = 2048,
// N = 1536): forward 306, input gradient 307, weight gradient 328 over seconds,
// as a training run sees it, when the power limit holds the clock down (floor
// 236 at the BF16 rate measured over seconds); 276, 274 and 288 to 291 in short
// bursts from a cold chip (floor 209 at the burst rate, 183 at the copy rate).
// In such bursts one expert for all rows takes 213 (98 % of the rate), 64 239,
// 128 even ones 266: beside the MMAs the weights come through HBM, 228 us
// without MMAs.
// Dense [16384, 2048] x [8192, 2048], GELU and checkpoint: 350 us = 1.57
// PFLOP/s over seconds, 295 = 1.87 in bursts.  The sweeps quoted below are
// bursts.  Two pairs sharing the token operand by multicast (clusters of four:
// 144 of 152 SMs) moved a quarter fewer bytes and were 0 to 3 % slower; an L2
// prefetch of the next tile's operands was 6 to 30 % slower.
//
// The weight gradient contracts over a segment's rows.  Its last 64-row block
// would hold rows of the next expert, whose Inf or NaN times a zero is NaN: it
// is copied in pieces of 32, 16, 8, 4, 2 and 1 rows that end with the segment,
// and filled up to a multiple of 16 by pieces that start beyond the tensor and
// read as zeros.  The pieces start on any 128-byte row: the swizzle goes by
// the shared-memory address.  (Zeroing the foreign rows after the copy, by
// stores or by copies, delayed the MMAs by 1500 to 3300 cycles a tile; adding
// those rows in the epilogue with mma.sync cost 100 us of 314.)
//
// Every wait is bounded; on expiry the CTA records a device status bit and
// unwinds.
#include "act.cuh"
#include "mx_internal.h"
#include "pair_common.cuh"

#include <atomic>
#include <type_traits>

namespace mx {

static __device__ unsigned g_ragged_status = 0;

namespace rg {
constexpr int THREADS = 384;  // warps: 0 and 3 copies, 1 MMAs, 2 hands out tiles, 4..11 epilogue
constexpr int ST = 6;         // 32 KB stages of 64 contraction steps
constexpr int BK = 64;
constexpr int P_BYTES = 16384, Q_BYTES = 16384;
constexpr int OFF_Q = ST * P_BYTES;
constexpr int STG = 2304;     // per epilogue warp; two share 32 rows x (128 + 16) bytes
constexpr int OFF_STG = OFF_Q + ST * Q_BYTES;
constexpr int OFF_SEG = OFF_STG + 8 * STG;                  // segment ends, [0] = 0
constexpr int OFF_PREF = OFF_SEG + 4 * (MAX_RAGGED_G + 1);  // row tiles before expert g
constexpr int OFF_ORD = OFF_PREF + 4 * (MAX_RAGGED_G + 1);  // experts by falling row count (uint16)
constexpr int SLOTS = 2;      // tile indices on their way from the hardware
constexpr int TILES = 4;      // tiles on their way to the roles
// Blocks of a tile still to be copied when the next tile is asked for: the answer
// comes in time, and a pair takes on no tile long before it is free for it
// (us with 8, and asked for at a tile's begin: weight gradient, skewed, 286, 293;
// 16384 rows, 512 -> 8192, 84.5, 95).
constexpr int AHEAD = 8;
constexpr int OFF_NEXT = (OFF_ORD + 2 * MAX_RAGGED_G + 15) / 16 * 16;
constexpr int OFF_TILES = OFF_NEXT + 16 * (SLOTS + 1);
constexpr int OFF_BAR = OFF_TILES + 48 * TILES;
constexpr int NUM_BARS = 2 * ST + 5 + 2 * SLOTS + 1 + 3 * TILES;
constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
constexpr int SMEM = OFF_MISC + 16 + 1024;                  // + slack for 1024-byte alignment
static_assert(SMEM <= 232448, "shared memory per CTA");
}  // namespace rg

enum RaggedMode : int { RAGGED_NK = 0, RAGGED_KN = 1, RAGGED_WGRAD = 2 };

struct RaggedK {
  int G;
  const int32_t* offsets;
  int64_t R;
  int64_t N;               // output columns (the P side's extent)
  int64_t K;               // contraction (WGRAD: the Q side's extent instead)
  int n_f;                 // 256-column tiles of the output
  int n_t;                 // WGRAD: row tiles of an expert's output
  int tw;                  // rows of a tile, a multiple of 32 up to 256
  int splits;              // NK, KN: pairs that share a tile; WGRAD: parts of a segment, each with an output [G, ...]
  void* out;
  int64_t ld_out;          // elements; WGRAD: N
  int accumulate;
  int fetch_old;           // bring what a tile is added to into L2 first
  int w_once;              // the weights are read by about one tile each
  RaggedEpi epi;
};

struct alignas(16) RaggedTile {
  int64_t t0;              // first output row (WGRAD: of the expert's matrix)
  int g;
  int valid;               // rows of the tile in the output
  int nt;                  // the MMA's N: valid rounded up to 32
  int f0;                  // first output column of the pair's 256
  int nk;                  // 64-step blocks of the contraction; -1: no tile, the last one was before
  int k0;                  // first step of the contraction
  int rem;                 // contraction steps in the last block (1..64)
  int part, parts;         // WGRAD into fp32: this pass over the tile, and how many it takes
  int split;               // WGRAD: which part of the segment
};
static_assert(sizeof(RaggedTile) == 48, "RaggedTile");

// Rows the fp32 weight gradient sums in tensor memory before it adds the sum
// to memory.  The tensor core's fp32 accumulation truncates, a drift towards
// zero of about 2^-26 per 16-row step: 7.6e-5 of the result after 65536 rows
// (measured), against the 1e-7 of fp32 sums rounded to nearest.  4096 rows
// keep it below 5e-6 and cost one read and write of the tile per 4 MB of
// operands.  A BF16 result (2e-3 from its own rounding) takes one pass.
constexpr int F32_ROWS = 4096;

// One poll that does not suspend the thread.
__device__ __forceinline__ uint32_t mbar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
               "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok;
}

// Bounded wait of a whole warp for a phase of a barrier (CLUSTER: with
// arrivals of the other CTA's).  The roles run as whole warps and elect one
// lane for what a single thread issues: in a branch on the lane's number every
// operand of a copy or an MMA goes through a register move that the loop waits
// for (measured: 97 cycles per MMA issued, 200 per wait, 720 a stage).
template <bool CLUSTER>
__device__ __forceinline__ bool ragged_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  uint64_t t0 = 0;
  for (uint32_t n = 1;; n++) {
    uint32_t ok;
    if constexpr (CLUSTER)
      asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                   "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    else
      ok = mbar_try_wait(bar, parity);
    if (__all_sync(0xFFFFFFFFu, ok != 0)) return true;
    if ((n & 63u) == 0u) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > WAIT_BUDGET_NS) *abort_flag = 1;
      if (__any_sync(0xFFFFFFFFu, *abort_flag != 0)) return false;
    }
  }
}

// The shared::cluster address of a local shared address in another CTA of the
// cluster, and the commit to both CTAs of the pair that starts at CTA `first`.
__device__ __forceinline__ uint32_t cta_addr(const void* p, uint32_t cta) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(cta));
  return r;
}
__device__ __forceinline__ void tc2_commit_pair(uint64_t* bar, uint32_t first) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               :: "r"(smem_u32(bar)), "h"((uint16_t)(3u << first)) : "memory");
}

// Hand an accumulator back: an arrival on a barrier of the leader CTA that
// orders no memory.  What it announces, this warp's tensor-memory loads, is
// complete (tcgen05.wait::ld); a release at cluster scope would also wait for
// the warp's stores to global memory, about 1100 cycles a tile.
__device__ __forceinline__ void arrive_on_leader_relaxed(uint32_t bar_cl) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar_cl) : "memory");
}

// Tiles are handed out by the hardware: the grid has a cluster for every tile,
// and a running pair takes over the next cluster that has not started yet
// (clusterlaunchcontrol.try_cancel), so pairs stay busy whatever the segments'
// lengths.  Experts come by falling row count, the long ones first.  A warp of
// each CTA does nothing else: the leader's asks for a tile once the last one's
// copies come to their end, the answer arrives in both CTAs, and each finds the
// expert and hands the finished description to its roles.  (Every role finding
// its tiles for itself held the copies up by 3000 cycles a tile, the lookups
// queueing behind the warp's own copies: 64 rows of each of 128 experts, weight
// gradient of [1536, 2048], 151 us, now 134; skewed training segments 301, now
// 287.)
struct RaggedSched {
  uint4* next;         // SLOTS answers, and one for the drain
  uint64_t* full;      // each CTA's: the answer is there
  uint64_t* empty;     // leader's: both CTAs have read it
};

__device__ __forceinline__ RaggedSched ragged_sched(uint8_t* smem) {
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + rg::OFF_BAR) + 2 * rg::ST + 5;
  return RaggedSched{reinterpret_cast<uint4*>(smem + rg::OFF_NEXT), bars, bars + rg::SLOTS};
}

// The first CTA of the cluster taken over, or false when none was left.
__device__ __forceinline__ bool taken_cta(const uint4* answer, uint32_t* cta) {
  uint32_t ok, x = 0;
  asm volatile("{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%2];\n\t"
               "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\t"
               "mov.u32 %1, 0;\n\t"
               "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, r;\n\t}"
               : "=r"(ok), "=r"(x) : "r"(smem_u32(answer)) : "memory");
  *cta = x;
  return ok != 0;
}

// The way through the pair's passes: each of its tiles, and of a tile each part.
// Tile indices only grow, so the expert is searched for from the last one on, 32
// at a time (one by one the 38 short experts between a pair's tiles took 8000
// cycles: 8113 rows of 128 experts, 104 -> 64, 14.0 us, now 8.0).
template <int MODE, bool F32, bool SPLIT>
struct RaggedWalk {
  const RaggedK& p;
  const int32_t *seg, *pref;
  const uint16_t* ord;
  RaggedSched sched;
  volatile int* abort_flag;
  uint32_t t, base;  // current tile; first tile of the expert at place `at`
  int at, part, slot;
  uint32_t phase;
  bool fetch;        // the next pass is another tile's
  bool asked;        // an answer is on its way
  bool more;         // a cluster was taken over for the last tile asked for (else none is left)
  __device__ RaggedWalk(const RaggedK& p_, uint8_t* smem)
      : p(p_), seg(reinterpret_cast<int32_t*>(smem + rg::OFF_SEG)), pref(reinterpret_cast<int32_t*>(smem + rg::OFF_PREF)),
        ord(reinterpret_cast<uint16_t*>(smem + rg::OFF_ORD)), sched(ragged_sched(smem)),
        abort_flag(reinterpret_cast<volatile int*>(smem + rg::OFF_MISC + 4)),
        t(SPLIT ? blockIdx.x / (2 * p_.splits) : blockIdx.x >> 1), base(0), at(0),
        part(0), slot(0), phase(0), fetch(false), asked(false), more(true) {}
  __device__ bool next(RaggedTile* T) {
    if (SPLIT && fetch) return false;  // a cluster's only tile
    if (!SPLIT && fetch) {
      if (!ragged_wait<false>(&sched.full[slot], phase, abort_flag)) return false;
      uint32_t cta;
      more = taken_cta(&sched.next[slot], &cta);
      asked = false;
      if (!more) return false;
      t = cta >> 1;
      fence_proxy_async_smem();
      __syncwarp();
      if (elect_one_lane()) arrive_on_leader_relaxed(leader_addr(&sched.empty[slot]));
      if (++slot == rg::SLOTS) { slot = 0; phase ^= 1u; }
    }
    const uint32_t n_f = (uint32_t)p.n_f;
    // past the end: told from the total, not by walking through every expert
    const uint32_t all = MODE == RAGGED_WGRAD ? (uint32_t)p.G * n_f * (uint32_t)p.n_t : (uint32_t)pref[p.G] * n_f;
    if (t >= (MODE == RAGGED_WGRAD ? all * (uint32_t)p.splits : all)) return false;
    uint32_t u = t;  // the tile within its part of the segments
    if (MODE == RAGGED_WGRAD && p.splits > 1) {
      T->split = (int)(t / all);
      u = t - (uint32_t)T->split * all;
    } else {
      T->split = 0;
    }
    if constexpr (MODE == RAGGED_WGRAD) {
      at = (int)(u / (n_f * (uint32_t)p.n_t));
      base = (uint32_t)at * n_f * (uint32_t)p.n_t;
    } else {
      const int lane = threadIdx.x & 31;
      const auto tiles_of = [&](int place) {
        const int e = ord[place];
        return (uint32_t)(pref[e + 1] - pref[e]) * n_f;
      };
      uint32_t count = tiles_of(at);
      if (u - base >= count) {
        for (base += count, at++;; at += 32) {
          count = at + lane < p.G ? tiles_of(at + lane) : 0;
          uint32_t upto = count;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += v;
          }
          const unsigned there = __ballot_sync(0xFFFFFFFFu, u - base < upto);
          if (there) {
            const int l = __ffs(there) - 1;
            base += __shfl_sync(0xFFFFFFFFu, upto - count, l);
            at += l;
            break;
          }
          base += __shfl_sync(0xFFFFFFFFu, upto, 31);
        }
      }
    }
    const int g = ord[at];
    const uint32_t mt = (u - base) / n_f;
    const int32_t seg0 = seg[g];
    T->g = g;
    T->f0 = (int)(u - base - mt * n_f) * 256;
    T->parts = 1;
    int64_t left;
    if constexpr (MODE == RAGGED_WGRAD) {
      T->t0 = (int64_t)mt * p.tw;
      left = p.K - T->t0;
      int rows = pref[g + 1] - pref[g];  // rows of the segment, 0 if malformed
      T->k0 = seg0;
      if (p.splits > 1) {
        const int per = ((rows + p.splits - 1) / p.splits + rg::BK - 1) / rg::BK * rg::BK, from = per * T->split;
        T->k0 += from < rows ? from : 0;
        rows = from < rows ? (rows - from < per ? rows - from : per) : 0;
      }
      if constexpr (F32) {
        T->parts = rows > F32_ROWS ? (rows + F32_ROWS - 1) / F32_ROWS : 1;
        T->k0 += part * F32_ROWS;
        rows -= part * F32_ROWS;
        if (rows > F32_ROWS) rows = F32_ROWS;
      }
      T->nk = (rows + rg::BK - 1) / rg::BK;
      T->rem = rows - (T->nk - 1) * rg::BK;
    } else {
      T->t0 = (int64_t)seg0 + p.tw * (int64_t)mt;
      left = (int64_t)seg[g + 1] - T->t0;
      T->k0 = 0;
      T->nk = (int)((p.K + rg::BK - 1) / rg::BK);
      T->rem = (int)p.K - (T->nk - 1) * rg::BK;
      if constexpr (SPLIT) {  // this pair's blocks of the contraction
        const int pair = (int)(cluster_rank() >> 1), from = T->nk * pair / p.splits, to = T->nk * (pair + 1) / p.splits;
        T->k0 = from * rg::BK;
        if (to < T->nk) T->rem = rg::BK;
        T->nk = to - from;
      }
    }
    T->valid = left < p.tw ? (int)left : p.tw;
    T->nt = (T->valid + 31) & ~31;
    T->part = part;
    fetch = ++part >= T->parts;
    if (fetch) part = 0;
    return true;
  }
};

// A role's view of the tiles handed to it (a whole warp).
struct RaggedFeed {
  const RaggedTile* tiles;
  uint64_t *full, *empty, *ending;  // the tile is there; all roles have read it; its copies come to their end
  volatile int* abort_flag;
  int slot;
  uint32_t phase;
  __device__ RaggedFeed(const RaggedK&, uint8_t* smem)
      : tiles(reinterpret_cast<const RaggedTile*>(smem + rg::OFF_TILES)),
        full(reinterpret_cast<uint64_t*>(smem + rg::OFF_BAR) + 2 * rg::ST + 5 + 2 * rg::SLOTS + 1),
        empty(full + rg::TILES), ending(empty + rg::TILES),
        abort_flag(reinterpret_cast<volatile int*>(smem + rg::OFF_MISC + 4)), slot(0), phase(0) {}
  __device__ bool next(RaggedTile* T) {
    if (!ragged_wait<false>(&full[slot], phase, abort_flag)) return false;
    *T = tiles[slot];
    __syncwarp();
    if (elect_one_lane()) mbar_arrive(&empty[slot]);
    if (++slot == rg::TILES) { slot = 0; phase ^= 1u; }
    return T->nk >= 0;
  }
  // The copying warp's word that the next tile may be asked for.
  __device__ void near_end() {
    if (elect_one_lane()) mbar_arrive(&ending[slot == 0 ? rg::TILES - 1 : slot - 1]);
  }
};
template <int MODE, bool F32, bool SPLIT>  // a cluster's only tile: every role works it out for itself
using RaggedSource = std::conditional_t<SPLIT, RaggedWalk<MODE, F32, SPLIT>, RaggedFeed>;

// The warp that hands out the tiles.
template <int MODE, bool F32>
__device__ __forceinline__ void ragged_tiles(const RaggedK& p, uint8_t* smem, bool leader) {
  using namespace rg;
  RaggedWalk<MODE, F32, false> walk(p, smem);
  RaggedFeed feed(p, smem);
  const RaggedSched sched = walk.sched;
  volatile int* abort_flag = walk.abort_flag;
  RaggedTile* const tiles = reinterpret_cast<RaggedTile*>(smem + OFF_TILES);
  const int lane = threadIdx.x & 31;
  int ask = 0, at = 0;                      // slots of the next request and of the tile that ends next
  uint32_t ask_phase = 1, at_phase = 0;
  bool ok = true;
  while (true) {
    RaggedTile T;
    const bool more = walk.next(&T);
    if (!more) T.nk = -1;
    if (!ragged_wait<false>(&feed.empty[feed.slot], feed.phase ^ 1u, abort_flag)) { ok = false; break; }
    if (lane == 0) tiles[feed.slot] = T;
    __syncwarp();
    if (elect_one_lane()) mbar_arrive(&feed.full[feed.slot]);
    if (++feed.slot == TILES) { feed.slot = 0; feed.phase ^= 1u; }
    if (!more) break;
    if (leader) {
      if (!ragged_wait<false>(&feed.ending[at], at_phase, abort_flag)) { ok = false; break; }
      if (++at == TILES) { at = 0; at_phase ^= 1u; }
    }
    if (walk.fetch) {  // ask for the tile after this one
      if (leader) {
        if (!ragged_wait<true>(&sched.empty[ask], ask_phase, abort_flag)) { ok = false; break; }
        if (elect_one_lane()) {
          mbar_arrive_expect_tx(&sched.full[ask], 16);
          asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], 16;"
                       :: "r"(peer_addr(&sched.full[ask])) : "memory");
          asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
                       ".multicast::cluster::all.b128 [%0], [%1];"
                       :: "r"(smem_u32(&sched.next[ask])), "r"(smem_u32(&sched.full[ask])) : "memory");
        }
        __syncwarp();
        if (++ask == SLOTS) { ask = 0; ask_phase ^= 1u; }
      }
      walk.asked = true;
    }
  }
  volatile int no_abort = 0;
  if (walk.asked) {  // given up while an answer is on its way: it lands first
    ragged_wait<false>(&sched.full[walk.slot], walk.phase, &no_abort);
  } else if (leader && ok && walk.more) {
    // The tile taken over last lies past the end: the grid counts a tile more
    // than there may be for every segment.  Take over the rest as well, so
    // that they do not start only to find nothing to do.
    uint64_t* bar = sched.empty + SLOTS;
    for (uint32_t parity = 0;; parity ^= 1u) {
      if (elect_one_lane()) {
        mbar_arrive_expect_tx(bar, 16);
        asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                     :: "r"(smem_u32(&sched.next[SLOTS])), "r"(smem_u32(bar)) : "memory");
      }
      __syncwarp();
      uint32_t cta;
      if (!ragged_wait<false>(bar, parity, &no_abort) || !taken_cta(&sched.next[SLOTS], &cta)) break;
      fence_proxy_async_smem();
      __syncwarp();
    }
  }
}

__device__ __forceinline__ void tma2_load_3d_hint(void* dst, const CUtensorMap* m, int c0, int c1, int c2,
                                                  uint32_t bar_cl, uint64_t pol) {
  asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
               " [%0], [%1, {%2, %3, %4}], [%5], %6;"
               :: "r"(smem_u32(dst)), "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(bar_cl), "l"(pol) : "memory");
}

__device__ __forceinline__ void tc2_mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
               :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

// 16 lanes x 32 columns of tensor memory as four 8-column groups: registers
// 4j, 4j + 1 hold columns 8j + 2 (lane % 4) + {0, 1} of lane lane / 4,
// registers 4j + 2, 4j + 3 those of lane lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, float (&r)[16]) {
  uint32_t u[16];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
                 "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; i++) r[i] = __uint_as_float(u[i]);
}

// Four 8x8 matrices of 16-bit values, transposed on the way: lane 8m + i
// gives the address of the row that receives column i of matrix m.
__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
               :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

template <int ACT>
__device__ __forceinline__ void act_values(float (&v)[2][16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    act2<ACT>(&v[0][i], &v[0][i + 1]);
    act2<ACT>(&v[1][i], &v[1][i + 1]);
  }
}

// The 8-bit checkpoint of a 32-feature x 32-token block (one scale block per
// token).  A thread holds four features of eight tokens: the amax of a token
// is a maximum over those and over the eight lanes that share its tokens.
// Codes of features f and f + 8 (one thread's) travel as one 16-bit value
// through stmatrix.trans and are separated again on the way out.
__device__ __forceinline__ void ckpt_block(const RaggedK& p, const float (&v)[2][16], uint8_t* stg, int lane,
                                           int64_t row0, int valid, int64_t col) {
  const uint32_t base = smem_u32(stg);
  uint8_t* sbytes = stg + 32 * 48;
#pragma unroll
  for (int jj = 0; jj < 2; jj++) {
    uint32_t w[2][2];
#pragma unroll
    for (int j2 = 0; j2 < 2; j2++) {
      const int j = 2 * jj + j2;
      uint32_t code[2][2];  // [features' half][token]
#pragma unroll
      for (int e = 0; e < 2; e++) {
        float m = max_abs_nan(max_abs_nan(v[0][4 * j + e], v[0][4 * j + 2 + e]),
                              max_abs_nan(v[1][4 * j + e], v[1][4 * j + 2 + e]));
        m = max_abs_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
        m = max_abs_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
        m = max_abs_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
        const uint32_t sb = rceil_scale_byte_sel<E4M3>(__float_as_uint(m) & 0x7FFFFFFFu);
        if (lane < 4) sbytes[8 * j + 2 * lane + e] = (uint8_t)sb;
        const float s = inv_scale_from_byte(sb & 0xFFu);
#pragma unroll
        for (int h = 0; h < 2; h++)
          code[h][e] = sb == 0xFFu ? 0x7F7Fu : cvt_e4m3x2(v[h][4 * j + e] * s, v[h][4 * j + 2 + e] * s);
      }
      w[j2][0] = code[0][0] | (code[0][1] << 16);
      w[j2][1] = code[1][0] | (code[1][1] << 16);
    }
    // matrices: (tokens 8 (2 jj + m / 2) .., features' half m % 2)
    stmatrix4_trans(base + (16 * jj + 8 * (lane >> 4) + (lane & 7)) * 48 + ((lane >> 3) & 1) * 16, w[0][0], w[0][1],
                    w[1][0], w[1][1]);
  }
  __syncwarp();
  if (col < p.N) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int t = 16 * i + (lane >> 1);
      const uint4 c = *reinterpret_cast<const uint4*>(stg + t * 48 + (lane & 1) * 16);
      if (t < valid)
        *reinterpret_cast<uint4*>(p.epi.q + (row0 + t) * p.N + col + 16 * (lane & 1)) =
            make_uint4(__byte_perm(c.x, c.y, 0x6420), __byte_perm(c.z, c.w, 0x6420), __byte_perm(c.x, c.y, 0x7531),
                       __byte_perm(c.z, c.w, 0x7531));
    }
  }
  // scales; the padding of the blocked layout (rows to 128, columns to 4) is zero
  const int64_t sc = p.N / 32, c = col / 32;
  if (c < (sc + 3) / 4 * 4) {
    if (lane < valid) p.epi.q_scale[blocked_offset(row0 + lane, c, sc)] = c < sc ? sbytes[lane] : 0;
    const int64_t end = row0 + valid;
    if (end == p.R && valid > 0)
      for (int64_t r = end + lane; r < (p.R + 127) / 128 * 128; r += 32) p.epi.q_scale[blocked_offset(r, c, sc)] = 0;
  }
  __syncwarp();
}

// The residual's part of a block, 16 bytes of 8 rows a load: fetched a block
// ahead, so that its latency is not the epilogue's.
__device__ __forceinline__ void load_residual(const RaggedK& p, uint4 (&x)[4], int lane, int64_t row0, int valid,
                                              int64_t col) {
  const int64_t c = col + 8 * (lane & 3);
  const uint16_t* at = p.epi.res + (row0 + (lane >> 2)) * p.epi.ld_res + c;
#pragma unroll
  for (int i = 0; i < 4; i++)
    x[i] = 8 * i + (lane >> 2) < valid && c < p.N ? *reinterpret_cast<const uint4*>(at + 8 * i * p.epi.ld_res)
                                                  : make_uint4(0, 0, 0, 0);
}

// One 32-feature x 32-token block of the accumulator -> BF16 rows, with the
// linear layer's epilogue when EPI.  Two warps whose features are neighbours
// share a staging buffer (32 rows of 128 + 16 bytes; stg, this warp's features
// 64 bytes into it or not) and store whole 128-byte lines of 16 rows each.
template <bool EPI>
__device__ __forceinline__ void store_block_bf16(const RaggedK& p, float (&v)[2][16], uint8_t* stg, int lane,
                                                 int odd, int bar, const float (&bias)[4], const uint4 (&res)[4],
                                                 uint16_t* out, int64_t row0, int valid, int64_t col) {
  const uint32_t base = smem_u32(stg);
  const uint32_t frag = base + (lane & 7) * 144 + (lane >> 3) * 16 + odd * 64;
  if constexpr (EPI) {
#pragma unroll
    for (int i = 0; i < 16; i++) {
      v[0][i] += bias[(i >> 1) & 1];
      v[1][i] += bias[2 + ((i >> 1) & 1)];
    }
    if (p.epi.q) ckpt_block(p, v, stg + odd * 2304, lane, row0, valid, col);
    if (p.epi.q) named_bar(bar, 64);
    if (p.epi.act == MX_ACT_GELU_TANH) act_values<MX_ACT_GELU_TANH>(v);
    else if (p.epi.act == MX_ACT_SILU) act_values<MX_ACT_SILU>(v);
    else if (p.epi.act == MX_ACT_RELU) act_values<MX_ACT_RELU>(v);
    if (p.epi.res) {
#pragma unroll
      for (int i = 0; i < 4; i++)
        *reinterpret_cast<uint4*>(stg + (8 * i + (lane >> 2)) * 144 + (lane & 3) * 16 + odd * 64) = res[i];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; j++) {
        uint32_t r[4];
        ldmatrix4_trans(frag + 8 * j * 144, r);
#pragma unroll
        for (int m = 0; m < 4; m++) {
          v[m >> 1][4 * j + 2 * (m & 1)] += bf16_bits_to_float(r[m] & 0xFFFFu);
          v[m >> 1][4 * j + 2 * (m & 1) + 1] += bf16_bits_to_float(r[m] >> 16);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; j++)
    stmatrix4_trans(frag + 8 * j * 144, float2_to_bf16x2(v[0][4 * j], v[0][4 * j + 1]),
                    float2_to_bf16x2(v[0][4 * j + 2], v[0][4 * j + 3]),
                    float2_to_bf16x2(v[1][4 * j], v[1][4 * j + 1]),
                    float2_to_bf16x2(v[1][4 * j + 2], v[1][4 * j + 3]));
  named_bar(bar, 64);
  const int64_t c = col - 32 * odd + 8 * (lane & 7);
  const int t0 = 16 * odd + (lane >> 3);
  uint16_t* at = out + (row0 + t0) * p.ld_out + c;
  uint4 x[4];
#pragma unroll
  for (int i = 0; i < 4; i++) x[i] = *reinterpret_cast<const uint4*>(stg + (t0 + 4 * i) * 144 + (lane & 7) * 16);
  if (valid >= 32 && col - 32 * odd + 64 <= p.N) {
#pragma unroll
    for (int i = 0; i < 4; i++) *reinterpret_cast<uint4*>(at + 4 * i * p.ld_out) = x[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (t0 + 4 * i < valid && c < p.N) *reinterpret_cast<uint4*>(at + 4 * i * p.ld_out) = x[i];
  }
  named_bar(bar, 64);  // the buffer is free
}

// Whether both of a pair's warps have `ok`; both always come here, so neither
// waits at a later barrier for one that gave up.
__device__ __forceinline__ bool both_ok(bool ok, int bar) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, %2, 64, p;\n\t"
               "selp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"((uint32_t)ok), "r"(bar) : "memory");
  return r != 0;
}

// The same block in fp32, stored or added.  A lane holds a feature's 32 tokens
// (tcgen05.ld 32x32b), so each token's row piece is a whole 128-byte line
// without staging.  Loads and whole blocks' stores have no conditions: under a
// condition of its own each became a branch of its own and waited for the one
// before (128 experts, 805 MB added to: 895 us, without 702).
struct F32Block {
  float* at;  // this lane's first value
  int rows;   // valid ones from there on, at least one
  bool in;    // the lane's feature is one
};
__device__ __forceinline__ F32Block f32_block(const RaggedK& p, float* out, int lane, int64_t row0, int valid,
                                              int64_t col) {
  return F32Block{out + row0 * p.ld_out + col + lane, valid, col + lane < p.N};
}
__device__ __forceinline__ void load_block_f32(const RaggedK& p, const F32Block& b, float (&old)[32]) {
  if (!b.in) return;
  if (b.rows >= 32) {
#pragma unroll
    for (int t = 0; t < 32; t++) old[t] = __ldcg(b.at + t * p.ld_out);
  } else {
#pragma unroll
    for (int t = 0; t < 32; t++) old[t] = __ldcg(b.at + (t < b.rows ? t : 0) * p.ld_out);
  }
}
__device__ __forceinline__ void store_block_f32(const RaggedK& p, const F32Block& b, const float (&v)[32]) {
  if (!b.in) return;
  if (b.rows >= 32) {
#pragma unroll
    for (int t = 0; t < 32; t++) b.at[t * p.ld_out] = v[t];
  } else {
#pragma unroll
    for (int t = 0; t < 32; t++)
      if (t < b.rows) b.at[t * p.ld_out] = v[t];
  }
}

// Ask for bytes [a, a + n) in L2; a and n are multiples of 16.
__device__ __forceinline__ void prefetch_l2(const void* a, uint32_t n) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" :: "l"(a), "r"(n) : "memory");
}

// Segment ends -> shared memory: seg[g] .. seg[g + 1] is expert g's segment,
// pref[g] the row tiles (WGRAD: the rows) of the experts before g.  A
// segment that decreases, begins before an earlier one's end or passes R
// counts nothing and is reported.
template <int MODE>
__device__ __forceinline__ void ragged_tables(const RaggedK& p, int32_t* seg, int32_t* pref, uint16_t* ord, int32_t* count,
                                              bool report) {
  if (p.offsets == nullptr) {  // one segment
    if (threadIdx.x == 0) {
      seg[0] = pref[0] = 0;
      seg[1] = (int32_t)p.R;
      pref[1] = MODE == RAGGED_WGRAD ? (int32_t)p.R : (int32_t)((p.R + p.tw - 1) / p.tw);
      ord[0] = 0;
    }
    return;
  }
  pdl_wait();
  bool wrong = false;
  for (int g = threadIdx.x; g < p.G; g += rg::THREADS) {
    const int32_t s0 = g ? *(p.offsets + g - 1) : 0, s1 = *(p.offsets + g);
    seg[g + 1] = s1;
    wrong |= s0 < 0 || s1 < s0 || (int64_t)s1 > p.R;
  }
  if (threadIdx.x == 0) seg[0] = 0;
  wrong = __syncthreads_or(wrong) != 0;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x >> 5 == 2) {  // the order, beside warp 0's scan and warp 1's allocation
    // A counting sort by the number of bits of the row count, long segments
    // first: within a factor of two is enough for the balance at the end.
    count[lane] = 0;
    __syncwarp();
    for (int g = lane; g < p.G; g += 32) atomicAdd(&count[__clz(max(seg[g + 1] - seg[g], 1))], 1);
    __syncwarp();
    int32_t upto = count[lane];  // class `lane`: 32 - lane bits
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += u;
    }
    count[lane] = upto - count[lane];  // place of the class's next expert
    __syncwarp();
    for (int b = 0; b < p.G; b += 32) {
      const int g = b + lane;
      const int key = g < p.G ? __clz(max(seg[g + 1] - seg[g], 1)) : 32;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, key), below = same & ((1u << lane) - 1u);
      const int first = g < p.G ? count[key] : 0;
      __syncwarp();
      if (g < p.G) {
        ord[first + __popc(below)] = (uint16_t)g;
        if (below == 0) count[key] = first + __popc(same);
      }
      __syncwarp();
    }
  }
  if (threadIdx.x >= 32) return;
  int32_t run = 0, high = 0;  // count and largest end so far
  bool bad = false;
  if (lane == 0) pref[0] = 0;
  for (int b = 0; b < p.G; b += 32) {
    const int g = b + lane;
    const int32_t s0 = g < p.G ? seg[g] : 0, s1 = g < p.G ? seg[g + 1] : 0;
    int32_t top = s0;  // the largest end before segment g
    if (wrong) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xFFFFFFFFu, top, o);
        if (lane >= o && u > top) top = u;
      }
      if (high > top) top = high;
      high = __shfl_sync(0xFFFFFFFFu, top, 31);
    }
    int32_t v = 0;
    if (g < p.G) {
      if (s0 < top || s1 < s0 || (int64_t)s1 > p.R) bad = true;
      else v = MODE == RAGGED_WGRAD ? s1 - s0 : (int32_t)(((uint32_t)(s1 - s0) + (uint32_t)p.tw - 1) / (uint32_t)p.tw);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += u;
    }
    if (g < p.G) pref[g + 1] = run + v;
    run += __shfl_sync(0xFFFFFFFFu, v, 31);
  }
  if (wrong && __any_sync(0xFFFFFFFFu, bad) && lane == 0 && report) atomicOr(&g_ragged_status, DEV_BAD_OFFSETS);
}

// The operands' maps.  P: NK and KN use box[0] only, 3-D (inner, outer,
// expert).  Q: boxes of half a tile's rows, and of 64, 32 and 16 for the
// narrower ones (a CTA's half is a multiple of 16 tokens).  WGRAD, both: boxes
// of 64, 32, 16, 8, 4, 2 and 1 rows of 64 columns.
struct RaggedMaps {
  CUtensorMap box[7];
};

// One operand's copies into the stage ring of this CTA (one warp).  Warp 0
// copies P, warp 3 Q: one thread issuing both was the limit where a stage
// takes four copies (weight gradient, G = 128: 397 -> 367 us).
template <int MODE, bool F32, bool IS_P, bool SPLIT>
__device__ __forceinline__ void ragged_copies(const RaggedMaps& tm, const RaggedK& p,
                                              uint8_t* smem, uint32_t rank, uint32_t first) {
  using namespace rg;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* empty = full + ST;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  // Operands stay in L2 ahead of the outputs, which would push them out while
  // other tiles still need them (us, and under the default policy: forward 276,
  // 280, weight gradient 287, 301); weights that meet one tile of rows only do not
  // stay (61 tokens 125.2 -> 120.0 us).
  const uint64_t pol = IS_P && MODE != RAGGED_WGRAD && p.w_once ? l2_policy_evict_first() : l2_policy_evict_last();
  uint8_t* const ring = smem + (IS_P ? 0 : OFF_Q);
  const bool leader = rank == 0;
  RaggedTile T;
  RaggedSource<MODE, F32, SPLIT> feed(p, smem);
  int stage = 0;
  uint32_t phase = 0, used = 0;  // stages copied into
  bool ready = false;  // the next stage has already been seen to be free
  const uint32_t full0 = SPLIT ? cta_addr(&full[0], first) : leader_addr(&full[0]);
  bool ok = true;
  while (ok && feed.next(&T)) {
    const int half = T.nt >> 1;                       // Q rows of this CTA
    const int boxes = IS_P ? 2 : (half + 63) >> 6;    // MN-major boxes of 64
    const uint32_t bytes = IS_P ? P_BYTES : (MODE == RAGGED_WGRAD ? boxes * 8192u : half * 128u);
    const int x = IS_P ? T.f0 + 128 * (int)rank : (int)T.t0 + half * (int)rank;
    int k = T.k0;
    const int tell = T.nk > AHEAD ? T.nk - AHEAD : 0;
    if constexpr (IS_P && !SPLIT) {
      if (T.nk == 0) feed.near_end();
    }
    for (int kb = 0; kb < T.nk; kb++, k += BK) {
      if constexpr (IS_P && !SPLIT) {
        if (kb == tell) feed.near_end();
      }
      if (!ready && !ragged_wait<false>(&empty[stage], phase ^ 1u, abort_flag)) { ok = false; break; }
      uint8_t* const dst = ring + stage * P_BYTES;
      const int here = stage;
      used |= 1u << here;
      if (++stage == ST) { stage = 0; phase ^= 1u; }
      const uint32_t free_next = mbar_try(&empty[stage], phase ^ 1u);  // polled while this stage's copies are issued
      const uint32_t fb = full0 + 8u * here;
      const bool pieces = MODE == RAGGED_WGRAD && kb == T.nk - 1 && (T.rem & 15) != 0;
      if (MODE == RAGGED_WGRAD && pieces) {
        // A lane per piece: the segment's last rows by the bits of their number
        // (lanes 0..5 of a box's 16: 32, 16, .. 1 rows), then the zeros (6..9: 8, 4, 2, 1).
        // (One lane issuing them in turn took 3000 cycles a tile.)
        const int lane = threadIdx.x & 31, i = lane & 15, zeros = 16 - (T.rem & 15);
        if (leader && elect_one_lane()) mbar_arrive_expect_tx(&full[here], (uint32_t)(boxes * 256 * ((T.rem + 15) & ~15)));
        __syncwarp();
        const int rows = i < 6 ? 32 >> i : 8 >> (i - 6);  // of this lane's piece
        const int of = i < 6 ? T.rem : zeros, before = of & -(2 * rows);
        if (i < 10 && (of & rows) && lane >> 4 < boxes)
          tma2_load_2d(dst + (lane >> 4) * 8192 + (before + (i < 6 ? 0 : T.rem)) * 128, &tm.box[i < 6 ? i + 1 : i - 3],
                       i < 6 ? x + 64 * (lane >> 4) : 0, i < 6 ? k + before : (int)p.R, fb, pol);
        __syncwarp();
      } else if (elect_one_lane()) {
        if (leader) mbar_arrive_expect_tx(&full[here], 2u * bytes);
        if constexpr (MODE == RAGGED_WGRAD) {
          tma2_load_2d(dst, &tm.box[0], x, k, fb, pol);
          if (boxes > 1) tma2_load_2d(dst + 8192, &tm.box[0], x + 64, k, fb, pol);
        } else if constexpr (IS_P && MODE == RAGGED_NK) {
          tma2_load_3d_hint(dst, &tm.box[0], k, x, T.g, fb, pol);
        } else if constexpr (IS_P) {
          tma2_load_3d_hint(dst, &tm.box[0], x, k, T.g, fb, pol);
          tma2_load_3d_hint(dst + 8192, &tm.box[0], x + 64, k, T.g, fb, pol);
        } else if (2 * half == p.tw) {
          tma2_load_2d(dst, &tm.box[0], k, x, fb, pol);
        } else {
          int row = 0;
#pragma unroll
          for (int j = 1; j < 4; j++) {
            if (half & (128 >> j)) {
              tma2_load_2d(dst + row * 128, &tm.box[j], k, x + row, fb, pol);
              row += 128 >> j;
            }
          }
        }
      }
      ready = __all_sync(0xFFFFFFFFu, free_next != 0);
    }
  }
  volatile int no_abort = 0;
  // Every copy has landed before the CTA leaves (the drain ignores the abort
  // flag).  Stages before the current one were last filled in this round of
  // the ring, the others in the one before.
  for (int s = 0; s < ST; s++)
    if (leader && (used >> s & 1u)) ragged_wait<false>(&full[s], s < stage ? phase : phase ^ 1u, &no_abort);
}

// The end of a tile whose contraction `splits` pairs of a cluster have shared:
// 32-token block b is one pair's to finish; the others hand it their sums
// through its shared memory (the stage ring: every pair's loads and MMAs are
// done), and it adds them in the pairs' order.  All threads of the cluster
// come here, also those that have given up or have no tile.
template <bool EPI>
__device__ __forceinline__ void ragged_join(const RaggedK& p, const RaggedTile& T, uint8_t* smem, uint32_t tmem_base,
                                            int warp, int lane, uint32_t rank, uint32_t first, bool mine) {
  using namespace rg;
  const int S = p.splits, pair = (int)(first >> 1), nb = mine ? T.nt >> 5 : 0;
  const int q = warp & 3, h = warp < 8 ? 0 : 1;  // nb is 0 for the other warps
  // both parities of blocks go to each pair where there are enough
  const bool twos = nb >= 2 * S;
  const auto owner = [&](int b) { return (twos ? b >> 1 : b) % S; };
  const auto slot = [&](int b, int from, int to) {  // 16 KB each: 4 warps x 32 lanes x 32 sums
    const int place = twos ? (b >> 1) / S * 2 + (b & 1) : b / S;
    return (place * (S - 1) + (from < to ? from : from - 1)) * 16384 + q * 4096 + lane * 16;
  };
  const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16);
  __syncwarp();
  cluster_sync_all();  // every pair's sums are ready
  tc_fence_after();
  for (int b = h; b < nb; b += 2) {
    const int to = owner(b);
    if (to == pair) continue;
    float v[2][16];
    tmem_ld_16x32(tb + 32 * b, v[0]);
    tmem_ld_16x32(tb + 32 * b + (16u << 16), v[1]);
    tmem_wait_ld();
    const uint32_t dst = cta_addr(smem + slot(b, pair, to), 2u * (uint32_t)to + rank);
#pragma unroll
    for (int j = 0; j < 8; j++)
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};"
                   :: "r"(dst + 512u * j), "f"(v[j >> 2][4 * (j & 3)]), "f"(v[j >> 2][4 * (j & 3) + 1]),
                      "f"(v[j >> 2][4 * (j & 3) + 2]), "f"(v[j >> 2][4 * (j & 3) + 3]) : "memory");
  }
  __syncwarp();
  cluster_sync_all();  // every block's sums are with its owner
  const int64_t col = T.f0 + 128 * rank + 32 * q;
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if constexpr (EPI) {
    if (mine && p.epi.bias) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int64_t f = col + (lane >> 2) + 8 * i;
        if (f < p.N) bias[i] = bf16_bits_to_float(*(p.epi.bias + f));
      }
    }
  }
  for (int b = h; b < nb; b += 2) {
    if (owner(b) != pair) continue;
    const int64_t row0 = T.t0 + 32 * b;
    const int valid = T.valid - 32 * b < 32 ? T.valid - 32 * b : 32;
    uint4 res[4];
    if (EPI && p.epi.res) load_residual(p, res, lane, row0, T.valid - 32 * b, col);
    float v[2][16];
    tmem_ld_16x32(tb + 32 * b, v[0]);
    tmem_ld_16x32(tb + 32 * b + (16u << 16), v[1]);
    tmem_wait_ld();
    for (int from = 0; from < S; from++) {
      if (from == pair) continue;
      const float4* src = reinterpret_cast<const float4*>(smem + slot(b, from, pair));
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float4 x = src[32 * j];
        v[j >> 2][4 * (j & 3)] += x.x;
        v[j >> 2][4 * (j & 3) + 1] += x.y;
        v[j >> 2][4 * (j & 3) + 2] += x.z;
        v[j >> 2][4 * (j & 3) + 3] += x.w;
      }
    }
    store_block_bf16<EPI>(p, v, smem + OFF_STG + ((warp - 4) & ~1) * STG, lane, warp & 1, 1 + ((warp - 4) >> 1), bias,
                          res, static_cast<uint16_t*>(p.out), row0, valid, col);
  }
}

template <int MODE, bool EPI, bool F32, bool SPLIT>
__device__ __forceinline__ void ragged_body(const RaggedMaps& tmP, const RaggedMaps& tmQ, const RaggedK& p) {
  using namespace rg;
  constexpr bool P_MN = MODE != RAGGED_NK, Q_MN = MODE == RAGGED_WGRAD;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);  // leader's: the stage is in both CTAs' shared memory
  uint64_t* empty = full + ST;      // both CTAs: the stage's MMAs are done
  uint64_t* acc_full = empty + ST;  // both CTAs: the tile's MMAs are done
  uint64_t* acc_empty = acc_full + 2;  // leader's: both CTAs' epilogue warps have read the accumulator
  uint64_t* final_bar = acc_empty + 2;
  int32_t* seg = reinterpret_cast<int32_t*>(smem + OFF_SEG);
  int32_t* pref = reinterpret_cast<int32_t*>(smem + OFF_PREF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  const uint32_t rank = SPLIT ? cluster_rank() & 1u : cluster_rank();  // in the pair
  const uint32_t first = SPLIT ? cluster_rank() & ~1u : 0;             // the pair's leader
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int j = 0; j < (Q_MN ? 7 : 1); j++) prefetch_tensormap(&tmP.box[j]);
    for (int j = 0; j < (Q_MN ? 7 : 4); j++) prefetch_tensormap(&tmQ.box[j]);
    for (int s = 0; s < ST; s++) { mbar_init(&full[s], 2); mbar_init(&empty[s], 1); }
    for (int a = 0; a < 2; a++) { mbar_init(&acc_full[a], 1); mbar_init(&acc_empty[a], 16); }
    mbar_init(final_bar, 1);
    const RaggedSched sched = ragged_sched(smem);
    for (int i = 0; i < SLOTS; i++) { mbar_init(&sched.full[i], 1); mbar_init(&sched.empty[i], 2); }
    mbar_init(sched.empty + SLOTS, 1);
    const RaggedFeed tiles(p, smem);
    for (int i = 0; i < TILES; i++) {
      mbar_init(&tiles.full[i], 1);
      mbar_init(&tiles.empty[i], leader ? 11 : 10);  // the copy and epilogue warps, the leader's MMA warp
      mbar_init(&tiles.ending[i], 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  pdl_trigger();
  ragged_tables<MODE>(p, seg, pref, reinterpret_cast<uint16_t*>(smem + OFF_ORD),
                      reinterpret_cast<int32_t*>(smem + OFF_STG), blockIdx.x == 0);
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers are initialised before any remote arrive or copy; the tables are built
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem_base = *tmem_slot;
  RaggedTile T;
  RaggedSource<MODE, F32, SPLIT> feed(p, smem);
  bool mine = false;  // SPLIT, epilogue warps: the pair's sums are there

  if (warp == 0) {
    ragged_copies<MODE, F32, true, SPLIT>(tmP, p, smem, rank, first);
  } else if (!SPLIT && warp == 2) {
    ragged_tiles<MODE, F32>(p, smem, leader);
  } else if (warp == 3) {
    ragged_copies<MODE, F32, false, SPLIT>(tmQ, p, smem, rank, first);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs (leader)
    if (leader) {
      // K-major: 8-row groups 1024 bytes apart, a 16-step 32 bytes on.
      // MN-major: 64-wide column blocks 8192 bytes apart, groups of 8 steps
      // 1024 bytes apart, a 16-step 2048 bytes on.
      const uint64_t pd0 = smem_desc(smem_u32(smem), P_MN ? 8192 : 16, 1024, 2);
      const uint64_t qd0 = smem_desc(smem_u32(smem + OFF_Q), Q_MN ? 8192 : 16, 1024, 2);
      constexpr uint64_t p_step = P_MN ? 128 : 2, q_step = Q_MN ? 128 : 2;
      // fp32 accumulator, BF16 operands, M = 256
      constexpr uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | ((P_MN ? 1u : 0u) << 15) |
                                  ((Q_MN ? 1u : 0u) << 16) | (16u << 24);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, ready = false;  // the next stage has already been seen to be full
      while (ok && feed.next(&T)) {
        if (T.nk == 0) continue;
        if (!ragged_wait<true>(&acc_empty[acc], acc_phase ^ 1u, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t idesc = idesc0 | ((uint32_t)(T.nt >> 3) << 17);
        const uint32_t d = tmem_base + (uint32_t)(acc * 256);
        for (int kb = 0; kb < T.nk; kb++) {
          const bool last = kb == T.nk - 1;
          if (!ready && !ragged_wait<false>(&full[stage], phase, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint64_t pd = pd0 + (uint64_t)((stage * P_BYTES) >> 4), qd = qd0 + (uint64_t)((stage * Q_BYTES) >> 4);
          uint64_t* const done = &empty[stage];
          if (++stage == ST) { stage = 0; phase ^= 1u; }
          const uint32_t next = mbar_try(&full[stage], phase);  // polled while this stage's MMAs are issued
          if (elect_one_lane()) {
            tc2_mma_bf16(d, pd, qd, idesc, kb != 0 ? 1u : 0u);
            if (!last) {
              tc2_mma_bf16(d, pd + p_step, qd + q_step, idesc, 1u);
              tc2_mma_bf16(d, pd + 2 * p_step, qd + 2 * q_step, idesc, 1u);
              tc2_mma_bf16(d, pd + 3 * p_step, qd + 3 * q_step, idesc, 1u);
              tc2_commit_pair(done, first);
            } else {
              if (T.rem > 16) tc2_mma_bf16(d, pd + p_step, qd + q_step, idesc, 1u);
              if (T.rem > 32) tc2_mma_bf16(d, pd + 2 * p_step, qd + 2 * q_step, idesc, 1u);
              if (T.rem > 48) tc2_mma_bf16(d, pd + 3 * p_step, qd + 3 * q_step, idesc, 1u);
              tc2_commit_pair(done, first);
              tc2_commit_pair(&acc_full[acc], first);
            }
          }
          ready = __all_sync(0xFFFFFFFFu, next != 0);
        }
        if (!ok) break;
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok) *abort_flag = 1;
      // No MMA may still be writing either CTA's tensor memory when it is freed.
      volatile int no_abort = 0;
      if (elect_one_lane()) tc2_commit_local(final_bar);
      __syncwarp();
      ragged_wait<false>(final_bar, 0, &no_abort);
    }
  } else if (SPLIT && warp >= 4) {
    if (feed.next(&T)) mine = both_ok(ragged_wait<false>(&acc_full[0], 0, abort_flag), 1 + ((warp - 4) >> 1));
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3, h = (warp - 4) >> 2;  // lane quarter (32 features), parity of the 32-token blocks
    const int odd = warp & 1, bar = 1 + ((warp - 4) >> 1);  // the warp's place in its pair, the pair's barrier
    uint8_t* stg = smem + OFF_STG + ((warp - 4) & ~1) * STG;
    int acc = 0;
    uint32_t acc_phase = 0;
    while (feed.next(&T)) {
      const int64_t col = T.f0 + 128 * rank + 32 * q;
      float bias[4] = {0.f, 0.f, 0.f, 0.f};
      if constexpr (EPI) {
        if (p.epi.bias) {
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int64_t f = col + (lane >> 2) + 8 * i;
            if (f < p.N) bias[i] = bf16_bits_to_float(*(p.epi.bias + f));
          }
        }
      }
      const int nb = T.nt >> 5;
      uint4 res[4];
      const auto valid_of = [&](int b) { return T.valid - 32 * b < 32 ? T.valid - 32 * b : 32; };
      const int64_t base = MODE == RAGGED_WGRAD ? ((int64_t)T.split * p.G + T.g) * p.K * p.ld_out : 0;
      const bool add = F32 && (p.accumulate || T.part > 0);
      if (add && T.nk == 0) continue;  // nothing to add
      float old[32] = {};
      if (F32 && add && h < nb)
        load_block_f32(p, f32_block(p, static_cast<float*>(p.out) + base, lane, T.t0 + 32 * h, valid_of(h), col), old);
      if (EPI && p.epi.res && h < nb) load_residual(p, res, lane, T.t0 + 32 * h, T.valid - 32 * h, col);
      if (T.nk > 0) {
        if (!both_ok(ragged_wait<false>(&acc_full[acc], acc_phase, abort_flag), bar)) break;
        tc_fence_after();
      }
      if (F32 && p.fetch_old && add && T.part == 0) {
        const int row = 64 + (warp - 4) * 32 + lane;
        const int64_t f = T.f0 + 128 * rank;
        if (row < T.valid && f < p.N)
          prefetch_l2(static_cast<const float*>(p.out) + base + (T.t0 + row) * p.ld_out + f,
                      (uint32_t)(p.N - f < 128 ? p.N - f : 128) * 4u);
      }
      const uint32_t tb = tmem_base + (uint32_t)(acc * 256) + ((uint32_t)(q * 32) << 16);
      const uint32_t hand_back = leader_addr(&acc_empty[acc]);
      if (T.nk > 0 && h >= nb && lane == 0) arrive_on_leader_relaxed(hand_back);
      for (int b = h; b < nb; b += 2) {
        float v[2][16], w[32];  // of one block, w in fp32 outputs' order
        if (T.nk > 0) {
          if constexpr (F32) {
            uint32_t u[32];
            tmem_ld32(tb + 32 * b, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i++) w[i] = __uint_as_float(u[i]);
          } else {
            tmem_ld_16x32(tb + 32 * b, v[0]);
            tmem_ld_16x32(tb + 32 * b + (16u << 16), v[1]);
            tmem_wait_ld();
          }
          if (b + 2 >= nb) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_on_leader_relaxed(hand_back);
          }
        } else {  // an expert without rows: zeros
#pragma unroll
          for (int i = 0; i < 16; i++) v[0][i] = v[1][i] = w[i] = w[16 + i] = 0.f;
        }
        const int64_t row0 = T.t0 + 32 * b;
        const int valid = valid_of(b);
        uint4 next[4];
        if (EPI && p.epi.res && b + 2 < nb) load_residual(p, next, lane, row0 + 64, T.valid - 32 * b - 64, col);
        if constexpr (F32) {
          if (add) {
#pragma unroll
            for (int i = 0; i < 32; i++) w[i] += old[i];
            if (b + 2 < nb)
              load_block_f32(p, f32_block(p, static_cast<float*>(p.out) + base, lane, row0 + 64, valid_of(b + 2), col),
                             old);
          }
          store_block_f32(p, f32_block(p, static_cast<float*>(p.out) + base, lane, row0, valid, col), w);
        } else
          store_block_bf16<EPI>(p, v, stg, lane, odd, bar, bias, res, static_cast<uint16_t*>(p.out) + base, row0,
                                valid, col);
        if (EPI && p.epi.res) {
#pragma unroll
          for (int i = 0; i < 4; i++) res[i] = next[i];
        }
      }
      if (T.nk > 0) {
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
    }
  }
  if constexpr (SPLIT) ragged_join<EPI>(p, T, smem, tmem_base, warp, lane, rank, first, mine);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) atomicOr(&g_ragged_status, DEV_TIMEOUT);
  cluster_sync_all();  // neither CTA frees tensor memory or exits while the other still uses the pair
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" :: "r"(tmem_base) : "memory");
}

template <int MODE, bool EPI, bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(rg::THREADS, 1)
ragged_kernel(const __grid_constant__ RaggedMaps tmP, const __grid_constant__ RaggedMaps tmQ, const RaggedK p) {
  ragged_body<MODE, EPI, F32, false>(tmP, tmQ, p);
}
template <int MODE, bool EPI>
__global__ void __launch_bounds__(rg::THREADS, 1)
ragged_split_kernel(const __grid_constant__ RaggedMaps tmP, const __grid_constant__ RaggedMaps tmQ, const RaggedK p) {
  ragged_body<MODE, EPI, false, true>(tmP, tmQ, p);
}

// The tile width for `rows` output rows in `segments` pieces under n_f column
// tiles: the one with the least waves x (width + 64).  A tile costs its width
// in MMA time and about 64 columns' worth besides; narrow tiles pay where wide
// ones leave pairs idle (777 rows, 5120 -> 2048, a pair to each tile: 32 tiles of
// 256 on 76 pairs, 31 us; 72 of 96, 22 us; that shape's tiles are shared by now,
// tile_shape below).  Past four waves the width is 256: fewer bytes
// to load per product.
static int tile_width(int64_t rows, int64_t segments, int64_t n_f, int pairs) {
  int best = 256;
  int64_t cost = -1;
  for (int w = 256; w >= 32; w -= 32) {
    const int64_t tiles = (rows + (int64_t)segments * w - 1) / w * n_f, waves = (tiles + pairs - 1) / pairs;
    if (w == 256 && waves > 4) break;
    if (cost < 0 || waves * (w + 64) < cost) {
      cost = waves * (w + 64);
      best = w;
    }
  }
  return best;
}

// Row tiles of width w for `rows` rows in up to `segments` pieces (0: one
// piece), at most.
static int64_t row_tiles(int64_t rows, int64_t segments, int64_t w) {
  return segments ? rows / w + segments : (rows + w - 1) / w;
}

// Clusters of 2 x splits CTAs that run at the same time.
constexpr int MAX_SPLITS = 4;
static cudaError_t resident_clusters(int splits, int* n) {
  static std::atomic<int> known[MAX_SPLITS + 1];
  if ((*n = known[splits].load(std::memory_order_relaxed)) != 0) return cudaSuccess;
  cudaError_t e = ensure_smem_attr<ragged_split_kernel<RAGGED_NK, true>>(rg::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2u * (unsigned)splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2u * (unsigned)splits);
  cfg.blockDim = dim3(rg::THREADS);
  cfg.dynamicSmemBytes = rg::SMEM;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(n, ragged_split_kernel<RAGGED_NK, true>, &cfg);
  if (e == cudaSuccess) known[splits].store(*n, std::memory_order_relaxed);
  return e;
}

// A tile's width and the pairs that share its contraction.  Where the tiles
// leave pairs idle, clusters of 2, 3 or 4 pairs take a tile each, a part of
// the contraction per pair, and join their sums through shared memory.  The
// cost in units of 0.4 ns, from sweeps of widths and splits: a 64-step block
// w + 450 (how long its loads are on their way), joining 4000 + 15 w splits,
// and all clusters must run at once (36, 23 and 15 of them).  Whole against
// split, us: 16 rows, 16384 -> 4096, 54.1, 29.5 (three pairs a tile); 128 rows,
// 5120 -> 2048, 19.2, 12.8; 777 rows, 21.2, 19.7 (20.0 to 20.6 on other boards); 600 rows, 8192 -> 1024, 29.1,
// 17.6; 53 rows, 2944 -> 128, 10.9, 7.7; 64 rows, 512 -> 256, 4.7, 6.0.
struct TileShape { int width, splits; };
static cudaError_t tile_shape(int64_t rows, int64_t segments, int64_t n_f, int64_t nk, int pairs, TileShape* best) {
  *best = TileShape{tile_width(rows, segments ? segments : 1, n_f, pairs), 1};
  const int64_t whole = row_tiles(rows, segments, best->width) * n_f;
  if (whole > pairs) return cudaSuccess;
  int64_t least = nk * (best->width + 450) * 19 / 20;
  for (int s = 2; s <= MAX_SPLITS && 2 * s <= nk; s++) {
    int clusters;
    const cudaError_t e = resident_clusters(s, &clusters);
    if (e != cudaSuccess) return e;
    for (int w = 32; w <= 256; w += 32) {
      const int64_t cost = (nk + s - 1) / s * (w + 450) + 4000 + 15 * w * s;
      if (row_tiles(rows, segments, w) * n_f <= clusters && cost < least) {
        least = cost;
        *best = TileShape{w, s};
      }
    }
  }
  return cudaSuccess;
}

template <int MODE, bool EPI, bool F32>
static cudaError_t launch_ragged(const RaggedK& p, const RaggedMaps& tp, const RaggedMaps& tq, int64_t tiles,
                                 cudaStream_t s) {
  if (tiles >= (1ll << 30)) return cudaErrorInvalidValue;
  const cudaError_t e = ensure_smem_attr<ragged_kernel<MODE, EPI, F32>>(rg::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(ragged_kernel<MODE, EPI, F32>, dim3((unsigned)(2 * tiles)), rg::THREADS, rg::SMEM, s, dim3(1), tp, tq, p);
}
template <int MODE, bool EPI>
static cudaError_t launch_split(const RaggedK& p, const RaggedMaps& tp, const RaggedMaps& tq, int64_t tiles,
                                cudaStream_t s) {
  const cudaError_t e = ensure_smem_attr<ragged_split_kernel<MODE, EPI>>(rg::SMEM);
  if (e != cudaSuccess) return e;
  const unsigned ctas = 2u * (unsigned)p.splits;
  return launch_pdl(ragged_split_kernel<MODE, EPI>, dim3((unsigned)tiles * ctas), rg::THREADS, rg::SMEM, s, dim3(ctas), tp,
                    tq, p);
}

// BF16 matrix [outer, inner] (row stride ld elements), optionally a stack of
// `batch` of them, as 128-byte swizzled boxes of 64 x box_rows.
static bool bf16_map(CUtensorMap* m, const void* base, int64_t inner, int64_t outer, int64_t ld, int64_t batch,
                     int box_rows) {
  TensorMapShape s{};
  s.rank = batch > 0 ? 3 : 2;
  s.dims[0] = (uint64_t)inner; s.dims[1] = (uint64_t)outer; s.dims[2] = (uint64_t)batch;
  s.strides[0] = (uint64_t)ld * 2; s.strides[1] = (uint64_t)outer * (uint64_t)ld * 2;
  s.box[0] = 64; s.box[1] = (uint32_t)box_rows; s.box[2] = 1;
  return encode_bf16_map(m, base, s) == MX_OK;
}

// Whether the kernel for few rows is the faster one (us there, on tiles).
static bool few_rows(const RaggedParams& p, int pairs) {
  if (p.R <= 8) return true;
  const int64_t n_f = (p.N + 255) / 256, weights = 2 * p.N * p.K;
  if (p.offsets) {
    // Mostly empty experts (16 rows of 128 experts, 2048 -> 1536: 19.5, 25.0; 64
    // rows 58.0, 57.6), or few tiles of which each meets a handful of rows (16 rows
    // of 8 experts 10.8, 12.9; 32 rows 12.0, 13.7; 64 rows 15.3, 13.8; 64 rows of
    // 64 experts, 512 -> 768, 13.4, 11.3).
    return 2 * p.R <= p.G || (p.R <= 4 * (int64_t)p.G && (p.G < p.R ? p.G : p.R) * n_f <= pairs);
  }
  // 16 rows, 2048 -> 2048: 4.9, 8.4; 16384 -> 4096: 26.1, 29.6; 4096 -> 16384, where
  // the tiles fill the pairs: 28.4, 25.2.  32 rows, 2048 -> 2048: 6.9, 8.4; 512 ->
  // 512: 2.4, 4.7; 5120 -> 2048: 13.0, 11.1.
  if (p.R <= 16) return weights <= 64000000 || 3 * n_f < 2 * pairs;
  return p.R <= 32 && weights <= 12000000;
}

cudaError_t launch_ragged_gemm(const RaggedParams& p, int num_sms, cudaStream_t s) {
  if (!p.w_kn && few_rows(p, num_sms / 2)) return launch_skinny(p, s);
  RaggedK k{};
  k.G = p.G; k.offsets = p.offsets;
  k.R = p.R; k.N = p.N; k.K = p.K;
  k.n_f = (int)((p.N + 255) / 256);
  k.out = p.out; k.ld_out = p.ld_out;
  k.epi = p.epi;
  // each segment ends in one tile of its own at most
  const int64_t own = p.offsets ? (p.G < p.R ? p.G : p.R) : 1;
  TileShape shape;
  const cudaError_t e = tile_shape(p.R, p.offsets ? own : 0, k.n_f, (p.K + rg::BK - 1) / rg::BK, num_sms / 2, &shape);
  if (e != cudaSuccess) return e;
  k.tw = shape.width;
  k.splits = shape.splits;
  k.w_once = p.R <= 32 * (p.offsets ? (int64_t)p.G : 1);
  RaggedMaps tp, tq;
  if (!(p.w_kn ? bf16_map(&tp.box[0], p.w, p.N, p.K, p.N, p.G, 64)
               : bf16_map(&tp.box[0], p.w, p.K, p.N, p.K, p.G, 128)) ||
      !bf16_map(&tq.box[0], p.a, p.K, p.R, p.ld_a, 0, k.tw / 2))
    return cudaErrorInvalidValue;
  for (int j = 1; j < 4; j++)
    if (!bf16_map(&tq.box[j], p.a, p.K, p.R, p.ld_a, 0, 128 >> j)) return cudaErrorInvalidValue;
  const int64_t tiles = row_tiles(p.R, p.offsets ? own : 0, k.tw) * k.n_f;
  const bool epi = p.epi.bias || p.epi.act != MX_ACT_NONE || p.epi.res || p.epi.q;
  if (k.splits > 1)
    return p.w_kn ? launch_split<RAGGED_KN, false>(k, tp, tq, tiles, s)
           : epi  ? launch_split<RAGGED_NK, true>(k, tp, tq, tiles, s)
                  : launch_split<RAGGED_NK, false>(k, tp, tq, tiles, s);
  if (p.w_kn) return launch_ragged<RAGGED_KN, false, false>(k, tp, tq, tiles, s);
  return epi ? launch_ragged<RAGGED_NK, true, false>(k, tp, tq, tiles, s)
             : launch_ragged<RAGGED_NK, false, false>(k, tp, tq, tiles, s);
}

// Parts that every segment is cut into when an output has few tiles: a single
// [512, 512] gradient is 4 tiles on 76 pairs, each summing all rows.  Every
// part sums its rows into an fp32 gradient of its own in the workspace, and a
// second launch adds them in order.  Worth it where it takes 2048 rows or more
// off a pair's sums (whole against split, us: [512, 512] from 65536 rows 210,
// 38; from 4096 rows 17.1, 12.6; two halves of 2048 rows 11.2, 12.1; 8
// gradients of [512, 512] from 16384 rows 14.9, 17.6).
constexpr int PAIRS = 76;  // GB300: 152 SMs
static int wgrad_splits(int64_t N, int64_t K, int64_t R, int64_t G) {
  const int64_t tiles = G * ((K + 255) / 256) * ((N + 255) / 256);
  int64_t s = PAIRS / tiles;
  if (s > R / (G * 1024)) s = R / (G * 1024);
  return s < 2 || R / G * (s - 1) / s < 2048 ? 1 : (int)s;
}

size_t ragged_wgrad_workspace(int64_t N, int64_t K, int64_t R, int G) {
  const int s = wgrad_splits(N, K, R, G);
  return s > 1 ? (size_t)s * (size_t)G * (size_t)N * (size_t)K * sizeof(float) : 0;
}

// grad (+)= the parts' sums, in order; n is a multiple of 4.
template <bool F32>
__global__ void __launch_bounds__(256) wgrad_sum_kernel(const float* parts, int splits, int64_t n, void* grad,
                                                        int accumulate) {
  pdl_trigger();
  pdl_wait();
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * 1024) {
    float4 t = *reinterpret_cast<const float4*>(parts + i);
#pragma unroll 4
    for (int s = 1; s < splits; s++) {
      const float4 v = *reinterpret_cast<const float4*>(parts + s * n + i);
      t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
    }
    if constexpr (F32) {
      float4* g = reinterpret_cast<float4*>(static_cast<float*>(grad) + i);
      if (accumulate) {
        // zero leaves the bits alone, as an empty segment has to
        const float4 v = *g;
        t.x = t.x == 0.f ? v.x : t.x + v.x;
        t.y = t.y == 0.f ? v.y : t.y + v.y;
        t.z = t.z == 0.f ? v.z : t.z + v.z;
        t.w = t.w == 0.f ? v.w : t.w + v.w;
      }
      *g = t;
    } else {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(grad) + i) =
          make_uint2(float2_to_bf16x2(t.x, t.y), float2_to_bf16x2(t.z, t.w));
    }
  }
}

cudaError_t launch_ragged_wgrad(const RaggedWgradParams& p, int num_sms, cudaStream_t s) {
  RaggedK k{};
  k.G = p.G; k.offsets = p.offsets;
  k.R = p.R;
  k.N = p.K;  // the output's columns
  k.K = p.N;  // its rows
  k.n_f = (int)((p.K + 255) / 256);
  k.splits = wgrad_splits(p.N, p.K, p.R, p.G);
  k.tw = k.splits > 1 ? 256 : tile_width(p.N, 1, k.n_f * (int64_t)p.G, num_sms / 2);
  k.n_t = (int)((p.N + k.tw - 1) / k.tw);
  k.out = k.splits > 1 ? p.workspace : p.grad ? static_cast<void*>(p.grad) : p.grad_f32;
  k.ld_out = p.K;
  k.accumulate = k.splits > 1 ? 0 : p.accumulate;
  // What a tile is added to is asked for in one go, in pieces of 512 bytes,
  // once its sums are ready (not before, when its operands are on their way).
  // Pays where pairs go through several tiles (us without and with: 128
  // experts of [1536, 2048], 702, 605; 64 of [1024, 1024] with few rows, 103,
  // 84); in one or two narrower tiles it does not (8 of [1000, 520]: 16.2, 17.7).
  k.fetch_old = k.accumulate && k.tw == 256;
  RaggedMaps tp, tq;
  for (int j = 0; j < 7; j++)
    if (!bf16_map(&tp.box[j], p.x, p.K, p.R, p.ld_x, 0, 64 >> j) ||
        !bf16_map(&tq.box[j], p.dy, p.N, p.R, p.ld_dy, 0, 64 >> j))
      return cudaErrorInvalidValue;
  const int64_t tiles = (int64_t)p.G * k.n_f * k.n_t * k.splits;
  if (k.splits == 1)
    return p.grad ? launch_ragged<RAGGED_WGRAD, false, false>(k, tp, tq, tiles, s)
                  : launch_ragged<RAGGED_WGRAD, false, true>(k, tp, tq, tiles, s);
  const cudaError_t e = launch_ragged<RAGGED_WGRAD, false, true>(k, tp, tq, tiles, s);
  if (e != cudaSuccess) return e;
  const int64_t n = (int64_t)p.G * p.N * p.K, blocks = (n / 4 + 255) / 256;
  const dim3 grid((unsigned)(blocks < num_sms * 8 ? blocks : num_sms * 8));
  const float* parts = static_cast<const float*>(p.workspace);
  return p.grad ? launch_pdl(wgrad_sum_kernel<false>, grid, 256, 0, s, dim3(1), parts, k.splits, n, (void*)p.grad, 0)
                : launch_pdl(wgrad_sum_kernel<true>, grid, 256, 0, s, dim3(1), parts, k.splits, n, (void*)p.grad_f32,
                             p.accumulate);
}

cudaError_t read_ragged_status(unsigned* out) { return cudaMemcpyFromSymbol(out, g_ragged_status, sizeof(unsigned)); }
cudaError_t reset_ragged_status() {
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_ragged_status, &zero, sizeof(unsigned));
}

}  // namespace mx
