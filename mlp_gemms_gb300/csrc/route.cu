// The expert routing: each token's k experts from its logits, their weights,
// and the logits' gradient.
#include "mx_internal.h"
#include "vec8.cuh"

namespace mx {

static __device__ unsigned g_route_status = 0;

// A warp takes a token; its lanes hold V consecutive experts each (expert
// lane * V + i, so that the lowest lane and the lowest slot are the lowest
// index), and lane j the j-th choice.

// Floating values as integers in the same order; -0 counts as +0, a NaN above
// everything, and 0 is free for "not there".
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);  // a NaN comes out of the sum as 0x7FFFFFFF
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  if ((b & 0x7FFFFFFFFFFFFFFFull) > 0x7FF0000000000000ull) return ~0ull;
  return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ uint32_t warp_max_key(uint32_t k) { return __reduce_max_sync(0xFFFFFFFFu, k); }
__device__ __forceinline__ uint64_t warp_max_key(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (uint64_t)hi << 32 | lo;
}

// The value of a 32-bit key.
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <typename F> __device__ __forceinline__ F minus_inf();
template <> __device__ __forceinline__ float minus_inf<float>() { return __uint_as_float(0xFF800000u); }
template <> __device__ __forceinline__ double minus_inf<double>() { return __longlong_as_double(0xFFF0000000000000ll); }
template <typename F> struct KeyOf { typedef uint32_t type; };
template <> struct KeyOf<double> { typedef uint64_t type; };

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }
// A sum that is never joined with the product before it: a score and its sum with a bias
// are the same bits in every slot of a lane, so that equal ones tie (joined in some slots
// of the unrolled loops and not in others, they did not).
__device__ __forceinline__ float add_alone(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ double add_alone(double a, double b) { return __dadd_rn(a, b); }
template <typename F> __device__ __forceinline__ F sigmoid_of(F v) { return (F)1 / add_alone((F)1, exp_of(-v)); }

template <typename F>
__device__ __forceinline__ F warp_sum_of(F v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
template <typename F>
__device__ __forceinline__ F warp_max_of(F v) {  // a NaN need not survive
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const F u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = u > v ? u : v;
  }
  return v;
}

__device__ __forceinline__ float load_logit(const RouteParams& p, int64_t t, int e) {
  if (p.x_f32) return *(static_cast<const float*>(p.logits) + t * p.ld + e);
  return bf16_bits_to_float(*(static_cast<const uint16_t*>(p.logits) + t * p.ld + e));
}

// The lane's logits, -Inf past its last expert.
template <int V>
__device__ __forceinline__ void load_logits(const RouteParams& p, int64_t t, int lane, float (&x)[V]) {
  const int e0 = lane * p.per_lane;
  if (p.wide) {  // per_lane == V, every lane's piece aligned to its size (at most 16 bytes)
    if (e0 >= p.G) {
#pragma unroll
      for (int i = 0; i < V; i++) x[i] = minus_inf<float>();
      return;
    }
    constexpr int E = V < 8 ? V : 8;
    if (p.x_f32) {
      const float* q = static_cast<const float*>(p.logits) + t * p.ld + e0;
      if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const uint4 w = load_stream16(q + i);
          x[i] = __uint_as_float(w.x); x[i + 1] = __uint_as_float(w.y);
          x[i + 2] = __uint_as_float(w.z); x[i + 3] = __uint_as_float(w.w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; i++) x[i] = q[i];
      }
    } else {
      const uint16_t* q = static_cast<const uint16_t*>(p.logits) + t * p.ld + e0;
      if constexpr (E == 8) {
#pragma unroll
        for (int i = 0; i < V; i += 8) {
          Raw8<false> r;
          float f[8];
          r.q[0] = load_stream16(q + i);
          unpack_raw8<false>(r, f);
#pragma unroll
          for (int j = 0; j < 8; j++) x[i + j] = f[j];
        }
      } else if constexpr (E == 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(q);
        x[0] = bf16_bits_to_float(w.x & 0xFFFFu); x[1] = __uint_as_float(w.x & 0xFFFF0000u);
        x[2] = bf16_bits_to_float(w.y & 0xFFFFu); x[3] = __uint_as_float(w.y & 0xFFFF0000u);
      } else {
#pragma unroll
        for (int i = 0; i < V; i++) x[i] = bf16_bits_to_float(q[i]);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; i++) {
    const int e = e0 + i;
    x[i] = i < p.per_lane && e < p.G ? load_logit(p, t, e) : minus_inf<float>();
  }
}

// The scores' two numbers for a token: softmax: the largest logit (0 if all are
// -Inf) and 1 / sum of exp(x - it) (0 if that sum is 0); sigmoid: not used.
template <typename F> struct Softmax { F top, inv; };
template <typename F, int V>
__device__ __forceinline__ Softmax<F> softmax_of(const float (&x)[V]) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < V; i++) m = fmaxf(m, x[i]);
  m = warp_max_of(m);
  Softmax<F> s;
  s.top = m == minus_inf<float>() ? (F)0 : (F)m;
  F sum = 0;
#pragma unroll
  for (int i = 0; i < V; i++) sum += exp_of((F)x[i] - s.top);
  sum = warp_sum_of(sum);
  s.inv = sum == (F)0 ? (F)0 : (F)1 / sum;
  return s;
}
// Where scores are weighed and not compared: exp(x - top) as the hardware's power
// of two of the scaled difference (a relative error of 2^-22 and 2 |x - top|
// roundings of 2^-24; results below 2^-126 are 0), an eighth of expf's
// instructions.
__device__ __forceinline__ float exp_near(float d) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d * LOG2E));
  return r;
}
// The exponentials of a row above `top`, its largest logit, and 1 / their sum.
template <int V>
__device__ __forceinline__ float exps_of(const float (&x)[V], float top, float (&e)[V]) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; i++) {
    e[i] = exp_near(x[i] - top);
    sum += e[i];
  }
  sum = warp_sum(sum);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(sum));
  return sum == 0.f ? 0.f : inv;
}
// The largest logit for exps_of; 0 where none is open.
template <int V>
__device__ __forceinline__ float top_of(const float (&x)[V]) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < V; i++) m = fmaxf(m, x[i]);
  m = key_value(__reduce_max_sync(0xFFFFFFFFu, order_key(m)));
  return m == minus_inf<float>() ? 0.f : m;
}
template <typename F, bool SIG>
__device__ __forceinline__ F score_of(float x, const Softmax<F>& s) {
  if constexpr (SIG) return sigmoid_of((F)x);
  else return exp_of((F)x - s.top) * s.inv;
}

// Each lane's share of the softmax over the lanes' own values (-Inf: none): the
// chosen scores over their sum, without the row's sum and without its underflow.
__device__ __forceinline__ float share_above(float xj, float top) {  // top: the largest
  const float e = exp_near(xj - top), total = warp_sum(e);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(total));
  return total == 0.f ? 0.f : e * inv;
}
__device__ __forceinline__ float chosen_share(float xj) {
  const float m = key_value(__reduce_max_sync(0xFFFFFFFFu, order_key(xj)));
  return share_above(xj, m == minus_inf<float>() ? 0.f : m);
}

// Below this sum of sigmoids each of them is below 2^-26, and exp(x) to 2^-26 of
// itself: their shares are a softmax's, where sigmoids leave fp32's range (below -87)
// included.
// (A vote, so that the branch is known to be the warp's: 16384 x 256 sigmoids with bias
// and groups 28.9 us, 29.4 without it.)
constexpr float LOW_SIGMOIDS = 1.f / (1 << 26);

// Each lane's sigmoid over the sum of the lanes' (not `there`: none, xj -Inf; 1 / Inf is
// the division's long way).
__device__ __forceinline__ float sigmoid_share(float xj, bool there) {
  const float w = there ? sigmoid_of(xj) : 0.f, total = warp_sum(w);
  if (__any_sync(0xFFFFFFFFu, total < LOW_SIGMOIDS)) return chosen_share(xj);
  return w / total;
}
// The sigmoids of a row, 0 past its last expert, and 1 / their sum; a low row's in units
// of its largest.
template <int V>
__device__ __forceinline__ float sigmoids_of(const RouteParams& p, const float (&x)[V], int e0, float (&s)[V]) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; i++) {
    s[i] = i < p.per_lane && e0 + i < p.G ? sigmoid_of(x[i]) : 0.f;
    sum += s[i];
  }
  sum = warp_sum(sum);
  if (__any_sync(0xFFFFFFFFu, sum < LOW_SIGMOIDS)) return exps_of<V>(x, top_of<V>(x), s);
  return 1.f / sum;
}

// The largest keys one after the other, the lowest index of equal ones: lane j
// gets the j-th index.  Taken keys become 0.
template <int V, typename K>
__device__ __forceinline__ int take_largest(K (&key)[V], int per_lane, int count, int lane) {
  int mine = 0;
  for (int j = 0; j < count; j++) {
    K m = key[0];
#pragma unroll
    for (int i = 1; i < V; i++) m = key[i] > m ? key[i] : m;
    const K w = warp_max_key(m);
    const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, m == w)) - 1;
    int slot = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; i--) slot = key[i] == w ? i : slot;
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i < V; i++) key[i] = i == slot ? 0 : key[i];
    }
    const int id = owner * per_lane + __shfl_sync(0xFFFFFFFFu, slot, owner);
    mine = lane == j ? id : mine;
  }
  return mine;
}

// Which groups are kept, as a bit mask; *close (fp32): some kept group's value less its
// error is not above some dropped one's with its error.  A group's error goes by its own
// terms, so one far from the border may be the one that is out of place (1000 and -999
// beside groups whose terms are around 1).  `tol`: the scores' part of the error.  c: the
// values of all experts in shared memory.
template <typename F>
__device__ __forceinline__ uint32_t keep_groups(const RouteParams& p, const F* c, int lane, F tol, bool* close) {
  const int size = p.G / p.groups;
  F a = minus_inf<F>(), b = a;
  bool nan = false;
  if (lane < p.groups) {
    int i = lane % size;  // each lane begins elsewhere: its group's start is the same bank as the others'
    for (int n = 0; n < size; n++) {
      const F v = c[lane * size + i];
      nan |= v != v;
      b = v > a ? a : (v > b ? v : b);
      a = v > a ? v : a;
      i = i + 1 == size ? 0 : i + 1;
    }
  }
  F value = p.group_top == 2 ? a + b : a;
  typename KeyOf<F>::type key = nan ? ~(typename KeyOf<F>::type)0 : order_key(value);
  int rank = 0;
  for (int g = 0; g < p.groups; g++) {
    const typename KeyOf<F>::type other = __shfl_sync(0xFFFFFFFFu, key, g);
    rank += other > key || (other == key && g < lane) ? 1 : 0;
  }
  const bool in = lane < p.groups;
  const uint32_t kept = __ballot_sync(0xFFFFFFFFu, in && rank < p.topk_groups);
  *close = false;
  if constexpr (sizeof(F) == 4) {
    // closed groups and those with a NaN are in their exact places
    const bool real = in && !nan && fabsf(value) <= 3e38f;
    const float err = tol + 2.5e-7f * (fabsf(a) + (p.group_top == 2 ? fabsf(b) : 0.f));
    const uint32_t low = __reduce_min_sync(0xFFFFFFFFu, real && rank < p.topk_groups ? order_key(value - err) : ~0u);
    const uint32_t high = __reduce_max_sync(0xFFFFFFFFu, real && rank >= p.topk_groups ? order_key(value + err) : 0u);
    *close = high >= low;
  }
  return kept;
}

// The choice by values that are computed (scores, biased scores) in F.  In
// fp32 two values nearer to each other than their error leave the order open:
// *open is set, and the caller repeats the choice in fp64.
template <int V, bool SIG, typename F>
__device__ __forceinline__ int choose(const RouteParams& p, int64_t t, const float (&x)[V], F* shared, int lane,
                                      bool* open) {
  constexpr bool FAST = sizeof(F) == 4;
  // relative error of a score and of the values compared, twice over: exp's
  // (2 units), the sum's (V + 5 roundings, softmax), the quotient's
  const F err = SIG ? (F)1e-6 : (F)6e-6;
  const int e0 = lane * p.per_lane;
  Softmax<F> s{};
  const bool scored = p.bias != nullptr || (p.groups > 1 && p.group_top == 2);  // else the logits order everything
  if constexpr (!SIG)
    if (scored) s = softmax_of<F, V>(x);
  typename KeyOf<F>::type key[V];
  F c[V];
#pragma unroll
  for (int i = 0; i < V; i++) {
    const int e = e0 + i;
    const bool there = i < p.per_lane && e < p.G;
    c[i] = !scored || x[i] == minus_inf<float>()
               ? (F)x[i]
               : add_alone(score_of<F, SIG>(x[i], s), p.bias != nullptr && there ? (F)*(p.bias + e) : (F)0);
    // without a bias the logits have the scores' order, exactly
    key[i] = there ? order_key(p.bias == nullptr ? (F)x[i] : c[i]) : 0;
  }
  *open = false;
  if (p.groups > 1) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; i++)
      if (i < p.per_lane && e0 + i < p.G)
        shared[e0 + i] = c[i];
    __syncwarp();
    bool close;
    const uint32_t kept = keep_groups<F>(p, shared, lane, err, &close);
    *open = FAST && close && scored;
    const int size = p.G / p.groups;
    int g = e0 / size, in = e0 - g * size;
#pragma unroll
    for (int i = 0; i < V; i++) {
      if (key[i] != 0 && !(kept >> g & 1u)) key[i] = order_key(minus_inf<F>());
      if (++in == size) { in = 0; g++; }
    }
  }
  // one more than k: the first that is left out
  const bool look = FAST && p.bias != nullptr && p.k < p.G && p.k < 32;
  const int id = take_largest(key, p.per_lane, p.k + (look ? 1 : 0), lane);
  if (FAST && p.bias != nullptr) {
    const int count = p.k + (look ? 1 : 0);
    const float xi = lane < count ? load_logit(p, t, id) : 0.f, bi = lane < count ? *(p.bias + id) : 0.f;
    const F si = score_of<F, SIG>(xi, s), ci = si + (F)bi;
    const F ux = __shfl_up_sync(0xFFFFFFFFu, xi, 1), ub = __shfl_up_sync(0xFFFFFFFFu, bi, 1);
    const F us = __shfl_up_sync(0xFFFFFFFFu, si, 1), uc = __shfl_up_sync(0xFFFFFFFFu, ci, 1);
    F most = si > us ? si : us;
    // Behind the first that is left out any expert may stand, with a score up to the
    // largest, that its bias cancels.
    if (look && lane == p.k) most = SIG ? (F)1 : s.inv;
    // equal logits with equal biases are equal for certain; closed experts are -Inf
    const bool near = lane > 0 && lane < count && !(xi == ux && bi == ub) && xi != minus_inf<float>() &&
                      uc - ci <= err * most + (F)2.5e-7 * ((uc < 0 ? -uc : uc) + (ci < 0 ? -ci : ci));
    *open = *open || __any_sync(0xFFFFFFFFu, near) || (p.k == 32 && p.G > 32);
  }
  return id;
}

// Compare-exchange of a descending sort, and the networks of up to eight values
// (Batcher's odd-even merge sort).
__device__ __forceinline__ void order_pair(uint32_t& a, uint32_t& b) {
  const uint32_t hi = a > b ? a : b;
  b = a > b ? b : a;
  a = hi;
}
template <int V>
__device__ __forceinline__ void sort_down(uint32_t (&k)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; i++)
          if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p)) order_pair(k[i + j], k[i + j + q]);
}

// The choice by the logits alone, where nothing else orders them.  A key is the
// logit's upper bits with the index below them, the lower one larger, so that
// one warp maximum gives a choice with its index and equal logits go by index.
// BF16 logits fit whole.  Of fp32 ones the last bits make room: where two of the
// k + 1 first keys differ in the index alone, *open is set, and the caller
// chooses by the whole logits.  *own: lane j's key.
template <int V>
__device__ __forceinline__ int choose_plain(const RouteParams& p, const float (&x)[V], int lane, bool* open, uint32_t* own) {
  constexpr uint32_t MASK = 32 * V - 1;
  const int e0 = lane * p.per_lane;
  uint32_t key[V], mine = 0;
#pragma unroll
  for (int i = 0; i < V; i++)
    key[i] = i < p.per_lane && e0 + i < p.G ? (order_key(x[i]) & ~MASK) | (MASK - (uint32_t)(e0 + i)) : 0u;
  constexpr bool SORTED = V <= 8;  // heads of sorted lists are popped; longer lists are searched each time
  if constexpr (SORTED) sort_down<V>(key);
  const int count = p.x_f32 && p.k < 32 && p.k < p.G ? p.k + 1 : p.k;
  for (int j = 0; j < count; j++) {
    uint32_t m = key[0];
    if constexpr (!SORTED) {
#pragma unroll
      for (int i = 1; i < V; i++) m = key[i] > m ? key[i] : m;
    }
    const uint32_t w = __reduce_max_sync(0xFFFFFFFFu, m);
    if constexpr (SORTED) {
      if (m == w) {
#pragma unroll
        for (int i = 0; i + 1 < V; i++) key[i] = key[i + 1];
        key[V - 1] = 0;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; i++) key[i] = key[i] == w ? 0u : key[i];
    }
    mine = lane == j ? w : mine;
  }
  const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, mine, 1);
  *open = p.x_f32 && (__any_sync(0xFFFFFFFFu, lane > 0 && lane < count && ((mine ^ up) & ~MASK) == 0u) ||
                      (p.k == 32 && p.G > 32));
  *own = mine;
  return (int)(MASK - (mine & MASK));
}

// sigmoid(x) where fp32's last bits do not matter: off by s (1 - s) (2 |x| + 4) +
// 2 s roundings of 2^-24.
__device__ __forceinline__ float sigmoid_near(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp_near(-x)));
  return r;
}

// The softmax in FP64 of a row with the largest logit `top`.  Rows that need it are few, so
// the loop is not unrolled: instructions that are fetched for one row cost more
// than they compute.
__device__ __forceinline__ Softmax<double> softmax_exact(const RouteParams& p, int64_t t, float top, int lane) {
  Softmax<double> s;
  s.top = (double)top;
  double sum = 0.;
#pragma unroll 1
  for (int e = lane; e < p.G; e += 32) sum += exp_of((double)load_logit(p, t, e) - s.top);
  sum = warp_sum_of(sum);
  s.inv = sum == 0. ? 0. : 1. / sum;
  return s;
}

// The place of the lane's group (of `lanes` lanes) by exact values; `bad`: it has a NaN.
template <bool SIG>
__device__ __forceinline__ int group_rank_exact(const RouteParams& p, int64_t t, float top, int lane, int lanes, bool bad) {
  const double closed = minus_inf<double>();
  double first = closed, second = closed;
  Softmax<double> s{};
  if constexpr (!SIG) s = softmax_exact(p, t, top, lane);
#pragma unroll 1
  for (int i = 0; i < p.per_lane; i++) {
    const int e = lane * p.per_lane + i;
    const float x = load_logit(p, t, e);
    const double c = x == minus_inf<float>()
                         ? closed
                         : add_alone(score_of<double, SIG>(x, s), p.bias != nullptr ? (double)*(p.bias + e) : 0.);
    second = c > first ? first : (c > second ? c : second);
    first = c > first ? c : first;
  }
#pragma unroll 1
  for (int o = 1; o < lanes; o <<= 1) {
    const double a = __shfl_xor_sync(0xFFFFFFFFu, first, o), b = __shfl_xor_sync(0xFFFFFFFFu, second, o);
    const double low = a < first ? a : first;
    second = low > second ? low : second;
    second = b > second ? b : second;
    first = a > first ? a : first;
  }
  const uint64_t order = bad ? ~0ull : order_key(p.group_top == 2 ? first + second : first);
  int rank = 0;
#pragma unroll 1
  for (int l = 0; l < 32; l += lanes) {
    const uint64_t other = __shfl_sync(0xFFFFFFFFu, order, l);
    rank += other > order || (other == order && l + lanes <= lane) ? 1 : 0;
  }
  return rank;
}

// The choice by scores, biases and groups in fp32 with the hardware's functions, for
// groups that are whole lanes (`by_lanes`).  A key's last bits hold the slot.  Where
// choices or groups are nearer than their errors, or keys equal but for the slot, exact
// values order them; *open is set where that does not settle it, and the caller
// takes choose().
// s: the softmax's top and 1 / sum, own[]: exp(x - top), bias: the lane's.
template <int V, bool SIG>
__device__ __forceinline__ int choose_scored(const RouteParams& p, int64_t t, const float (&x)[V], const float (&own)[V],
                                             const Softmax<float>& s, const float (&bias)[V], bool scored, int lane,
                                             bool* open) {
  constexpr uint32_t MASK = V - 1;
  const float closed = minus_inf<float>();
  const int e0 = lane * p.per_lane;
  uint32_t key[V];
  float first = closed, second = closed;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < V; i++) {
    const bool there = i < p.per_lane && e0 + i < p.G;
    float c = x[i];
    if (scored && x[i] != closed) c = SIG ? sigmoid_near(x[i]) + bias[i] : fmaf(own[i], s.inv, bias[i]);
    key[i] = there ? (order_key(p.bias == nullptr ? x[i] : c) & ~MASK) | (MASK - (uint32_t)i) : 0u;
    if (there) {
      nan |= c != c;
      second = c > first ? first : (c > second ? c : second);
      first = c > first ? c : first;
    }
  }
  if (p.groups > 1) {
    const int lanes = 32 / p.groups, mine = lane / lanes;
    for (int o = 1; o < lanes; o <<= 1) {
      const float a = __shfl_xor_sync(0xFFFFFFFFu, first, o), b = __shfl_xor_sync(0xFFFFFFFFu, second, o);
      const float low = a < first ? a : first;
      second = low > second ? low : second;
      second = b > second ? b : second;
      first = a > first ? a : first;
    }
    const float value = p.group_top == 2 ? first + second : first;
    const uint32_t bad = __ballot_sync(0xFFFFFFFFu, nan) >> (mine * lanes) & (lanes == 32 ? ~0u : (1u << lanes) - 1u);
    const uint32_t order = bad ? 0xFFFFFFFFu : order_key(value);
    int rank = 0;
    for (int g = 0; g < p.groups; g++) {
      const uint32_t other = __shfl_sync(0xFFFFFFFFu, order, g * lanes);
      rank += other > order || (other == order && g < mine) ? 1 : 0;
    }
    if (scored) {
      // As in keep_groups.  Units of 2^-24: two sigmoids are off by at most 10, the
      // softmax's scores, which sum to 1, by 70 together (16 and 100 here); the sums
      // by 2 of their size (4 here).
      const bool real = !bad && fabsf(value) <= 3e38f;
      const float err = (SIG ? 1e-6f : 6e-6f) + 2.5e-7f * (fabsf(first) + (p.group_top == 2 ? fabsf(second) : 0.f));
      const uint32_t low = __reduce_min_sync(0xFFFFFFFFu, real && rank < p.topk_groups ? order_key(value - err) : ~0u);
      const uint32_t high = __reduce_max_sync(0xFFFFFFFFu, real && rank >= p.topk_groups ? order_key(value + err) : 0u);
      if (high >= low) rank = group_rank_exact<SIG>(p, t, s.top, lane, lanes, bad != 0);
    }
    if (rank >= p.topk_groups) {
#pragma unroll
      for (int i = 0; i < V; i++)
        if (key[i] != 0) key[i] = (order_key(closed) & ~MASK) | (MASK - (uint32_t)i);
    }
  }
  constexpr bool SORTED = V <= 8;
  if constexpr (SORTED) sort_down<V>(key);
  uint32_t mine = 0;
  int id = 0;
  const auto take = [&](int from, int to) {  // lane j: the j-th largest key and its index, of equal keys the lowest
    for (int j = from; j < to; j++) {
      uint32_t m = key[0];
      if constexpr (!SORTED) {
#pragma unroll
        for (int i = 1; i < V; i++) m = key[i] > m ? key[i] : m;
      }
      const uint32_t w = __reduce_max_sync(0xFFFFFFFFu, m & ~MASK);
      const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, (m & ~MASK) == w)) - 1;
      const int taken = owner * p.per_lane + (int)(MASK - (__shfl_sync(0xFFFFFFFFu, m, owner) & MASK));
      if (lane == owner) {
        if constexpr (SORTED) {
#pragma unroll
          for (int i = 0; i + 1 < V; i++) key[i] = key[i + 1];
          key[V - 1] = 0;
        } else {
#pragma unroll
          for (int i = 0; i < V; i++) key[i] = key[i] == m ? 0u : key[i];
        }
      }
      mine = lane == j ? w : mine;
      id = lane == j ? taken : id;
    }
  };
  // The lane's choice and the one that lane `from` (not above its own) has: may exact
  // values order them otherwise?  Below the last key taken nothing is larger by more
  // than the bits that hold the slot; but a score there may be any, and its error with
  // it, so `last` stands for all behind it: units of 2^-24, two sigmoids are off by 10
  // (20 here), two of the softmax's scores by 74 of the largest (92 here).
  const float any_score = SIG ? 1.2e-6f : 5.5e-6f * s.inv;
  const uint32_t last_key = order_key(closed) & ~MASK;  // closed ones go by index
  float xi = 0.f, bi = 0.f;
  const auto close_to = [&](int from, bool asked, bool last) {
    const uint32_t up = __shfl_sync(0xFFFFFFFFu, mine, from);
    bool near;
    if (p.bias == nullptr) {  // BF16 logits fit whole
      near = p.x_f32 && mine == up;
    } else {
      const float si = SIG ? sigmoid_near(xi) : exp_near(xi - s.top) * s.inv, ci = si + bi;
      // units of 2^-24 of a score: 7 + 2.5 |x| (softmax: from the top), here 10 + 2.7 |x|,
      // each of its own score, so that a finite mask, far away with a score of 0, adds
      // nothing (by the larger of both every token with a mask of -1e9 needed exact values:
      // 32768 x 128 softmax with a bias 176 us instead of 28); a sum with a bias 1; the
      // slot's bits 2 V of the value; the softmax's sum 60, the same part of both scores
      const float ei = (6e-7f + 1.6e-7f * fabsf(SIG ? xi : xi - s.top)) * si;
      const float us = __shfl_sync(0xFFFFFFFFu, si, from), uc = __shfl_sync(0xFFFFFFFFu, ci, from);
      const float pair = ei + __shfl_sync(0xFFFFFFFFu, ei, from) + (SIG ? 0.f : 4e-6f * fabsf(us - si));
      const float tol = last ? fmaxf(pair, any_score) : pair;
      near = uc - ci <= tol + (2.5e-7f + V * 1.2e-7f) * (fabsf(uc) + fabsf(ci)) + 1e-36f;
    }
    return __any_sync(0xFFFFFFFFu, asked && near && mine != last_key) != 0;
  };
  const auto reload = [&](int from, int to) {
    if (lane >= from && lane < to) {
      xi = load_logit(p, t, id);
      if (p.bias != nullptr) bi = *(p.bias + id);
    }
  };
  const int count = p.k < 32 && p.k < p.G ? p.k + 1 : p.k;  // with the first that is left out
  take(0, count);
  if (p.bias != nullptr) reload(0, count);
  *open = p.k == 32 && p.G > 32;
  if (*open || !close_to(lane > 0 ? lane - 1 : 0, lane > 0 && lane < count, lane == p.k)) return id;
  // Eight more, and the order of these by exact values, a lane each: an eighth of the
  // FP64 instructions of all experts' (at 8 a lane), of which an SM does two a clock.
  const int n = min(count + 8, min(p.G, 32));
  take(count, n);
  reload(p.bias != nullptr ? count : 0, n);
  *open = n < p.G && close_to(p.k - 1, lane == n - 1, true);
  if (*open) return id;
  double value = (double)xi;
  if (p.bias != nullptr) {
    Softmax<double> exact{};
    if constexpr (!SIG) exact = softmax_exact(p, t, s.top, lane);
    value = add_alone(score_of<double, SIG>(xi, exact), (double)bi);
  }
  const uint64_t order = lane >= n ? 0 : mine == last_key ? order_key((double)closed) : order_key(value);
  int rank = 0;
  for (int j = 0; j < n; j++) {
    const uint64_t other = __shfl_sync(0xFFFFFFFFu, order, j);
    const int other_id = __shfl_sync(0xFFFFFFFFu, id, j);
    rank += other > order || (other == order && other_id < id) ? 1 : 0;
  }
  int chosen = 0;
  for (int j = 0; j < n; j++) {
    const int to = __shfl_sync(0xFFFFFFFFu, rank, j), what = __shfl_sync(0xFFFFFFFFu, id, j);
    chosen = lane == to ? what : chosen;
  }
  return chosen;
}

// Forward.  The order is that of the exact values: by the logits themselves
// where there is no bias (both scores grow with them), else by score + bias in
// fp32 and, for the few tokens where two of them are nearer than their error,
// in fp64: with all values of such a token again in fp64, 16384 x 256 sigmoids with
// bias and groups took 57 us, a token alone 20 of them; with the candidates' and the
// groups' alone 28.  32768 x 128 fp32 with a bias: 24 us (softmax 28), without 13.
// PLAIN: neither bias nor groups; of 257 to 512 experts held to the registers of two
// blocks an SM (138 of its own accord, one block: 8192 x 512 17.8 us, 12.5 this way).
template <int V, bool SIG, bool PLAIN>
__global__ void __launch_bounds__(256, V == 16 && PLAIN ? 2 : 0) route_fwd_kernel(const RouteParams p) {
  extern __shared__ char route_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e0 = lane * p.per_lane;
  double* const values = reinterpret_cast<double*>(route_smem) + (p.groups > 1 ? warp * p.G : 0);  // groups: G per warp
  int32_t* const load = reinterpret_cast<int32_t*>(route_smem + (p.groups > 1 ? 8 * p.G * sizeof(double) : 0));
  float* const sums = reinterpret_cast<float*>(load + p.G);
  float share[V] = {};
  const bool stats = p.partial_load != nullptr;
  if (stats)
    for (int e = threadIdx.x; e < p.G; e += blockDim.x) {
      load[e] = 0;
      sums[e] = 0.f;
    }
  __syncthreads();
  pdl_trigger();
  pdl_wait();
  const bool scored = p.bias != nullptr || (p.groups > 1 && p.group_top == 2);  // else the logits order everything
  float bias[PLAIN ? 1 : V];
#pragma unroll
  for (int i = 0; i < (PLAIN ? 1 : V); i++)
    bias[i] = !PLAIN && p.bias != nullptr && i < p.per_lane && e0 + i < p.G ? *(p.bias + e0 + i) : 0.f;
  for (int64_t t = (int64_t)blockIdx.x * 8 + warp; t < p.T; t += (int64_t)gridDim.x * 8) {
    float x[V];
    load_logits<V>(p, t, lane, x);
    bool open;
    int id;
    const bool mine = lane < p.k;
    float xj, own[V], norm = 1.f;
    Softmax<float> s{};
    if constexpr (PLAIN) {
      uint32_t key;
      id = choose_plain<V>(p, x, lane, &open, &key);
      // a BF16 logit is its key's upper half
      xj = p.x_f32 ? 0.f : key_value((key & 0x80000000u) ? key & 0xFFFF0000u : key | 0xFFFFu);
      if (open) id = choose<V, SIG, float>(p, t, x, reinterpret_cast<float*>(values), lane, &open);
      if (p.x_f32 && mine) xj = load_logit(p, t, id);
      if constexpr (!SIG) {
        // The first choice's logit, whole: the cut bits of a key are worth hundreds where
        // the logits are 1e9 (a finite mask).  Nothing open: 0 instead of -Inf.
        const float top = __shfl_sync(0xFFFFFFFFu, xj, 0);
        s.top = top == minus_inf<float>() ? 0.f : top;
      }
    } else {
      if constexpr (!SIG) {
        s.top = top_of<V>(x);
        if (scored) s.inv = exps_of<V>(x, s.top, own);
      }
      if (p.by_lanes) {
        id = choose_scored<V, SIG>(p, t, x, own, s, bias, scored, lane, &open);
      } else {
        open = true;
      }
      if (open) id = choose<V, SIG, float>(p, t, x, reinterpret_cast<float*>(values), lane, &open);
      if (open) id = choose<V, SIG, double>(p, t, x, values, lane, &open);
      xj = mine ? load_logit(p, t, id) : 0.f;
      if constexpr (!SIG) {  // a NaN or +Inf anywhere in the row is one in all of its scores
        bool bad = false;
#pragma unroll
        for (int i = 0; i < V; i++) bad |= !(x[i] < __uint_as_float(0x7F800000u));
        if (__any_sync(0xFFFFFFFFu, bad)) xj = __uint_as_float(0x7FC00000u);
      }
    }
    if (!mine) xj = minus_inf<float>();
    if (!SIG && (stats || !p.renorm) && (PLAIN || !scored)) s.inv = exps_of<V>(x, s.top, own);
    float w;
    if constexpr (SIG) {
      w = p.renorm ? sigmoid_share(xj, mine) : mine ? sigmoid_of(xj) : 0.f;
    } else if (p.renorm) {
      w = PLAIN ? share_above(xj, s.top) : chosen_share(xj);
    } else {
      w = exp_near(xj - s.top) * s.inv;
    }
    if (mine) {
      p.weights[t * p.k + lane] = w * p.scale;
      p.ids[t * p.k + lane] = id;
    }
    if (stats) {
      if constexpr (SIG) {
        norm = sigmoids_of<V>(p, x, e0, own);
      } else {
        norm = s.inv;
      }
#pragma unroll
      for (int i = 0; i < V; i++) share[i] = fmaf(own[i], norm, share[i]);
      if (mine) atomicAdd(&load[id], 1);
    }
  }
  if (!stats) return;
  for (int w = 0; w < 8; w++) {  // the warps' sums in warp order
    __syncthreads();
    if (warp == w) {
#pragma unroll
      for (int i = 0; i < V; i++)
        if (i < p.per_lane && e0 + i < p.G) sums[e0 + i] += share[i];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.G; e += blockDim.x) {
    p.partial_load[(int64_t)blockIdx.x * p.G + e] = load[e];
    p.partial_sum[(int64_t)blockIdx.x * p.G + e] = sums[e];
  }
}

// The blocks' counts and sums added in order: a block takes 32 experts, its 32
// warps every 32nd block each, with eight of them in flight at a time.
__global__ void __launch_bounds__(1024) route_stats_kernel(const RouteParams p, int blocks) {
  __shared__ float s[32][32];
  __shared__ int32_t n[32][32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.x * 32 + lane;
  float t = 0.f;
  int32_t c = 0;
  pdl_trigger();
  pdl_wait();
  if (e < p.G) {
#pragma unroll 8
    for (int b = w; b < blocks; b += 32) {
      t += p.partial_sum[(int64_t)b * p.G + e];
      c += p.partial_load[(int64_t)b * p.G + e];
    }
  }
  s[w][lane] = t;
  n[w][lane] = c;
  __syncthreads();
  if (w == 0 && e < p.G) {
    t = 0.f;
    c = 0;
#pragma unroll
    for (int i = 0; i < 32; i++) {
      t += s[i][lane];
      c += n[i][lane];
    }
    p.load[e] = c;
    p.score_sum[e] = t;
  }
}

// Backward.  With a_j = scale * dweights_j, s the scores, r_j = s_j / S the
// renormalised ones (S the choices' sum) and A = sum a_j r_j, the choices give
//   softmax: r_j (a_j - A), or s_e ([e chosen] a_e - sum a_j s_j) without renorm;
//   sigmoid: r_j (a_j - A) (1 - s_j), or a_j s_j (1 - s_j),
// and the gradient v of the scores' sums, with p = softmax, or sigmoid / its sum:
//   p_e (v_e - sum v p), for the sigmoid times (1 - s_e).
// (1 - s = sigmoid(-x), without cancellation; 0 where a score is 0, as of a closed
// expert.)
template <int V, bool SIG>
__global__ void __launch_bounds__(256) route_bwd_kernel(const RouteParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e0 = lane * p.per_lane;
  pdl_trigger();
  pdl_wait();
  // With renormalised weights and no gradient of the sums, all but the choices' get 0.
  const bool dense = p.dsum != nullptr || (!SIG && !p.renorm);
  for (int64_t t = (int64_t)blockIdx.x * 8 + warp; t < p.T; t += (int64_t)gridDim.x * 8) {
    float x[V], d[V];
    if (dense) load_logits<V>(p, t, lane, x);
    int id = -1;
    float a = 0.f;
    if (lane < p.k) {
      id = *(p.ids + t * p.k + lane);
      if (id < 0 || id >= p.G) {  // a dropped choice (-1) has no part
        if (id != -1) atomicOr(&g_route_status, DEV_BAD_INDEX);
        id = -1;
      } else {
        a = *(p.dweights + t * p.k + lane) * p.scale;
      }
    }
    const float xj = id >= 0 ? load_logit(p, t, id) : minus_inf<float>();
    float own[V], norm = 1.f, v_mean = 0.f, top = 0.f, inv = 0.f;
    if (!SIG && dense) {
      top = top_of<V>(x);
      inv = exps_of<V>(x, top, own);
    }
    float r, all = 0.f;
    if constexpr (SIG) {
      r = p.renorm ? sigmoid_share(xj, id >= 0) : id >= 0 ? sigmoid_of(xj) : 0.f;
    } else {
      r = p.renorm ? chosen_share(xj) : exp_near(xj - top) * inv;
    }
    if (p.renorm) a -= warp_sum_of(a * r);
    else if (!SIG) all = warp_sum_of(a * r);  // taken from every expert below
    float g = r == 0.f ? 0.f : r * a;
    if (SIG) g *= sigmoid_of(-xj);
#pragma unroll
    for (int i = 0; i < V; i++) d[i] = 0.f;
    if (dense) {
      if constexpr (SIG) {
        norm = sigmoids_of<V>(p, x, e0, own);
      } else {
#pragma unroll
        for (int i = 0; i < V; i++) own[i] *= inv;
      }
      if (p.dsum != nullptr) {
#pragma unroll
        for (int i = 0; i < V; i++) {
          d[i] = i < p.per_lane && e0 + i < p.G ? *(p.dsum + e0 + i) : 0.f;
          v_mean = fmaf(d[i], own[i] * norm, v_mean);
        }
        v_mean = warp_sum_of(v_mean);
      }
#pragma unroll
      for (int i = 0; i < V; i++) {
        d[i] = own[i] == 0.f ? 0.f : own[i] * ((d[i] - v_mean) * norm - all);
        if (SIG) d[i] *= sigmoid_of(-x[i]);
      }
    }
#pragma unroll 4
    for (int j = 0; j < p.k; j++) {  // each choice's part to the lane that has its expert
      const int e = __shfl_sync(0xFFFFFFFFu, id, j) - e0;
      const float part = __shfl_sync(0xFFFFFFFFu, g, j);
#pragma unroll
      for (int i = 0; i < V; i++) d[i] += e == i ? part : 0.f;
    }
    if (p.x_f32) {
      float* const out = static_cast<float*>(p.dlogits) + t * p.ld_d + e0;
      if (p.wide && V >= 4) {
        if (e0 < p.G) {
#pragma unroll
          for (int i = 0; i + 3 < V; i += 4) *reinterpret_cast<float4*>(out + i) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; i++)
          if (i < p.per_lane && e0 + i < p.G) out[i] = d[i];
      }
    } else {
      uint16_t* const out = static_cast<uint16_t*>(p.dlogits) + t * p.ld_d + e0;
      if (p.wide && V >= 4) {
        if (e0 < p.G) {
#pragma unroll
          for (int i = 0; i + 3 < V; i += 4)
            *reinterpret_cast<uint2*>(out + i) = make_uint2(float2_to_bf16x2(d[i], d[i + 1]), float2_to_bf16x2(d[i + 2], d[i + 3]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; i++)
          if (i < p.per_lane && e0 + i < p.G) out[i] = (uint16_t)float2_to_bf16x2(d[i], 0.f);
      }
    }
  }
}

int64_t route_blocks(int64_t T) {
  const int64_t want = (T + 7) / 8;
  return want < 152 * 4 ? want : 152 * 4;
}

// Lane layout of G experts: V slots, per_lane of them used.
static int slots(int G) {
  int v = 1;
  while (32 * v < G) v *= 2;
  return v;
}
static void set_layout(RouteParams& p) {
  const int v = slots(p.G), bytes = v * (p.x_f32 ? 4 : 2) < 16 ? v * (p.x_f32 ? 4 : 2) : 16;
  p.per_lane = (p.G + 31) / 32;
  if (p.G % v == 0) p.per_lane = v;  // whole pieces for fewer lanes
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.logits) | (uintptr_t)(p.ld * (p.x_f32 ? 4 : 2)) |
                       reinterpret_cast<uintptr_t>(p.dlogits) | (uintptr_t)(p.ld_d * (p.x_f32 ? 4 : 2));
  // groups of whole lanes, 32 lanes in all
  p.by_lanes = p.groups <= 1 || (p.G == 32 * p.per_lane && 32 % p.groups == 0);
  p.wide = p.G % v == 0 && (at & (uintptr_t)(bytes - 1)) == 0;
}

template <int V, bool SIG>
static cudaError_t launch_v(const RouteParams& p, bool bwd, cudaStream_t s) {
  const dim3 grid((unsigned)route_blocks(p.T));
  if (bwd) return launch_pdl(route_bwd_kernel<V, SIG>, dim3((unsigned)(p.T < 152 * 64 ? (p.T + 7) / 8 : 152 * 8)), 256, 0, s, dim3(1), p);
  const int smem = (p.groups > 1 ? 8 * p.G * 8 : 0) + (p.partial_load ? 8 * p.G : 0);
  if (p.bias == nullptr && p.groups <= 1) return launch_pdl(route_fwd_kernel<V, SIG, true>, grid, 256, smem, s, dim3(1), p);
  if (smem > 32 * 1024) {
    const cudaError_t e = ensure_smem_attr<route_fwd_kernel<V, SIG, false>>(8 * 1024 * 8 + 8 * 1024);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(route_fwd_kernel<V, SIG, false>, grid, 256, smem, s, dim3(1), p);
}
template <bool SIG>
static cudaError_t launch_slots(const RouteParams& p, bool bwd, cudaStream_t s) {
  switch (slots(p.G)) {
    case 1: return launch_v<1, SIG>(p, bwd, s);
    case 2: return launch_v<2, SIG>(p, bwd, s);
    case 4: return launch_v<4, SIG>(p, bwd, s);
    case 8: return launch_v<8, SIG>(p, bwd, s);
    case 16: return launch_v<16, SIG>(p, bwd, s);
    default: return launch_v<32, SIG>(p, bwd, s);
  }
}

cudaError_t launch_route_fwd(RouteParams p, cudaStream_t s) {
  set_layout(p);
  const cudaError_t e = p.sigmoid ? launch_slots<true>(p, false, s) : launch_slots<false>(p, false, s);
  if (e != cudaSuccess || p.partial_load == nullptr) return e;
  return launch_pdl(route_stats_kernel, dim3((unsigned)((p.G + 31) / 32)), 1024, 0, s, dim3(1), p, (int)route_blocks(p.T));
}

cudaError_t launch_route_bwd(RouteParams p, cudaStream_t s) {
  set_layout(p);
  return p.sigmoid ? launch_slots<true>(p, true, s) : launch_slots<false>(p, true, s);
}

cudaError_t read_route_status(unsigned* out) { return cudaMemcpyFromSymbol(out, g_route_status, sizeof(unsigned)); }
cudaError_t reset_route_status() {
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_route_status, &zero, sizeof(unsigned));
}

}  // namespace mx
