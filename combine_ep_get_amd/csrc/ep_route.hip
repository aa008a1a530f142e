// ep_route.hip -- the router: gate logits to expert ids and weights
// (include/ep_get.h, ep_route, states the formula).
//
// One wavefront per token, lane l holds the logits of experts l*V .. l*V+V-1
// (so the lowest lane with a value has the lowest expert, and a lane is inside
// one group where the sizes allow).  The num_topk maxima are taken one after
// another: the wavefront's maximum of 32-bit keys by DPP, the winner by ballot.
//
// Without a bias the experts order as their float32 logits do, exactly.  With one
// (or with groups scored by the sum of two) the scores decide, and neighbours
// at the border of the selection differ by less than float32's roundings about
// once in 10^3 tokens: the selection is made in float32 and stands if every
// decision was clear by more than the error bound (error_of).  Experts that were
// not clear of each other are ranked again by their 64-bit scores, one per lane;
// a wavefront whose groups were not clear, or that has more such experts than lanes,
// repeats the whole selection in 64 bits (choose_exact).  4096 tokens of 256 experts with
// a bias, no groups: 8 us, and 38 where no token is clear (all scores 1 in float32).
//
// One wavefront's chain of num_topk maxima is latency, so is a call: 5.8 us for one
// token of 256 experts, of which an empty launch is 3.5.  4096 tokens of 256 experts (4.5
// MB) take 11.2 us with VALU busy 63% of the time and 16384 of 256 in bf16 (9.4 MB)
// 13.7 us with 97%: this selection's instructions are what counts, not HBM (1.3 us).
#include "ep_host.h"

#include <algorithm>
#include <type_traits>

namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / 64;

// Integers that order like the numbers they come from (never 0 for a number; -0
// as 0).
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return (b >> 63) ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b >> 31) ? ~b : b | (1u << 31);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ double value_of(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? k & ~(1ull << 63) : ~k));
}

// ---------------------------------------------------------------- wavefront reductions
// Lane 63 collects the others: shifts by 1, 2, 4, 8 inside rows of 16 lanes, then
// the rows' last lanes.  Lanes without a source read 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, true);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = dpp<CTRL, ROWS>((uint32_t)b), hi = dpp<CTRL, ROWS>((uint32_t)(b >> 32));
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ uint32_t read_lane(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ __forceinline__ uint64_t read_lane(uint64_t v, int lane) {
  return ((uint64_t)read_lane((uint32_t)(v >> 32), lane) << 32) | read_lane((uint32_t)v, lane);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(dpp<CTRL, ROWS>(__float_as_uint(v)));
}
template <typename T, typename Op>
__device__ __forceinline__ T collect(T v, Op op) {
  v = op(v, dpp<0x111, 0xF>(v));               // row_shr:1
  v = op(v, dpp<0x112, 0xF>(v));
  v = op(v, dpp<0x114, 0xF>(v));
  v = op(v, dpp<0x118, 0xF>(v));
  v = op(v, dpp<0x142, 0xA>(v));               // row_bcast:15 into rows 1 and 3
  v = op(v, dpp<0x143, 0xC>(v));               // row_bcast:31 into rows 2 and 3
  return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  return read_lane(collect(v, [](uint32_t a, uint32_t b) { return max(a, b); }), 63);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  const uint32_t hi = wave_max((uint32_t)(v >> 32));
  const uint32_t lo = wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ float wave_sum(float v) {
  const float s = collect(v, [](float a, float b) { return a + b; });
  return __uint_as_float(read_lane(__float_as_uint(s), 63));
}
__device__ __forceinline__ double wave_sum(double v) {
  const double s = collect(v, [](double a, double b) { return a + b; });
  return __longlong_as_double((long long)read_lane((uint64_t)__double_as_longlong(s), 63));
}

// ---------------------------------------------------------------- the parts
struct RouteParams {
  const float* bias;
  float* weights;
  int N, E, K, G, keep, top, softmax, renorm;
  float scale;
};

template <typename L>
struct Pack;
template <>
struct Pack<float> {
  static __device__ __forceinline__ float value(float v) { return v; }
};
template <>
struct Pack<uint16_t> {
  static __device__ __forceinline__ float value(uint16_t v) {
    return __uint_as_float((uint32_t)v << 16);
  }
};

// The score of a logit: sigmoid, or softmax given the row's maximum and sum.
__device__ __forceinline__ double score(double l, bool softmax, double m, double z) {
  return softmax ? exp(l - m) / z : 1.0 / (1.0 + exp(-l));
}

// The same in float32, and how far it is off.  With u = 2^-24: the product
// l * log2(e) is off by u of itself, which moves a sigmoid by at most
// |l| s (1 - s) u < 0.3 u; v_exp is off by 2 u of its value, which moves it by at
// most 0.5 u; the sum in the denominator by u, v_rcp by 2 u: 3.8 u in all.  A
// softmax: x e^-x 2 u < 0.8 u, v_exp 2 u, the quotient u, the sum of up to 1024
// terms (16 per lane, then a tree of six levels) with their errors 26 u: 30 u.
// Adding the bias rounds by u of the result.  error_of is about twice that.
__device__ __forceinline__ float fast_exp(float v) {
  return __builtin_amdgcn_exp2f(v * 1.44269504088896340736f);
}
__device__ __forceinline__ float error_of(float v, bool softmax) {
  return (softmax ? 0x1p-18f : 0x1p-21f) + 0x1p-23f * fabsf(v);
}

__device__ __forceinline__ void fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The logit of an expert; false where it is masked.
template <typename L>
__device__ __forceinline__ bool logit_of(L raw, float& l) {
  l = Pack<L>::value(raw);
  const bool live = l > -INFINITY;             // false for NaN too
  l = fminf(l, 3.402823466e38f);               // +inf counts as the largest float
  return live;
}

template <int V>
__device__ __forceinline__ double sum_of_exp(const float* l, const bool* live, double m) {
  double z = 0.0;
#pragma unroll
  for (int v = 0; v < V; v++) z += live[v] ? exp((double)l[v] - m) : 0.0;
  return wave_sum(z);
}

struct Choice {
  int expert;                                  // in lane k the k-th, -1: none
  float logit;                                 // its logit
  bool settled;                                // MARGIN: the selection is that of 64-bit scores
};

// The V keys of a lane.  Up to 4 are sorted once, descending and stable, with
// their places (a byte each) beside them; the next one is then always the first.
template <int V, typename U>
struct Keys {
  static constexpr bool sorted = V > 1 && V <= 4;
  U k[V];
  uint32_t order;
  __device__ __forceinline__ void sort() {
    order = 0x03020100u;
    if constexpr (sorted) {
      uint32_t at[V];
#pragma unroll
      for (int v = 0; v < V; v++) at[v] = v;
#pragma unroll
      for (int n = V - 1; n > 0; n--)
#pragma unroll
        for (int v = 0; v < n; v++) {
          const bool swap = k[v + 1] > k[v];
          const U lo = swap ? k[v] : k[v + 1];
          k[v] = swap ? k[v + 1] : k[v];
          k[v + 1] = lo;
          const uint32_t la = swap ? at[v] : at[v + 1];
          at[v] = swap ? at[v + 1] : at[v];
          at[v + 1] = la;
        }
      order = 0;
#pragma unroll
      for (int v = 0; v < V; v++) order |= at[v] << (8 * v);
    }
  }
  __device__ __forceinline__ U largest() const {
    U best = k[0];
    if constexpr (!sorted) {
#pragma unroll
      for (int v = 1; v < V; v++) best = max(best, k[v]);
    }
    return best;
  }
  // Take the largest key, `top`, of lane w away; its place in that lane.
  __device__ __forceinline__ int take(U top, int w) {
    const bool mine = (int)(threadIdx.x & 63) == w;
    if constexpr (sorted) {
      const int at = (int)read_lane(order, w) & 3;
#pragma unroll
      for (int v = 0; v < V; v++) k[v] = mine ? (v + 1 < V ? k[v + 1] : U(0)) : k[v];
      order = mine ? order >> 8 : order;
      return at;
    } else {
      int at = V - 1;
#pragma unroll
      for (int v = V - 2; v >= 0; v--) at = k[v] == top ? v : at;
      at = __builtin_amdgcn_readlane(at, w);
#pragma unroll
      for (int v = 0; v < V; v++) k[v] = mine && v == at ? U(0) : k[v];
      return at;
    }
  }
};

// The selection, with U = uint32_t keys of floats or uint64_t keys of doubles: val[]
// scores the groups, by orders the experts, 0 is masked.  MARGIN: float32 scores
// that may be off by error_of.  Experts that might change places are ranked by
// their 64-bit scores (m, z: the softmax's maximum and sum in 64 bits, z read
// through exact_z only then).  Not settled: the groups' decision might not stand, or
// more experts than there are lanes might change places.
template <int V, bool MARGIN, typename U, typename Z>
__device__ __forceinline__ Choice choose(const U* val, Keys<V, U> by, const float* l,
                                         const RouteParams& p, U* lds, double m, Z exact_z) {
  typedef decltype(value_of(U(0))) Num;
  const int lane = threadIdx.x & 63;
  Choice c{-1, 0.f, true};
  if (p.G > 1) {
    const int per = p.E / p.G, lanes = per / V;
    U gk = 0;                                  // of the lane's group (inside) or group `lane`
    Num first, second;                         // its two largest, where gk is not 0
    const bool two = p.top == 2;
    // whole lanes per group, a power of two of them: butterflies; else through LDS
    const bool inside = per % V == 0 && (lanes & (lanes - 1)) == 0;
    if (inside) {
      Num a = -INFINITY, b = -INFINITY;        // the two largest of the lane, then of the group
#pragma unroll
      for (int v = 0; v < V; v++) {
        const Num x = val[v] ? value_of(val[v]) : (Num)-INFINITY;
        b = fmax(b, fmin(a, x));
        a = fmax(a, x);
      }
      for (int d = 1; d < lanes; d <<= 1) {
        const Num oa = __shfl_xor(a, d);
        if (two) b = fmax(fmin(a, oa), fmax(b, __shfl_xor(b, d)));
        a = fmax(a, oa);
      }
      first = a, second = b;
      // no group without its terms (their sum may be -inf in float32)
      if (lane * V < p.E && (two ? b : a) > -INFINITY) gk = ordered(two ? a + b : a);
    } else {
      fence();
#pragma unroll
      for (int v = 0; v < V; v++)
        if (lane * V + v < p.E) lds[lane * V + v] = val[v];
      fence();
      U a = 0, b = 0;
      if (lane < p.G)
        for (int i = 0; i < per; i++) {
          const U k = lds[lane * per + i];
          b = k > a ? a : (k > b ? k : b);
          a = k > a ? k : a;
        }
      first = value_of(a), second = value_of(b);
      gk = !two ? a : b ? ordered(first + second) : U(0);
    }
    // rank of the lane's group: those with a larger score, or an equal one and before it
    const int step = inside ? lanes : 1, own = inside ? lane / lanes : lane;
    int rank = 0;
    for (int g = 0; g < p.G; g++) {
      const U o = read_lane(gk, g * step);
      rank += (o > gk || (o == gk && g < own)) ? 1 : 0;
    }
    const bool stays = own < p.G && rank < p.keep;
    const uint64_t kept = __ballot(stays);
    if constexpr (MARGIN) {
      // The least that a group that stays may have (~: the minimum) against the most of
      // one that goes.  Of a sum both terms may be off, however small it is itself: the
      // bias may be large and of either sign.  error_of(s) covers the rounding of the sum
      // and of s -+ off.  (inf - inf: not clear.)
      const float s = value_of(gk);
      const float off = error_of(s, p.softmax) +
                        (two ? error_of(first, p.softmax) + error_of(second, p.softmax) : 0.f);
      const U least = ordered(fmaxf(s - off, -INFINITY)), most = ordered(fminf(s + off, INFINITY));
      const U in = ~wave_max(stays && gk ? ~least : U(0));
      const U out = wave_max(own < p.G && !stays && gk ? most : U(0));
      if (out) c.settled = in > out;           // else all that go are masked
    }
#pragma unroll
    for (int v = 0; v < V; v++) {
      const int g = inside ? lane : (lane * V + v) / per;
      if (lane * V + v < p.E && !((kept >> g) & 1)) by.k[v] = 0;
    }
  }
  by.sort();
  const bool scored = MARGIN && p.bias;
  float before = 0.f;
  bool clear = true;
  int n = 0;                                   // chosen so far, in the lanes 0 .. n-1
  for (;; n++) {
    const U best = by.largest();
    const U top = wave_max(best);
    if (top == 0) break;
    if (scored) {                              // clear of the one before?
      const float now = value_of(top);
      const bool far = before - now > error_of(before, p.softmax) + error_of(now, p.softmax);
      if (n >= p.K && far) break;              // and of all after: they are smaller still
      if (n == 64) {                           // a lane for each, and the run goes on
        c.settled = false;
        break;
      }
      clear &= n == 0 || far;
      before = now;
    } else if (n == p.K) {
      break;
    }
    const int w = __ffsll((unsigned long long)__ballot(best == top)) - 1;
    const int at = by.take(top, w);
    float logit = (float)value_of(top);        // without a bias the keys are the logits
    if (p.bias) {
      uint32_t bits = 0;
#pragma unroll
      for (int v = 0; v < V; v++) bits |= v == at ? __float_as_uint(l[v]) : 0u;
      logit = __uint_as_float(read_lane(bits, w));
    }
    if (lane == n) c.expert = w * V + at, c.logit = logit;
  }
  if constexpr (MARGIN) {
    if (!clear && c.settled) {
      const double z = exact_z();
      double s = 0.0;
      if (lane < n) s = score(c.logit, p.softmax, m, z) + (double)p.bias[c.expert];
      const uint64_t key = lane < n ? ordered(s) : 0;
      int rank = 0;
      for (int j = 0; j < n; j++) {
        const uint64_t o = read_lane(key, j);
        const int e = __builtin_amdgcn_readlane(c.expert, j);
        rank += (o > key || (o == key && e < c.expert)) ? 1 : 0;
      }
      const int to = 4 * (lane < n ? rank : lane);
      c.expert = __builtin_amdgcn_ds_permute(to, c.expert);
      c.logit = __int_as_float(__builtin_amdgcn_ds_permute(to, __float_as_int(c.logit)));
    }
  }
  if (lane >= p.K) c.expert = -1;
  return c;
}

// The selection in 64 bits.  Not inlined, and with the row read again, so that the
// usual path keeps its registers.
template <int V, typename L>
__device__ __noinline__ Choice choose_exact(const L* row, RouteParams p, double m, uint64_t* lds) {
  const int lane = threadIdx.x & 63;
  float l[V];
  bool live[V];
#pragma unroll
  for (int v = 0; v < V; v++) {
    l[v] = 0.f;
    live[v] = lane * V + v < p.E && logit_of(row[lane * V + v], l[v]);
  }
  const double z = p.softmax ? sum_of_exp<V>(l, live, m) : 1.0;
  uint64_t val[V];
  Keys<V, uint64_t> by;
#pragma unroll
  for (int v = 0; v < V; v++) {
    val[v] = by.k[v] = 0;
    if (live[v]) {
      double s = score(l[v], p.softmax, m, z);
      if (p.bias) s += (double)p.bias[lane * V + v];
      val[v] = ordered(s);
      by.k[v] = p.bias ? val[v] : ordered((double)l[v]);
    }
  }
  return choose<V, false>(val, by, l, p, lds, m, [] { return 1.0; });
}

// V experts per lane; L the logits' type, I the type of the ids.  SCORED: scores, not
// logits, decide.  wide: a row of logits is aligned for V at a time.
template <int V, typename L, typename I, bool SCORED>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(const L* __restrict__ logits,
                                                              I* __restrict__ idx, RouteParams p,
                                                              bool wide) {
  extern __shared__ uint64_t lds[];            // [waves][E], only with groups
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * kRouteWaves + wave;
  if (t >= p.N) return;                        // no barrier below: waves are independent
  const L* row = logits + (int64_t)t * p.E;

  float l[V], bias[V];
  bool live[V];
  {
    typedef L Row __attribute__((ext_vector_type(V)));
    L raw[V];
    if (wide && V > 1) {                       // E % V == 0: a lane has all or none
      if (lane * V < p.E) {
        const Row r = *reinterpret_cast<const Row*>(row + lane * V);
#pragma unroll
        for (int v = 0; v < V; v++) raw[v] = r[v];
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; v++)
        if (lane * V + v < p.E) raw[v] = row[lane * V + v];
    }
#pragma unroll
    for (int v = 0; v < V; v++)
      bias[v] = SCORED && p.bias && lane * V + v < p.E ? p.bias[lane * V + v] : 0.f;
#pragma unroll
    for (int v = 0; v < V; v++) {
      l[v] = 0.f;
      live[v] = lane * V + v < p.E && logit_of(raw[v], l[v]);
    }
  }
  float m = 0.f, z = 1.f;                      // softmax: the row's maximum and sum
  if (p.softmax) {
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < V; v++) top = live[v] ? max(top, ordered(l[v])) : top;
    m = value_of(wave_max(top));
    if (SCORED || !p.renorm) {
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; v++) sum += live[v] ? fast_exp(l[v] - m) : 0.f;
      z = wave_sum(sum);
    }
  }

  // keys by which experts are chosen, and the values that score the groups
  uint32_t val[V];
  Keys<V, uint32_t> by;
#pragma unroll
  for (int v = 0; v < V; v++) {
    by.k[v] = val[v] = live[v] ? ordered(l[v]) : 0u;
    if (SCORED && live[v]) {
      const float s = p.softmax ? fast_exp(l[v] - m) / z
                                : __builtin_amdgcn_rcpf(1.f + fast_exp(-l[v]));
      val[v] = ordered(s + bias[v]);
      if (p.bias) by.k[v] = val[v];
    }
  }
  uint64_t* own = lds + wave * p.E;
  Choice c = choose<V, SCORED>(val, by, l, p, reinterpret_cast<uint32_t*>(own), m, [&] {
    return p.softmax ? sum_of_exp<V>(l, live, m) : 1.0;
  });
  if (SCORED && !c.settled) c = choose_exact<V>(row, p, m, own);

  // The weights in float32.  Scores that are divided by their sum only need a common
  // factor, so exponentials are taken from the largest logit chosen, and a softmax's sum
  // z is left out: nothing underflows that counts.  sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)).
  float s = 0.f;
  const bool any = c.expert >= 0;
  if (p.softmax) {
    const float from = p.renorm ? value_of(wave_max(any ? ordered(c.logit) : 0u)) : m;
    s = any ? expf(c.logit - from) : 0.f;
    if (any && !p.renorm) s /= z;
  } else {
    const float from = p.renorm ? fminf(value_of(wave_max(any ? ordered(c.logit) : 0u)), 0.f) : 0.f;
    s = any ? expf(fminf(c.logit, 0.f) - from) / (1.f + expf(-fabsf(c.logit))) : 0.f;
  }
  if (p.renorm) {
    const float sum = wave_sum(s);
    s = any ? s / sum : 0.f;                   // the sum is at least 1/2 where one is chosen
  }
  if (lane < p.K) {
    idx[(int64_t)t * p.K + lane] = (I)c.expert;
    p.weights[(int64_t)t * p.K + lane] = s * p.scale;
  }
}

// A grid has less than 2^32 threads in all, 2^26 tokens: more tokens take several launches.
constexpr int kTokensPerLaunch = 1 << 24;

template <typename L, typename I, bool SCORED>
int launch_route(const ep_route_args_t* a, hipStream_t st) {
  RouteParams p{a->bias, nullptr, 0, a->num_experts, a->num_topk,
                a->num_groups, a->topk_groups, a->group_top, a->scoring == EP_SCORE_SOFTMAX,
                a->renormalize != 0, a->scale};
  const size_t lds = p.G > 1 ? sizeof(uint64_t) * kRouteWaves * p.E : 0;
  const int v = (p.E + 63) / 64;
  EP_LOG("route: N=%d E=%d K=%d groups=%d/%d", a->num_tokens, p.E, p.K, p.keep, p.G);
  for (int64_t t = 0; t < a->num_tokens; t += kTokensPerLaunch) {
    p.N = (int)std::min<int64_t>(a->num_tokens - t, kTokensPerLaunch);
    p.weights = a->topk_weights + t * p.K;
    const L* lg = (const L*)a->logits + t * p.E;
    I* ix = (I*)a->topk_idx + t * p.K;
    const int grid = (p.N + kRouteWaves - 1) / kRouteWaves;
    const auto go = [&](auto V) {
      constexpr int n = decltype(V)::value;
      const bool wide = p.E % n == 0 && ((uintptr_t)lg & (n * sizeof(L) - 1)) == 0;
      route_kernel<n, L, I, SCORED><<<grid, kRouteThreads, lds, st>>>(lg, ix, p, wide);
    };
    if (v <= 1) go(std::integral_constant<int, 1>());
    else if (v <= 2) go(std::integral_constant<int, 2>());
    else if (v <= 4) go(std::integral_constant<int, 4>());
    else if (v <= 8) go(std::integral_constant<int, 8>());
    else go(std::integral_constant<int, 16>());
    const int rc = check_launch("route_kernel");
    if (rc != EP_OK) return rc;
  }
  return EP_OK;
}

template <typename L, typename I>
int launch_route(const ep_route_args_t* a, hipStream_t st) {
  return a->bias || (a->group_top == 2 && a->num_groups > 1) ? launch_route<L, I, true>(a, st)
                                                            : launch_route<L, I, false>(a, st);
}

}  // namespace

extern "C" int ep_route(const ep_route_args_t* a, void* stream) {
  if (!a) return EP_ERR_INVALID_ARG;
  const int64_t N = a->num_tokens, E = a->num_experts, K = a->num_topk, G = a->num_groups;
  if (N < 0 || E < 1 || E > EP_MAX_EXPERTS || K < 1 || K > EP_MAX_TOPK) return EP_ERR_INVALID_ARG;
  if (G < 1 || G > EP_MAX_GROUPS || E % G != 0) return EP_ERR_INVALID_ARG;
  if (a->topk_groups < 1 || a->topk_groups > G) return EP_ERR_INVALID_ARG;
  if (a->group_top < 1 || a->group_top > 2 || a->group_top > E / G) return EP_ERR_INVALID_ARG;
  if (K > a->topk_groups * (E / G)) return EP_ERR_INVALID_ARG;
  if (a->scoring != EP_SCORE_SIGMOID && a->scoring != EP_SCORE_SOFTMAX) return EP_ERR_INVALID_ARG;
  if (a->renormalize != 0 && a->renormalize != 1) return EP_ERR_INVALID_ARG;
  if (a->logits_bytes != 4 && a->logits_bytes != 2) return EP_ERR_INVALID_ARG;
  if (a->topk_idx_bytes != 0 && a->topk_idx_bytes != 4 && a->topk_idx_bytes != 8)
    return EP_ERR_INVALID_ARG;
  if (N * K > INT32_MAX) return EP_ERR_INVALID_ARG;
  if (N > 0 && (!a->logits || !a->topk_idx || !a->topk_weights)) return EP_ERR_INVALID_ARG;
  const int rc = check_device();
  if (rc != EP_OK || N == 0) return rc;
  hipStream_t st = (hipStream_t)stream;
  if (a->logits_bytes == 4)
    return a->topk_idx_bytes == 8 ? launch_route<float, int64_t>(a, st)
                                  : launch_route<float, int32_t>(a, st);
  return a->topk_idx_bytes == 8 ? launch_route<uint16_t, int64_t>(a, st)
                                : launch_route<uint16_t, int32_t>(a, st);
}
