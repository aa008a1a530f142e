// ep_route.hip -- the router: gate logits to expert ids and weights
// (include/ep_get.h, ep_route, states the formula).
//
// One wavefront per token.  Lane l holds the logits of experts v*64 + l, v = 0,
// 1, ..; the values that decide are 64-bit (neighbours at the border of the
// selection differ by less than a float32 rounding about once in 10^4 tokens),
// mapped to integers that order like them, with 0 for "not to be chosen".  The
// num_topk maxima are taken one after another by butterflies over the wavefront.
#include "ep_host.h"

namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / 64;

// Integers that order like the doubles they come from (never 0 for a number).
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);  // -0 equals 0
  return (b >> 63) ? ~b : b | (1ull << 63);
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int m) {
  const uint32_t lo = __shfl_xor((uint32_t)v, m), hi = __shfl_xor((uint32_t)(v >> 32), m);
  return ((uint64_t)hi << 32) | lo;
}

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}

struct RouteParams {
  const float* bias;
  float* weights;
  int N, E, K, G, keep, top, softmax, renorm;
  float scale;
};

// The score of a logit: sigmoid, or softmax given the row's maximum and sum.
__device__ __forceinline__ double score(double l, bool softmax, double m, double z) {
  return softmax ? exp(l - m) / z : 1.0 / (1.0 + exp(-l));
}

// V experts per lane; L the logits' type, I the type of the ids.
template <int V, typename L, typename I>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(const L* __restrict__ logits,
                                                              I* __restrict__ idx,
                                                              RouteParams p) {
  extern __shared__ uint64_t lds[];            // [waves][E] keys, only with groups
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * kRouteWaves + wave;
  if (t >= p.N) return;                        // no barrier below: waves are independent
  const L* row = logits + (int64_t)t * p.E;

  float l[V];
  bool live[V];
#pragma unroll
  for (int v = 0; v < V; v++) {
    const int e = v * 64 + lane;
    l[v] = e < p.E ? load_logit(row + e) : -INFINITY;
    live[v] = l[v] > -INFINITY;                // false for NaN too
    l[v] = fminf(l[v], 3.402823466e38f);       // +inf counts as the largest float
  }
  double m = 0.0, z = 1.0;
  if (p.softmax) {
    float mf = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; v++) mf = live[v] ? fmaxf(mf, l[v]) : mf;
    m = wave_max(mf);
    double zz = 0.0;
#pragma unroll
    for (int v = 0; v < V; v++) zz += live[v] ? exp((double)l[v] - m) : 0.0;
    z = wave_sum(zz);
  }
  uint64_t key[V], by[V];                      // by value (groups), by order (experts)
#pragma unroll
  for (int v = 0; v < V; v++) {
    const int e = v * 64 + lane;
    key[v] = by[v] = 0;
    if (live[v]) {
      by[v] = ordered((double)l[v]);
      if (p.bias || p.top == 2) {
        double s = score(l[v], p.softmax, m, z);
        if (p.bias) s += (double)p.bias[e];
        key[v] = ordered(s);
        if (p.bias) by[v] = key[v];
      } else {
        key[v] = by[v];
      }
    }
  }

  if (p.G > 1) {                               // lane g scores group g
    uint64_t* mine = lds + wave * p.E;
#pragma unroll
    for (int v = 0; v < V; v++) {
      const int e = v * 64 + lane;
      if (e < p.E) mine[e] = key[v];
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int per = p.E / p.G;
    uint64_t gk = 0;
    if (lane < p.G) {
      uint64_t a = 0, b = 0;                   // the two largest
      for (int i = 0; i < per; i++) {
        const uint64_t k = mine[lane * per + i];
        b = k > a ? a : (k > b ? k : b);
        a = k > a ? k : a;
      }
      gk = a;
      if (p.top == 2) {
        const auto value = [](uint64_t k) {
          return __longlong_as_double((long long)((k >> 63) ? k & ~(1ull << 63) : ~k));
        };
        gk = b ? ordered(value(a) + value(b)) : 0;
      }
    }
    // rank of the group: those with a larger score, or an equal one and before it
    int rank = 0;
    for (int g = 0; g < p.G; g++) {
      const uint32_t lo = __shfl((uint32_t)gk, g), hi = __shfl((uint32_t)(gk >> 32), g);
      const uint64_t o = ((uint64_t)hi << 32) | lo;
      rank += (o > gk || (o == gk && g < lane)) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < p.G && rank < p.keep);
#pragma unroll
    for (int v = 0; v < V; v++) {
      const int e = v * 64 + lane;
      if (e < p.E && !((kept >> (e / per)) & 1)) by[v] = 0;
    }
  }

  int chosen = -1;                             // lane k keeps the k-th
  float clogit = 0.0f;
  for (int k = 0; k < p.K; k++) {
    uint64_t a = 0;
    int ai = INT_MAX;
    float al = 0.0f;
#pragma unroll
    for (int v = 0; v < V; v++)
      if (by[v] > a) a = by[v], ai = v * 64 + lane, al = l[v];   // ties: the lowest v stays
#pragma unroll
    for (int d = 32; d; d >>= 1) {
      const uint64_t o = shfl_xor64(a, d);
      const int oi = __shfl_xor(ai, d);
      const float ol = __shfl_xor(al, d);
      if (o > a || (o == a && oi < ai)) a = o, ai = oi, al = ol;
    }
    if (a == 0) break;
    if (lane == k) chosen = ai, clogit = al;
#pragma unroll
    for (int v = 0; v < V; v++)
      if (v * 64 + lane == ai) by[v] = 0;
  }

  // the weights, in 64 bits up to the one rounding
  double s = chosen >= 0 ? score(clogit, p.softmax, m, z) : 0.0;
  if (p.renorm) {
    const double sum = wave_sum(s);
    s = sum > 0.0 ? s / sum : 0.0;
  }
  if (lane < p.K) {
    idx[(int64_t)t * p.K + lane] = (I)chosen;
    p.weights[(int64_t)t * p.K + lane] = (float)(s * (double)p.scale);
  }
}

template <typename L, typename I>
int launch_route(const ep_route_args_t* a, hipStream_t st) {
  RouteParams p{a->bias, a->topk_weights, a->num_tokens, a->num_experts, a->num_topk,
                a->num_groups, a->topk_groups, a->group_top, a->scoring == EP_SCORE_SOFTMAX,
                a->renormalize != 0, a->scale};
  const int grid = (p.N + kRouteWaves - 1) / kRouteWaves;
  const size_t lds = p.G > 1 ? sizeof(uint64_t) * kRouteWaves * p.E : 0;
  const L* lg = (const L*)a->logits;
  I* ix = (I*)a->topk_idx;
  const int v = (p.E + 63) / 64;
  EP_LOG("route: N=%d E=%d K=%d groups=%d/%d grid=%d", p.N, p.E, p.K, p.keep, p.G, grid);
  if (v <= 1) route_kernel<1, L, I><<<grid, kRouteThreads, lds, st>>>(lg, ix, p);
  else if (v <= 2) route_kernel<2, L, I><<<grid, kRouteThreads, lds, st>>>(lg, ix, p);
  else if (v <= 4) route_kernel<4, L, I><<<grid, kRouteThreads, lds, st>>>(lg, ix, p);
  else if (v <= 8) route_kernel<8, L, I><<<grid, kRouteThreads, lds, st>>>(lg, ix, p);
  else route_kernel<16, L, I><<<grid, kRouteThreads, lds, st>>>(lg, ix, p);
  return check_launch("route_kernel");
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
