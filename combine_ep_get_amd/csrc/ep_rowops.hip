// ep_rowops.hip -- rows as 8-bit integers, and combine's gradient (include/ep_get.h
// states the contracts).  Both read each row once and are bound by HBM.
#include "ep_host.h"
#include "ep_rows.h"

#include <algorithm>

namespace {

// ---------------------------------------------------------------- 8-bit integers
// A row by WAVES wavefronts, which hold up to CH 16-byte chunks per lane in registers (of a
// longer row the rest is read twice); blocks (segment, part): segments are the experts, or the
// sub-blocks of ep_ll_dispatch, whose rows are shared out over the parts.  4096 rows of
// 7168: 18.7 us over and over on the same rows, one wavefront per row 24.7; 21 on new rows.
template <int WAVES, int CH>
__global__ __launch_bounds__(256) void quantize_kernel(Rows rows, const uint8_t* x, int cols,
                                                       uint8_t* codes, float* scales) {
  __shared__ uint32_t tops[2][4];
  constexpr int kRows = 4 / WAVES, kLanes = 64 * WAVES;
  const int seg = blockIdx.x, l = threadIdx.x % kLanes;
  int first, n;
  if (rows.count && !rows.offset) {
    first = seg * rows.M;
    n = max(0, min(rows.count[seg], rows.M));
  } else {
    first = rows.first_slot(seg);
    n = rows.rows_of(seg);
  }
  const int chunks = cols / 8;
  int turn = 0;                          // rows alternate between two sets of maxima
  for (int64_t j = (int64_t)blockIdx.y * kRows + threadIdx.x / kLanes; j < n;
       j += gridDim.y * kRows) {
    const int64_t slot = first + j;
    const u32x4* in = (const u32x4*)(x + slot * cols * 2);
    u32x2* out = (u32x2*)(codes + slot * cols);
    u32x4 held[CH];
#pragma unroll
    for (int i = 0; i < CH; i++)
      held[i] = i * kLanes + l < chunks ? in[i * kLanes + l] : u32x4{0, 0, 0, 0};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < CH; i++) top = max(top, largest8(held[i]));
    for (int c = CH * kLanes + l; c < chunks; c += kLanes) top = max(top, largest8(in[c]));
    top = wave_max(top);
    if constexpr (WAVES == 4) {          // the whole workgroup has the same rows
      if ((l & 63) == 0) tops[turn][l >> 6] = top;
      __syncthreads();
      top = max(max(tops[turn][0], tops[turn][1]), max(tops[turn][2], tops[turn][3]));
      turn ^= 1;
    }
    const RowScale s = RowScale::of(top);
    if (l == 0) scales[slot] = s.scale;
#pragma unroll
    for (int i = 0; i < CH; i++)
      if (i * kLanes + l < chunks) out[i * kLanes + l] = s.codes8(held[i]);
    for (int c = CH * kLanes + l; c < chunks; c += kLanes) out[c] = s.codes8(in[c]);
  }
}

// ---------------------------------------------------------------- combine's gradient
constexpr int kMostWaves = 16, kPairs = 4;
// A grid has less than 2^32 threads along an axis (with more, the count wraps and tokens
// stay undone without an error), 2^22 workgroups of 1024: more tokens take several launches.
constexpr int kTokensPerLaunch = 1 << 21;

// A workgroup per token and four of its pairs, a thread per 16-byte chunk of the row (or
// per several): all loads of a chunk are in flight at once, and dy's row is read once
// for these pairs.  The sums meet in LDS at the end, in a fixed order.  4096 tokens of 8
// pairs by 7168: 189 us, 5.3 TB/s of mixed reads and writes (a copy of 1 GiB: 5.15), whatever
// the pairs (8: 190, 2: 188, 1: 225) or wavefronts per workgroup; 128 tokens: 7.4 us, with
// eight pairs 10.9.
__global__ __launch_bounds__(1024) void combine_backward_kernel(
    const u32x4* dy, const u32x4* eo, const int* slot_of, const float* wts, u32x4* deo,
    float* dwts, int H8, int K, int cap) {
  __shared__ float sums[kMostWaves][kPairs];
  const int64_t t = blockIdx.x;
  const int k0 = blockIdx.y * kPairs, tid = threadIdx.x, waves = blockDim.x >> 6;
  int slot[kPairs];
  float w[kPairs], sum[kPairs];
#pragma unroll
  for (int k = 0; k < kPairs; k++) {
    const bool in = k0 + k < K;
    slot[k] = in ? slot_of[t * K + k0 + k] : -1;
    if (slot[k] >= cap) slot[k] = -1;
    w[k] = in ? wts[t * K + k0 + k] : 0.f;
    sum[k] = 0.f;
  }
  for (int c = tid; c < H8; c += blockDim.x) {
    const u32x4 g = dy[t * H8 + c];
    u32x4 o[kPairs];
#pragma unroll
    for (int k = 0; k < kPairs; k++)
      if (slot[k] >= 0) o[k] = __builtin_nontemporal_load(eo + (int64_t)slot[k] * H8 + c);
    float gf[8];
    unpack8(g, gf);
#pragma unroll
    for (int k = 0; k < kPairs; k++) {
      if (slot[k] < 0) continue;
      float of[8];
      unpack8(o[k], of);
      u32x4 r;
#pragma unroll
      for (int i = 0; i < 4; i++) r[i] = pack2(w[k] * gf[2 * i], w[k] * gf[2 * i + 1]);
#pragma unroll
      for (int i = 0; i < 8; i++) sum[k] = fmaf(of[i], gf[i], sum[k]);
      __builtin_nontemporal_store(r, deo + (int64_t)slot[k] * H8 + c);
    }
  }
#pragma unroll
  for (int k = 0; k < kPairs; k++) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum[k] += __shfl_xor(sum[k], d);
    if ((tid & 63) == 0) sums[tid >> 6][k] = sum[k];
  }
  __syncthreads();
  if (tid < kPairs && k0 + tid < K) {
    float total = 0.f;
    for (int v = 0; v < waves; v++) total += sums[v][tid];
    dwts[t * K + k0 + tid] = total;
  }
}

}  // namespace

namespace ep {

int quantize_rows(const Rows& rows, int max_rows, const void* x, int cols, void* codes,
                  float* scales, hipStream_t st) {
  const int segments = rows.count && !rows.offset ? rows.E * rows.R : rows.E;
  // at most about 16 workgroups per CU; at least twice the average segment, so that an
  // uneven one takes few passes
  const int rows_per = cols <= 2048 ? 4 : 1;
  const int64_t per = ((int64_t)max_rows / segments + 1) * 2;
  int64_t parts = (per + rows_per - 1) / rows_per;
  const int64_t most = segments >= 4096 ? 1 : 4096 / segments;
  if (parts > most) parts = most;
  const dim3 grid(segments, (int)parts);
  const uint8_t* in = (const uint8_t*)x;
  if (cols <= 2048)
    quantize_kernel<1, 4><<<grid, 256, 0, st>>>(rows, in, cols, (uint8_t*)codes, scales);
  else
    quantize_kernel<4, 4><<<grid, 256, 0, st>>>(rows, in, cols, (uint8_t*)codes, scales);
  return check_launch("quantize_rows");
}

}  // namespace ep

extern "C" {

int ep_quantize_rows(int64_t num_rows, int32_t cols, const void* x, int8_t* codes, float* scales,
                     void* stream) {
  if (num_rows < 0 || num_rows > INT32_MAX || !valid_width(cols, EP_WEIGHT_INT8))
    return EP_ERR_INVALID_ARG;
  if (num_rows == 0) return EP_OK;
  if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned(scales, 4) ||
      overlap(codes, num_rows * cols, x, num_rows * cols * 2))
    return EP_ERR_INVALID_ARG;
  int rc = check_device();
  if (rc != EP_OK) return rc;
  const Rows r{nullptr, nullptr, (int)num_rows, 1, 1, 0, (int)num_rows};
  return quantize_rows(r, (int)num_rows, x, cols, codes, scales, (hipStream_t)stream);
}

int ep_combine_backward(const ep_problem_t* p, const void* dy, const void* expert_out,
                        const int32_t* slot_of, const float* topk_weights, void* d_expert_out,
                        float* d_topk_weights, int64_t recv_capacity, void* stream) {
  int rc = validate_layout(p);
  if (rc != EP_OK) return rc;
  const int H = p->hidden, N = p->num_tokens;
  if (H <= 0 || H > EP_MAX_HIDDEN || H % 8 != 0 || (p->use_fp8 != 0 && p->use_fp8 != 1) ||
      recv_capacity < 0 || recv_capacity > INT32_MAX)
    return EP_ERR_INVALID_ARG;
  if (N == 0) return EP_OK;
  if (!dy || !slot_of || !topk_weights || !d_topk_weights ||
      (recv_capacity > 0 && (!expert_out || !d_expert_out)) || !aligned16(dy) ||
      !aligned16(expert_out) || !aligned16(d_expert_out))
    return EP_ERR_INVALID_ARG;
  const int64_t rows = recv_capacity * 2 * H, own = (int64_t)N * 2 * H;
  if (overlap(d_expert_out, rows, dy, own) ||
      (d_expert_out != expert_out && overlap(d_expert_out, rows, expert_out, rows)))
    return EP_ERR_INVALID_ARG;
  rc = check_device();
  if (rc != EP_OK) return rc;
  EP_LOG("combine_backward N=%d H=%d K=%d cap=%lld", N, H, p->num_topk, (long long)recv_capacity);
  const int K = p->num_topk, q = (H / 8 + 63) / 64;
  const int passes = (q + kMostWaves - 1) / kMostWaves, waves = (q + passes - 1) / passes;
  for (int64_t t = 0; t < N; t += kTokensPerLaunch) {
    const int n = (int)std::min<int64_t>(N - t, kTokensPerLaunch);
    combine_backward_kernel<<<dim3(n, (K + kPairs - 1) / kPairs), dim3(64 * waves), 0,
                              (hipStream_t)stream>>>(
        (const u32x4*)dy + t * (H / 8), (const u32x4*)expert_out, slot_of + t * K,
        topk_weights + t * K, (u32x4*)d_expert_out, d_topk_weights + t * K, H / 8, K,
        (int)recv_capacity);
    rc = check_launch("combine_backward");
    if (rc != EP_OK) return rc;
  }
  return EP_OK;
}

}  // extern "C"
