// ep_moe.hip -- the experts' products for a few tokens (include/ep_get.h states
// the contracts): the whole expert layer in two kernels, and the product of a few
// rows with a 4-bit weight.
//
// All of it is one loop, `Stream`: 16-row tiles of a weight flow from HBM
// through registers into v_mfma_f32_16x16x32_bf16, whose other operand is rows
// of x.  The weights are the bytes that count (a decode batch has too few
// tokens for the products to matter: 16 tokens are 16 flops per weight byte in
// bf16, HBM's rate allows about 400), so every choice serves the stream:
//   - a wavefront loads its tile straight into the operand layout (lane r + 16 g
//     holds row r), with no LDS and no barrier on the way, several steps ahead;
//   - the wavefronts of a workgroup split the contraction and meet once, at the
//     end, in LDS;
//   - where an access falls outside (columns behind the end, rows behind the
//     last, absent tokens) its buffer offset is out of range and the hardware
//     returns zeros, so the loop has no branches.
//
// The contraction runs in steps of 128 columns, four MFMAs each.  Which eight
// columns lane group g feeds to MFMA j is free as long as both operands agree;
// it is chosen so that the weight's loads are as wide as its format allows
// (`Fmt::col`).  A 4-bit weight is scaled per (row, group): lane r holds row r's
// column of the 16x16 result, so one factor per lane does it, after the sum
// over the group, in float32.  int4 codes become bf16 by putting the nibble
// under the exponent of 128 (exact: 128 + code); the 128 and the zero point
// leave again as (128 + zero) * sum(x), whose sum comes from an MFMA with ones.
// E2M1 codes with their power-of-two scale are exact bf16 values already.
//
// Up to four tokens (`Quad`): rows t*4 + j of the MFMA's 16 hold the four
// column pieces j of token t, so one load per step brings all of x and every
// lane takes part; MFMA j's row t*4 + j is the product wanted, the other rows
// are ignored.
#include "ep_host.h"

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kStep = 128;                 // columns per step
constexpr int kBufferWord3 = 0x00020000;   // raw buffer, 32-bit data format
constexpr int kOutside = 0x7FFFFFFF;       // offset out of every buffer's range
constexpr int kNonTemporal = 2;            // NT in the cache-policy operand

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// ---------------------------------------------------------------- formats
// Weight format and group; Z: int4 with zero points.
enum { kBf16, kMx, kInt128, kInt64, kInt32, kInt128Z, kInt64Z, kInt32Z };

template <int F>
struct Fmt {
  static constexpr bool quant = F != kBf16, integer = F >= kInt128, zeros = F >= kInt128Z;
  static constexpr int group = F == kInt128 || F == kInt128Z ? 128
                               : F == kInt64 || F == kInt64Z ? 64 : 32;
  // words a lane loads at a time, and how many such loads make a step
  static constexpr int words = integer ? group / 32 : 4;
  static constexpr int loads = F == kBf16 ? 4 : 4 / words;
  static constexpr int groups = F == kMx ? 1 : quant ? kStep / group : 0;  // scale loads per step
  static constexpr int step_bytes = quant ? kStep / 2 : kStep * 2;
  // first of the eight columns that lane group g feeds to MFMA j
  static __device__ __forceinline__ int col(int g, int j) {
    if constexpr (F == kMx || (integer && words == 4)) return g * 32 + j * 8;
    else if constexpr (words == 2) return (j >> 1) * 64 + g * 16 + (j & 1) * 8;
    else return j * 32 + g * 8;
  }
};

// ---------------------------------------------------------------- one weight tile
// 16 rows of a weight as buffers; rows behind the last are out of range.
struct Tile {
  __amdgpu_buffer_rsrc_t data, scale, zero;
};

// Bytes of a row of codes (or bf16 values) and of its scales and zeros.
template <int F>
__device__ __forceinline__ int row_bytes(int cols) { return Fmt<F>::quant ? cols / 2 : cols * 2; }
template <int F>
__device__ __forceinline__ int row_groups(int cols) { return Fmt<F>::quant ? cols / Fmt<F>::group : 0; }

struct Weight {           // kernel argument: ep_weight_t without what the kernel's type says
  const uint8_t* data;
  const uint8_t* scale;
  const uint8_t* zero;
};

template <int F>
__device__ __forceinline__ Tile make_tile(const Weight& w, int64_t row, int rows, int cols) {
  Tile t;
  const int n = max(0, min(16, rows));
  const int rb = row_bytes<F>(cols), rg = row_groups<F>(cols);
  t.data = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(w.data) + row * rb, 0, n * rb,
                                             kBufferWord3);
  if constexpr (Fmt<F>::quant) {
    constexpr int size = F == kMx ? 1 : 2;
    t.scale = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(w.scale) + row * rg * size, 0,
                                                n * rg * size, kBufferWord3);
    if constexpr (Fmt<F>::zeros)
      t.zero = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(w.zero) + row * rg, 0,
                                                 n * rg, kBufferWord3);
  }
  return t;
}

// ---------------------------------------------------------------- the stream
// RT weight tiles times T token tiles of 16 (T == 0: Quad, up to 4 tokens).
template <int F, int RT, int T>
struct Stream {
  static constexpr bool quad = T == 0;
  static constexpr int TT = quad ? 1 : T;
  // Steps in flight: enough that the loads of a CU's wavefronts cover HBM's
  // latency, as far as the registers go.
  static constexpr int depth = Fmt<F>::quant ? (TT <= 1 ? 4 : 2) : (quad ? 3 : 2);

  struct Slot {
    u32x4 w[RT][Fmt<F>::loads];
    uint32_t s[RT][Fmt<F>::groups ? Fmt<F>::groups : 1];
    uint32_t z[RT][Fmt<F>::groups ? Fmt<F>::groups : 1];
    u32x4 x[TT][quad ? 1 : 4];
  };

  // acc[i][j]: Quad: MFMA j's own rows (bf16), or [i][0] the whole sum (4-bit);
  // otherwise token tile j.  In the MFMA's result layout: lane r + 16 g holds
  // weight row r of tokens g*4 .. g*4+3.
  f32x4 acc[RT][quad ? 4 : TT];
  Slot slot[depth];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
      for (int j = 0; j < (quad ? 4 : TT); j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // Load step s (columns s*128 ..) of the tiles and of x; nothing if s >= end.
  __device__ __forceinline__ void load(Slot& b, int s, int end, int cols, const Tile* tile,
                                       __amdgpu_buffer_rsrc_t xr, const int* xoff) {
    using M = Fmt<F>;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const bool in = s < end;
    const int c0 = in ? s * kStep : 0;
    const int left = in ? cols - c0 : 0;                   // columns left from here
    const int rb = row_bytes<F>(cols);
#pragma unroll
    for (int q = 0; q < M::loads; q++) {
      // columns of this load: 8 * words-in-codes (4-bit) or 8 values (bf16)
      const int c = M::quant ? q * (kStep / M::loads) + g * (8 * M::words) : M::col(g, q);
      const int off = c < left ? r * rb + (M::quant ? c / 2 : c * 2) : kOutside;
      const int so = c0 / kStep * M::step_bytes;
#pragma unroll
      for (int i = 0; i < RT; i++) {
        if constexpr (M::words == 4)
          b.w[i][q] = __builtin_amdgcn_raw_buffer_load_b128(tile[i].data, off, so, kNonTemporal);
        else if constexpr (M::words == 2) {
          const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(tile[i].data, off, so, 0);
          b.w[i][q].x = v.x, b.w[i][q].y = v.y;
        } else
          b.w[i][q].x = __builtin_amdgcn_raw_buffer_load_b32(tile[i].data, off, so, 0);
      }
    }
    if constexpr (M::quant) {
      const int rg = row_groups<F>(cols);
#pragma unroll
      for (int q = 0; q < M::groups; q++) {
        const int c = F == kMx ? g * 32 : q * M::group;
        const int at = r * rg + (c0 + c) / M::group;
#pragma unroll
        for (int i = 0; i < RT; i++) {
          if constexpr (F == kMx)
            b.s[i][q] = __builtin_amdgcn_raw_buffer_load_b8(tile[i].scale, c < left ? at : kOutside,
                                                            0, 0);
          else
            b.s[i][q] = __builtin_amdgcn_raw_buffer_load_b16(
                tile[i].scale, c < left ? at * 2 : kOutside, 0, 0);
          if constexpr (M::zeros)
            b.z[i][q] = __builtin_amdgcn_raw_buffer_load_b8(tile[i].zero, c < left ? at : kOutside,
                                                            0, 0);
        }
      }
    }
    if constexpr (quad) {
      const int c = M::col(g, lane & 3);
      b.x[0][0] = __builtin_amdgcn_raw_buffer_load_b128(xr, c < left ? xoff[0] + c * 2 : kOutside,
                                                        c0 * 2, 0);
    } else {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int c = M::col(g, j);
#pragma unroll
        for (int k = 0; k < TT; k++)
          b.x[k][j] = __builtin_amdgcn_raw_buffer_load_b128(
              xr, c < left ? xoff[k] + c * 2 : kOutside, c0 * 2, 0);
      }
    }
  }

  // The eight bf16 weights of MFMA j.
  __device__ __forceinline__ static u32x4 operand(const Slot& b, int i, int j) {
    using M = Fmt<F>;
    if constexpr (!M::quant) {
      return b.w[i][j];
    } else {
      const u32x4 v = b.w[i][j / M::words];
      const uint32_t w = M::words == 4 ? v[j] : M::words == 2 ? v[j & 1] : v[0];
      u32x4 o;
      if constexpr (M::integer) {
#pragma unroll
        for (int q = 0; q < 4; q++) o[q] = ((w >> (4 * q)) & 0x000F000Fu) | 0x43004300u;
      } else {
        const float s = __uint_as_float(b.s[i][0] << 23);
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
      }
      return o;
    }
  }

  // What is taken off the codes as the operand holds them (128 + code).
  __device__ __forceinline__ static float zero_of(const Slot& b, int i, int q) {
    return Fmt<F>::zeros ? 128.f + (float)b.z[i][q] : 136.f;
  }

  __device__ __forceinline__ void compute(const Slot& b) {
    using M = Fmt<F>;
    const f32x4 none{0.f, 0.f, 0.f, 0.f};
    constexpr uint32_t kOnes = 0x3F803F80u;
    const u32x4 ones{kOnes, kOnes, kOnes, kOnes};
    if constexpr (!M::integer) {
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int i = 0; i < RT; i++) {
          const u32x4 w = operand(b, i, j);
          if constexpr (quad) {
            acc[i][j] = mfma(b.x[0][0], w, acc[i][j]);
          } else {
#pragma unroll
            for (int k = 0; k < TT; k++) acc[i][k] = mfma(b.x[k][j], w, acc[i][k]);
          }
        }
    } else {
      constexpr int per = 4 / M::groups;       // MFMAs per group
      if constexpr (quad) {
        const f32x4 sx = mfma(b.x[0][0], ones, none);      // register j: sum of piece j
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
          for (int q = 0; q < M::groups; q++) {
            float sum = 0.f, xs = 0.f;
#pragma unroll
            for (int j = q * per; j < (q + 1) * per; j++) {
              const f32x4 d = mfma(b.x[0][0], operand(b, i, j), none);
              sum += d[j];
              xs += sx[j];
            }
            const float z = zero_of(b, i, q);
            acc[i][0][0] = fmaf(bf16_value(b.s[i][q]), fmaf(-z, xs, sum), acc[i][0][0]);
          }
      } else {
#pragma unroll
        for (int q = 0; q < M::groups; q++)
#pragma unroll
          for (int k = 0; k < TT; k++) {
            f32x4 xs = none;
#pragma unroll
            for (int j = q * per; j < (q + 1) * per; j++) xs = mfma(b.x[k][j], ones, xs);
#pragma unroll
            for (int i = 0; i < RT; i++) {
              f32x4 d = none;
#pragma unroll
              for (int j = q * per; j < (q + 1) * per; j++) d = mfma(b.x[k][j], operand(b, i, j), d);
              const float s = bf16_value(b.s[i][q]), z = zero_of(b, i, q);
#pragma unroll
              for (int e = 0; e < 4; e++) acc[i][k][e] = fmaf(s, fmaf(-z, xs[e], d[e]), acc[i][k][e]);
            }
          }
      }
    }
  }

  // Add steps first, first + by, .. < end of x times the tiles to acc.  xoff:
  // the lane's row(s) of x as byte offsets (kOutside: no token), from `xrow`.
  __device__ __forceinline__ void run(int first, int by, int end, int cols, const Tile* tile,
                                      __amdgpu_buffer_rsrc_t xr, const int* xoff) {
#pragma unroll
    for (int d = 0; d < depth; d++) load(slot[d], first + d * by, end, cols, tile, xr, xoff);
    for (int s = first; s < end; s += depth * by) {
#pragma unroll
      for (int d = 0; d < depth; d++) {
        compute(slot[d]);                       // a step behind the end adds zeros
        load(slot[d], s + (depth + d) * by, end, cols, tile, xr, xoff);
      }
    }
  }

  // Which token (of this call's tokens) the lane loads rows of x for, tile k.
  static __device__ __forceinline__ int token(int k) {
    const int lane = threadIdx.x & 63;
    return quad ? (lane & 15) >> 2 : k * 16 + (lane & 15);
  }

  // Results: values(i, f) calls f(token, value) for every token row this lane
  // holds of weight tile i (weight row lane & 15).
  template <typename Fn>
  __device__ __forceinline__ void values(int i, Fn&& f) const {
    const int g = (threadIdx.x & 63) >> 4;
    if constexpr (quad) {
      if constexpr (Fmt<F>::integer) f(g, acc[i][0][0]);
      else f(g, acc[i][0][0] + acc[i][1][1] + acc[i][2][2] + acc[i][3][3]);
    } else {
#pragma unroll
      for (int k = 0; k < TT; k++)
#pragma unroll
        for (int e = 0; e < 4; e++) f(k * 16 + g * 4 + e, acc[i][k][e]);
    }
  }
  static constexpr int tokens = quad ? 4 : 16 * TT;
};

// ---------------------------------------------------------------- y = x W^T
constexpr int kLinWaves = 8;

// One workgroup: RT*16 rows of the weight, all columns split over the waves, 16 T
// rows of x (blockIdx.y).
template <int F, int RT, int T>
__global__ __launch_bounds__(64 * kLinWaves) void linear_kernel(
    const uint16_t* __restrict__ x, Weight w, uint16_t* __restrict__ y, int n, int cols, int rows) {
  using S = Stream<F, RT, T>;
  __shared__ float red[kLinWaves][RT][S::tokens][16];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int row0 = blockIdx.x * (RT * 16), t0 = blockIdx.y * S::tokens;
  const int nt = min(n - t0, S::tokens);
  Tile tile[RT];
#pragma unroll
  for (int i = 0; i < RT; i++)
    tile[i] = make_tile<F>(w, min(row0 + i * 16, rows), rows - row0 - i * 16, cols);
  const auto xr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(x) + (int64_t)t0 * cols,
                                                    0, nt * cols * 2, kBufferWord3);
  int xoff[S::TT];
#pragma unroll
  for (int k = 0; k < S::TT; k++) xoff[k] = S::token(k) < nt ? S::token(k) * cols * 2 : kOutside / 2;
  S st;
  st.clear();
  st.run(wave, kLinWaves, (cols + kStep - 1) / kStep, cols, tile, xr, xoff);
#pragma unroll
  for (int i = 0; i < RT; i++)
    st.values(i, [&](int t, float v) { red[wave][i][t][lane & 15] = v; });
  __syncthreads();
  for (int q = threadIdx.x; q < nt * RT * 16; q += 64 * kLinWaves) {
    const int t = q / (RT * 16), c = q % (RT * 16);
    float v = 0.f;
#pragma unroll
    for (int u = 0; u < kLinWaves; u++) v += red[u][c >> 4][t][c & 15];
    if (row0 + c < rows) y[(int64_t)(t0 + t) * rows + row0 + c] = bf16_bits(v);
  }
}

// ---------------------------------------------------------------- the expert layer
// Workspace: what the first kernel finds out about the routing, and the rows
// between the two products.
struct MoePlan {
  int32_t experts;                        // most experts that can be active: min(E, N*K)
  int64_t o_expert, o_count, o_pairs, o_hidden, bytes;   // byte offsets
};
// word 0: error bits (ep_layout_error), word 1: active experts

__host__ __device__ inline int64_t align256(int64_t v) { return (v + 255) & ~int64_t(255); }

MoePlan make_moe_plan(const ep_problem_t* p, int inter) {
  const int64_t N = p->num_tokens, pairs = N * p->num_topk;
  MoePlan m;
  m.experts = (int32_t)(pairs < p->num_experts ? pairs : p->num_experts);
  m.o_expert = 256;
  m.o_count = m.o_expert + align256((int64_t)m.experts * 4);
  m.o_pairs = m.o_count + align256((int64_t)m.experts * 4);
  m.o_hidden = m.o_pairs + align256(m.experts * N * 4);
  m.bytes = m.o_hidden + align256(pairs * inter * 2);
  return m;
}

struct MoeArgs {
  const uint16_t* x;
  const void* idx;
  const float* weights;
  Weight w13, w2;
  uint16_t* y;
  int32_t* words;                         // [0] error bits, [1] active experts
  int32_t* expert;                        // [experts] ids of the active experts, ascending
  int32_t* count;                         // [experts] tokens of each
  int32_t* pairs;                         // [experts][N]: token << 8 | k, in token order
  uint16_t* hidden;                       // [N*K][I] bf16: weight * silu(gate) * up
  int N, H, K, E, I, wide;                // wide: 64-bit ids
};

// A routing entry as an expert id; whatever is no expert becomes -1, and bad
// tells entries outside [-1, E).
__device__ __forceinline__ int expert_at(const MoeArgs& a, int q, bool& bad) {
  if (a.wide) {
    const int64_t v = ((const int64_t*)a.idx)[q];
    bad = v < -1 || v >= a.E;
    return bad ? -1 : (int)v;
  }
  const int v = ((const int32_t*)a.idx)[q];
  bad = v < -1 || v >= a.E;
  return bad ? -1 : v;
}

constexpr int kUpThreads = EP_MAX_FEW_TOKENS;         // one thread per token in the preamble
constexpr int kUpWaves = kUpThreads / 64;

// What a workgroup of the first kernel knows about its expert.
struct Routing {
  uint32_t bitmap[EP_MAX_EXPERTS / 32];
  int32_t pair[EP_MAX_FEW_TOKENS];        // token << 8 | k
  float weight[EP_MAX_FEW_TOKENS];
  int32_t wave_count[kUpWaves];
  int32_t bad;
};

// The j-th (from 0) expert that some token names, and how many there are.
__device__ __forceinline__ int nth_active(const uint32_t* bitmap, int j, int& total) {
  const int lane = threadIdx.x & 63;
  const uint32_t w = lane < EP_MAX_EXPERTS / 32 ? bitmap[lane] : 0;
  int sum = __popc(w);
#pragma unroll
  for (int d = 1; d < EP_MAX_EXPERTS / 32; d <<= 1) {
    const int o = __shfl_up(sum, d);
    if (lane >= d) sum += o;
  }
  total = __builtin_amdgcn_readlane(sum, EP_MAX_EXPERTS / 32 - 1);
  if (j >= total) return -1;
  const int l = __ffsll((unsigned long long)__ballot(sum > j)) - 1;   // l < 32: lane 31 has total
  uint32_t word = __builtin_amdgcn_readlane(w, l);
  int n = j - __builtin_amdgcn_readlane(sum - __popc(w), l);
  while (n-- > 0) word &= word - 1;
  return l * 32 + __ffs(word) - 1;
}

// Finds expert number blockIdx.y among the active ones, its tokens in order and
// their weights.  Returns the id (-1: none), the tokens' count in n.
__device__ __forceinline__ int find_expert(const MoeArgs& a, Routing& r, int j, int& n,
                                           int& total) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid < EP_MAX_EXPERTS / 32) r.bitmap[tid] = 0;
  if (tid == 0) r.bad = 0;
  __syncthreads();
  for (int q = tid; q < a.N * a.K; q += kUpThreads) {
    bool bad;
    const int e = expert_at(a, q, bad);
    if (e >= 0) atomicOr(&r.bitmap[e >> 5], 1u << (e & 31));
    if (bad) r.bad = EP_LAYOUT_ERR_INDEX;
  }
  __syncthreads();
  const int e = uniform(nth_active(r.bitmap, j, total));
  if (e < 0) return -1;
  int k0 = -1;
  float w = 0.f;
  if (tid < a.N)
    for (int k = 0; k < a.K; k++) {
      bool bad;
      if (expert_at(a, tid * a.K + k, bad) == e) {
        if (k0 < 0) k0 = k;
        w += a.weights[tid * a.K + k];        // an expert named twice: the weights add up
      }
    }
  const uint64_t has = __ballot(k0 >= 0);
  if (lane == 0) r.wave_count[wave] = __popcll(has);
  __syncthreads();
  int at = __popcll(has & ((1ull << lane) - 1));
  n = 0;
#pragma unroll
  for (int v = 0; v < kUpWaves; v++) {
    if (v < wave) at += r.wave_count[v];
    n += r.wave_count[v];
  }
  if (k0 >= 0) {
    r.pair[at] = tid << 8 | k0;
    r.weight[at] = w;
  }
  __syncthreads();
  n = uniform(n);
  return e;
}

__device__ __forceinline__ float silu(float g) { return g / (1.f + expf(-g)); }

// Tokens pos0 .. of the expert's list through 16 gate and 16 up rows.
template <int F, int T>
__device__ __forceinline__ void up_tokens(const MoeArgs& a, const Routing& r,
                                          float (*red)[2][64][16], const Tile* tile, int i0,
                                          int pos0, int n) {
  using S = Stream<F, 2, T>;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int nt = min(n - pos0, S::tokens);
  const auto xr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(a.x), 0,
                                                    a.N * a.H * 2, kBufferWord3);
  int xoff[S::TT];
#pragma unroll
  for (int k = 0; k < S::TT; k++) {
    const int t = S::token(k);
    xoff[k] = t < nt ? (r.pair[pos0 + t] >> 8) * a.H * 2 : kOutside / 2;
  }
  S st;
  st.clear();
  st.run(wave, kUpWaves, (a.H + kStep - 1) / kStep, a.H, tile, xr, xoff);
  if (pos0 > 0) __syncthreads();              // red of the tokens before is consumed
#pragma unroll
  for (int i = 0; i < 2; i++)
    st.values(i, [&](int t, float v) { red[wave][i][t][lane & 15] = v; });
  __syncthreads();
  for (int q = threadIdx.x; q < nt * 16; q += kUpThreads) {
    const int t = q >> 4, c = q & 15;
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int v = 0; v < kUpWaves; v++) g += red[v][0][t][c], u += red[v][1][t][c];
    const int pair = r.pair[pos0 + t];
    // the one rounding between the products: the second one's operand is bf16
    if (i0 + c < a.I)
      a.hidden[(int64_t)((pair >> 8) * a.K + (pair & 255)) * a.I + i0 + c] =
          bf16_bits(r.weight[pos0 + t] * (silu(g) * u));
  }
}

// First kernel: blockIdx.x the tile of 16 gate and up rows, blockIdx.y the
// expert among the active ones.  BIG: lists of more than 16 tokens occur.
template <int F, bool BIG>
__global__ __launch_bounds__(kUpThreads) void moe_up_kernel(MoeArgs a) {
  __shared__ Routing r;
  __shared__ float red[kUpWaves][2][64][16];
  int n = 0, total = 0;
  const int j = blockIdx.y, i0 = blockIdx.x * 16;
  const int e = find_expert(a, r, j, n, total);
  if (blockIdx.x == 0 && j == 0 && threadIdx.x == 0) {
    a.words[0] = r.bad;
    a.words[1] = total;
  }
  if (e < 0) return;
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) a.expert[j] = e, a.count[j] = n;
    if ((int)threadIdx.x < n) a.pairs[j * a.N + threadIdx.x] = r.pair[threadIdx.x];
  }
  Tile tile[2];
  const int64_t row = (int64_t)e * 2 * a.I + i0;
  tile[0] = make_tile<F>(a.w13, row, a.I - i0, a.H);
  tile[1] = make_tile<F>(a.w13, row + a.I, a.I - i0, a.H);
  if (n <= 4) return up_tokens<F, 0>(a, r, red, tile, i0, 0, n);
  if (n <= 16) return up_tokens<F, 1>(a, r, red, tile, i0, 0, n);
  if constexpr (BIG) {
    if (n <= 32) return up_tokens<F, 2>(a, r, red, tile, i0, 0, n);
    for (int p = 0; p < n; p += 64) up_tokens<F, 4>(a, r, red, tile, i0, p, n);
  }
}

// ---- second product.  One workgroup owns 16 columns of y and walks the active
// experts; its wavefronts share the steps of all experts' contractions evenly
// and each adds its part to a tile [N][16] of its own in LDS, which are summed
// in order at the end: no atomics, the same sums on every run.
template <int F, int T>
__device__ __forceinline__ void down_tokens(const MoeArgs& a, float (*mine)[16], const Tile* tile,
                                            __amdgpu_buffer_rsrc_t hr, const int32_t* pairs,
                                            int pos0, int n, int first, int end) {
  using S = Stream<F, 1, T>;
  const int lane = threadIdx.x & 63;
  const int nt = min(n - pos0, S::tokens);
  int xoff[S::TT], tok[S::TT];
#pragma unroll
  for (int k = 0; k < S::TT; k++) {
    const int t = S::token(k);
    const int pair = t < nt ? pairs[pos0 + t] : 0;
    tok[k] = pair >> 8;
    xoff[k] = t < nt ? ((pair >> 8) * a.K + (pair & 255)) * a.I * 2 : kOutside / 2;
  }
  S st;
  st.clear();
  st.run(first, 1, end, a.I, tile, hr, xoff);
  st.values(0, [&](int t, float v) {
    // the lane that loaded token t's row knows its number
    const int k = S::quad ? 0 : t >> 4;
    const int row = __shfl(tok[k], S::quad ? t * 4 : t & 15);
    if (t < nt) mine[row][lane & 15] += v;
  });
}

template <int F, bool BIG>
__global__ __launch_bounds__(512) void moe_down_kernel(MoeArgs a) {
  extern __shared__ float lds[];              // [waves][N][16]
  const int waves = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  float(*mine)[16] = reinterpret_cast<float(*)[16]>(lds + (int64_t)wave * a.N * 16);
  for (int q = lane; q < a.N * 16; q += 64) mine[q >> 4][q & 15] = 0.f;
  const int h0 = blockIdx.x * 16;
  const int steps = (a.I + kStep - 1) / kStep;
  const int total = uniform(a.words[1]) * steps;
  const auto hr = __builtin_amdgcn_make_buffer_rsrc(a.hidden, 0, a.N * a.K * a.I * 2, kBufferWord3);
  int s = (int)((int64_t)total * wave / waves);
  const int stop = (int)((int64_t)total * (wave + 1) / waves);
  while (s < stop) {
    const int j = s / steps, first = s - j * steps, end = min(steps, first + stop - s);
    s += end - first;
    const int e = uniform(a.expert[j]), n = uniform(a.count[j]);
    const int32_t* pairs = a.pairs + (int64_t)j * a.N;
    const Tile tile = make_tile<F>(a.w2, (int64_t)e * a.H + h0, a.H - h0, a.I);
    if (n <= 4) down_tokens<F, 0>(a, mine, &tile, hr, pairs, 0, n, first, end);
    else if (n <= 16) down_tokens<F, 1>(a, mine, &tile, hr, pairs, 0, n, first, end);
    else if constexpr (BIG) {
      for (int p = 0; p < n; p += 32)
        down_tokens<F, 2>(a, mine, &tile, hr, pairs, p, n, first, end);
    }
  }
  __syncthreads();
  for (int q = threadIdx.x; q < a.N * 16; q += blockDim.x) {
    const int c = q & 15;
    float v = 0.f;
    for (int u = 0; u < waves; u++) v += lds[(int64_t)u * a.N * 16 + q];
    if (h0 + c < a.H) a.y[(int64_t)(q >> 4) * a.H + h0 + c] = bf16_bits(v);
  }
}

// ---------------------------------------------------------------- host side
// The kernel's weight format, or -1 where the descriptor is not valid for a
// contraction over `cols`.
int format_of(const ep_weight_t& w, int cols) {
  if (!w.data || ((uintptr_t)w.data & 15) || cols < 1 || cols > EP_MAX_CONTRACTION) return -1;
  if (w.format == EP_WEIGHT_BF16) return cols % 8 == 0 ? kBf16 : -1;
  if (!w.scales) return -1;
  if (w.format == EP_WEIGHT_INT4) {
    if ((uintptr_t)w.scales & 1) return -1;
    if (w.group != 32 && w.group != 64 && w.group != 128) return -1;
    if (cols % w.group != 0) return -1;
    const int z = w.zeros ? kInt128Z - kInt128 : 0;
    return z + (w.group == 128 ? kInt128 : w.group == 64 ? kInt64 : kInt32);
  }
  if (w.format == EP_WEIGHT_MXFP4)
    return w.group == 32 && cols % 32 == 0 && !w.zeros ? kMx : -1;
  return -1;
}

Weight kernel_weight(const ep_weight_t& w) {
  const bool q = w.format != EP_WEIGHT_BF16;
  return Weight{(const uint8_t*)w.data, q ? (const uint8_t*)w.scales : nullptr,
                w.format == EP_WEIGHT_INT4 ? w.zeros : nullptr};
}

int validate_moe(const ep_problem_t* p, int inter) {
  const int rc = validate_layout(p);
  if (rc != EP_OK) return rc;
  if (p->num_tokens > EP_MAX_FEW_TOKENS) return EP_ERR_INVALID_ARG;
  if (p->hidden < 8 || p->hidden % 8 != 0 || p->hidden > EP_MAX_CONTRACTION)
    return EP_ERR_INVALID_ARG;
  if (inter < 8 || inter % 8 != 0 || inter > EP_MAX_CONTRACTION) return EP_ERR_INVALID_ARG;
  // the rows between the products are indexed in 32 bits of bytes
  if ((int64_t)p->num_tokens * p->num_topk * inter * 2 > INT32_MAX / 2) return EP_ERR_INVALID_ARG;
  return EP_OK;
}

template <int F>
int launch_moe(const MoeArgs& a, int experts, hipStream_t st) {
  const dim3 up((a.I + 15) / 16, experts);
  const int down = (a.H + 15) / 16;
  const int waves = a.N > 128 ? 4 : 8;
  const size_t lds = sizeof(float) * 16 * a.N * waves;
  EP_LOG("moe: N=%d H=%d I=%d E=%d K=%d up=%ux%u down=%d", a.N, a.H, a.I, a.E, a.K, up.x, up.y,
         down);
  if (a.N <= 16) {
    moe_up_kernel<F, false><<<up, kUpThreads, 0, st>>>(a);
    moe_down_kernel<F, false><<<down, 64 * waves, lds, st>>>(a);
  } else {
    moe_up_kernel<F, true><<<up, kUpThreads, 0, st>>>(a);
    moe_down_kernel<F, true><<<down, 64 * waves, lds, st>>>(a);
  }
  return check_launch("moe_layer");
}

template <int F>
int launch_linear(int n, int cols, int rows, const void* x, const Weight& w, void* y,
                  hipStream_t st) {
  constexpr int RT = 2;
  const int gx = (rows + RT * 16 - 1) / (RT * 16);
  const uint16_t* xp = (const uint16_t*)x;
  uint16_t* yp = (uint16_t*)y;
  EP_LOG("quant_linear: n=%d cols=%d rows=%d grid=%d", n, cols, rows, gx);
  constexpr int B = 64 * kLinWaves;
  if (n <= 4) linear_kernel<F, RT, 0><<<dim3(gx, 1), B, 0, st>>>(xp, w, yp, n, cols, rows);
  else if (n <= 16) linear_kernel<F, RT, 1><<<dim3(gx, 1), B, 0, st>>>(xp, w, yp, n, cols, rows);
  else
    linear_kernel<F, RT, 2><<<dim3(gx, (n + 31) / 32), B, 0, st>>>(xp, w, yp, n, cols, rows);
  return check_launch("quant_linear");
}

}  // namespace

extern "C" {

int64_t ep_moe_workspace_bytes(const ep_problem_t* p, int32_t inter) {
  if (validate_moe(p, inter) != EP_OK) return -1;
  return make_moe_plan(p, inter).bytes;
}

int ep_moe_layer(const ep_problem_t* p, const ep_moe_args_t* a, void* stream) {
  if (!a) return EP_ERR_INVALID_ARG;
  int rc = validate_moe(p, a->inter);
  if (rc != EP_OK) return rc;
  const int f = format_of(a->w13, p->hidden);
  if (f < 0 || f != format_of(a->w2, a->inter)) return EP_ERR_INVALID_ARG;
  if (!a->workspace || ((uintptr_t)a->workspace & 255)) return EP_ERR_INVALID_ARG;
  if (p->num_tokens > 0 && (!a->x || ((uintptr_t)a->x & 15) || !a->topk_idx || !a->topk_weights ||
                            !a->y || ((uintptr_t)a->y & 1)))
    return EP_ERR_INVALID_ARG;
  rc = check_device();
  if (rc != EP_OK || p->num_tokens == 0) return rc;
  const MoePlan m = make_moe_plan(p, a->inter);
  char* ws = (char*)a->workspace;
  const MoeArgs k{(const uint16_t*)a->x, a->topk_idx, a->topk_weights, kernel_weight(a->w13),
                  kernel_weight(a->w2), (uint16_t*)a->y, (int32_t*)ws,
                  (int32_t*)(ws + m.o_expert), (int32_t*)(ws + m.o_count),
                  (int32_t*)(ws + m.o_pairs), (uint16_t*)(ws + m.o_hidden), p->num_tokens,
                  p->hidden, p->num_topk, p->num_experts, a->inter, p->topk_idx_bytes == 8};
  hipStream_t st = (hipStream_t)stream;
  switch (f) {
    case kBf16: return launch_moe<kBf16>(k, m.experts, st);
    case kInt128: return launch_moe<kInt128>(k, m.experts, st);
    case kInt64: return launch_moe<kInt64>(k, m.experts, st);
    case kInt32: return launch_moe<kInt32>(k, m.experts, st);
    case kInt128Z: return launch_moe<kInt128Z>(k, m.experts, st);
    case kInt64Z: return launch_moe<kInt64Z>(k, m.experts, st);
    case kInt32Z: return launch_moe<kInt32Z>(k, m.experts, st);
    default: return launch_moe<kMx>(k, m.experts, st);
  }
}

int ep_quant_linear(int32_t num_rows, int32_t cols, int32_t out_rows, const void* x,
                    const ep_weight_t* w, void* y, void* stream) {
  if (!w || num_rows < 0 || num_rows > EP_MAX_FEW_TOKENS || out_rows < 1 ||
      out_rows > EP_MAX_HIDDEN)
    return EP_ERR_INVALID_ARG;
  const int f = format_of(*w, cols);
  if (f < 0 || f == kBf16) return EP_ERR_INVALID_ARG;
  if (num_rows > 0 && (!x || ((uintptr_t)x & 15) || !y || ((uintptr_t)y & 1)))
    return EP_ERR_INVALID_ARG;
  const int rc = check_device();
  if (rc != EP_OK || num_rows == 0) return rc;
  const Weight k = kernel_weight(*w);
  hipStream_t st = (hipStream_t)stream;
  switch (f) {
    case kInt128: return launch_linear<kInt128>(num_rows, cols, out_rows, x, k, y, st);
    case kInt64: return launch_linear<kInt64>(num_rows, cols, out_rows, x, k, y, st);
    case kInt32: return launch_linear<kInt32>(num_rows, cols, out_rows, x, k, y, st);
    case kInt128Z: return launch_linear<kInt128Z>(num_rows, cols, out_rows, x, k, y, st);
    case kInt64Z: return launch_linear<kInt64Z>(num_rows, cols, out_rows, x, k, y, st);
    case kInt32Z: return launch_linear<kInt32Z>(num_rows, cols, out_rows, x, k, y, st);
    default: return launch_linear<kMx>(num_rows, cols, out_rows, x, k, y, st);
  }
}

}  // extern "C"
