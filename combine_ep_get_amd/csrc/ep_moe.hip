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

constexpr int kBufferWord3 = 0x00020000;   // raw buffer, 32-bit data format
constexpr int kOutside = 0x7FFFFFFF;       // offset out of every buffer's range
constexpr int kAbsent = 0x60000000;        // the same, with columns added
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
#ifndef EP_DQ
#define EP_DQ 2
#endif
#ifndef EP_D1
#define EP_D1 2
#endif
#ifndef EP_DB
#define EP_DB 2
#endif
#ifndef EP_UPW
#ifndef EP_W0
#define EP_W0 3
#endif
#define EP_UPW(F, T) (T == 0 ? EP_W0 : 2)
#endif
#ifndef EP_DNW
#define EP_DNW(F, T) 2
#endif
#ifndef EP_TWO
#define EP_TWO 64
#endif
#ifndef EP_UT
#define EP_UT 2
#endif
#ifndef EP_D2
#define EP_D2 1
#endif
#ifndef EP_DWAVES
#define EP_DWAVES 8
#endif
enum { kBf16, kMx, kInt128, kInt64, kInt32, kInt128Z, kInt64Z, kInt32Z };

template <int F>
struct Fmt {
  static constexpr bool quant = F != kBf16, integer = F >= kInt128, zeros = F >= kInt128Z;
  static constexpr int group = F == kInt128 || F == kInt128Z ? 128
                               : F == kInt64 || F == kInt64Z ? 64 : 32;
  static constexpr int step = quant ? 256 : 128;     // columns per step
  static constexpr int halves = step / 128;          // of 128 columns, four MFMAs each
  static constexpr int chunks = quant ? 8 : 16;      // 16-byte chunks of a row per step
  static constexpr int loads = chunks / 4;           // 1 KiB loads per tile and step
  // words of a row's codes that a lane feeds to MFMAs one after the other
  static constexpr int words = integer ? group / 32 : 4;
  static constexpr int groups = F == kMx ? 1 : quant ? 128 / group : 0;   // scales per half
  // first of the eight columns (of a half) that lane group g feeds to MFMA j
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
  // in a scalar register: a buffer descriptor that is not costs every load a loop
  const int n = uniform(max(0, min(16, rows)));
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
//
// Where the steps come from is the caller's cursor: `step` (which 128
// columns), `live` (false: load nothing, which adds zeros), `tile[RT]`, `xoff[TT]`
// (the lane's rows of x as byte offsets, kAbsent for none) and advance().
template <int F, int RT, int T>
struct Stream {
  static constexpr bool quad = T == 0;
  static constexpr int TT = quad ? 1 : T;
  static constexpr int tokens = quad ? 4 : 16 * TT;
  // Steps in flight: enough that the loads of a CU's wavefronts cover HBM's
  // latency, as far as the registers go.
  static constexpr int depth = Fmt<F>::quant ? (quad ? EP_DQ : TT <= 1 ? EP_D1 : EP_D2) : (quad ? EP_DB : 2);

  struct Slot {
    u32x4 w[RT][Fmt<F>::loads];                      // as loaded: see load()
    uint32_t s[RT][Fmt<F>::halves][Fmt<F>::groups ? Fmt<F>::groups : 1];
    uint32_t z[RT][Fmt<F>::halves][Fmt<F>::groups ? Fmt<F>::groups : 1];
    u32x4 x[TT][Fmt<F>::halves][quad ? 1 : 4];
  };

  // acc[i][j]: Quad: MFMA j's own rows (bf16, mxfp4), or [i][0] the whole sum
  // (int4); otherwise token tile j.  In the MFMA's result layout: lane r + 16 g
  // holds weight row r of tokens g*4 .. g*4+3.
  f32x4 acc[RT][quad ? 4 : TT];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
      for (int j = 0; j < (quad ? 4 : TT); j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // A step's loads.  One load instruction reads whole 128-byte lines: 16 lanes a
  // row's 256 bytes (bf16 weights and x: four rows per load), 8 lanes 128 bytes
  // (codes: eight rows).  xoff[k][j]: row j*4 + lane/16 of token tile k (Quad:
  // the row that token() names), in bytes.
  template <typename Cursor>
  __device__ __forceinline__ void load(Slot& b, const Cursor& at, int cols,
                                       __amdgpu_buffer_rsrc_t xr) {
    using M = Fmt<F>;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int step = uniform(at.live ? at.step : 0);
    const int c0 = step * M::step;
    const int left = at.live ? cols - c0 : 0;              // columns left from here
    const int rb = row_bytes<F>(cols);
    {
      const int chunk = lane & (M::chunks - 1), row = lane / M::chunks;
      const bool in = chunk * (M::quant ? 32 : 8) < left;
#pragma unroll
      for (int q = 0; q < M::loads; q++) {
        const int off = in ? (q * (64 / M::chunks) + row) * rb + chunk * 16 : kOutside;
#pragma unroll
        for (int i = 0; i < RT; i++)
          b.w[i][q] = __builtin_amdgcn_raw_buffer_load_b128(at.tile[i].data, off,
                                                            step * (M::chunks * 16), kNonTemporal);
      }
    }
    if constexpr (M::quant) {
      const int rg = row_groups<F>(cols);
#pragma unroll
      for (int m = 0; m < M::halves; m++)
#pragma unroll
        for (int q = 0; q < M::groups; q++) {
          const int c = m * 128 + (F == kMx ? g * 32 : q * M::group);
          const int n = r * rg + (c0 + c) / M::group;
#pragma unroll
          for (int i = 0; i < RT; i++) {
            if constexpr (F == kMx)
              b.s[i][m][q] = __builtin_amdgcn_raw_buffer_load_b8(at.tile[i].scale,
                                                                 c < left ? n : kOutside, 0, 0);
            else
              b.s[i][m][q] = __builtin_amdgcn_raw_buffer_load_b16(at.tile[i].scale,
                                                                  c < left ? n * 2 : kOutside, 0, 0);
            if constexpr (M::zeros)
              b.z[i][m][q] = __builtin_amdgcn_raw_buffer_load_b8(at.tile[i].zero,
                                                                 c < left ? n : kOutside, 0, 0);
          }
        }
    }
#pragma unroll
    for (int m = 0; m < M::halves; m++) {
      const int c = m * 128 + (quad ? M::col(g, lane & 3) : r * 8);
#pragma unroll
      for (int k = 0; k < TT; k++)
#pragma unroll
        for (int j = 0; j < (quad ? 1 : 4); j++)
          b.x[k][m][j] = __builtin_amdgcn_raw_buffer_load_b128(
              xr, c < left ? at.xoff[k][j] + c * 2 : kOutside, c0 * 2, 0);
    }
  }

  // From loaded rows to MFMA operands, through 4 KiB of LDS that are the
  // wavefront's own (its LDS accesses execute in order, so the fences only bind
  // the compiler).  Chunk c of row r lies at slot c ^ r of its row: the 8 lanes
  // of an access phase fall on different banks when they write (one row, 8
  // chunks) and when they read (8 rows, one chunk).
  static __device__ __forceinline__ void fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  template <int CHUNKS>
  static __device__ __forceinline__ int place(int row, int chunk) {
    return row * CHUNKS + (chunk ^ (row & (CHUNKS - 1)));
  }
  template <int CHUNKS>
  static __device__ __forceinline__ void put(u32x4* buf, const u32x4* v) {
    const int lane = threadIdx.x & 63;
    fence();
#pragma unroll
    for (int q = 0; q < CHUNKS / 4; q++)
      buf[place<CHUNKS>(q * (64 / CHUNKS) + lane / CHUNKS, lane & (CHUNKS - 1))] = v[q];
    fence();
  }

  // The four operands of x for a half that lies in buf.
  static __device__ __forceinline__ void take_x(const u32x4* buf, u32x4* o) {
    const int r = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int j = 0; j < 4; j++) o[j] = buf[place<16>(r, Fmt<F>::col(g, j) / 8)];
  }

  // Half m of a weight tile that lies in buf: bf16 the four operands, else the
  // four words of codes.
  static __device__ __forceinline__ void take_w(const u32x4* buf, int m, u32x4* o) {
    using M = Fmt<F>;
    const int r = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    if constexpr (!M::quant) {
#pragma unroll
      for (int j = 0; j < 4; j++) o[j] = buf[place<16>(r, j * 4 + g)];
    } else if constexpr (M::words == 4) {
      o[0] = buf[place<8>(r, m * 4 + g)];
    } else if constexpr (M::words == 2) {
#pragma unroll
      for (int q = 0; q < 2; q++) {
        const u32x2 v = reinterpret_cast<const u32x2*>(
            buf + place<8>(r, m * 4 + q * 2 + (g >> 1)))[g & 1];
        o[0][q * 2] = v.x, o[0][q * 2 + 1] = v.y;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; q++)
        o[0][q] = reinterpret_cast<const uint32_t*>(buf + place<8>(r, m * 4 + q))[g];
    }
  }

  // The eight bf16 weights of a word of codes (int4: 128 + code; mxfp4: scaled).
  static __device__ __forceinline__ u32x4 operand(uint32_t w, uint32_t scale) {
    u32x4 o;
    if constexpr (Fmt<F>::integer) {
#pragma unroll
      for (int q = 0; q < 4; q++) o[q] = ((w >> (4 * q)) & 0x000F000Fu) | 0x43004300u;
    } else {
      const float s = __uint_as_float(scale << 23);
      o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
      o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
      o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
      o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
    }
    return o;
  }

  // The products of a step.
  __device__ __forceinline__ void compute(const Slot& b, u32x4* buf) {
    using M = Fmt<F>;
    const f32x4 none{0.f, 0.f, 0.f, 0.f};
    constexpr uint32_t kOnes = 0x3F803F80u;
    const u32x4 ones{kOnes, kOnes, kOnes, kOnes};
    constexpr int per = M::integer ? 4 / M::groups : 4;      // MFMAs per group
    u32x4 w[RT][M::halves];                      // codes
    if constexpr (M::quant) {
#pragma unroll
      for (int i = 0; i < RT; i++) {
        put<M::chunks>(buf, b.w[i]);
#pragma unroll
        for (int m = 0; m < M::halves; m++) take_w(buf, m, &w[i][m]);
      }
    }
#pragma unroll
    for (int m = 0; m < M::halves; m++) {
      u32x4 x[TT][4];
#pragma unroll
      for (int k = 0; k < TT; k++) {
        if constexpr (quad) {
          x[k][0] = x[k][1] = x[k][2] = x[k][3] = b.x[k][m][0];
        } else {
          put<16>(buf, b.x[k][m]);
          take_x(buf, x[k]);
        }
      }
      if constexpr (!M::integer) {
#pragma unroll
        for (int i = 0; i < RT; i++) {
          u32x4 o[4];
          if constexpr (M::quant) {
#pragma unroll
            for (int j = 0; j < 4; j++) o[j] = operand(w[i][m][j], b.s[i][m][0]);
          } else {
            put<M::chunks>(buf, b.w[i]);
            take_w(buf, 0, o);
          }
#pragma unroll
          for (int j = 0; j < 4; j++)
#pragma unroll
            for (int k = 0; k < TT; k++) {
              f32x4& c = acc[i][quad ? j : k];
              c = mfma(x[k][j], o[j], c);
            }
        }
      } else if constexpr (quad) {
        const f32x4 sx = mfma(x[0][0], ones, none);      // register j: sum of piece j
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
          for (int q = 0; q < M::groups; q++) {
            float sum = 0.f, xs = 0.f;
#pragma unroll
            for (int j = q * per; j < (q + 1) * per; j++) {
              const f32x4 d = mfma(x[0][0], operand(w[i][m][j], 0), none);
              sum += d[j];
              xs += sx[j];
            }
            acc[i][0][0] = fmaf(bf16_value(b.s[i][m][q]), fmaf(-zero_of(b, i, m, q), xs, sum),
                                acc[i][0][0]);
          }
      } else {
#pragma unroll
        for (int q = 0; q < M::groups; q++) {
          f32x4 xs[TT], d[RT][TT];
#pragma unroll
          for (int k = 0; k < TT; k++) {
            xs[k] = none;
#pragma unroll
            for (int i = 0; i < RT; i++) d[i][k] = none;
          }
#pragma unroll
          for (int j = q * per; j < (q + 1) * per; j++) {
#pragma unroll
            for (int k = 0; k < TT; k++) xs[k] = mfma(x[k][j], ones, xs[k]);
#pragma unroll
            for (int i = 0; i < RT; i++) {
              const u32x4 o = operand(w[i][m][j], 0);
#pragma unroll
              for (int k = 0; k < TT; k++) d[i][k] = mfma(x[k][j], o, d[i][k]);
            }
          }
#pragma unroll
          for (int i = 0; i < RT; i++) {
            const float s = bf16_value(b.s[i][m][q]), z = zero_of(b, i, m, q);
#pragma unroll
            for (int k = 0; k < TT; k++)
#pragma unroll
              for (int e = 0; e < 4; e++)
                acc[i][k][e] = fmaf(s, fmaf(-z, xs[k][e], d[i][k][e]), acc[i][k][e]);
          }
        }
      }
    }
  }

  // What is taken off the codes as the operand holds them (128 + code).
  static __device__ __forceinline__ float zero_of(const Slot& b, int i, int m, int q) {
    return Fmt<F>::zeros ? 128.f + (float)b.z[i][m][q] : 136.f;
  }

  // Add `count` steps of the cursor to acc; after(i) follows step i's products.
  template <typename Cursor, typename After>
  __device__ __forceinline__ void run(int count, Cursor& at, int cols, __amdgpu_buffer_rsrc_t xr,
                                      u32x4* buf, After&& after) {
    Slot slot[depth];
#pragma unroll
    for (int d = 0; d < depth; d++) {
      at.live = d < count;
      load(slot[d], at, cols, xr);
      at.advance();
    }
    for (int i = 0; i < count; i += depth) {
#pragma unroll
      for (int d = 0; d < depth; d++) {
        compute(slot[d], buf);
        at.live = i + d + depth < count;
        load(slot[d], at, cols, xr);
        at.advance();
        after(i + d);
      }
    }
  }

  // Which token row the lane's load j of x is for in token tile k.
  static constexpr int rows = quad ? 1 : 4;            // such loads per half
  static __device__ __forceinline__ int token(int k, int j) {
    const int lane = threadIdx.x & 63;
    return quad ? (lane & 15) >> 2 : k * 16 + j * 4 + (lane >> 4);
  }

  // f(token, value) for every token row this lane holds of weight tile i (its
  // weight row is lane & 15).
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
};

constexpr int kBuffer = 256;               // 16-byte words of LDS per wavefront (Stream::put)

// The cursor over every by-th step of the same tiles and rows.
template <int RT, typename S>
struct Strided {
  Tile tile[RT];
  int xoff[S::TT][S::rows];
  int step, by;
  bool live;
  __device__ __forceinline__ void advance() { step += by; }
};

template <int F>
__device__ __forceinline__ int steps_of(int cols) {
  return (cols + Fmt<F>::step - 1) / Fmt<F>::step;
}

// How many of `steps` a wave takes that starts at `first` and goes on by `by`.
__device__ __forceinline__ int share_of(int steps, int first, int by) {
  return first < steps ? (steps - first + by - 1) / by : 0;
}

// ---------------------------------------------------------------- y = x W^T
constexpr int kLinWaves = 8;

// One workgroup: RT*16 rows of the weight, all columns split over the waves, 16 T
// rows of x (blockIdx.y).
template <int F, int RT, int T>
__global__ __launch_bounds__(64 * kLinWaves) void linear_kernel(
    const uint16_t* __restrict__ x, Weight w, uint16_t* __restrict__ y, int n, int cols, int rows) {
  using S = Stream<F, RT, T>;
  __shared__ float red[kLinWaves][RT][S::tokens][16];
  __shared__ u32x4 buf[kLinWaves][kBuffer];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int row0 = blockIdx.x * (RT * 16), t0 = blockIdx.y * S::tokens;
  const int nt = min(n - t0, S::tokens);
  Strided<RT, S> at;
#pragma unroll
  for (int i = 0; i < RT; i++)
    at.tile[i] = make_tile<F>(w, min(row0 + i * 16, rows), rows - row0 - i * 16, cols);
  const auto xr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(x) + (int64_t)t0 * cols,
                                                    0, nt * cols * 2, kBufferWord3);
#pragma unroll
  for (int k = 0; k < S::TT; k++)
#pragma unroll
    for (int q = 0; q < S::rows; q++) {
      const int t = S::token(k, q);
      at.xoff[k][q] = t < nt ? t * cols * 2 : kAbsent;
    }
  at.step = wave;
  at.by = kLinWaves;
  S st;
  st.clear();
  st.run(share_of(steps_of<F>(cols), wave, kLinWaves), at, cols, xr, buf[wave], [](int) {});
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
// Two ways through it.  Few (N <= 16): row t of an MFMA is token t for every
// expert, so a token that an expert does not have is a row of zeros, and the
// second product adds up over the experts in its accumulators.  Many: each
// expert's tokens are listed and packed into the rows.
constexpr int kFew = 16;
constexpr int kPairShift = 8;                // a listed pair: token << 8 | k

// Workspace: what the first kernel finds out about the routing, and the rows
// between the two products.
struct MoePlan {
  int32_t experts;                        // most experts that can be active: min(E, N*K)
  int64_t o_expert, o_count, o_start, o_pairs, o_hidden, bytes;   // byte offsets
};
// word 0: error bits (ep_layout_error), word 1: active experts

__host__ __device__ inline int64_t align256(int64_t v) { return (v + 255) & ~int64_t(255); }

MoePlan make_moe_plan(const ep_problem_t* p, int inter) {
  const int64_t N = p->num_tokens, pairs = N * p->num_topk;
  MoePlan m;
  m.experts = (int32_t)(pairs < p->num_experts ? pairs : p->num_experts);
  const int64_t list = align256((int64_t)m.experts * 4);
  m.o_expert = 256;
  m.o_count = m.o_expert + list;
  m.o_start = m.o_count + list;
  m.o_pairs = m.o_start + list;
  // many: uint16 [N*K]; few: bytes [experts][16]
  m.o_hidden = m.o_pairs + align256(N > kFew ? pairs * 2 : (int64_t)m.experts * kFew);
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
  int32_t* count;                         // [experts] many: tokens of each
  int32_t* start;                         // [experts] many: first of its pairs
  void* pairs;                            // many: pairs by expert; few: k + 1 (0: none) of
                                          // [expert][token]
  uint16_t* hidden;                       // [N*K][I] bf16: weight * silu(gate) * up
  int N, H, K, E, I, wide;                // wide: 64-bit ids
  int experts;
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

// The j-th (from 0) expert of the bitmap, -1 if it has fewer; and how many it has.
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

// What a workgroup of the first kernel knows about its expert's tokens.
struct Routing {
  uint32_t bitmap[EP_MAX_EXPERTS / 32];
  int32_t pair[EP_MAX_FEW_TOKENS];        // many: token << 8 | k; few: by token, -1 for none
  float weight[EP_MAX_FEW_TOKENS];
  int32_t wave_count[kUpWaves], wave_before[kUpWaves];
  int32_t bad;
};

// Finds the j-th active expert, its tokens (in order) with their weights, and
// how many pairs name lower experts.  ids: LDS for N*K entries.  Returns the
// id, -1 if there are fewer.
template <bool MANY>
__device__ __forceinline__ int find_expert(const MoeArgs& a, Routing& r, int16_t* ids, int j,
                                           int& n, int& before, int& total) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid < EP_MAX_EXPERTS / 32) r.bitmap[tid] = 0;
  if (tid == 0) r.bad = 0;
  __syncthreads();
  for (int q = tid; q < a.N * a.K; q += kUpThreads) {
    bool bad;
    const int e = expert_at(a, q, bad);
    ids[q] = (int16_t)e;
    if (e >= 0) atomicOr(&r.bitmap[e >> 5], 1u << (e & 31));
    if (bad) r.bad = EP_LAYOUT_ERR_INDEX;
  }
  __syncthreads();
  const int e = uniform(nth_active(r.bitmap, j, total));
  if (e < 0) return -1;
  int k0 = -1, below = 0;
  float w = 0.f;
  if (tid < a.N)
    for (int k = 0; k < a.K; k++) {
      const int o = ids[tid * a.K + k];
      if (o == e) {
        if (k0 < 0) k0 = k;
        w += a.weights[tid * a.K + k];        // an expert named twice: the weights add up
      }
      below += o >= 0 && o < e ? 1 : 0;
    }
  if constexpr (!MANY) {
    if (tid < kFew) {
      r.pair[tid] = k0 >= 0 ? tid << kPairShift | k0 : -1;
      r.weight[tid] = w;
    }
    n = a.N;
  } else {
    const uint64_t has = __ballot(k0 >= 0);
#pragma unroll
    for (int d = 32; d; d >>= 1) below += __shfl_xor(below, d);
    if (lane == 0) r.wave_count[wave] = __popcll(has), r.wave_before[wave] = below;
    __syncthreads();
    int at = __popcll(has & ((1ull << lane) - 1));
    n = before = 0;
#pragma unroll
    for (int v = 0; v < kUpWaves; v++) {
      if (v < wave) at += r.wave_count[v];
      n += r.wave_count[v];
      before += r.wave_before[v];
    }
    if (k0 >= 0) {
      r.pair[at] = tid << kPairShift | k0;
      r.weight[at] = w;
    }
    n = uniform(n);
  }
  __syncthreads();
  return e;
}

__device__ __forceinline__ float silu(float g) { return g / (1.f + expf(-g)); }

// Entries pos0 .. of the expert's list through 16 gate and 16 up rows.
template <int F, int T>
__device__ __forceinline__ void up_tokens(const MoeArgs& a, const Routing& r,
                                          float (*red)[16], u32x4 (*buf)[kBuffer],
                                          const Tile* tile, int i0, int pos0, int n) {
  using S = Stream<F, 2, T>;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int nt = min(n - pos0, S::tokens);
  const auto xr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(a.x), 0,
                                                    a.N * a.H * 2, kBufferWord3);
  Strided<2, S> at;
  at.tile[0] = tile[0], at.tile[1] = tile[1];
#pragma unroll
  for (int k = 0; k < S::TT; k++)
#pragma unroll
    for (int q = 0; q < S::rows; q++) {
      const int t = S::token(k, q), pair = t < nt ? r.pair[pos0 + t] : -1;
      at.xoff[k][q] = pair >= 0 ? (pair >> kPairShift) * a.H * 2 : kAbsent;
    }
  at.step = wave;
  at.by = kUpWaves;
  S st;
  st.clear();
  st.run(share_of(steps_of<F>(a.H), wave, kUpWaves), at, a.H, xr, buf[wave], [](int) {});
  if (pos0 > 0) __syncthreads();              // red of the tokens before is consumed
  // red[(wave * 2 + tile) * tokens + token][row]
#pragma unroll
  for (int i = 0; i < 2; i++)
    st.values(i, [&](int t, float v) { red[(wave * 2 + i) * S::tokens + t][lane & 15] = v; });
  __syncthreads();
  for (int q = threadIdx.x; q < nt * 16; q += kUpThreads) {
    const int t = q >> 4, c = q & 15;
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int v = 0; v < kUpWaves; v++) {
      g += red[v * 2 * S::tokens + t][c];
      u += red[(v * 2 + 1) * S::tokens + t][c];
    }
    const int pair = r.pair[pos0 + t];
    // the one rounding between the products: the second one's operand is bf16
    if (pair >= 0 && i0 + c < a.I)
      a.hidden[(int64_t)((pair >> kPairShift) * a.K + (pair & ((1 << kPairShift) - 1))) * a.I +
               i0 + c] = bf16_bits(r.weight[pos0 + t] * (silu(g) * u));
  }
}

// First kernel: blockIdx.x the tile of 16 gate and up rows, blockIdx.y the
// expert among the active ones.  T: token tiles per pass; 0 and 1 without MANY:
// few tokens.
template <int F, int T, bool MANY>
__global__ __launch_bounds__(kUpThreads, EP_UPW(F, T)) void moe_up_kernel(MoeArgs a) {
  __shared__ Routing r;
  __shared__ float red[kUpWaves * 2 * (T == 0 ? 4 : 16 * T)][16];
  __shared__ u32x4 buf[kUpWaves][kBuffer];
  extern __shared__ int16_t ids[];            // [N*K]
  int n = 0, before = 0, total = 0;
  const int j = blockIdx.y, i0 = blockIdx.x * 16;
  const int e = find_expert<MANY>(a, r, ids, j, n, before, total);
  if (blockIdx.x == 0 && j == 0 && threadIdx.x == 0) {
    a.words[0] = r.bad;
    a.words[1] = total;
  }
  if (e < 0) return;
  if (blockIdx.x == 0) {                      // what the second kernel wants to know
    const int tid = threadIdx.x;
    if (tid == 0) a.expert[j] = e;
    if constexpr (MANY) {
      if (tid == 0) a.count[j] = n, a.start[j] = before;
      if (tid < n) ((uint16_t*)a.pairs)[before + tid] = (uint16_t)r.pair[tid];
    } else if (tid < kFew) {
      const int pair = tid < a.N ? r.pair[tid] : -1;
      ((uint8_t*)a.pairs)[j * kFew + tid] =
          (uint8_t)(pair < 0 ? 0 : (pair & ((1 << kPairShift) - 1)) + 1);
    }
  }
  Tile tile[2];
  const int64_t row = (int64_t)e * 2 * a.I + i0;
  tile[0] = make_tile<F>(a.w13, row, a.I - i0, a.H);
  tile[1] = make_tile<F>(a.w13, row + a.I, a.I - i0, a.H);
  if constexpr (!MANY) {
    up_tokens<F, T>(a, r, red, buf, tile, i0, 0, n);
  } else {
    if (T == 1 || n > 16)
      for (int p = 0; p < n; p += 16 * T) up_tokens<F, T>(a, r, red, buf, tile, i0, p, n);
    else
      up_tokens<F, 1>(a, r, red, buf, tile, i0, 0, n);
  }
}

// ---- second product.  One workgroup owns 16 columns of y and walks the active
// experts; its wavefronts share the steps of all of them evenly, one stream of
// loads each that does not stop between experts.  The parts meet in LDS and are
// added in the wavefronts' order: no atomics, the same sums on every run.

// Few: token rows are the same for every expert, the accumulators go through.
template <int F, typename S>
struct FewCursor {
  const MoeArgs* a;
  const int32_t* expert;                  // LDS
  const uint8_t* map;                     // LDS [experts][16]
  int64_t row0;
  int rows, j, step, steps, n, rot;
  Tile tile[1];
  int xoff[1][S::rows];
  bool live;
  __device__ __forceinline__ void enter() {
    const int at = min(j, a->experts - 1);
    tile[0] = make_tile<F>(a->w2, (int64_t)uniform(expert[at]) * a->H + row0, rows, a->I);
#pragma unroll
    for (int q = 0; q < S::rows; q++) {
      const int t = S::token(0, q), k1 = map[at * kFew + t];
      xoff[0][q] = k1 ? (t * a->K + k1 - 1) * a->I * 2 : kAbsent;
    }
  }
  __device__ __forceinline__ void turn() {
    step = n + rot;
    if (step >= steps) step -= steps;
  }
  __device__ __forceinline__ void advance() {
    if (++n == steps) {
      n = 0;
      j++;
      enter();
    }
    turn();
  }
};

template <int F, int T>
__global__ __launch_bounds__(512, EP_DNW(F, T)) void moe_down_few_kernel(MoeArgs a) {
  using S = Stream<F, 1, T>;
  extern __shared__ u32x4 lds4[];
  int32_t* lds = reinterpret_cast<int32_t*>(lds4);
  const int waves = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  u32x4* buf = reinterpret_cast<u32x4*>(lds) + wave * kBuffer;
  float(*red)[S::tokens][16] =
      reinterpret_cast<float(*)[S::tokens][16]>(lds + waves * kBuffer * 4);
  int32_t* expert = lds + waves * (kBuffer * 4 + S::tokens * 16);
  uint8_t* map = reinterpret_cast<uint8_t*>(expert + a.experts);
  const int active = a.words[1];
  for (int q = threadIdx.x; q < a.experts; q += blockDim.x) expert[q] = a.expert[q];
  for (int q = threadIdx.x; q < a.experts * (kFew / 4); q += blockDim.x)
    reinterpret_cast<uint32_t*>(map)[q] = ((const uint32_t*)a.pairs)[q];
  __syncthreads();
  const int h0 = blockIdx.x * 16, steps = steps_of<F>(a.I);
  const int total = uniform(active) * steps;
  const int first = (int)((int64_t)total * wave / waves);
  const int count = (int)((int64_t)total * (wave + 1) / waves) - first;
  FewCursor<F, S> at;
  at.a = &a, at.expert = expert, at.map = map, at.row0 = h0, at.rows = a.H - h0;
  at.j = first / steps, at.n = first % steps, at.steps = steps;
  at.rot = blockIdx.x % steps;           // the same for all that share an expert's steps
  at.turn();
  S st;
  st.clear();
  if (count > 0) {
    at.enter();
    const auto hr = __builtin_amdgcn_make_buffer_rsrc(a.hidden, 0, a.N * a.K * a.I * 2,
                                                      kBufferWord3);
    st.run(count, at, a.I, hr, buf, [](int) {});
  }
  st.values(0, [&](int t, float v) { red[wave][t][lane & 15] = v; });
  __syncthreads();
  for (int q = threadIdx.x; q < a.N * 16; q += blockDim.x) {
    const int t = q >> 4, c = q & 15;
    float v = 0.f;
    for (int u = 0; u < waves; u++) v += red[u][t][c];
    if (h0 + c < a.H) a.y[(int64_t)t * a.H + h0 + c] = bf16_bits(v);
  }
}

// Many: an item is up to 16 T listed tokens of an expert.  The wavefronts share the
// steps of all items evenly, a contiguous range each; what a wavefront has of
// an item when it leaves it (a segment) goes to rows in LDS that nobody else
// writes: the item's own rows, by list position, if the segment begins the
// item, else the wavefront's extra rows (only its first segment can begin
// inside an item).  In the end every (token, column) sums up its own rows, in
// a fixed order.  LDS holds kRows listed pairs at a time; longer lists take
// several rounds.
// item: expert | first pair << 10 | tokens << 23.
constexpr int kManyWaves = 8;
constexpr int kRows = 384;

template <int F, int T>
struct ManyCursor {
  const MoeArgs* a;
  const uint32_t* items;                  // LDS
  const uint16_t* pairs;                  // LDS
  int64_t row0;
  int rows, steps, item, last, tail, rot;   // tail: the last item's end
  int begin, end, left, step;
  Tile tile[1];
  int xoff[T][4];
  bool live;
  __device__ __forceinline__ void enter(int from) {
    const uint32_t it = uniform(items[min(item, last)]);
    const int e = it & 1023, first = (it >> 10) & 8191, n = it >> 23;
    begin = from;
    end = item >= last ? tail : steps;
    left = end - begin;
    // wavefronts and workgroups start at different columns: rows of 4 KiB would
    // otherwise have them all in the same few memory channels
    step = begin + rot % left;
    tile[0] = make_tile<F>(a->w2, (int64_t)e * a->H + row0, rows, a->I);
#pragma unroll
    for (int k = 0; k < T; k++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int t = Stream<F, 1, T>::token(k, q);
        const int pair = t < n ? pairs[first + t] : 0;
        xoff[k][q] = t < n ? ((pair >> kPairShift) * a->K + (pair & ((1 << kPairShift) - 1))) *
                                 a->I * 2
                           : kAbsent;
      }
  }
  __device__ __forceinline__ void advance() {
    if (--left == 0) {
      item++;
      enter(0);
    } else if (++step == end) {
      step = begin;
    }
  }
};

// LDS of the kernel below: buffers, rows, items, list, positions.
__host__ __device__ inline int most_items(int experts, int pairs, int T) {
  return experts + pairs / (16 * T);
}
__host__ __device__ inline int list_words(int pairs) { return (pairs + 1) / 2; }
size_t many_lds(int N, int K, int experts, int T) {
  return (size_t)kManyWaves * kBuffer * 16 + (kRows + 16 * T + kManyWaves * 16 * T) * 64 +
         4 * ((size_t)most_items(experts, N * K, T) + 2 * list_words(N * K));
}

template <int F, int T>
__global__ __launch_bounds__(64 * kManyWaves, EP_DNW(F, T)) void moe_down_many_kernel(MoeArgs a) {
  using S = Stream<F, 1, T>;
  constexpr int kOut = EP_MAX_FEW_TOKENS * 16 / (64 * kManyWaves);   // results per thread
  extern __shared__ u32x4 lds4[];       // (the type aligns it: behind the variables below)
  int32_t* lds = reinterpret_cast<int32_t*>(lds4);
  __shared__ int n_items;
  __shared__ uint32_t extra_item[kManyWaves];        // item of the extra rows, 0: none
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int NK = a.N * a.K;
  u32x4* buf = reinterpret_cast<u32x4*>(lds) + wave * kBuffer;
  float(*own)[16] = reinterpret_cast<float(*)[16]>(lds + kManyWaves * kBuffer * 4);
  float(*extra)[16] = own + kRows + 16 * T;          // [waves][16 T]
  uint32_t* items = reinterpret_cast<uint32_t*>(extra + kManyWaves * 16 * T);
  uint16_t* pairs = reinterpret_cast<uint16_t*>(items + most_items(a.experts, NK, T));
  uint16_t* place = pairs + 2 * list_words(NK);      // where in the list (token, k) is
  const int active = uniform(a.words[1]);
  for (int q = threadIdx.x; q < list_words(NK); q += blockDim.x) {
    reinterpret_cast<uint32_t*>(pairs)[q] = ((const uint32_t*)a.pairs)[q];
    reinterpret_cast<uint32_t*>(place)[q] = ~0u;
  }
  if (wave == 0) {                        // the items, in the experts' order
    int base = 0;
    for (int j0 = 0; j0 < active; j0 += 64) {
      const int j = j0 + lane;
      const int n = j < active ? a.count[j] : 0, e = j < active ? a.expert[j] : 0;
      const int first = j < active ? a.start[j] : 0;
      const int mine = (n + 16 * T - 1) / (16 * T);
      int up_to = mine;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(up_to, d);
        if (lane >= d) up_to += o;
      }
      int at = base + up_to - mine;
      for (int p = 0; p < n; p += 16 * T)
        items[at++] = e | (first + p) << 10 | (uint32_t)min(16 * T, n - p) << 23;
      base += __builtin_amdgcn_readlane(up_to, 63);
    }
    if (lane == 0) n_items = base;
  }
  __syncthreads();
  const int all = uniform(n_items);
  for (int i = threadIdx.x; i < all; i += blockDim.x) {
    const uint32_t it = items[i];
    for (int q = 0; q < (int)(it >> 23); q++) {
      const int at = ((it >> 10) & 8191) + q, pair = pairs[at];
      place[(pair >> kPairShift) * a.K + (pair & ((1 << kPairShift) - 1))] = (uint16_t)at;
    }
  }
  const int h0 = blockIdx.x * 16, steps = steps_of<F>(a.I);
  const auto hr = __builtin_amdgcn_make_buffer_rsrc(a.hidden, 0, NK * a.I * 2, kBufferWord3);
  float out[kOut];
#pragma unroll
  for (int i = 0; i < kOut; i++) out[i] = 0.f;
  // a round: the items whose first pair is in [from, from + kRows)
  for (int from = 0, i0 = 0, i1 = 0; i0 < all; from += kRows, i0 = i1) {
    for (bool more = true; more;) {
      const int i = i1 + lane;
      const int in = __popcll(
          __ballot(i < all && (int)((items[min(i, all - 1)] >> 10) & 8191) < from + kRows));
      i1 += in;
      more = in == 64;
    }
    if (i1 == i0) continue;
    const int total = (i1 - i0) * steps;
    const int s0 = (int)((int64_t)total * wave / kManyWaves);
    const int s1 = (int)((int64_t)total * (wave + 1) / kManyWaves);
    if (lane == 0) extra_item[wave] = 0;
    if (s1 > s0) {
      ManyCursor<F, T> at;
      at.a = &a, at.items = items, at.pairs = pairs, at.row0 = h0, at.rows = a.H - h0;
      at.steps = steps, at.rot = blockIdx.x + wave;
      at.item = i0 + s0 / steps;
      at.last = i0 + (s1 - 1) / steps;
      at.tail = (s1 - 1) % steps + 1;
      at.enter(s0 % steps);
      if (at.begin && lane == 0) extra_item[wave] = items[at.item];
      int item = at.item, left = at.left;            // where the products are, behind the loads
      bool whole = at.begin == 0;
      S st;
      st.clear();
      st.run(s1 - s0, at, a.I, hr, buf, [&](int i) {
        if (i >= s1 - s0 || --left > 0) return;
        const uint32_t it = uniform(items[item]);
        const int n = it >> 23;
        float(*to)[16] = whole ? own + ((it >> 10) & 8191) - from : extra + wave * 16 * T;
        st.values(0, [&](int t, float v) {
          if (t < n) to[t][lane & 15] = v;
        });
        st.clear();
        whole = true;
        left = ++item < at.last ? steps : at.tail;
      });
    }
    __syncthreads();
    const uint32_t last = items[i1 - 1];
    const int lo = (items[i0] >> 10) & 8191, hi = ((last >> 10) & 8191) + (last >> 23);
#pragma unroll
    for (int i = 0; i < kOut; i++) {
      const int q = threadIdx.x + i * 64 * kManyWaves, t = q >> 4, c = q & 15;
      if (t >= a.N) break;
      for (int k = 0; k < a.K; k++) {
        const int p = place[t * a.K + k];
        if (p < lo || p >= hi) continue;             // another round's, or no pair
        out[i] += own[p - from][c];
#pragma unroll
        for (int u = 0; u < kManyWaves; u++) {
          const int at = p - (int)((extra_item[u] >> 10) & 8191);
          if (at >= 0 && at < (int)(extra_item[u] >> 23)) out[i] += extra[u * 16 * T + at][c];
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kOut; i++) {
    const int q = threadIdx.x + i * 64 * kManyWaves, t = q >> 4, c = q & 15;
    if (t < a.N && h0 + c < a.H) a.y[(int64_t)t * a.H + h0 + c] = bf16_bits(out[i]);
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

template <int F, int T, bool MANY>
void launch_moe(const MoeArgs& a, hipStream_t st) {
  const dim3 up((a.I + 15) / 16, a.experts);
  const int down = (a.H + 15) / 16;
  const size_t ids = sizeof(int16_t) * a.N * a.K;
  moe_up_kernel<F, (MANY ? EP_UT : T), MANY><<<up, kUpThreads, ids, st>>>(a);
  if constexpr (MANY) {
    moe_down_many_kernel<F, T><<<down, 64 * kManyWaves, many_lds(a.N, a.K, a.experts, T), st>>>(a);
  } else {
    constexpr int waves = EP_DWAVES;
    const size_t lds = sizeof(float) * waves * (kBuffer * 4 + Stream<F, 1, T>::tokens * 16) +
                       (size_t)a.experts * (4 + kFew);
    moe_down_few_kernel<F, T><<<down, 64 * waves, lds, st>>>(a);
  }
}

template <int F>
int launch_moe(const MoeArgs& a, hipStream_t st) {
  const int64_t pairs = (int64_t)a.N * a.K;
  EP_LOG("moe: N=%d H=%d I=%d E=%d K=%d", a.N, a.H, a.I, a.E, a.K);
  if (a.N <= 4) launch_moe<F, 0, false>(a, st);
  else if (a.N <= kFew) launch_moe<F, 1, false>(a, st);
  else if (pairs <= EP_TWO * a.E) launch_moe<F, 1, true>(a, st);
  else launch_moe<F, 2, true>(a, st);
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
                  (int32_t*)(ws + m.o_start), ws + m.o_pairs, (uint16_t*)(ws + m.o_hidden),
                  p->num_tokens, p->hidden, p->num_topk, p->num_experts, a->inter,
                  p->topk_idx_bytes == 8, m.experts};
  hipStream_t st = (hipStream_t)stream;
  switch (f) {
    case kBf16: return launch_moe<kBf16>(k, st);
    case kInt128: return launch_moe<kInt128>(k, st);
    case kInt64: return launch_moe<kInt64>(k, st);
    case kInt32: return launch_moe<kInt32>(k, st);
    case kInt128Z: return launch_moe<kInt128Z>(k, st);
    case kInt64Z: return launch_moe<kInt64Z>(k, st);
    case kInt32Z: return launch_moe<kInt32Z>(k, st);
    default: return launch_moe<kMx>(k, st);
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
