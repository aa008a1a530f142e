// ep_moe.hip -- the experts' products for a few tokens (include/ep_get.h states
// the contracts): the whole expert layer in two kernels, and the product of a few
// rows with a 4-bit weight.
//
// All of it is one loop, `Stream`: 16-row tiles of a weight flow from HBM
// into v_mfma_f32_16x16x32_bf16, whose other operand is rows of x.  The weights
// are the bytes that count (a decode batch has too few tokens for the products to
// matter: 16 tokens are 16 flops per weight byte in bf16, HBM's rate allows
// about 400), so every choice serves the stream:
//   - a load instruction reads whole 128-byte lines: 16 lanes 256 bytes of a bf16
//     row, 8 lanes 128 bytes of a row of codes.  The MFMA wants lane r + 16 g
//     to hold columns of row r; loading that directly touches 64 bytes of 16
//     rows at a time, which reached 5.1 TB/s where whole lines reach 7.0 (493 MB,
//     both as bare loads).  The loaded tile is turned through LDS, private to the
//     wavefront, so there is no barrier (but see SHARED);
//   - loads run `depth` steps ahead in registers;
//   - the wavefronts of a workgroup split the contraction and meet once, at the
//     end;
//   - where an access falls outside (columns behind the end, rows behind the
//     last, absent tokens) its buffer offset is out of range and the hardware
//     returns zeros, so the loop has no branches.
//
// A step is 128 columns of bf16 or 256 of codes, four MFMAs per 128.  Which eight
// columns of these 128 lane group g feeds to MFMA j is free as long as both operands
// agree (Fmt::col): it is what a lane reads from LDS at once.  A 4-bit weight is
// scaled per (row, group): lane r holds row r's column of the 16x16 result,
// so one factor per lane does it, after the sum over the group, in float32.  int4
// codes become bf16 by putting the nibble under the exponent of 128 (exact:
// 128 + code); the 128 and the zero point leave again as (128 + zero) * sum(x),
// whose sum comes from an MFMA with ones.  E2M1 codes with their power-of-two
// scale are exact bf16 values already.
//
// Up to four tokens (`Quad`): rows t*4 + j of the MFMA's 16 hold the four
// column pieces j of token t, so one load per half brings all of x and every
// lane takes part; MFMA j's row t*4 + j is the product wanted, the other rows
// are ignored.
//
// What it reaches (weights' bytes over the whole call, HBM reads at 7.0 TB/s at best):
// bf16 6.5 TB/s at one token and 6.2 at 256; 4-bit 4.6 at one token, 5.1 at 16, 3.7
// at 64, where the SIMDs run VALU (codes to bf16) 40% and MFMA 20% of the time and two
// wavefronts each do not cover the rest: the first product has no registers for more
// (233), the second no workgroups (224 of eight wavefronts for 256 CUs).  Calls under 50
// MB are the two launches' and three dependent loads' latency (routing, weights, sums).
//
// Times in the comments below compare two builds that differ in that point alone;
// later steps may have made both faster.
//
// Weights are taken to be finite: a column or token that is not there is a zero
// of x, and zero times an infinite weight would not be zero.
#include "ep_host.h"

#include <type_traits>

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kBufferWord3 = 0x00020000;   // raw buffer, 32-bit data format
constexpr int kOutside = 0x7FFFFFFF;       // offset out of every buffer's range
constexpr int kAbsent = 0x60000000;        // the same, with columns added
constexpr int kNonTemporal = 2;            // NT in the cache-policy operand

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Loads outside [0, bytes) return zeros.  The scalar offset counts as part of what is
// checked, also where it is behind the end by itself (0 bytes and an offset: all zeros).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, kBufferWord3);
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

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
  static constexpr int step = quant ? 256 : 128;     // columns per step
  static constexpr int halves = step / 128;          // of 128 columns, four MFMAs each
  static constexpr int chunks = quant ? 8 : 16;      // 16-byte chunks of a row per step
  static constexpr int loads = chunks / 4;           // 1 KiB loads per tile and step
  // words of a row's codes that a lane reads together and feeds to MFMAs one after
  // the other: as many as stay inside a group, so that an MFMA's 32 columns are of
  // one group (mxfp4 scales each lane's codes by themselves)
  static constexpr int words = integer ? group / 32 : 4;
  // first of the eight columns (of a half) that lane group g feeds to MFMA j
  static __device__ __forceinline__ int col(int g, int j) {
    if constexpr (quant && words == 4) return g * 32 + j * 8;
    else if constexpr (words == 2) return (j >> 1) * 64 + g * 16 + (j & 1) * 8;
    else return j * 32 + g * 8;
  }
  static constexpr int groups = quant ? 128 / group : 1;    // scales per half
  static constexpr int scales = quant ? step / group : 0;   // scales of a row per step
  static constexpr int scale_bytes = F == kMx ? 1 : 2;
  // steps whose scales of a row are 16 bytes (their zeros 8)
  static constexpr int chunk = quant ? 16 / (scales * scale_bytes) : 1;
};

// Bytes of a row of codes (or bf16 values), and its number of groups.
template <int F>
__device__ __forceinline__ int row_bytes(int cols) { return Fmt<F>::quant ? cols / 2 : cols * 2; }
template <int F>
__device__ __forceinline__ int row_groups(int cols) {
  return Fmt<F>::quant ? cols / Fmt<F>::group : 0;
}
template <int F>
__device__ __forceinline__ int steps_of(int cols) {
  return (cols + Fmt<F>::step - 1) / Fmt<F>::step;
}

struct Weight {           // kernel argument: ep_weight_t without what the kernel's type says
  const uint8_t* data;
  const uint8_t* scale;
  const uint8_t* zero;
};

// ---------------------------------------------------------------- weight tiles
// RT tiles of 16 rows: tile i starts at row `row` + i*16, or, where the tiles are
// pairs of gate and up rows (`far` > 0), at row + (i/2)*16 + (i%2)*far.  `rows` is
// how many rows there are from `row` on (for pairs: of each kind; none if negative);
// those behind are out of range.  The scales of all tiles share one buffer; what it
// returns for rows that are not there only reaches results that nobody stores.
template <int F, int RT>
struct Tiles {
  const uint8_t* data[RT];
  const uint8_t *scale, *zero;
  int bytes[RT], scale_end;
  __device__ __forceinline__ void set(const Weight& w, int64_t row, int rows, int far, int cols) {
    const int rb = row_bytes<F>(cols), rg = row_groups<F>(cols);
    rows = max(0, rows);
#pragma unroll
    for (int i = 0; i < RT; i++) {
      const int at = far ? (i >> 1) * 16 : i * 16;
      // in a scalar register: a descriptor that is not costs every load a loop
      bytes[i] = uniform(max(0, min(16, rows - at))) * rb;
      data[i] = w.data + (row + at + (far ? (i & 1) * far : 0)) * rb;
    }
    if constexpr (Fmt<F>::quant) {
      const int span = uniform(far ? far + min(rows, RT * 8) : min(rows, RT * 16));
      scale_end = span * rg;
      scale = w.scale + row * rg * Fmt<F>::scale_bytes;
      if constexpr (Fmt<F>::zeros) zero = w.zero + row * rg;
    }
  }
};

// ---------------------------------------------------------------- the stream
// RT weight tiles times T token tiles of 16 (T == 0: Quad, up to 4 tokens); PART: the
// last step may have fewer columns, the last chunk fewer steps.
//
// Scales come 16 bytes of a row at a time, for Fmt::chunk steps (PART: value by value
// at every step).  A load of them touches as many lines as four of codes do: 64 tokens,
// 4-bit, 7168 x 2048: 214 us for the layer, with one for every step 236; one row
// by 7168 x 7168 of mxfp4, which has eight scales a step: 7.9 us, value by value 10.1.
//
// Where the steps come from is the caller's cursor: `step` (which columns), `serial`
// (another one for every run of steps inside a chunk and the same tiles), `live`
// (false: load nothing, which adds zeros), `tiles`, `xoff[TT][rows]` (the row of x
// of token(k, j) in bytes, kAbsent for none) and advance().
//
// SHARED: the four wavefronts of a workgroup take the same steps of the same rows of x
// and different tiles.  Each loads a quarter of a step's x into LDS for all, and as
// registers hold neither it nor the codes during the products, the next step's loads
// go out before them.  One barrier a step: x alternates between two places, and who is
// past the barrier of a step has read the step before.  64 tokens, 4-bit, 7168 x 2048:
// 196 us for the layer, with each wavefront's own x 214.
template <int F, int RT, int T, bool PART, bool SHARED = false>
struct Stream {
  using M = Fmt<F>;
  static constexpr bool quad = T == 0;
  static constexpr int TT = quad ? 1 : T;
  static constexpr int tokens = quad ? 4 : 16 * TT;
  static constexpr int rows = quad || SHARED ? 1 : 4;             // loads of x per tile and half
  static constexpr int shared_words = SHARED ? TT * M::halves * 256 : 0;   // a step's x
  static constexpr int values_per_row = RT * M::scales;           // scales of a step, all tiles
  static constexpr int scale_loads = (values_per_row + 3) / 4;    // a value per lane group
  // Steps in flight: enough that the loads of a CU's wavefronts cover HBM's latency, as
  // far as the registers go.  Codes with token tiles have one, where a second step's x
  // would leave fewer wavefronts (the layer with 4-bit experts: 13 tokens, 1952 x 992:
  // 32.1 us, with two steps 36.7; 16 tokens, 7168 x 2048: 157 and 162; 64 tokens with
  // pairs of tiles, which spill then: 245 and 339).
  static constexpr int depth = M::quant && !quad ? 1 : 2;
  // 16-byte words of LDS per wavefront: the tiles of a step, then scales and zeros.
  // x passes through the same words, and in the end the sums.
  static constexpr int tile_words = 16 * M::chunks;
  // Scales by chunks?  Not where it gains nothing: Quad has one load per step either way
  // with groups of 128 (one token: 41.4 us, by chunks 44.2); nor where the registers are
  // out: 352 bytes spilled, 256 tokens 529 us against 333.
  static constexpr bool wide =
      M::quant && !PART && !(quad && M::group == 128) && !(F == kInt32Z && TT > 1);
  static constexpr int scale_words = M::integer ? 16 * scale_loads : wide ? 8 * RT : 0;
  static constexpr int results = RT * tokens * 16;                // floats of a wavefront's sums
  static constexpr int most(int a, int b) { return a > b ? a : b; }
  static constexpr int buffer_words = most(
      most(RT * tile_words + scale_words * (M::zeros ? 2 : 1), quad ? 0 : 256), results / 4);

  struct Slot {
    u32x4 w[RT][M::loads];                           // as loaded: see load()
    uint32_t s[M::quant && !wide ? scale_loads : 1], z[M::zeros && !wide ? scale_loads : 1];
    u32x4 sc;                                        // wide: the chunk of row lane & 15 of
    u32x2 zc;                                        // tile lane >> 4
    int serial, step;
    u32x4 x[TT][M::halves][rows];                    // as loaded (Quad: the MFMA operand)
  };

  // acc[i][j]: Quad: MFMA j's own rows (bf16, mxfp4), or [i][0] the whole sum
  // (int4); otherwise token tile j.  In the MFMA's result layout: lane r + 16 g
  // holds weight row r of tokens g*4 .. g*4+3.
  f32x4 acc[RT][quad ? 4 : TT];
  // The lane's offsets: loads of the tiles, of the scales (in values), of x.
  int woff[M::loads], soff[M::quant && !wide ? scale_loads : 1], xcol;

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
      for (int j = 0; j < (quad ? 4 : TT); j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // far: as in Tiles::set
  __device__ __forceinline__ void init(int cols, int far) {
    clear();
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int rb = row_bytes<F>(cols), rg = row_groups<F>(cols);
#pragma unroll
    for (int q = 0; q < M::loads; q++)
      woff[q] = (q * (64 / M::chunks) + lane / M::chunks) * rb + (lane & (M::chunks - 1)) * 16;
    if constexpr (wide) {
      const int row = r + (far ? (g >> 1) * 16 + (g & 1) * far : g * 16);
      soff[0] = g < RT ? row * rg : kOutside / 2;
    } else if constexpr (M::quant) {
#pragma unroll
      for (int q = 0; q < scale_loads; q++) {        // lane group g has value q*4 + g of its row
        const int v = q * 4 + g, i = v / M::scales;
        const int row = r + (far ? (i >> 1) * 16 + (i & 1) * far : i * 16);
        soff[q] = v < values_per_row ? row * rg + v % M::scales : kOutside / 2;
      }
    }
    xcol = quad ? M::col(g, lane & 3) : r * 8;
  }

  // A step's loads.  x comes as the weights do: 256 bytes of four rows per load (a load
  // in the MFMA's layout, 64 bytes of 16 rows, takes four times as long in L1).
  template <typename Cursor>
  __device__ __forceinline__ void load(Slot& b, Cursor& at, bool live, int cols, const void* x,
                                       int xbytes) {
    at.live = live;
    const int step = uniform(at.live ? at.step : 0);
#pragma unroll
    for (int i = 0; i < RT; i++) {
      const auto rs = buffer(at.tiles.data[i], at.live ? at.tiles.bytes[i] : 0);
#pragma unroll
      for (int q = 0; q < M::loads; q++)
        b.w[i][q] = __builtin_amdgcn_raw_buffer_load_b128(rs, woff[q], step * (M::chunks * 16),
                                                          kNonTemporal);
    }
    if constexpr (wide) {
      b.step = step;
      // Quad: at every step, as a load that may not be there would have the other
      // step's wait include it
      if (quad || (at.live && b.serial != at.serial)) {
        b.serial = at.serial;
        const int c = (uint32_t)step / M::chunk;
        const int n = at.live ? at.tiles.scale_end : 0;
        b.sc = __builtin_amdgcn_raw_buffer_load_b128(buffer(at.tiles.scale, n * M::scale_bytes),
                                                     soff[0] * M::scale_bytes, c * 16, 0);
        if constexpr (M::zeros)
          b.zc = __builtin_amdgcn_raw_buffer_load_b64(buffer(at.tiles.zero, n), soff[0], c * 8, 0);
      }
    } else if constexpr (M::quant) {
      const int n = at.live ? at.tiles.scale_end : 0;
      const auto ss = buffer(at.tiles.scale, n * M::scale_bytes);
#pragma unroll
      for (int q = 0; q < scale_loads; q++) {
        if constexpr (M::scale_bytes == 1)
          b.s[q] = __builtin_amdgcn_raw_buffer_load_b8(ss, soff[q], step * M::scales, 0);
        else
          b.s[q] = __builtin_amdgcn_raw_buffer_load_b16(ss, soff[q] * 2, step * (M::scales * 2), 0);
      }
      if constexpr (M::zeros) {
        const auto zs = buffer(at.tiles.zero, n);
#pragma unroll
        for (int q = 0; q < scale_loads; q++)
          b.z[q] = __builtin_amdgcn_raw_buffer_load_b8(zs, soff[q], step * M::scales, 0);
      }
    }
    const auto xr = buffer(x, at.live ? xbytes : 0);
    const int left = cols - step * M::step;          // columns left from here
#pragma unroll
    for (int m = 0; m < M::halves; m++) {
      const int c = m * 128 + xcol;
      const bool in = !PART || c < left;
#pragma unroll
      for (int k = 0; k < TT; k++)
#pragma unroll
        for (int j = 0; j < rows; j++)
          b.x[k][m][j] = __builtin_amdgcn_raw_buffer_load_b128(
              xr, in ? at.xoff[k][j] + c * 2 : kOutside, step * (M::step * 2), 0);
    }
  }

  // The wavefront's LDS accesses execute in order; the fences bind the compiler.
  static __device__ __forceinline__ void fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }

  // Where chunk c of row r lies in its tile: permuted so that the 8 lanes of an
  // access phase fall on different banks when they write (a row's chunks) and when
  // they read (8 rows, one chunk).
  static __device__ __forceinline__ int place(int r, int c) {
    return r * M::chunks + (c ^ (r & (M::chunks - 1)));
  }

  // Write the step's tiles and scales to LDS.
  __device__ __forceinline__ void put(const Slot& b, u32x4* buf) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    fence();
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
      for (int q = 0; q < M::loads; q++)
        buf[i * tile_words +
            place(q * (64 / M::chunks) + lane / M::chunks, lane & (M::chunks - 1))] = b.w[i][q];
    if constexpr (wide) {
      // of each row: its values of all tiles
      const int in = (uint32_t)b.step % M::chunk;    // step of the chunk
      if (g < RT) {
        if constexpr (!M::integer) {
          reinterpret_cast<u32x2*>(buf + RT * tile_words)[r * RT + g] =
              in ? u32x2{b.sc[2], b.sc[3]} : u32x2{b.sc[0], b.sc[1]};
        } else {
          float* sb = reinterpret_cast<float*>(buf + RT * tile_words) + r * 4 * scale_loads +
                      g * M::scales;
          uint32_t v[M::scales / 2];                 // pairs of bf16
#pragma unroll
          for (int q = 0; q < M::scales / 2; q++) {
            v[q] = b.sc[q];
#pragma unroll
            for (int c = 1; c < M::chunk; c++)
              if (in == c) v[q] = b.sc[c * (M::scales / 2) + q];
            sb[q * 2] = __uint_as_float(v[q] << 16);
            sb[q * 2 + 1] = __uint_as_float(v[q] & 0xFFFF0000u);
          }
          if constexpr (M::zeros) {
            float* zb = sb + scale_words * 4;
            const uint64_t z = ((uint64_t)b.zc.y << 32 | b.zc.x) >> (in * M::scales * 8);
#pragma unroll
            for (int q = 0; q < M::scales; q++) zb[q] = 128.f + (float)(uint8_t)(z >> (q * 8));
          }
        }
      }
    } else if constexpr (M::integer) {
      float* sb = reinterpret_cast<float*>(buf + RT * tile_words) + r * 4 * scale_loads + g;
#pragma unroll
      for (int q = 0; q < scale_loads; q++) {
        sb[q * 4] = __uint_as_float(b.s[q] << 16);
        if constexpr (M::zeros) sb[scale_words * 4 + q * 4] = 128.f + (float)b.z[q];
      }
    }
    fence();
  }

  // The row's scales (or zeros: 128 + zero) of the step, by tile and group.
  static __device__ __forceinline__ void take_scales(const u32x4* at, f32x4* v) {
    const int r = threadIdx.x & 15;
#pragma unroll
    for (int q = 0; q < scale_loads; q++)
      v[q] = reinterpret_cast<const f32x4*>(at)[r * scale_loads + q];
  }

  // Half m of tile i: the four words of codes for the MFMAs.
  static __device__ __forceinline__ u32x4 take_codes(const u32x4* buf, int i, int m) {
    const int r = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    buf += i * tile_words;
    u32x4 v;
    if constexpr (M::words == 4) {
      v = buf[place(r, m * 4 + g)];
    } else if constexpr (M::words == 2) {
#pragma unroll
      for (int q = 0; q < 2; q++) {
        const u32x4* at = buf + place(r, m * 4 + q * 2 + (g >> 1));
        const u32x2 t = reinterpret_cast<const u32x2*>(at)[g & 1];
        v[q * 2] = t.x, v[q * 2 + 1] = t.y;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; q++)
        v[q] = reinterpret_cast<const uint32_t*>(buf + place(r, m * 4 + q))[g];
    }
    return v;
  }

  // The eight bf16 weights of a word of codes (int4: 128 + code; mxfp4: scaled).
  static __device__ __forceinline__ u32x4 operand(uint32_t w, float scale) {
    u32x4 o;
    if constexpr (M::integer) {
      // one v_and_or each: it takes no literals, and one scalar register at most
      uint32_t mask = 0x000F000Fu, exponent = 0x43004300u;
      asm("" : "+v"(mask));
      asm("" : "+s"(exponent));
#pragma unroll
      for (int q = 0; q < 4; q++) o[q] = ((w >> (4 * q)) & mask) | exponent;
    } else {
      o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
      o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
      o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
      o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
    }
    return o;
  }

  // The products of a step.  SHARED: next() once b's registers are free.
  template <typename Next>
  __device__ __forceinline__ void compute(const Slot& b, u32x4* buf, u32x4* xs, Next&& next) {
    const int r = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    const f32x4 none{0.f, 0.f, 0.f, 0.f};
    constexpr uint32_t kOnes = 0x3F803F80u;
    const u32x4 ones{kOnes, kOnes, kOnes, kOnes};
    constexpr int per = 4 / M::groups;               // MFMAs per group
    if constexpr (M::quant) put(b, buf);
    // mxfp4, value by value: the scales stay in registers
    uint32_t sm[M::quant && !wide && !M::integer ? scale_loads : 1];
    if constexpr (M::quant && !wide && !M::integer) {
#pragma unroll
      for (int q = 0; q < scale_loads; q++) sm[q] = b.s[q];
    }
    if constexpr (SHARED) {
      const int lane = threadIdx.x & 63, row = (threadIdx.x >> 6) * 4 + (lane >> 4);
#pragma unroll
      for (int k = 0; k < TT; k++)
#pragma unroll
        for (int m = 0; m < M::halves; m++)
          xs[(k * M::halves + m) * 256 + row * 16 + ((lane & 15) ^ row)] = b.x[k][m][0];
      __syncthreads();
      next();
    }
    f32x4 sv[M::integer ? scale_loads : 1], zv[M::zeros ? scale_loads : 1];
    if constexpr (M::integer) take_scales(buf + RT * tile_words, sv);
    if constexpr (M::zeros) take_scales(buf + RT * tile_words + scale_words, zv);
    u32x2 mx[wide && !M::integer ? RT : 1];          // the row's eight scales, by tile
    if constexpr (wide && !M::integer) {
#pragma unroll
      for (int i = 0; i < RT; i++)
        mx[i] = reinterpret_cast<const u32x2*>(buf + RT * tile_words)[r * RT + i];
    }
    u32x4 codes[RT][M::halves];
    if constexpr (M::quant) {
#pragma unroll
      for (int i = 0; i < RT; i++)
#pragma unroll
        for (int m = 0; m < M::halves; m++) codes[i][m] = take_codes(buf, i, m);
    }
    const auto weight = [&](int i, int m, int j) {   // operand of MFMA j
      if constexpr (!M::quant) return buf[i * tile_words + place(r, j * 4 + g)];
      // mxfp4: lane group g's codes are under the half's scale g (PART: which it loaded)
      else return operand(codes[i][m][j],
                          M::integer ? 0.f
                          : wide ? __uint_as_float(__builtin_amdgcn_ubfe(mx[i][m], g * 8, 8) << 23)
                                 : __uint_as_float(sm[i * M::halves + m] << 23));
    };
    const auto scale = [&](int i, int m, int q) {
      const int v = i * M::scales + m * M::groups + q;
      return sv[v / 4][v % 4];
    };
    const auto zero = [&](int i, int m, int q) {     // off the codes as the operand has them
      const int v = i * M::scales + m * M::groups + q;
      return M::zeros ? zv[v / 4][v % 4] : 136.f;
    };
#pragma unroll
    for (int m = 0; m < M::halves; m++) {
      u32x4 xo[TT][4];
#pragma unroll
      for (int k = 0; k < TT; k++) {
        if constexpr (quad) {
#pragma unroll
          for (int j = 0; j < 4; j++) xo[k][j] = b.x[k][m][0];
        } else if constexpr (SHARED) {
#pragma unroll
          for (int j = 0; j < 4; j++)
            xo[k][j] = xs[(k * M::halves + m) * 256 + r * 16 + ((M::col(g, j) / 8) ^ r)];
        } else {
          const int lane = threadIdx.x & 63;
          fence();
#pragma unroll
          for (int j = 0; j < 4; j++)
            buf[(j * 4 + (lane >> 4)) * 16 + ((lane & 15) ^ (j * 4 + (lane >> 4)))] = b.x[k][m][j];
          fence();
#pragma unroll
          for (int j = 0; j < 4; j++) xo[k][j] = buf[r * 16 + ((M::col(g, j) / 8) ^ r)];
        }
      }
      if constexpr (!M::quant) put(b, buf);
      const auto x = [&](int k, int, int j) { return xo[k][j]; };
      if constexpr (!M::integer) {
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const u32x4 o = weight(i, m, j);
#pragma unroll
            for (int k = 0; k < TT; k++) {
              f32x4& c = acc[i][quad ? j : k];
              c = mfma(x(k, m, j), o, c);
            }
          }
      } else if constexpr (quad) {
        const f32x4 sx = mfma(x(0, m, 0), ones, none);   // register j: sum of piece j
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
          for (int q = 0; q < M::groups; q++) {
            float sum = 0.f, xs = 0.f;
#pragma unroll
            for (int j = q * per; j < (q + 1) * per; j++) {
              const f32x4 d = mfma(x(0, m, j), weight(i, m, j), none);
              sum += d[j];
              xs += sx[j];
            }
            acc[i][0][0] = fmaf(scale(i, m, q),
                                fmaf(-zero(i, m, q), xs, sum), acc[i][0][0]);
          }
      } else {
#pragma unroll
        for (int q = 0; q < M::groups; q++) {
          // without zero points the sums start at -136 sum(x), the same for all tiles
          f32x4 xs[TT], start[TT];
#pragma unroll
          for (int k = 0; k < TT; k++) {
            xs[k] = none;
#pragma unroll
            for (int j = q * per; j < (q + 1) * per; j++) xs[k] = mfma(x(k, m, j), ones, xs[k]);
            start[k] = M::zeros ? none : xs[k] * -136.f;
          }
#pragma unroll
          for (int i = 0; i < RT; i++) {
            f32x4 d[TT];
#pragma unroll
            for (int k = 0; k < TT; k++) d[k] = start[k];
#pragma unroll
            for (int j = q * per; j < (q + 1) * per; j++) {
              const u32x4 o = weight(i, m, j);
#pragma unroll
              for (int k = 0; k < TT; k++) d[k] = mfma(x(k, m, j), o, d[k]);
            }
            const float s = scale(i, m, q), z = zero(i, m, q);
#pragma unroll
            for (int k = 0; k < TT; k++)
#pragma unroll
              for (int e = 0; e < 4; e++)
                acc[i][k][e] = fmaf(s, M::zeros ? fmaf(-z, xs[k][e], d[k][e]) : d[k][e],
                                    acc[i][k][e]);
          }
        }
      }
    }
  }

  // Add `count` steps of the cursor to acc; after(i) follows step i's products.  SHARED:
  // the same count in all wavefronts; xs: LDS, two times shared_words.
  template <typename Cursor, typename After>
  __device__ __forceinline__ void run(int count, Cursor& at, int cols, const void* x, int xbytes,
                                      u32x4* buf, After&& after, u32x4* xs = nullptr) {
    if constexpr (SHARED) {
      Slot slot;
      slot.serial = -1;
      load(slot, at, count > 0, cols, x, xbytes);
      at.advance();
      for (int i = 0; i < count; i++) {
        compute(slot, buf, xs + (i & 1) * shared_words, [&] {
          load(slot, at, i + 1 < count, cols, x, xbytes);
          at.advance();
        });
        after(i);
      }
    } else {
      Slot slot[depth];
#pragma unroll
      for (int d = 0; d < depth; d++) {
        slot[d].serial = -1;
        load(slot[d], at, d < count, cols, x, xbytes);
        at.advance();
      }
      for (int i = 0; i < count; i += depth) {
#pragma unroll
        for (int d = 0; d < depth; d++) {
          if (d > 0 && i + d >= count) break;
          compute(slot[d], buf, nullptr, [] {});
          load(slot[d], at, i + d + depth < count, cols, x, xbytes);
          at.advance();
          after(i + d);
        }
      }
    }
  }

  // The token row that the lane's load j of x is of in token tile k.
  static __device__ __forceinline__ int token(int k, int j) {
    const int lane = threadIdx.x & 63;
    if (SHARED) j = threadIdx.x >> 6;
    return quad ? (lane & 15) >> 2 : k * 16 + j * 4 + (lane >> 4);
  }

  // f(token, value) for every token row this lane holds of weight tile i (its
  // weight row is lane & 15).
  template <typename Fn>
  __device__ __forceinline__ void values(int i, Fn&& f) const {
    const int g = (threadIdx.x & 63) >> 4;
    if constexpr (quad) {
      if constexpr (M::integer) f(g, acc[i][0][0]);
      else f(g, acc[i][0][0] + acc[i][1][1] + acc[i][2][2] + acc[i][3][3]);
    } else {
#pragma unroll
      for (int k = 0; k < TT; k++)
#pragma unroll
        for (int e = 0; e < 4; e++) f(k * 16 + g * 4 + e, acc[i][k][e]);
    }
  }
};

// The cursor over every by-th step of the same tiles and rows.
template <int F, int RT, typename S>
struct Strided {
  Tiles<F, RT> tiles;
  int xoff[S::TT][S::rows];
  int step, by, from, end, serial;                   // behind the last step: from the first again
  bool live;
  // The wavefront `part` of `of` that share the steps, beginning with its `turn`-th one
  // (modulo their number, which is returned).
  __device__ __forceinline__ int share(int steps, int part, int of, int turn) {
    const int n = part < steps ? (steps - part + of - 1) / of : 0;
    from = part, by = of, end = steps;
    step = part + (n ? turn % n * of : 0);
    serial = 0;
    return n;
  }
  __device__ __forceinline__ void advance() {
    step += by;
    if (by > 1 || (uint32_t)step % Fmt<F>::chunk == 0 || step >= end) serial++;
    if (step >= end) step = from;
  }
};

// ---------------------------------------------------------------- y = x W^T
constexpr int kLinWaves = 8;

// One workgroup: RT*16 rows of the weight, all columns split over the waves, 16 T
// rows of x (blockIdx.y).  Eight wavefronts, so that 7168 columns are four steps each:
// one row by 7168 x 7168 int4 takes 7.3 us (3.6 TB/s of 26.5 MB, 4 us of it latency),
// 64 rows by 7168 x 2048 with zero points 9.9 us (each of two row groups reads all
// codes, from L2 the second time).
template <int F, int RT, int T, bool PART>
__global__ __launch_bounds__(64 * kLinWaves) void linear_kernel(
    const uint16_t* __restrict__ x, Weight w, uint16_t* __restrict__ y, int n, int cols, int rows) {
  using S = Stream<F, RT, T, PART>;
  __shared__ u32x4 buf[kLinWaves][S::buffer_words];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int row0 = blockIdx.x * (RT * 16), t0 = blockIdx.y * S::tokens;
  const int nt = min(n - t0, S::tokens);
  Strided<F, RT, S> at;
  at.tiles.set(w, row0, rows - row0, 0, cols);
#pragma unroll
  for (int k = 0; k < S::TT; k++)
#pragma unroll
    for (int q = 0; q < S::rows; q++) {
      const int t = S::token(k, q);
      at.xoff[k][q] = t < nt ? t * cols * 2 : kAbsent;
    }
  const int count = at.share(steps_of<F>(cols), wave, kLinWaves, 0);
  S st;
  st.init(cols, 0);
  st.run(count, at, cols, x + (int64_t)t0 * cols,
         nt * cols * 2, buf[wave], [](int) {});
  float* sums = reinterpret_cast<float*>(buf[wave]);         // [RT][tokens][16]
  S::fence();
#pragma unroll
  for (int i = 0; i < RT; i++)
    st.values(i, [&](int t, float v) { sums[(i * S::tokens + t) * 16 + (lane & 15)] = v; });
  __syncthreads();
  for (int q = threadIdx.x; q < nt * RT * 16; q += 64 * kLinWaves) {
    const int t = q / (RT * 16), c = q % (RT * 16);
    float v = 0.f;
#pragma unroll
    for (int u = 0; u < kLinWaves; u++)
      v += reinterpret_cast<const float*>(buf[u])[((c >> 4) * S::tokens + t) * 16 + (c & 15)];
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
  // many: uint16 [N*K]; few: bytes [experts][16]; room for both, so that a workspace
  // does for fewer tokens as well
  const int64_t few = (int64_t)m.experts * kFew;
  m.o_hidden = m.o_pairs + align256(pairs * 2 > few ? pairs * 2 : few);
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
  int split;                              // first kernel: wavefronts per contraction
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

// What thread `tid` keeps of token tid's weight until the products are there: the
// load is on its way meanwhile.
struct Gate {
  uint32_t named;
  int at;                                     // place in the expert's list, -1: not there
  float weight;
  __device__ __forceinline__ void put(const MoeArgs& a, Routing& r) const {
    if (at < 0) return;
    float w = weight;
    for (uint32_t more = named & (named - 1); more; more &= more - 1)
      w += a.weights[threadIdx.x * a.K + __ffs(more) - 1];   // named twice: the weights add up
    r.weight[at] = w;
  }
};

// Finds the j-th active expert, its tokens (in order) with their weights, and
// how many pairs name lower experts.  ids: LDS for N*K entries.  Returns the
// id, -1 if there are fewer.
template <bool MANY>
__device__ __forceinline__ int find_expert(const MoeArgs& a, Routing& r, int16_t* ids, int j,
                                           Gate& gate, int& n, int& before, int& total) {
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
  int below = 0;
  uint32_t named = 0;                         // the choices of token tid that are e
  if (tid < a.N)
    for (int k = 0; k < a.K; k++) {
      const int o = ids[tid * a.K + k];
      named |= o == e ? 1u << k : 0u;
      below += o >= 0 && o < e ? 1 : 0;
    }
  const int k0 = __ffs(named) - 1;
  gate.named = named;
  gate.at = -1;
  if (k0 >= 0) gate.weight = a.weights[tid * a.K + k0];   // waited for in Gate::put
  if constexpr (!MANY) {
    if (tid < kFew) r.pair[tid] = k0 >= 0 ? tid << kPairShift | k0 : -1;
    if (k0 >= 0) gate.at = tid;
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
      gate.at = at;
    }
    n = uniform(n);
  }
  __syncthreads();
  return e;
}

__device__ __forceinline__ float silu(float g) { return g / (1.f + expf(-g)); }

// A workgroup's four wavefronts share 4/split groups of tiles (RT/2 pairs of 16 gate
// and 16 up rows), split of them the contraction of each.
// Entries pos0 .. of the expert's list.
template <int F, int RT, int T, bool PART, bool SHARED>
__device__ __forceinline__ void up_tokens(const MoeArgs& a, Routing& r, const Gate& gate,
                                          u32x4* buf, u32x4* xs, const Tiles<F, RT>& tiles, int i0,
                                          int pos0, int n) {
  using S = Stream<F, RT, T, PART, SHARED>;
  const int split = SHARED ? 1 : a.split;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int nt = min(n - pos0, S::tokens);
  Strided<F, RT, S> at;
  at.tiles = tiles;
#pragma unroll
  for (int k = 0; k < S::TT; k++)
#pragma unroll
    for (int q = 0; q < S::rows; q++) {
      const int t = S::token(k, q), pair = t < nt ? r.pair[pos0 + t] : -1;
      at.xoff[k][q] = pair >= 0 ? (pair >> kPairShift) * a.H * 2 : kAbsent;
    }
  // Wavefronts at the same columns of rows of 4 KiB or 8 KiB are all in the same few
  // memory channels, so workgroups start at different ones (64 tokens, bf16, 4096 x 1024:
  // 265 us, without 294).  Where the wavefronts are apart already it only costs (one
  // token, 4-bit: 41.4 us, with 42.4).
  const int turn = split < kUpWaves ? blockIdx.x : 0;
  const int count = at.share(steps_of<F>(a.H), wave & (split - 1), split, turn);
  S st;
  st.init(a.H, a.I);
  st.run(count, at, a.H, a.x, a.N * a.H * 2,
         buf + wave * S::buffer_words, [](int) {}, xs);
  if (pos0 == 0) gate.put(a, r);
  float* sums = reinterpret_cast<float*>(buf + wave * S::buffer_words);   // [RT][tokens][16]
  S::fence();
#pragma unroll
  for (int i = 0; i < RT; i++)
    st.values(i, [&](int t, float v) { sums[(i * S::tokens + t) * 16 + (lane & 15)] = v; });
  __syncthreads();
  const int wide = kUpWaves / split * RT * 8;      // rows of hidden per workgroup
  for (int q = threadIdx.x; q < nt * wide; q += kUpThreads) {
    const int t = q / wide, c = q - t * wide;
    const int w0 = c / (RT * 8) * split, i = c % (RT * 8) / 16 * 2;
    float g = 0.f, u = 0.f;
    for (int v = w0; v < w0 + split; v++) {
      const float* part = reinterpret_cast<const float*>(buf + v * S::buffer_words);
      g += part[(i * S::tokens + t) * 16 + (c & 15)];
      u += part[((i + 1) * S::tokens + t) * 16 + (c & 15)];
    }
    const int pair = r.pair[pos0 + t];
    // The one rounding between the products: the second one's MFMA takes bf16, and a
    // second operand for what that loses would double its products and its reads of
    // these rows.  Off by 2^-8 of a value at most, the layer by 0.0024 of y's norm
    // (0.0017 is y's own rounding).
    if (pair >= 0 && i0 + c < a.I)
      a.hidden[(int64_t)((pair >> kPairShift) * a.K + (pair & ((1 << kPairShift) - 1))) * a.I +
               i0 + c] = bf16_bits(r.weight[pos0 + t] * (silu(g) * u));
  }
  if (pos0 + S::tokens < n) __syncthreads();    // the next tokens' tiles go where the sums are
}

// First kernel: blockIdx.x the groups of tiles, blockIdx.y the expert among the
// active ones.  T: token tiles per pass; 0 and 1 without MANY: few tokens.  Each
// workgroup finds its expert and tokens itself, from the ids in L2, rather than wait for
// a kernel that lists them.  7168 x 2048, 32 experts: one token (8 experts) 470 MB of
// bf16 in 70 us (6.7 TB/s) or 121 MB of int4 in 25 us (4.8); 64 tokens int4 485 MB in
// 96 us (5.1); 256 tokens bf16 1.88 GB in 290 us (6.5).
template <int F, int RT, int T, bool MANY, bool PART, bool SHARED>
__global__ __launch_bounds__(kUpThreads, T == 0 && F != kInt32Z ? 3 : 2) void moe_up_kernel(
    MoeArgs a) {
  using S = Stream<F, RT, T, PART, SHARED>;
  const int split = SHARED ? 1 : a.split;
  __shared__ Routing r;
  __shared__ u32x4 buf[kUpWaves * S::buffer_words];
  __shared__ u32x4 xs[SHARED ? 2 * S::shared_words : 1];
  extern __shared__ int16_t ids[];            // [N*K]
  int n = 0, before = 0, total = 0;
  const int j = blockIdx.y, i0 = blockIdx.x * (kUpWaves / split * RT * 8);
  Gate gate;
  const int e = find_expert<MANY>(a, r, ids, j, gate, n, before, total);
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
  Tiles<F, RT> tiles;
  const int own = i0 + uniform(threadIdx.x >> 6) / split * (RT * 8);
  tiles.set(a.w13, (int64_t)e * 2 * a.I + min(own, a.I), a.I - own, a.I, a.H);
  if constexpr (!MANY) {
    up_tokens<F, RT, T, PART, SHARED>(a, r, gate, buf, xs, tiles, i0, 0, n);
  } else {
    if (T == 1 || n > 16)
      for (int p = 0; p < n; p += 16 * T)
        up_tokens<F, RT, T, PART, SHARED>(a, r, gate, buf, xs, tiles, i0, p, n);
    else
      up_tokens<F, RT, 1, PART, SHARED>(a, r, gate, buf, xs, tiles, i0, 0, n);
  }
}

// No tokens: only what the workspace says about the routing.
__global__ void moe_none_kernel(int32_t* words) { words[0] = words[1] = 0; }

// ---- second product.  One workgroup owns RT*16 columns of y and walks the active
// experts; its wavefronts share the steps of all of them evenly, one stream of
// loads each that does not stop between experts.  The parts meet in LDS and are
// added in the wavefronts' order: no atomics, the same sums on every run.
// 7168 x 2048, 32 experts: one token (8 experts) 235 MB of bf16 in 38 us (6.2 TB/s) or
// 61 MB of int4 in 16 us (3.8); 64 tokens int4 243 MB in 110 us (2.2; experts of more
// than 16 tokens are read twice, 343 MB); 256 tokens bf16 0.94 GB in 181 us (5.2).

// Few: token rows are the same for every expert, the accumulators go through.
// 16 wavefronts where there are fewer than 256 workgroups: no faster (1952 columns,
// 13 tokens: 35.4 us for the layer, with eight 34.8).
constexpr int kFewWaves = 8;

template <int F, int RT, typename S>
struct FewCursor {
  const MoeArgs* a;
  const int32_t* expert;                  // LDS
  const uint8_t* map;                     // LDS [experts][16]
  int64_t row0;
  int rows, j, step, steps, n, rot, serial;
  Tiles<F, RT> tiles;
  int xoff[1][S::rows];
  bool live;
  __device__ __forceinline__ void enter() {
    const int at = min(j, a->experts - 1);
    tiles.set(a->w2, (int64_t)uniform(expert[at]) * a->H + row0, rows, 0, a->I);
#pragma unroll
    for (int q = 0; q < S::rows; q++) {
      const int t = S::token(0, q), k1 = map[at * kFew + t];
      xoff[0][q] = k1 ? (t * a->K + k1 - 1) * a->I * 2 : kAbsent;
    }
  }
  __device__ __forceinline__ void turn() {
    step = n + rot;
    if (step >= steps) step -= steps;
    if (n == 0 || (uint32_t)step % Fmt<F>::chunk == 0) serial++;
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

template <int F, int RT, int T, bool PART>
__global__ __launch_bounds__(64 * kFewWaves, 2) void moe_down_few_kernel(MoeArgs a) {
  using S = Stream<F, RT, T, PART>;
  constexpr int wide = RT * 16;               // columns of y per workgroup
  extern __shared__ u32x4 lds4[];
  int32_t* lds = reinterpret_cast<int32_t*>(lds4);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  u32x4* buf = lds4 + wave * S::buffer_words;
  int32_t* expert = lds + kFewWaves * S::buffer_words * 4;
  uint8_t* map = reinterpret_cast<uint8_t*>(expert + a.experts);
  const int active = a.words[1];
  for (int q = threadIdx.x; q < a.experts; q += blockDim.x) expert[q] = a.expert[q];
  for (int q = threadIdx.x; q < a.experts * (kFew / 4); q += blockDim.x)
    reinterpret_cast<uint32_t*>(map)[q] = ((const uint32_t*)a.pairs)[q];
  __syncthreads();
  const int h0 = blockIdx.x * wide, steps = steps_of<F>(a.I);
  const int total = uniform(active) * steps;
  const int first = (int)((int64_t)total * wave / kFewWaves);
  const int count = (int)((int64_t)total * (wave + 1) / kFewWaves) - first;
  FewCursor<F, RT, S> at;
  at.a = &a, at.expert = expert, at.map = map, at.row0 = h0, at.rows = a.H - h0;
  at.j = first / steps, at.n = first % steps, at.steps = steps;
  at.serial = 0;
  at.rot = blockIdx.x % steps;           // the same for all that share an expert's steps
  at.turn();
  S st;
  st.init(a.I, 0);
  if (count > 0) {
    at.enter();
    st.run(count, at, a.I, a.hidden, a.N * a.K * a.I * 2, buf, [](int) {});
  }
  float* sums = reinterpret_cast<float*>(buf);               // [tokens][wide]
  S::fence();
#pragma unroll
  for (int i = 0; i < RT; i++)
    st.values(i, [&](int t, float v) { sums[t * wide + i * 16 + (lane & 15)] = v; });
  __syncthreads();
  for (int q = threadIdx.x; q < a.N * wide; q += blockDim.x) {
    const int t = q / wide, c = q % wide;
    float v = 0.f;
    for (int u = 0; u < kFewWaves; u++)
      v += reinterpret_cast<const float*>(lds4 + u * S::buffer_words)[t * wide + c];
    if (h0 + c < a.H) a.y[(int64_t)t * a.H + h0 + c] = bf16_bits(v);
  }
}

// Many: an item is up to 16 T listed tokens of an expert.  The wavefronts share the
// steps of all items evenly, a contiguous range each; what a wavefront has of
// an item when it leaves it (a segment) goes to rows in LDS that nobody else
// writes: the item's own rows, by list position, if the segment begins the
// item, else the wavefront's extra rows (only its first segment can begin
// inside an item).  In the end every (token, column) sums up its own rows, in
// a fixed order.  LDS holds rows_kept listed pairs at a time; longer lists take
// several rounds.
// item: expert | first pair << 10 | tokens << 23.
constexpr int kManyWaves = 8;
constexpr int rows_kept(int RT) { return 384 / RT; }

template <int F, int RT, int T>
struct ManyCursor {
  const MoeArgs* a;
  const uint32_t* items;                  // LDS
  const uint16_t* pairs;                  // LDS
  int64_t row0;
  int rows, steps, item, last, tail, rot;   // tail: the last item's end
  int begin, end, left, step, serial;
  Tiles<F, RT> tiles;
  int xoff[T][4];
  bool live;
  __device__ __forceinline__ void enter(int from) {
    const uint32_t it = uniform(items[min(item, last)]);
    const int e = it & 1023, first = (it >> 10) & 8191, n = it >> 23;
    serial++;
    begin = from;
    end = item >= last ? tail : steps;
    left = end - begin;
    // wavefronts and workgroups start at different columns: rows of 4 KiB would
    // otherwise have them all in the same few memory channels
    step = begin + rot % left;
    tiles.set(a->w2, (int64_t)e * a->H + row0, rows, 0, a->I);
#pragma unroll
    for (int k = 0; k < T; k++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int t = Stream<F, RT, T, false>::token(k, q);
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
    } else {
      if (++step == end) step = begin;
      if (step == begin || (uint32_t)step % Fmt<F>::chunk == 0) serial++;
    }
  }
};

// LDS of the kernel below: buffers, rows, items, list, positions.
__host__ __device__ inline int most_items(int experts, int pairs, int T) {
  return experts + pairs / (16 * T);
}
__host__ __device__ inline int list_words(int pairs) { return (pairs + 1) / 2; }
size_t many_lds(int buffer_words, int N, int K, int experts, int RT, int T) {
  return (size_t)kManyWaves * buffer_words * 16 +
         (size_t)(rows_kept(RT) + 16 * T + kManyWaves * 16 * T) * RT * 64 +
         4 * ((size_t)most_items(experts, N * K, T) + 2 * list_words(N * K));
}

template <int F, int RT, int T, bool PART>
__global__ __launch_bounds__(64 * kManyWaves, 2) void moe_down_many_kernel(MoeArgs a) {
  using S = Stream<F, RT, T, PART>;
  constexpr int wide = RT * 16, kRows = rows_kept(RT);     // columns of y; listed pairs at a time
  constexpr int kOut = EP_MAX_FEW_TOKENS * wide / (64 * kManyWaves);   // results per thread
  extern __shared__ u32x4 lds4[];       // (the type aligns it: behind the variables below)
  __shared__ int n_items;
  __shared__ uint32_t extra_item[kManyWaves];        // item of the extra rows, 0: none
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int NK = a.N * a.K;
  u32x4* buf = lds4 + wave * S::buffer_words;
  float(*own)[wide] = reinterpret_cast<float(*)[wide]>(lds4 + kManyWaves * S::buffer_words);
  float(*extra)[wide] = own + kRows + 16 * T;          // [waves][16 T]
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
  const int h0 = blockIdx.x * wide, steps = steps_of<F>(a.I);
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
      ManyCursor<F, RT, T> at;
      at.a = &a, at.items = items, at.pairs = pairs, at.row0 = h0, at.rows = a.H - h0;
      at.steps = steps, at.rot = blockIdx.x + wave, at.serial = 0;
      at.item = i0 + s0 / steps;
      at.last = i0 + (s1 - 1) / steps;
      at.tail = (s1 - 1) % steps + 1;
      at.enter(s0 % steps);
      if (at.begin && lane == 0) extra_item[wave] = items[at.item];
      int item = at.item, left = at.left;            // where the products are, behind the loads
      bool whole = at.begin == 0;
      S st;
      st.init(a.I, 0);
      st.run(s1 - s0, at, a.I, a.hidden, NK * a.I * 2, buf, [&](int i) {
        if (--left > 0) return;
        const uint32_t it = uniform(items[item]);
        const int n = it >> 23;
        float(*to)[wide] = whole ? own + ((it >> 10) & 8191) - from : extra + wave * 16 * T;
#pragma unroll
        for (int i = 0; i < RT; i++)
          st.values(i, [&](int t, float v) {
            if (t < n) to[t][i * 16 + (lane & 15)] = v;
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
      const int q = threadIdx.x + i * 64 * kManyWaves, t = q / wide, c = q % wide;
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
    const int q = threadIdx.x + i * 64 * kManyWaves, t = q / wide, c = q % wide;
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

// f(std::bool_constant<PART>): whole steps and, of codes, whole chunks of scales that
// lie where they can be loaded at once?
template <int F, typename Fn>
void with_part(const Weight& w, int cols, Fn&& f) {
  const bool whole = cols % (Fmt<F>::step * Fmt<F>::chunk) == 0 && (uintptr_t)w.scale % 16 == 0 &&
                     (uintptr_t)w.zero % 8 == 0;
  if (whole) f(std::false_type());
  else f(std::true_type());
}

template <int F, int RT, int T, bool MANY>
void launch_down(const MoeArgs& a, hipStream_t st) {
  const int grid = (a.H + RT * 16 - 1) / (RT * 16);
  with_part<F>(a.w2, a.I, [&](auto part) {
    using S = Stream<F, RT, T, part.value>;
    if constexpr (MANY) {
      moe_down_many_kernel<F, RT, T, part.value><<<
          grid, 64 * kManyWaves, many_lds(S::buffer_words, a.N, a.K, a.experts, RT, T), st>>>(a);
    } else {
      const size_t lds = (size_t)kFewWaves * S::buffer_words * 16 + (size_t)a.experts * (4 + kFew);
      moe_down_few_kernel<F, RT, T, part.value><<<grid, 64 * kFewWaves, lds, st>>>(a);
    }
  });
}

// T: token tiles per item of the second product.  The first one takes pairs of tiles
// for longer lists, its registers allow it (4-bit, 64 tokens: 245 us for the layer,
// with single tiles 308), and single ones where no list is longer than 16.
template <int F, int T, bool MANY>
void launch_moe(MoeArgs a, hipStream_t st) {
  constexpr bool quant = Fmt<F>::quant, coarse = F == kMx || Fmt<F>::group == 128;
  // Codes with token tiles: four row tiles per wavefront, which read x half as often
  // as two do (64 tokens 238 us for the layer, with two 262; 16 tokens 156 and 167).
  // Finer integer groups with their scales and zeros have no registers for that.
  constexpr int RT = T > 0 && coarse && quant ? 4 : 2, UT = MANY ? 2 : T;
  // A workgroup's four wavefronts share one contraction, which keeps the latency of
  // few tokens short (one token, 4-bit: 41.4 us, two on each 42.0, one on each 48.2).
  // Where there are more workgroups than CUs anyway, less splitting is better: longer
  // lists are made for more rows, and codes go through the SHARED stream with x loaded
  // once for all four.  256 tokens, bf16, 7168 x 2048: 467 us with four on each, 455
  // with two; 64 tokens, 4-bit: 236 with four, 196 shared; but 64 tokens, 2048 x 256, 16
  // experts: 25.7 with four, 40.4 with one on each.
  const auto groups = [&](int split) { return (a.I + kUpWaves / split * RT * 8 - 1) /
                                              (kUpWaves / split * RT * 8); };
  constexpr int apart = quant ? 1 : 2;
  bool enough = false;
  if constexpr (MANY) {
    enough = groups(apart) * a.experts >= 256;
  } else if constexpr (T == 1 && quant) {
    // 5 to 16 tokens: if most experts are likely to be named (16 tokens, 7168 x 2048,
    // 8 of 32 experts: 137 us, split 148; 2048 x 768 with zero points, 8 of 64: 54.2, 64.4; if
    // most choices are -1 it costs: 74.3, 69.1; and with 10 tokens, 4 of 32: 52.7, 49.1)
    enough = groups(apart) * a.experts >= 512 && 2 * a.N * a.K >= 3 * a.E;
  }
  a.split = enough ? apart : kUpWaves;
  const dim3 up(groups(a.split), a.experts);
  with_part<F>(a.w13, a.H, [&](auto part) {
    const size_t lds = sizeof(int16_t) * a.N * a.K;
    if constexpr (T > 0 && quant) {
      if (a.split == 1)
        return moe_up_kernel<F, RT, UT, MANY, part.value, true><<<up, kUpThreads, lds, st>>>(a);
    }
    moe_up_kernel<F, RT, UT, MANY, part.value, false><<<up, kUpThreads, lds, st>>>(a);
  });
  // Codes with one token tile: two row tiles per wavefront halve what x costs, if
  // the workgroups still fill the GPU (64 tokens, 7168 columns: 115 us against 145;
  // 13 tokens, 1952 columns: 22.7 against 15.0).
  if constexpr (T == 1 && quant && coarse)
    if (a.H >= 32 * 192) return launch_down<F, 2, T, MANY>(a, st);
  launch_down<F, 1, T, MANY>(a, st);
}

template <int F>
int launch_moe(const MoeArgs& a, hipStream_t st) {
  const int64_t pairs = (int64_t)a.N * a.K;
  EP_LOG("moe: N=%d H=%d I=%d E=%d K=%d", a.N, a.H, a.I, a.E, a.K);
  if (a.N <= 4) launch_moe<F, 0, false>(a, st);
  else if (a.N <= kFew) launch_moe<F, 1, false>(a, st);
  // Up to 64 tokens per expert if they were spread evenly: items of 16 for the second
  // product, which most lists fit (256 tokens, 8 of 256 experts, 32 of them here, bf16:
  // 455 us, with items of 32 500); longer lists would read the weights too often (64
  // tokens to each of 64 experts, 2048 x 1024, 4-bit: 281 us with items of 16, 271).
  else if (pairs <= 64 * a.E) launch_moe<F, 1, true>(a, st);
  // Groups of 32 with zero points would spill with two token tiles (256 tokens, 16
  // experts: 410 us against 333).
  else launch_moe<F, F == kInt32Z ? 1 : 2, true>(a, st);
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
  with_part<F>(w, cols, [&](auto part) {
    constexpr bool P = part.value;
    // fine groups and two token tiles: one row tile, or the registers spill
    constexpr int R2 = (Fmt<F>::integer && Fmt<F>::group == 32) || (F == kInt64Z && P) ? 1 : RT;
    const int g2 = (rows + R2 * 16 - 1) / (R2 * 16);
    if (n <= 4) linear_kernel<F, RT, 0, P><<<dim3(gx, 1), B, 0, st>>>(xp, w, yp, n, cols, rows);
    else if (n <= 16)
      linear_kernel<F, RT, 1, P><<<dim3(gx, 1), B, 0, st>>>(xp, w, yp, n, cols, rows);
    else
      linear_kernel<F, R2, 2, P><<<dim3(g2, (n + 31) / 32), B, 0, st>>>(xp, w, yp, n, cols, rows);
  });
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
  if (rc != EP_OK) return rc;
  const MoePlan m = make_moe_plan(p, a->inter);
  char* ws = (char*)a->workspace;
  hipStream_t st = (hipStream_t)stream;
  if (p->num_tokens == 0) {
    moe_none_kernel<<<1, 1, 0, st>>>((int32_t*)ws);
    return check_launch("moe_layer");
  }
  const MoeArgs k{(const uint16_t*)a->x, a->topk_idx, a->topk_weights, kernel_weight(a->w13),
                  kernel_weight(a->w2), (uint16_t*)a->y, (int32_t*)ws,
                  (int32_t*)(ws + m.o_expert), (int32_t*)(ws + m.o_count),
                  (int32_t*)(ws + m.o_start), ws + m.o_pairs, (uint16_t*)(ws + m.o_hidden),
                  p->num_tokens, p->hidden, p->num_topk, p->num_experts, a->inter,
                  p->topk_idx_bytes == 8, m.experts, 0};
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
  if (num_rows > 0) {
    if (!x || ((uintptr_t)x & 15) || !y || ((uintptr_t)y & 1)) return EP_ERR_INVALID_ARG;
    const uintptr_t x0 = (uintptr_t)x, y0 = (uintptr_t)y;
    if (x0 < y0 + (size_t)num_rows * out_rows * 2 && y0 < x0 + (size_t)num_rows * cols * 2)
      return EP_ERR_INVALID_ARG;         // workgroups read x while others write y
  }
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
