// ep_ffn.hip -- the experts' feed-forward block on dispatched rows, its gradient, and
// products in 8-bit integers (include/ep_get.h states the contracts).
//
// All of it is D = A B^T over a contraction, for the rows of every expert in one launch
// (the counts are on the device, so each workgroup finds its tiles itself):
//   block      h = silu(x Wg^T) * (x Wu^T), y = h W2^T      activations by a weight's rows
//   gradient   dh = dy W2 (dg, du and h in its epilogue), dx = [dg du] W13
//                                                           ... by its columns
//              dW13 = [dg du]^T x, dW2 = dy^T h             k runs over an expert's rows
//   integers   the same first form on bytes, the sums exact in 32 bits
// gate and up meet in one tile (128 columns of each), so that h leaves the kernel and 2 *
// inter values per row never do, unless a gradient will ask for them.
//
// Three kernels, chosen by run_rows and run_grad:
//   product_kernel  256 by 256 tiles, 8 wavefronts, one workgroup per CU that walks over
//                   tiles.  A tile's step (128 bytes of the contraction) is 2048 cycles of
//                   MFMA on each SIMD and 64 KiB of operands, which go straight to LDS two
//                   steps deep and are read with few bank conflicts.  Bound by the MFMAs and,
//                   with them, by the card's power: gate and up of 8192 rows of 8192, 4096
//                   columns, in bf16 1270 TFLOP/s at 1.59 GHz, the MFMAs busy 82 % of the
//                   cycles (a large library product: 1260 to 1550); 8192^3 int8 2220 TOP/s
//                   at 1.61 GHz, 71 % (2060 to 2120).  Not counted in the cycles: 8 % of the
//                   time, in which a CU has no work yet or none left.
//                   Tiles of at most 128 rows have a loop of their own (stream): bound by
//                   HBM, 6.9 TB/s of weights at 16 rows an expert.
//   few_kernel      few rows: weights as a stream, the contraction split over wavefronts
//   small_kernel    what lies between: 64 by 64 tiles on many CUs
// One workgroup computes a value from one fixed order of sums: the same bits on every run.
// h, dg and du are rounded to bf16 between the products, whose operands they are: float32
// operands have a sixteenth of the bf16 MFMAs' rate.  It is most of what the block's error has
// over that of one rounding of y (0.0023 of the norm, 0.0017).
#include "ep_host.h"
#include "ep_rows.h"

#include <algorithm>
#include <type_traits>

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

#define EP_LDS __attribute__((address_space(3)))

constexpr int kRange = 0x60000000;     // bytes that a buffer descriptor spans
constexpr int kAbsent = 0x7F000000;    // an offset outside of it: the load returns zeros
constexpr int kBM = 256, kBN = 256;    // rows and columns of a tile
constexpr int kHalf = 16384;           // bytes of half of either operand's tile (128 by 128 bytes)
constexpr int kStage = 4 * kHalf;      // a's two halves, b's two halves
constexpr int kSteps = 2;              // stages in LDS
constexpr int kGroupM = 8;             // row tiles that are neighbours in the order of tiles
constexpr int kLastTile = INT32_MAX - 1024;    // strides behind it are in 32 bits still

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// How the operands lie in memory (D = A B^T, contraction over k):
//   kRowsT  A [row][k], B [column][k]     activations by a weight's rows
//   kRows   A [row][k], B [k][column]     activations by a weight's columns
//   kOuter  A [k][row], B [k][column]     a weight's gradient: k runs over an expert's rows
enum { kRowsT, kRows, kOuter };

struct Outer {
  const uint8_t *a, *b;
  int64_t a_row, b_row;
  int m, n;
};

struct Product {            // kernel argument
  Rows rows;
  const uint8_t* a;
  const uint8_t* b;
  int64_t a_row, b_row;     // bytes per row of a and b
  int64_t b_expert;         // bytes per expert of b (kRowsT, kRows)
  int k;                    // contraction: bytes of a row of a (kRowsT, kRows)
  int m, n;                 // D's rows (kOuter) and columns
  int far;                  // > 0: column j of a tile's second half is b's row far + n0/2 + j
  Outer also;               // kOuter: a second product over the same rows
};

// 16 bytes per lane from global memory straight to LDS, lane l's at base + 16 l.  In asm,
// because the compiler would wait for all such loads before the next read of LDS; the
// waits are written out at the loops.  The s_nop covers a descriptor word or base that a
// VALU instruction has just written (five wait states), which the compiler cannot see
// here, and m0.  ONCE: the bytes are not kept in the caches for another workgroup.
template <bool ONCE>
__device__ __forceinline__ void load_lds(uint32_t lds, int offset, i32x4 desc) {
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
                 :
                 : "s"(uniform((int)lds)), "v"(offset), "s"(desc)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(uniform((int)lds)), "v"(offset), "s"(desc)
                 : "memory");
}
// Two of them, 1 KiB apart in LDS.
template <bool ONCE>
__device__ __forceinline__ void load_lds2(uint32_t lds, int offset0, int offset1, i32x4 desc) {
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %4, 0 offen nt lds\n\t"
                 "s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %4, 0 offen nt lds"
                 :
                 : "s"(uniform((int)lds)), "s"(uniform((int)lds + 1024)), "v"(offset0),
                   "v"(offset1), "s"(desc)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %4, 0 offen lds\n\t"
                 "s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %4, 0 offen lds"
                 :
                 : "s"(uniform((int)lds)), "s"(uniform((int)lds + 1024)), "v"(offset0),
                   "v"(offset1), "s"(desc)
                 : "memory");
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ void barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ i32x4 descriptor(const uint8_t* p) {
  const uint64_t a = (uint64_t)p;
  i32x4 d;
  d[0] = uniform((int)(uint32_t)a);
  d[1] = uniform((int)((a >> 32) & 0xFFFF));
  d[2] = kRange;
  d[3] = 0x00020000;
  return d;
}

// With the hardware's reciprocal, one ulp off: a whole quotient would be most of a gate's
// epilogue (ten instructions for each of its 32768 values).
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-g));
}

// Waits for loads into v here, whatever is done with it later: a wait that the compiler
// leaves to a path behind a branch comes back in the main loop as a wait for everything.
__device__ __forceinline__ void arrive(float& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void arrive(f32x4& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void arrive(u32x4& v) { asm volatile("" : "+v"(v)); }

// ---------------------------------------------------------------- epilogues
// Four values from p[c] on, of n (those behind the last are the last again).  Scales are
// aligned to 4 bytes only, which is enough for a load of 16.
typedef float f32x4_at_4 __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ f32x4 load4(const float* p, int c, int n) {
  if ((n & 3) == 0) return *(const f32x4_at_4*)(p + min(c, n - 4));
  f32x4 r;
#pragma unroll
  for (int j = 0; j < 4; j++) r[j] = p[min(c + j, n - 1)];
  return r;
}

// A sum of codes (at most 2^30) times a row's scale and a column's.  The first product would
// pass float32's range with scales of 2^96 on (rows near bf16's largest) though the result need
// not: those are taken 2^64 times smaller and the result larger again, both exact.
struct RowFactor {
  float s, back;
  __device__ __forceinline__ explicit RowFactor(float scale) {
    const bool large = fabsf(scale) >= 0x1p96f;
    s = large ? scale * 0x1p-64f : scale;
    back = large ? 0x1p64f : 1.f;
  }
  __device__ __forceinline__ float operator()(int sum, float column) const {
    return (float)sum * s * column * back;
  }
};

// What becomes of eight neighbouring columns of a row of D; put: of eight that store_block has
// rounded to bf16 (`rounds`).  `slot` is the row's slot (kOuter: its row of the expert's
// matrix), `e` the expert, `c` the first column; columns from n on are dropped.
// `stores` is how many of them a wavefront sends at least for a whole tile (16 calls, 8 of
// a gate).
struct StoreRows {
  static constexpr bool gate = false;
  static constexpr int stores = 16;
  __device__ __forceinline__ int columns(int) const { return n; }
  uint16_t* y;
  int n;
  const float *sx, *sw;    // 8-bit products: scales per slot and per expert and column
  static constexpr bool rounds = true;
  __device__ __forceinline__ void put(int, int slot, int c, u32x4 r, int more) const {
    c += more;
    if (c >= n) return;
    uint16_t* to = y + (int64_t)slot * n + c;
    if ((n & 7) == 0) {
      *(u32x4*)to = r;
    } else if ((n & 1) == 0) {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (c + 2 * i < n) *(uint32_t*)(to + 2 * i) = r[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++)
        if (c + i < n) to[i] = (uint16_t)(r[i >> 1] >> (16 * (i & 1)));
    }
  }
  // scales of four columns (whatever behind the last one)
  __device__ __forceinline__ f32x4 scales(int e, int c, int half) const {
    return load4(sw + (int64_t)e * n, c + half * 128, n);
  }
  template <class T>
  __device__ __forceinline__ void operator()(int e, int slot, int c, const T* v, const T*) const {
    if (c >= n) return;
    float f[8];
    if constexpr (std::is_same_v<T, int>) {
      const RowFactor row(sx[slot]);
      const f32x4 w[2] = {scales(e, c, 0), scales(e, c + 4, 0)};
#pragma unroll
      for (int i = 0; i < 8; i++) f[i] = row(v[i], w[i >> 2][i & 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) f[i] = v[i];
    }
    put(e, slot, c, pack8(f), 0);
  }
};

// kOuter: [e][m][n], and of a second product where e is `experts` more
struct StoreMatrix {
  static constexpr bool gate = false;
  static constexpr int stores = 16;
  uint16_t *y, *also;
  int experts, m, n, also_m, also_n;
  __device__ __forceinline__ int columns(int e) const { return e < experts ? n : also_n; }
  static constexpr bool rounds = true;
  __device__ __forceinline__ void put(int e, int row, int c, u32x4 r, int more) const {
    const bool first = e < experts;
    const int width = first ? n : also_n, of = first ? e * m : (e - experts) * also_m;
    c += more;
    if (c < width) *(u32x4*)((first ? y : also) + ((int64_t)of + row) * width + c) = r;
  }
  __device__ __forceinline__ void operator()(int e, int row, int c, const float* v,
                                             const float*) const {
    put(e, row, c, pack8(v), 0);
  }
};

// silu(gate) * up; the tile's columns are `c` of gate and of up.
struct StoreGate {
  static constexpr bool gate = true;
  static constexpr int stores = 8;
  __device__ __forceinline__ int columns(int) const { return inter; }
  uint16_t* h;             // [slot][inter]
  uint16_t* gu;            // [slot][2 inter] or NULL
  int inter;
  const float *sx, *sw;
  static constexpr bool rounds = true;
  __device__ __forceinline__ void put(int, int slot, int c, u32x4 r, int what) const {
    if (c >= inter) return;
    if (what == 0) *(u32x4*)(h + (int64_t)slot * inter + c) = r;
    else *(u32x4*)(gu + (int64_t)slot * 2 * inter + (what - 1) * inter + c) = r;
  }
  __device__ __forceinline__ f32x4 scales(int e, int c, int half) const {
    return load4(sw + ((int64_t)e * 2 + half) * inter, c, inter);
  }
  template <class T>
  __device__ __forceinline__ void operator()(int e, int slot, int c, const T* g, const T* u) const {
    if (c >= inter) return;
    float a[8], b[8], r[8];
    if constexpr (std::is_same_v<T, int>) {
      const RowFactor row(sx[slot]);
      const float* w = sw + (int64_t)e * 2 * inter + c;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        a[i] = row(g[i], w[i]);
        b[i] = row(u[i], w[inter + i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        a[i] = g[i];
        b[i] = u[i];
      }
    }
    if (gu) {
      uint16_t* to = gu + (int64_t)slot * 2 * inter + c;
      *(u32x4*)to = pack8(a);
      *(u32x4*)(to + inter) = pack8(b);
    }
#pragma unroll
    for (int i = 0; i < 8; i++) r[i] = a[i] * sigmoid(a[i]) * b[i];
    *(u32x4*)(h + (int64_t)slot * inter + c) = pack8(r);
  }
};

// v is the gradient of h: those of gate and up, and h itself again.
struct StoreGateGrad {
  static constexpr bool gate = false;
  static constexpr int stores = 48;
  static constexpr bool rounds = false;
  __device__ __forceinline__ int columns(int) const { return inter; }
  const uint16_t* gu;      // [slot][2 inter]
  uint16_t* dgu;           // [slot][2 inter]
  uint16_t* h;             // [slot][inter]
  int inter;
  struct Ahead {           // what it reads, asked for before v is there
    u32x4 g, u;
  };
  __device__ __forceinline__ Ahead ahead(int slot, int c) const {
    const int64_t at = (int64_t)slot * 2 * inter + min(c, inter - 8);
    return Ahead{*(const u32x4*)(gu + at), *(const u32x4*)(gu + at + inter)};
  }
  __device__ __forceinline__ void operator()(const Ahead& x, int slot, int c,
                                             const float* v) const {
    if (c >= inter) return;
    const int64_t at = (int64_t)slot * 2 * inter + c;
    float g[8], u[8], dg[8], du[8], hh[8];
    unpack8(x.g, g);
    unpack8(x.u, u);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float s = sigmoid(g[i]), silu = g[i] * s;
      dg[i] = v[i] * u[i] * (s * (1.f + g[i] * (1.f - s)));
      du[i] = v[i] * silu;
      hh[i] = silu * u[i];
    }
    *(u32x4*)(dgu + at) = pack8(dg);
    *(u32x4*)(dgu + at + inter) = pack8(du);
    *(u32x4*)(h + (int64_t)slot * inter + c) = pack8(hh);
  }
  __device__ __forceinline__ void operator()(int, int slot, int c, const float* v,
                                             const float*) const {
    (*this)(ahead(slot, c), slot, c, v);
  }
};

// ---------------------------------------------------------------- the product
template <bool I8>
struct Acc {
  using type = std::conditional_t<I8, i32x16, f32x16>;
  using scalar = std::conditional_t<I8, int, float>;
};

template <bool I8>
__device__ __forceinline__ typename Acc<I8>::type mfma(u32x4 a, u32x4 b,
                                                       typename Acc<I8>::type c) {
  if constexpr (I8)
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a),
                                                 __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// One operand's half tile in LDS: rows by 128 bytes of k (16-byte chunk c of row r at
// c ^ (r / 2 & 7)), or, where k is the slow axis, 64 k by 128 columns (256 bytes; chunk c of
// row k at c ^ 4 (k & 3)): no two lanes that LDS serves together share a bank.  (It
// serves lanes 0-3, 12-15 and 20-27 of a 16-byte read together: with c ^ (r & 7) conflicts
// were half of its busy cycles.)
template <bool SLOW_K>
__device__ __forceinline__ u32x4 fragment(const uint8_t* half, int lane_off, int ks) {
  if constexpr (SLOW_K) {
    // 4 k by 16 columns per 16 lanes, transposed on the way: lane l gets column l % 16
    EP_LDS bf16x4* p = (EP_LDS bf16x4*)(half + lane_off + ks * 4096);
    EP_LDS bf16x4* q = (EP_LDS bf16x4*)(half + lane_off + ks * 4096 + 1024);
    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(p));
    const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(q));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3);
  } else {
    return *(const u32x4*)(half + (lane_off ^ (ks * 32)));
  }
}

// The scales of 8-bit products for store_block, of N times 64 rows, 128 apart: all at once.  Loaded
// where each block needs them, one latency after the other made a tile's epilogue 22 us long
// instead of 8.
template <int N, class Epi, class RowAt>
__device__ __forceinline__ void load_scales(const Epi& epi, int e, int r0, int nrows, int c0, int v,
                                            RowAt row_at, float (&row)[N][2], f32x4 (&col)[2][4]) {
#pragma unroll
  for (int i = 0; i < 2 * N; i++) {
    const int r = r0 + (i >> 1) * 128 + (i & 1) * 32 + (v & 31);
    row[i >> 1][i & 1] = r < nrows ? epi.sx[row_at(r)] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; i++)
    col[i >> 2][i & 3] = epi.scales(e, c0 + 8 * (i & 3) + 4 * (v >> 5), i >> 2);
#pragma unroll
  for (int i = 0; i < 8; i++) arrive(col[i >> 2][i & 3]);
#pragma unroll
  for (int i = 0; i < 2 * N; i++) arrive(row[i >> 1][i & 1]);
}

// A wavefront's 64 rows (from r0 on, of nrows) by 32 columns of either half (from c0 on): blocks
// of 32 by 32, rounded to bf16, through 2 KiB of its own LDS at mine0 and at mine1, where a
// lane's four columns of a row become eight of another: stores of 64 bytes of a row.  Two
// blocks are under way.
template <class Epi, bool I8, class RowAt>
__device__ __forceinline__ void store_block(const Epi& epi, int e, int r0, int nrows, int c0,
                                            const typename Acc<I8>::type (&acc)[2][2],
                                            const float (&row_scale)[2], const f32x4 (&scales)[2][4],
                                            uint8_t* mine0, uint8_t* mine1, int v, RowAt row_at) {
  auto turn16 = [&](const f32x16& x, uint8_t* mine) {
#pragma unroll
    for (int i = 0; i < 4; i++)
      *(u32x2*)(mine + (v & 31) * 64 + ((i ^ ((v >> 2) & 3)) << 4) + (v >> 5) * 8) =
          u32x2{pack2(x[i * 4], x[i * 4 + 1]), pack2(x[i * 4 + 2], x[i * 4 + 3])};
  };
#pragma unroll
  for (int mb = 0; mb < 2; mb++) {
    const int first = r0 + mb * 32;
    if (first >= nrows) continue;
    auto values = [&](int half) {
      f32x16 x;
      if constexpr (I8) {
        const RowFactor row(row_scale[mb]);
#pragma unroll
        for (int j = 0; j < 16; j++) x[j] = row(acc[half][mb][j], scales[half][j >> 2][j & 3]);
      } else {
        x = acc[half][mb];
      }
      return x;
    };
    auto put = [&](const uint8_t* mine, int what) {
      u32x4 q[2];
#pragma unroll
      for (int it = 0; it < 2; it++)
        q[it] = *(const u32x4*)(mine + it * 1024 + (v >> 2) * 64 +
                                (((v & 3) ^ ((v >> 4) & 3)) << 4));
#pragma unroll
      for (int it = 0; it < 2; it++) {
        const int r = first + it * 16 + (v >> 2);
        if (r < nrows) epi.put(e, row_at(r), c0 + (v & 3) * 8, q[it], what);
      }
    };
    const f32x16 a = values(0), b = values(1);
    if constexpr (Epi::gate) {
      f32x16 x;
#pragma unroll
      for (int j = 0; j < 16; j++) x[j] = a[j] * sigmoid(a[j]) * b[j];
      turn16(x, mine0);
      put(mine0, 0);
      if (epi.gu) {
        turn16(a, mine0);
        turn16(b, mine1);
        put(mine0, 1);
        put(mine1, 2);
      }
    } else {
      turn16(a, mine0);
      turn16(b, mine1);
      put(mine0, 0);
      put(mine1, 128);
    }
  }
}

// Tiles of at most 128 rows by a weight's rows, which come from HBM: 48 KiB a step, three stages
// in LDS and all wavefronts in the same phase, so that two whole steps (96 KiB per CU) are on
// their way where the wide tiles' loop has one.  A workgroup takes them after its wide ones,
// from tile `tile` on; those before `wide` are wide.  Both products for 32 experts of 64 rows,
// 7168 x 2048: 495 us, with the wide tiles' loop 533; of 128 rows 546 : 582; of 64 in 8 bits 289 : 319.
constexpr int kStreamM = 128, kStream = 3 * kHalf;      // rows; bytes of a stage

template <class Epi, bool I8>
__device__ __forceinline__ void stream(const Product& p, const Epi& epi, uint8_t* lds,
                                       const Experts& experts, int tile, int wide, int total) {
  using acc_t = typename Acc<I8>::type;
  constexpr int kCols = Epi::gate ? 128 : kBN;
  const int tid = threadIdx.x, l = tid & 63, w = uniform(tid >> 6);
  const int wm = w >> 2, wn = w & 3;     // rows wm*64.., columns wn*32.. of each half
  const uint32_t lds0 = (uint32_t)(uintptr_t)(EP_LDS uint8_t*)lds;
  const int NT = (p.n + kCols - 1) / kCols, G = gridDim.x;
  const bool blocks = p.rows.count && !p.rows.offset;
  auto chunk_k = [&](int j) { return (l & 7) ^ ((j << 2) + (l >> 4)); };
  const int read_k = (l & 31) * 128 + (((l >> 5) ^ ((l >> 1) & 7)) << 4);
  const int read_a = wm * 64 * 128 + read_k, read_b = kHalf + wn * 32 * 128 + read_k;

  struct Tile {
    int e, nt, nrows, row0, slot0;
  };
  const uint8_t *a0 = nullptr, *b0 = nullptr;
  int left = 0;                          // contraction of what is loaded
  int off_a[2], off_b[2][2];
  const int64_t far = Epi::gate ? (int64_t)p.far * p.b_row : 0;
  const int KT = max(2, (p.k + 127) / 128);

  // step t, whose last bytes may be behind the contraction's end
  auto load = [&](int t, int stage) {
    int a[2], b[2][2];
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const bool in = chunk_k(j) * 16 < left - t * 128;
      a[j] = in ? off_a[j] : kAbsent;
      b[0][j] = in ? off_b[0][j] : kAbsent;
      b[1][j] = in ? off_b[1][j] : kAbsent;
    }
    const uint32_t to = lds0 + stage * kStream + w * 2048;
    const uint8_t* from = b0 + (int64_t)t * 128;
    load_lds2<true>(to + kHalf, b[0][0], b[0][1], descriptor(from));
    load_lds2<true>(to + 2 * kHalf, b[1][0], b[1][1], descriptor(from + far));
    load_lds2<false>(to, a[0], a[1], descriptor(a0 + (int64_t)t * 128));
  };
  // Finds tile `tile` and turns the loads to it; behind the last one they load zeros.
  auto locate = [&](int tile, Tile& x) {
    left = 0;
    if (tile >= total) return;
    const int at = (tile - wide) / NT;
    x.e = find_expert(experts.first_short, p.rows.E, at);
    x.nt = tile - wide - at * NT;
    x.row0 = (uniform(experts.first[x.e + 1]) - uniform(experts.first[x.e])) * kBM;
    x.nrows = uniform(experts.count[x.e]) - x.row0;
    x.slot0 = uniform(experts.slot[x.e]) + (blocks ? 0 : x.row0);
    a0 = p.a + (int64_t)x.slot0 * p.a_row;
    b0 = p.b + (int64_t)x.e * p.b_expert + (int64_t)x.nt * kCols * p.b_row;
    left = p.k;
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const int r = w * 16 + j * 8 + (l >> 3), c = chunk_k(j) * 16;
      int s = r;                         // slots behind slot0
      if (blocks && s < x.nrows) s = p.rows.slot(x.e, x.row0 + s) - x.slot0;
      off_a[j] = r < x.nrows ? s * (int)p.a_row + c : kAbsent;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int col = Epi::gate ? r : h * 128 + r;
        off_b[h][j] = x.nt * kCols + col < p.n ? col * (int)p.b_row + c : kAbsent;
      }
    }
  };

  Tile cur, next;
  locate(tile, cur);
  next = cur;
  load(0, 0);
  load(1, 1);
  int stage = 0, ahead = 2;
  bool stores = false;         // the last epilogue surely sent kStores of them
  constexpr int kStores = Epi::stores / 2;
  for (;;) {
    acc_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 4; i++) acc[i >> 1][i & 1] = acc_t{};
    const bool any = wm * 64 < cur.nrows;
    for (int t = 0; t < KT; t++) {
      // this step's loads have arrived and the last one's stage is read by all: it is loaded
      // again.  Behind an epilogue its stores stay under way for two steps.
      if (t < 2 && stores) wait_loads<6 + kStores>();
      else wait_loads<6>();
      barrier();
      if (t == KT - 2) locate(tile + G, next);
      load(t + 2 < KT ? t + 2 : t + 2 - KT, ahead);
      if (any) {
        const uint8_t* st = lds + stage * kStream;
        u32x4 fa[2][4], fb[2][4];
#pragma unroll
        for (int ks = 0; ks < 4; ks++)
#pragma unroll
          for (int i = 0; i < 2; i++) {
            fa[i][ks] = fragment<false>(st + i * 4096, read_a, ks);
            fb[i][ks] = fragment<false>(st + i * kHalf, read_b, ks);
          }
        wait_lds();
#pragma unroll
        for (int ks = 0; ks < 4; ks++)
#pragma unroll
          for (int i = 0; i < 4; i++)
            acc[i >> 1][i & 1] = mfma<I8>(fb[i >> 1][ks], fa[i & 1][ks], acc[i >> 1][i & 1]);
      }
      stage = stage == 2 ? 0 : stage + 1;
      ahead = ahead == 2 ? 0 : ahead + 1;
    }
    // ---- results, through the stage that was read last, each wavefront where its own next
    // loads go
    barrier();
    uint8_t* const mine0 = lds + ahead * kStream + w * 2048;
    uint8_t* const mine1 = mine0 + kHalf;
    auto row_at = [&](int r) {
      return blocks ? p.rows.slot(cur.e, cur.row0 + r) : cur.slot0 + r;
    };
    const int c0 = cur.nt * kCols + wn * 32;
    float row_scale[1][2];
    f32x4 scales[2][4];
    if constexpr (I8)
      load_scales(epi, cur.e, wm * 64, cur.nrows, c0, l, row_at, row_scale, scales);
    store_block<Epi, I8>(epi, cur.e, wm * 64, cur.nrows, c0, acc, row_scale[0], scales, mine0, mine1, l,
                         row_at);
    tile += G;
    if (tile >= total) break;
    stores = cur.nrows == kStreamM && (cur.nt + 1) * kCols <= epi.columns(cur.e);
    wait_lds();
    cur = next;
  }
  wait_loads<0>();             // zeros behind the last tile
}

template <int KIND, class Epi, bool I8>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
void product_kernel(Product p, Epi epi) {
  constexpr bool kSlowA = KIND == kOuter, kSlowB = KIND != kRowsT;
  using acc_t = typename Acc<I8>::type;
  using val_t = typename Acc<I8>::scalar;

  __shared__ __attribute__((aligned(1024))) uint8_t lds[kSteps * kStage + 8 * 2048];
  __shared__ Experts experts;

  const int tid = threadIdx.x, l = tid & 63, w = uniform(tid >> 6);
  const int wm = w >> 2, wn = w & 3;     // rows wm*64.., columns wn*32.. of each half
  const uint32_t lds0 = (uint32_t)(uintptr_t)(EP_LDS uint8_t*)lds;
  const int NT = KIND == kRowsT && p.far ? (p.n + 127) / 128 : (p.n + kBN - 1) / kBN;
  const int MT = (p.m + kBM - 1) / kBM;                    // kOuter, of its first product
  const bool blocks = p.rows.count && !p.rows.offset;      // rows of several sub-blocks
  experts.fill(p.rows, kBM);
  // Tiles, those of over 128 rows, and those of them that are taken as two halves of 128 rows:
  // what is left for the last round of the grid's workgroups, where the rounds then take
  // less time.  Half a tile takes about 0.6 of a tile's.  16 experts of 512 rows on average:
  // dh, 264 tall and 48 short tiles, 392 us without halves, 355 with them.
  const int G = gridDim.x;
  const int NT2 = (p.also.n + kBN - 1) / kBN, MT2 = (p.also.m + kBM - 1) / kBM;
  int total = p.rows.E * (MT * NT + MT2 * NT2), tall = 0, halved = 0, all = 0;
  if constexpr (KIND != kOuter) {
    tall = uniform(experts.first[p.rows.E]) * NT;
    total = tall + uniform(experts.first_short[p.rows.E]) * NT;
    const int rest = tall % G, shorts = total - tall;
    const int kept = 10 + 6 * ((max(0, shorts - (G - rest)) + G - 1) / G);
    if (rest > 0 && 6 * ((2 * rest + shorts + G - 1) / G) < kept) {
      halved = rest;
      total += rest;
    }
    all = total;
    if constexpr (KIND == kRowsT) total = tall + halved;   // the short ones: stream()
  }

  // where this lane's bytes of a load go (a wavefront sends two loads per half: rows
  // w*16 + 8 j + l/8, or k w*8 + 4 j + l/16), and where it reads
  const int chunk_n = (l & 15) ^ ((l >> 4) << 2);          // of 128 columns of a k
  auto chunk_k = [&](int j) { return (l & 7) ^ ((j << 2) + (l >> 4)); };   // of a row
  const int read_k = (l & 31) * 128 + (((l >> 5) ^ ((l >> 1) & 7)) << 4);
  const int i16 = l & 15;
  auto read_n = [&](int chunk) {
    return ((l >> 5) * 8 + (i16 >> 2)) * 256 +
           (((chunk + ((l >> 4) & 1) * 2 + ((i16 & 3) >> 1)) ^ ((i16 >> 2) << 2)) << 4) +
           (i16 & 1) * 8;
  };
  int read_a[2];
#pragma unroll
  for (int mb = 0; mb < 2; mb++)
    read_a[mb] = kSlowA ? read_n(wm * 8 + mb * 4) : (wm * 64 + mb * 32) * 128 + read_k;
  const int read_b = kSlowB ? read_n(wn * 4) : wn * 32 * 128 + read_k;

  struct Tile {
    int e, nt, nrows, row0, slot0, KT;
  };
  // ---- what the loads run over: the current tile, and from its last steps on the next
  const uint8_t *a0 = nullptr, *b0 = nullptr;
  int k_a = 0, k_b = 0;        // contraction of a and b in what their tail counts
  int off_a[2][2], off_b[2][2];
  const int64_t far = (int64_t)p.far * p.b_row;
  int64_t step_a = kSlowA ? 64 * p.a_row : 128, step_b = kSlowB ? 64 * p.b_row : 128;

  // step t of the operand at `at`; TAIL: its last bytes may be behind the contraction's end
  auto load_a = [&](auto tail, const uint8_t* at, int t, int stage, int h) {
    int o[2];
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const bool in = !decltype(tail)::value ||
                      (kSlowA ? w * 8 + j * 4 + (l >> 4) < k_a - t * 64
                              : chunk_k(j) * 16 < k_a - t * 128);
      o[j] = in ? off_a[h][j] : kAbsent;
    }
    load_lds2<false>(lds0 + stage * kStage + h * kHalf + w * 2048, o[0], o[1], descriptor(at));
  };
  auto load_b = [&](auto tail, const uint8_t* at, int t, int stage, int h) {
    int o[2];
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const bool in = !decltype(tail)::value ||
                      (kSlowB ? w * 8 + j * 4 + (l >> 4) < k_b - t * 64
                              : chunk_k(j) * 16 < k_b - t * 128);
      o[j] = in ? off_b[h][j] : kAbsent;
    }
    load_lds2<KIND == kRowsT>(lds0 + stage * kStage + (2 + h) * kHalf + w * 2048, o[0], o[1],
                              descriptor(at + h * far));
  };
  // what the first phase of step t reads
  auto load_first = [&](auto tail, const uint8_t* at_a, const uint8_t* at_b, int t, int stage) {
    load_b(tail, at_b, t, stage, 0);
    load_a(tail, at_a, t, stage, 0);
    load_b(tail, at_b, t, stage, 1);
  };
  constexpr std::true_type kTail{};
  constexpr std::false_type kWhole{};

  // Finds tile `tile` and turns the loads to it; behind the last one they load zeros.
  auto locate = [&](int tile, Tile& x) {
    x.KT = 2;
    k_a = k_b = 0;
    if (tile >= total) return;
    int64_t a_row = p.a_row, b_row = p.b_row;
    int n = p.n;
    if constexpr (KIND == kOuter) {
      const bool first = tile < p.rows.E * MT * NT;
      const int nts = first ? NT : NT2, mts = first ? MT : MT2;
      if (!first) {
        tile -= p.rows.E * MT * NT;
        a_row = p.also.a_row;
        b_row = p.also.b_row;
        n = p.also.n;
      }
      const int e = tile / (mts * nts), r = tile - e * mts * nts;
      const int g = r / (kGroupM * nts), f = g * kGroupM, gs = min(kGroupM, mts - f);
      const int q = r - g * kGroupM * nts;
      x.e = first ? e : e + p.rows.E;
      x.row0 = (f + q % gs) * kBM;
      x.nt = q / gs;
      x.nrows = min(kBM, (first ? p.m : p.also.m) - x.row0);
      k_a = k_b = uniform(experts.count[e]);
      x.slot0 = uniform(experts.slot[e]);
      a0 = (first ? p.a : p.also.a) + (int64_t)x.slot0 * a_row + (int64_t)x.row0 * 2;
      b0 = (first ? p.b : p.also.b) + (int64_t)x.slot0 * b_row + (int64_t)x.nt * kBN * 2;
      step_a = 64 * a_row;
      step_b = 64 * b_row;
      x.KT = max(2, (k_a + 63) / 64);
    } else {
      // the short ones last: they take half the time, and a workgroup whose share was all
      // tall ones would keep the others waiting
      const bool is_short = KIND != kRowsT && tile >= tall + halved;
      const int half = tile - (tall - halved);               // of a halved one
      const int at = is_short ? tile - (tall + halved) : half >= 0 ? tall - halved + half / 2 : tile;
      x.e = is_short ? find_expert(experts.first_short, p.rows.E, at / NT)
                     : find_expert(experts.first, p.rows.E, at / NT);
      const int f0 = uniform(experts.first[x.e]), mts = uniform(experts.first[x.e + 1]) - f0;
      if (is_short) {
        x.row0 = mts * kBM;
        x.nt = at % NT;
      } else {
        const int r = at - f0 * NT;
        const int g = r / (kGroupM * NT), f = g * kGroupM, gs = min(kGroupM, mts - f);
        const int q = r - g * kGroupM * NT;
        x.row0 = (f + q % gs) * kBM;
        x.nt = q / gs;
      }
      int most = kBM;
      if (!is_short && half >= 0) {
        most = kBM / 2;
        x.row0 += half % 2 * most;
      }
      x.nrows = min(most, uniform(experts.count[x.e]) - x.row0);
      x.slot0 = uniform(experts.slot[x.e]) + (blocks ? 0 : x.row0);
      a0 = p.a + (int64_t)x.slot0 * p.a_row;
      b0 = p.b + (int64_t)x.e * p.b_expert;
      if constexpr (KIND == kRowsT)
        b0 += (int64_t)x.nt * (p.far ? 128 : kBN) * p.b_row;
      else
        b0 += (int64_t)x.nt * kBN * 2;
      k_a = p.k;
      k_b = KIND == kRows ? p.k / 2 : p.k;    // rows of b, or bytes of its rows
      x.KT = max(2, (p.k + 127) / 128);
    }
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
      for (int j = 0; j < 2; j++) {
        const int r = w * 16 + j * 8 + (l >> 3), k = w * 8 + j * 4 + (l >> 4);
        const int c = h * 128 + chunk_n * 8;
        if constexpr (kSlowA) {
          off_a[h][j] = c < x.nrows ? k * (int)a_row + c * 2 : kAbsent;
        } else {
          int s = h * 128 + r;               // slots behind slot0
          const bool in = s < x.nrows;
          if (blocks && in) s = p.rows.slot(x.e, x.row0 + s) - x.slot0;
          off_a[h][j] = in ? s * (int)p.a_row + chunk_k(j) * 16 : kAbsent;
        }
        if constexpr (kSlowB)
          off_b[h][j] = x.nt * kBN + c < n ? k * (int)b_row + c * 2 : kAbsent;
        else if (p.far)
          off_b[h][j] = x.nt * 128 + r < p.n ? r * (int)p.b_row + chunk_k(j) * 16 : kAbsent;
        else
          off_b[h][j] = x.nt * kBN + h * 128 + r < p.n
                            ? (r + h * 128) * (int)p.b_row + chunk_k(j) * 16 : kAbsent;
      }
  };

  // workgroup ids go round robin over the 8 XCDs: give each XCD neighbouring tiles
  int tile = G % 8 == 0 ? (blockIdx.x % 8) * (G / 8) + blockIdx.x / 8 : blockIdx.x;
  if constexpr (KIND == kRowsT) {
    if (tile >= total) {
      if (tile < all) stream<Epi, I8>(p, epi, lds, experts, tile, total, all);
      return;
    }
  } else if (tile >= total) {
    return;
  }
  Tile cur, next;
  locate(tile, cur);
  next = cur;
  load_first(kTail, a0, b0, 0, 0);
  load_a(kTail, a0, 0, 0, 1);
  load_first(kTail, a0 + step_a, b0 + step_b, 1, 1);
  wait_loads<8>();
  barrier();
  if (wm == 1) barrier();
  int stage = 0;
  bool stores = false;         // the last epilogue surely sent kStores of them
  constexpr int kStores = Epi::stores;
  for (;;) {
    acc_t acc[2][2][2];
#pragma unroll
    for (int i = 0; i < 8; i++) acc[i >> 2][(i >> 1) & 1][i & 1] = acc_t{};

    // ---- the loop.  Two groups of four wavefronts, one of each group on every SIMD, half
    // a phase apart: while one group's MFMAs run, the other reads its next fragments and
    // sends loads.  Phases per step: b and a's first half, a's second half.  Loads run one
    // step and a phase ahead, across the tiles; a half tile is loaded again as soon as
    // both groups have read it: reads have returned (wait_lds) before the barrier behind
    // which the load is sent, and a load has arrived (wait_loads) one barrier before it is
    // read.  vmcnt counts the epilogue's stores as well, which a tile's first step leaves
    // under way.
    const bool any0 = wm * 64 < cur.nrows, any1 = 128 + wm * 64 < cur.nrows;
    const int KT = cur.KT;
    // One step; `load1` and `load2` send the loads of its two phases.
    auto step = [&](auto&& load1, auto&& load2, auto&& wait) {
      const uint8_t* st = lds + stage * kStage;
      u32x4 fa[2][4], fb[2][4];
      auto read_as = [&](int h) {
#pragma unroll
        for (int mb = 0; mb < 2; mb++)
#pragma unroll
          for (int ks = 0; ks < 4; ks++)
            fa[mb][ks] = fragment<kSlowA>(st + h * kHalf, read_a[mb], ks);
      };
      auto multiply = [&](int h) {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int ks = 0; ks < 4; ks++)
#pragma unroll
          for (int i = 0; i < 4; i++)
            acc[h][i >> 1][i & 1] =
                mfma<I8>(fb[i >> 1][ks], fa[i & 1][ks], acc[h][i >> 1][i & 1]);
        __builtin_amdgcn_s_setprio(0);
      };
      if (any0) {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int ks = 0; ks < 4; ks++)
            fb[h][ks] = fragment<kSlowB>(st + (2 + h) * kHalf, read_b, ks);
        read_as(0);
      }
      load1();
      wait();
      wait_lds();
      barrier();
      if (any0) multiply(0);
      barrier();
      if (any1) read_as(1);
      load2();
      wait();
      wait_lds();
      barrier();
      if (any1) multiply(1);
      barrier();
      stage ^= 1;
    };
    for (int t = 0; t < KT;) {
      // the first step, and the last three, whose loads reach the end or the next tile
      step([&] {
             const int s = t + 1 < KT ? t + 1 : 0;
             load_a(kTail, a0 + s * step_a, s, stage ^ 1, 1);
           },
           [&] {
             if (t == KT - 2) locate(tile + G, next);
             const int s = t + 2 < KT ? t + 2 : t + 2 - KT;
             load_first(kTail, a0 + s * step_a, b0 + s * step_b, s, stage);
           },
           [&] {
             if (t == 0 && stores) wait_loads<8 + kStores>();
             else wait_loads<8>();
           });
      t++;
      // those between, without branches or bounds
      const uint8_t *a1 = a0 + (t + 1) * step_a, *b2 = b0 + (t + 2) * step_b;
      for (; t < KT - 3; t++) {
        step([&] { load_a(kWhole, a1, 0, stage ^ 1, 1); },
             [&] {
               a1 += step_a;
               load_first(kWhole, a1, b2, 0, stage);
               b2 += step_b;
             },
             [] { wait_loads<8>(); });
      }
    }

    // ---- this tile's results are in registers, the next one's first loads under way.
    // They go through LDS: half of it where this wavefront's own next load goes, so that
    // no other one is waited for.
    uint8_t* const mine0 = lds + (stage ^ 1) * kStage + kHalf + w * 2048;
    uint8_t* const mine1 = lds + kSteps * kStage + w * 2048;
    // this lane as a value of its own: what follows from it is computed here, not before
    // the loop, whose registers are all in use
    int v = l;
    asm volatile("" : "+v"(v));
    const int swizzle = (v >> 1) & 7;        // of row v % 32, that is v % 16
    uint8_t* const to_row = (v & 16 ? mine1 : mine0) + (v & 15) * 128;
    const int take_at = (v >> 2) * 128, take_swizzle = (v >> 3) & 7;
    // blocks in 32 bits, for an epilogue that does not round first
    auto turn = [&](const acc_t& x) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        u32x4 q;
#pragma unroll
        for (int j = 0; j < 4; j++)
          q[j] = __builtin_bit_cast(uint32_t, (val_t)x[i * 4 + j]);
        *(u32x4*)(to_row + (((2 * i + (v >> 5)) ^ swizzle) << 4)) = q;
      }
    };
    auto take = [&](int it, val_t* to) {     // 16 rows `it`, row v / 4, columns 8 (v % 4) ..
#pragma unroll
      for (int q = 0; q < 2; q++) {
        const u32x4 x = *(const u32x4*)((it ? mine1 : mine0) + take_at +
                                        (((2 * (v & 3) + q) ^ take_swizzle) << 4));
#pragma unroll
        for (int j = 0; j < 4; j++) to[q * 4 + j] = __builtin_bit_cast(val_t, (uint32_t)x[j]);
      }
    };
    auto row_at = [&](int r) {
      return KIND == kOuter ? cur.row0 + r
             : blocks       ? p.rows.slot(cur.e, cur.row0 + r)
                            : cur.slot0 + r;
    };
    const int c00 = cur.nt * (Epi::gate ? 128 : kBN) + wn * 32, c0 = c00 + (v & 3) * 8;
    if constexpr (Epi::rounds) {
      float row_scale[2][2];
      f32x4 scales[2][4];
      if constexpr (I8)
        load_scales(epi, cur.e, wm * 64, cur.nrows, c00, v, row_at, row_scale, scales);
#pragma unroll
      for (int h = 0; h < 2; h++)
        store_block<Epi, I8>(epi, cur.e, h * 128 + wm * 64, cur.nrows, c00, acc[h], row_scale[h],
                             scales, mine0, mine1, v, row_at);
    } else {
#pragma unroll
      for (int b = 0; b < 4; b++) {
        const int r0 = (b >> 1) * 128 + wm * 64 + (b & 1) * 32;
        if (r0 >= cur.nrows) continue;
        // a block's operands together, one latency instead of four (rows behind the last:
        // the last again)
        typename Epi::Ahead ahead[4];
        int row[2];
#pragma unroll
        for (int it = 0; it < 2; it++) {
          row[it] = row_at(min(r0 + it * 16 + (v >> 2), cur.nrows - 1));
          ahead[it] = epi.ahead(row[it], c0);
          ahead[2 + it] = epi.ahead(row[it], c0 + 128);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
          arrive(ahead[i].g);
          arrive(ahead[i].u);
        }
#pragma unroll
        for (int qn = 0; qn < 2; qn++) {
          val_t x[2][8];
          turn(acc[b >> 1][qn][b & 1]);
          take(0, x[0]);
          take(1, x[1]);
#pragma unroll
          for (int it = 0; it < 2; it++)
            if (r0 + it * 16 + (v >> 2) < cur.nrows)
              epi(ahead[qn * 2 + it], row[it], c0 + qn * 128, x[it]);
        }
      }
    }
    tile += G;
    if (tile >= total) break;
    // whole tiles store the same number of times, and so do the ones behind this here
    stores = cur.nrows == kBM && (cur.nt + 1) * (Epi::gate ? 128 : kBN) <= epi.columns(cur.e);
    wait_lds();
    cur = next;
  }
  wait_loads<0>();             // zeros behind the last tile
  if (wm == 0) barrier();
  if constexpr (KIND == kRowsT) {
    if (tile < all) {
      wait_lds();
      barrier();
      stream<Epi, I8>(p, epi, lds, experts, tile, total, all);
    }
  }
}

// ---------------------------------------------------------------- few rows
// Rows that are too few to fill 256-row tiles: a workgroup takes 32 rows of the weight (16
// of gate and 16 of up) and 16 TT rows of x, its four wavefronts take every fourth 128
// bytes of the contraction, each with loads of its own running ahead in LDS of its own, so
// that there is no barrier before the sums meet at the end.
// FUSE: at most 16 rows of x in bf16, which every workgroup rounds to 8-bit integers
// itself while its first weights are on their way (51 MB of weights: 14 us; rounded by a
// launch before it, 4 + 11).
// Bound by HBM from about 50 MB of weights on (7168 x 2048 for 32 experts of 16 rows: 5.5
// TB/s), below that by the latency of counts, weights and sums one after the other: 5 us.
template <bool I8>
struct Acc4 {
  using type = std::conditional_t<I8, i32x4, f32x4>;
};

template <bool I8>
__device__ __forceinline__ typename Acc4<I8>::type mfma16(u32x4 a, u32x4 b,
                                                          typename Acc4<I8>::type c) {
  if constexpr (I8)
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                                 __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

constexpr int kFuseBytes = 32768;      // x in LDS, in bf16

template <class Epi, bool I8, int TT, bool FUSE>
__global__ __launch_bounds__(256) void few_kernel(Product p, Epi epi) {
  constexpr int kRowsX = 16 * TT, kCols = Epi::gate ? 16 : 32;
  constexpr int kW = 4096, kX = FUSE ? 0 : kRowsX * 128;     // bytes of a stage
  constexpr int kDepth = FUSE ? 7 : TT == 1 ? 3 : 2;
  constexpr int kLoads = 4 + (FUSE ? 0 : 2 * TT);
  constexpr int kMine = kDepth * (kW + kX);
  using acc_t = typename Acc4<I8>::type;
  using val_t = typename Acc<I8>::scalar;
  static_assert(kMine >= kRowsX * 32 * 4, "a wavefront's sums fit where its stages were");

  __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * kMine + (FUSE ? kFuseBytes : 0)];
  __shared__ int slots[kRowsX];
  __shared__ float scale[16];            // FUSE: of each row of x
  __shared__ RowScale scales[FUSE ? 16 : 1];
  __shared__ uint32_t tops[16];

  const int tid = threadIdx.x, l = tid & 63, w = uniform(tid >> 6);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(EP_LDS uint8_t*)lds;
  const uint32_t mine = lds0 + w * kMine;
  const uint8_t* my = lds + w * kMine;
  const int NT = (p.n + kCols - 1) / kCols, KT = (p.k + 127) / 128, NI = (KT + 3) / 4;
  const int64_t far = (int64_t)p.far * p.b_row;
  auto chunk_k = [&](int j) { return (l & 7) ^ (((j & 1) << 2) + (l >> 4)); };
  const int read = (l & 15) * 128 + (((l >> 4) ^ ((l >> 1) & 7)) << 4);
  const int G = gridDim.x;
  int tile = G % 8 == 0 ? (blockIdx.x % 8) * (G / 8) + blockIdx.x / 8 : blockIdx.x;
  const bool blocks = p.rows.count && !p.rows.offset;
  for (; tile <= kLastTile; tile += G) {
    int e = 0, nt = tile, nrows = p.rows.plain, slot0 = 0;
    if constexpr (!FUSE) {
      Found x;
      if (!find_rows(p.rows, kRowsX, tile / NT, x)) break;
      e = x.e;
      const int r = tile - x.first * NT;
      const int g = r / (kGroupM * NT), f = g * kGroupM, gs = min(kGroupM, x.tiles - f);
      const int q = r - g * kGroupM * NT;
      const int row0 = (f + q % gs) * kRowsX;
      nt = q / gs;
      nrows = min(kRowsX, x.count - row0);
      slot0 = x.slot + (blocks ? 0 : row0);
      if (tid < kRowsX)
        slots[tid] = tid >= nrows ? -1 : blocks ? p.rows.slot(e, row0 + tid) : slot0 + tid;
      __syncthreads();
    } else if (tile >= NT) {
      break;
    } else if (tid < kRowsX) {
      slots[tid] = tid < nrows ? tid : -1;
      tops[tid] = 0;
    }
    const uint8_t* a0 = p.a + (int64_t)slot0 * p.a_row;
    const uint8_t* b0 = p.b + (int64_t)e * p.b_expert + (int64_t)nt * kCols * p.b_row;
    int off_w[4], off_x[FUSE ? 1 : 2 * TT];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int r = (Epi::gate ? j & 1 : j) * 8 + (l >> 3);
      off_w[j] = nt * kCols + r < p.n ? (int)(r * p.b_row) + chunk_k(j) * 16 : kAbsent;
    }
    if constexpr (!FUSE) {
#pragma unroll
      for (int j = 0; j < 2 * TT; j++) {
        const int s = slots[j * 8 + (l >> 3)];
        off_x[j] = s >= 0 ? (int)((s - slot0) * p.a_row) + chunk_k(j) * 16 : kAbsent;
      }
    }
    // step i of this wavefront: bytes 128 (4 i + w) .. of the contraction
    auto load = [&](int i, int stage) {
      const int at = (i * 4 + w) * 128;
      const uint32_t to = mine + stage * (kW + kX);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const i32x4 d = descriptor(b0 + at + (Epi::gate && j >= 2 ? far : 0));
        load_lds<true>(to + j * 1024, chunk_k(j) * 16 < p.k - at ? off_w[j] : kAbsent, d);
      }
      if constexpr (!FUSE) {
        const i32x4 d = descriptor(a0 + at);
#pragma unroll
        for (int j = 0; j < 2 * TT; j++)
          load_lds<false>(to + kW + j * 1024, chunk_k(j) * 16 < p.k - at ? off_x[j] : kAbsent, d);
      }
    };
    // x is still bf16 (FUSE): p.a_row counts its bytes.  It is asked for before the weights,
    // since loads arrive in order.
    uint8_t* const xs = lds + 4 * kMine;
    if constexpr (FUSE) {
      const i32x4 d = descriptor(p.a);
#pragma unroll
      for (int j = 0; j < kFuseBytes / 4096; j++) {
        const int at = (j * 4 + w) * 1024;
        load_lds<false>(lds0 + 4 * kMine + at, at + l * 16 < nrows * (int)p.a_row ? at + l * 16 : kAbsent,
                        d);
      }
    }
#pragma unroll
    for (int i = 0; i < kDepth; i++) load(i, i);
    if constexpr (FUSE) {
      wait_loads<kDepth * kLoads>();
      __syncthreads();
      // every thread holds its chunks of all rows, so the codes may take their place
      constexpr int kHeld = kFuseBytes / 4096;
      const int per = p.k / 8, chunks = nrows * per;
      u32x4 held[kHeld];
      int row[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld; i++) {
        const int c = i * 256 + tid;
        row[i] = c / per;
        if (i * 256 >= chunks) break;
        held[i] = *(const u32x4*)(xs + min(c, chunks - 1) * 16);
        const uint32_t top = largest8(held[i]);
        const int r = min(row[i], nrows - 1), r0 = uniform(r);
        if (__all(r == r0)) {
          const uint32_t of_row = wave_max(top);
          if (l == 0) atomicMax(&tops[r0], of_row);
        } else {
          atomicMax(&tops[r], top);
        }
      }
      __syncthreads();
      if (tid < nrows) {
        const RowScale s = RowScale::of(tops[tid]);
        scales[tid] = s;
        scale[tid] = s.scale;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kHeld; i++) {
        const int c = i * 256 + tid;
        if (c < chunks) *(u32x2*)(xs + c * 8) = scales[row[i]].codes8(held[i]);
      }
      epi.sx = scale;
      __syncthreads();
    }

    acc_t acc[2][TT];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int j = 0; j < TT; j++) acc[i][j] = acc_t{};
    int stage = 0;
    for (int i = 0; i < NI; i++) {
      wait_loads<(kDepth - 1) * kLoads>();
      const uint8_t* st = my + stage * (kW + kX);
      u32x4 fw[2][2], fx[TT][2];
#pragma unroll
      for (int m = 0; m < 2; m++) {
#pragma unroll
        for (int r = 0; r < 2; r++) fw[r][m] = *(const u32x4*)(st + r * 2048 + (read ^ (m * 64)));
        if constexpr (FUSE) {
          const int at = (i * 4 + w) * 128 + m * 64 + (l >> 4) * 16;
          fx[0][m] = (l & 15) < nrows && at < p.k
                         ? *(const u32x4*)(xs + (l & 15) * p.k + at)
                         : u32x4{0, 0, 0, 0};
        } else {
#pragma unroll
          for (int j = 0; j < TT; j++)
            fx[j][m] = *(const u32x4*)(st + kW + j * 2048 + (read ^ (m * 64)));
        }
      }
      wait_lds();                       // read before the stage is loaded again
      load(i + kDepth, stage);
      stage = stage + 1 == kDepth ? 0 : stage + 1;
#pragma unroll
      for (int m = 0; m < 2; m++)
#pragma unroll
        for (int r = 0; r < 2; r++)
#pragma unroll
          for (int j = 0; j < TT; j++) acc[r][j] = mfma16<I8>(fw[r][m], fx[j][m], acc[r][j]);
    }
    wait_loads<0>();                    // those behind the last step: zeros

    // ---- lane l has weight rows 16 r + 4 (l / 16) + 0..3 of x's row 16 j + l % 16
#pragma unroll
    for (int r = 0; r < 2; r++)
#pragma unroll
      for (int j = 0; j < TT; j++)
        *(u32x4*)(lds + w * kMine + (j * 16 + (l & 15)) * 128 +
                  (((r * 4 + (l >> 4)) ^ ((l >> 1) & 7)) << 4)) =
            __builtin_bit_cast(u32x4, acc[r][j]);
    __syncthreads();
    constexpr int kChunks = kCols / 8;
    const int row = tid / kChunks, c = tid % kChunks;
    if (row < nrows && row < kRowsX) {
      val_t v[8], u[8];
      auto sum = [&](int chunk, val_t* to) {
#pragma unroll
        for (int q = 0; q < 2; q++) {
          acc_t t = {};
#pragma unroll
          for (int o = 0; o < 4; o++)
            t += *(const acc_t*)(lds + o * kMine + row * 128 +
                                 (((chunk + q) ^ ((row >> 1) & 7)) << 4));
#pragma unroll
          for (int j = 0; j < 4; j++) to[q * 4 + j] = t[j];
        }
      };
      sum(2 * c, v);
      if constexpr (Epi::gate) sum(4 + 2 * c, u);
      epi(e, slots[row], nt * kCols + c * 8, v, u);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- small products
// Products whose 256 by 256 tiles would leave most CUs idle: 64 by 64 tiles, each
// wavefront all of a tile over every fourth step of the contraction, with loads of its own
// in LDS of its own, as above.
constexpr int kST = 64;                // rows and columns of a tile

template <int KIND, class Epi, bool I8>
__global__ __launch_bounds__(256) void small_kernel(Product p, Epi epi) {
  constexpr bool kSlowA = KIND == kOuter, kSlowB = KIND != kRowsT;
  constexpr int kCols = Epi::gate ? kST / 2 : kST;         // of gate, and as many of up
  using acc_t = typename Acc<I8>::type;
  using val_t = typename Acc<I8>::scalar;
  typedef val_t val4 __attribute__((ext_vector_type(4)));
  constexpr int kOp = 8192, kSmallStage = 2 * kOp, kMine = 2 * kSmallStage, kLoads = 16;

  __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * kMine];
  __shared__ int slots[kST];

  const int tid = threadIdx.x, l = tid & 63, w = uniform(tid >> 6);
  const uint32_t mine = (uint32_t)(uintptr_t)(EP_LDS uint8_t*)lds + w * kMine;
  const uint8_t* my = lds + w * kMine;
  const int NT = (p.n + kCols - 1) / kCols, MT = (p.m + kST - 1) / kST;
  const int NT2 = (p.also.n + kST - 1) / kST, MT2 = (p.also.m + kST - 1) / kST;    // kOuter
  // chunk c of row r at c ^ (r / 2 & 7); where k is slow, of 128 bytes of a k at c ^ 4 (k / 2 & 1)
  auto chunk_k = [&](int j) { return (l & 7) ^ (((j & 1) << 2) + (l >> 4)); };
  const int chunk_n = (l & 7) ^ (((l >> 4) & 1) << 2);
  const int read_k = (l & 31) * 128 + (((l >> 5) ^ ((l >> 1) & 7)) << 4);
  const int i16 = l & 15;
  const int read_n = ((l >> 5) * 8 + (i16 >> 2)) * 128 +
                     (((((l >> 4) & 1) * 2 + ((i16 & 3) >> 1)) ^ ((i16 >> 3) << 2)) << 4) +
                     (i16 & 1) * 8;
  auto slow = [&](const uint8_t* op, int b, int ks) {      // columns 32 b .., k 16 ks ..
    const int at = (read_n ^ (b << 6)) + ks * 2048;
    const u32x2 lo = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((EP_LDS bf16x4*)(op + at)));
    const u32x2 hi = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((EP_LDS bf16x4*)(op + at + 512)));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3);
  };
  auto fast = [&](const uint8_t* op, int b, int ks) {
    return *(const u32x4*)(op + b * 4096 + (read_k ^ (ks * 32)));
  };

  const int G = gridDim.x;
  int tile = G % 8 == 0 ? (blockIdx.x % 8) * (G / 8) + blockIdx.x / 8 : blockIdx.x;
  const bool blocks = p.rows.count && !p.rows.offset;
  for (; tile <= kLastTile; tile += G) {
    int e, nt, nrows, row0, slot0, k_a, k_b, KT, n = p.n;
    int64_t a_row = p.a_row, b_row = p.b_row;
    const uint8_t *a0, *b0;
    if constexpr (KIND == kOuter) {
      const int before = p.rows.E * MT * NT;
      if (tile >= before + p.rows.E * MT2 * NT2) break;
      const bool first = tile < before;
      const int nts = first ? NT : NT2, per = first ? MT * NT : MT2 * NT2;
      if (!first) {
        a_row = p.also.a_row;
        b_row = p.also.b_row;
        n = p.also.n;
      }
      const int at = first ? tile : tile - before, of = at / per, r = at - of * per;
      e = first ? of : of + p.rows.E;
      row0 = r / nts * kST;
      nt = r % nts;
      nrows = min(kST, (first ? p.m : p.also.m) - row0);
      k_a = k_b = uniform(p.rows.rows_of(of));
      KT = (k_a + 63) / 64;
      slot0 = uniform(p.rows.first_slot(of));
      a0 = (first ? p.a : p.also.a) + (int64_t)slot0 * a_row + (int64_t)row0 * 2;
      b0 = (first ? p.b : p.also.b) + (int64_t)slot0 * b_row + (int64_t)nt * kST * 2;
    } else {
      Found x;
      if (!find_rows(p.rows, kST, tile / NT, x)) break;
      e = x.e;
      const int r = tile - x.first * NT;
      row0 = r / NT * kST;
      nt = r % NT;
      nrows = min(kST, x.count - row0);
      slot0 = x.slot + (blocks ? 0 : row0);
      if (tid < kST)
        slots[tid] = tid >= nrows ? -1 : blocks ? p.rows.slot(e, row0 + tid) : slot0 + tid;
      a0 = p.a + (int64_t)slot0 * p.a_row;
      b0 = p.b + (int64_t)e * p.b_expert + (int64_t)nt * kCols * (kSlowB ? 2 : p.b_row);
      k_a = p.k;
      k_b = kSlowB ? p.k / 2 : p.k;
      KT = (p.k + 127) / 128;
      __syncthreads();
    }
    const int64_t step_a = kSlowA ? 64 * a_row : 128, step_b = kSlowB ? 64 * b_row : 128;
    int off_a[8], off_b[8];
    const bool in_a = chunk_n * 8 < nrows, in_b = nt * kST + chunk_n * 8 < n;
#pragma unroll
    for (int j = 0; j < 8; j++) {
      if constexpr (kSlowA) {
        off_a[j] = in_a ? (j * 8 + (l >> 3)) * (int)a_row + chunk_n * 16 : kAbsent;
      } else {
        const int s = slots[j * 8 + (l >> 3)];
        off_a[j] = s >= 0 ? (int)((s - slot0) * a_row) + chunk_k(j) * 16 : kAbsent;
      }
      if constexpr (kSlowB) {
        off_b[j] = in_b ? (j * 8 + (l >> 3)) * (int)b_row + chunk_n * 16 : kAbsent;
      } else {
        const int r = (Epi::gate ? j & 3 : j) * 8 + (l >> 3);
        off_b[j] = nt * kCols + r < n ? r * (int)b_row + chunk_k(j) * 16 : kAbsent;
      }
    }
    const int64_t far = (int64_t)p.far * p.b_row;
    auto load = [&](int i, int stage) {
      const int64_t t = i * 4 + w;
      const uint32_t to = mine + stage * kSmallStage;
      const i32x4 da = descriptor(a0 + t * step_a), db = descriptor(b0 + t * step_b);
      const i32x4 du = Epi::gate ? descriptor(b0 + far + t * step_b) : db;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int k = j * 8 + (l >> 3);
        const bool ok = kSlowA ? k < k_a - t * 64 : chunk_k(j) * 16 < k_a - t * 128;
        load_lds<false>(to + j * 1024, ok ? off_a[j] : kAbsent, da);
        const bool ok_b = kSlowB ? k < k_b - t * 64 : chunk_k(j) * 16 < k_b - t * 128;
        load_lds<false>(to + kOp + j * 1024, ok_b ? off_b[j] : kAbsent,
                        Epi::gate && j >= 4 ? du : db);
      }
    };
    acc_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 4; i++) acc[i >> 1][i & 1] = acc_t{};
    load(0, 0);
    load(1, 1);
    for (int i = 0; i * 4 < KT; i++) {
      wait_loads<kLoads>();
      const uint8_t* st = my + (i & 1) * kSmallStage;
      u32x4 fa[2][4], fb[2][4];
#pragma unroll
      for (int ks = 0; ks < 4; ks++)
#pragma unroll
        for (int b = 0; b < 2; b++) {
          if constexpr (kSlowA) fa[b][ks] = slow(st, b, ks);
          else fa[b][ks] = fast(st, b, ks);
          if constexpr (kSlowB) fb[b][ks] = slow(st + kOp, b, ks);
          else fb[b][ks] = fast(st + kOp, b, ks);
        }
      wait_lds();
      load(i + 2, i & 1);
#pragma unroll
      for (int ks = 0; ks < 4; ks++)
#pragma unroll
        for (int b = 0; b < 4; b++)
          acc[b >> 1][b & 1] = mfma<I8>(fb[b >> 1][ks], fa[b & 1][ks], acc[b >> 1][b & 1]);
    }
    wait_loads<0>();

    // sums: row r's 16 chunks of four columns, chunk c at c ^ (r & 15)
#pragma unroll
    for (int b = 0; b < 4; b++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int r = (b & 1) * 32 + (l & 31), c = (b >> 1) * 8 + 2 * i + (l >> 5);
        val4 v;
#pragma unroll
        for (int j = 0; j < 4; j++) v[j] = acc[b >> 1][b & 1][i * 4 + j];
        *(val4*)(lds + w * kMine + r * 256 + ((c ^ (r & 15)) << 4)) = v;
      }
    __syncthreads();
    constexpr int kChunks = kCols / 8;
#pragma unroll
    for (int h = 0; h < kST * kChunks / 256; h++) {
      const int r = h * (256 / kChunks) + tid / kChunks, c = tid % kChunks;
      if (r >= nrows) continue;
      val_t v[8], u[8];
      auto sum = [&](int chunk, val_t* to) {
#pragma unroll
        for (int q = 0; q < 2; q++) {
          val4 t = {};
#pragma unroll
          for (int o = 0; o < 4; o++)
            t += *(const val4*)(lds + o * kMine + r * 256 + (((chunk + q) ^ (r & 15)) << 4));
#pragma unroll
          for (int j = 0; j < 4; j++) to[q * 4 + j] = t[j];
        }
      };
      sum(2 * c, v);
      if constexpr (Epi::gate) sum(8 + 2 * c, u);
      epi(e, KIND == kOuter ? row0 + r : slots[r], nt * kCols + c * 8, v, u);
    }
    __syncthreads();
  }
}

template <int KIND, class Epi, bool I8>
int launch(const Product& p, const Epi& epi, int64_t tiles, hipStream_t st) {
  // one workgroup per CU at most: each takes more than half of a CU's LDS
  // (twice the tiles: they may be taken by halves)
  const int grid = (int)(tiles < 128 ? 2 * tiles : 256);
  EP_LOG("  wide tiles: up to %lld", (long long)tiles);
  product_kernel<KIND, Epi, I8><<<dim3(grid), dim3(512), 0, st>>>(p, epi);
  return check_launch("ep_ffn product");
}

// ---------------------------------------------------------------- which kernel
// Times in us that the choice between the kernels goes by, fitted to measurements of both
// sides (MI355X, graph replays); only their order matters.  Row tiles are counted on the
// device, so they go by the bound of all rows, taken as spread evenly.
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Most row tiles that max_rows rows of E experts can make.
int64_t row_tiles(const Rows& r, int max_rows, int tile) { return (int64_t)max_rows / tile + r.E; }

// 256 by 256 tiles, `tiles` of them, `steps` of 128 bytes of the contraction: a step takes
// 0.86 us on half a tile's rows, 1.3 on a whole tile's, 1.2 where all CUs stream weights; rows
// of columns that are no whole 16 bytes are stored in parts.
double wide_us(int64_t tiles, int64_t steps, double rows, int cols) {
  const double parts = cols % 8 ? 5 : 0;
  if (tiles >= 200) return 4 + (double)ceil_div(tiles, 256) * ((double)steps * 1.2 + 6 + parts);
  return 10 + (double)steps * (rows > 128 ? 1.3 : 0.86) + parts;
}

// 64 by 64 tiles: a step of a workgroup's four wavefronts is 64 KiB from the caches, which all
// CUs together get at 12 TB/s (4.8 where it is weights from HBM), or 0.55 us of one alone.
double small_us(double tiles, int64_t steps, double weight_bytes) {
  const double rounds = std::max(1.0, tiles / 256),
               step = std::max(0.55, 1.37 * std::min(1.0, tiles / 256));
  return 3.5 + std::max(rounds * ((double)ceil_div(steps, 4) * step + 2.8), weight_bytes / 4.8e6);
}

// How many tiles of t rows the experts' rows are on average.
double row_tiles_mean(int experts, double rows, int t) {
  if (experts == 1) return (double)ceil_div((int64_t)rows, t);
  return experts * std::max(1.0, rows / t + (rows > t ? 0.5 : rows > t / 2 ? 0.25 : 0));
}

template <class Epi, bool I8, int TT, bool FUSE>
int launch_few(const Product& p, const Epi& epi, int64_t row_tiles, hipStream_t st) {
  const int64_t tiles = row_tiles * ceil_div(p.n, Epi::gate ? 16 : 32);
  const int grid = (int)(tiles < 512 ? tiles : 512);       // two workgroups per CU
  EP_LOG("  few rows: %d rows a tile%s, %lld tiles", 16 * TT, FUSE ? " of bf16" : "",
         (long long)tiles);
  few_kernel<Epi, I8, TT, FUSE><<<dim3(grid), dim3(256), 0, st>>>(p, epi);
  return check_launch("ep_ffn few rows");
}

template <int KIND, class Epi, bool I8>
int launch_small(const Product& p, const Epi& epi, int64_t tiles, hipStream_t st) {
  EP_LOG("  small tiles: up to %lld", (long long)tiles);
  small_kernel<KIND, Epi, I8><<<dim3((int)(tiles < 256 ? tiles : 256)), dim3(256), 0, st>>>(p, epi);
  return check_launch("ep_ffn small product");
}

// Activations by a weight's rows.  Measured, wide, few, small (us), 8-bit, rows x columns of the
// weight: 1 row by 7168 x 7168 53, 11, -; 16 rows 53, 12, 14; 64 rows 63, 20, 17; 256 rows 68, 66,
// 41; 980 rows by 861 x 7120 92, 52, 23; 4000 by 4000 x 512 23, 114, 70; 33 by 1237 x 2000 23, 6,
// 9.  Both products of a bf16 block: 512 rows, 2048 x 1024 64, 35, 25; 2048 rows 67, 124, 80; 32
// experts of about 16 rows, 7168 x 2048: first 273, 313, second 183, 171.  Row tiles are
// estimated as at least one for each expert, also of fewer rows than experts: counted as
// min(experts, rows) the choice is few rows, and slower (8-bit block, 512 experts, 2048 x 512,
// 10 rows 35 us by wide tiles, 44 by few rows; 80 rows 81 : 123; bf16 has few rows either way).
template <class Epi, bool I8>
int run_rows(const Product& p, const Epi& epi, int max_rows, hipStream_t st) {
  const int E = p.rows.E, wide = Epi::gate ? 128 : kBN;
  const double rows = (double)max_rows / E, cols = Epi::gate ? 2.0 * p.n : p.n;
  const int64_t steps = ceil_div(p.k, 128);
  const double weight = cols * p.k;                        // bytes of one expert
  const int few = rows <= 8 ? 16 : 32;
  const double few_tiles = row_tiles_mean(E, rows, few);
  const double few_rounds = few_tiles * (cols / 32) / 512, few_steps = (double)ceil_div(steps, 4);
  const double few_us =
      3.5 + std::max(few_tiles * weight / (few == 16 ? 7.0e6 : 6.2e6),
                     few_rounds <= 1 ? few_steps * 0.35 + 0.5 : few_rounds * (few_steps * 0.45 + 2.7));
  const double small = small_us(row_tiles_mean(E, rows, kST) * cols / kST, steps, E * weight);
  const int64_t wide_tiles = E * std::max<int64_t>(1, (int64_t)(rows / kBM + 0.5)) *
                             ceil_div(p.n, wide);
  if (std::min(few_us, small) < wide_us(wide_tiles, steps, rows, p.n)) {
    if (small < few_us)
      return launch_small<kRowsT, Epi, I8>(
          p, epi, row_tiles(p.rows, max_rows, kST) * ceil_div(p.n, Epi::gate ? kST / 2 : kST), st);
    if (few == 16) return launch_few<Epi, I8, 1, false>(p, epi, row_tiles(p.rows, max_rows, 16), st);
    return launch_few<Epi, I8, 2, false>(p, epi, row_tiles(p.rows, max_rows, 32), st);
  }
  return launch<kRowsT, Epi, I8>(p, epi, row_tiles(p.rows, max_rows, kBM) * ceil_div(p.n, wide),
                                 st);
}

// A gradient, or the two of the weights in one launch.  Measured, small tiles against wide ones: 12
// experts of 88 rows, 1000 x 344: dh 13 : 39, dx 16 : 20, dw13 33 : 15; one matrix of 1024 rows,
// 2048 x 1024, all four 88 : 149; 8 experts of 512 rows, 1024 x 1024, all four 187 : 126.
template <int KIND, class Epi>
int run_grad(const Product& p, const Epi& epi, int max_rows, hipStream_t st) {
  const int E = p.rows.E;
  const double rows = (double)max_rows / E;
  if constexpr (KIND == kOuter) {
    auto tiles = [&](int t) {
      return E * (ceil_div(p.m, t) * ceil_div(p.n, t) + ceil_div(p.also.m, t) * ceil_div(p.also.n, t));
    };
    const int64_t steps = (int64_t)(rows / 64) + 1;
    if (small_us((double)tiles(kST), steps, 0) < wide_us(tiles(kBM), steps, kBM, p.n))
      return launch_small<KIND, Epi, false>(p, epi, tiles(kST), st);
    return launch<KIND, Epi, false>(p, epi, tiles(kBM), st);
  } else {
    const int64_t steps = ceil_div(p.k, 128),
                  wide_rows = std::max<int64_t>(1, (int64_t)(rows / kBM + 0.5));
    if (small_us(row_tiles_mean(E, rows, kST) * ceil_div(p.n, kST), steps, (double)E * p.n * p.k) <
        wide_us(E * wide_rows * ceil_div(p.n, kBN), steps, rows, p.n))
      return launch_small<KIND, Epi, false>(
          p, epi, row_tiles(p.rows, max_rows, kST) * ceil_div(p.n, kST), st);
    return launch<KIND, Epi, false>(p, epi,
                                    row_tiles(p.rows, max_rows, kBM) * ceil_div(p.n, kBN), st);
  }
}

// Whether every workgroup rounds x to integers by itself.
bool fuses(const Rows& r, int max_rows, int cols) {
  return !r.count && max_rows <= 16 && (int64_t)max_rows * cols * 2 <= kFuseBytes;
}

// Rows of bf16 by an 8-bit weight: rounded by the product itself, or before it into
// `codes` and `scales`, which `epi` reads.
template <class Epi>
int run_int8(Product p, const Epi& epi, int max_rows, const void* x, uint8_t* codes, float* scales,
             hipStream_t st) {
  p.a = (const uint8_t*)x;
  p.a_row = 2 * p.k;
  if (fuses(p.rows, max_rows, p.k)) return launch_few<Epi, true, 1, true>(p, epi, 1, st);
  const int rc = quantize_rows(p.rows, max_rows, x, p.k, codes, scales, st);
  if (rc != EP_OK) return rc;
  p.a = codes;
  p.a_row = p.k;
  return run_rows<Epi, true>(p, epi, max_rows, st);
}

template <class Epi>
int run_bf16(Product p, const Epi& epi, int max_rows, const void* x, hipStream_t st) {
  p.a = (const uint8_t*)x;
  p.a_row = p.k;
  return run_rows<Epi, false>(p, epi, max_rows, st);
}

// Tiles are counted in 32 bits, the smallest of them of 16 rows by 16 columns.  Regions that
// overlap (counts that nobody wrote, say) may be the whole buffer for every expert: then
// row tiles and wide tiles still fit, and few_kernel and small_kernel stop at the last that does.
bool few_enough(const Rows& r, int cols) {
  const int64_t most = (int64_t)r.E * r.cap;
  return row_tiles(r, r.cap, 16) * ceil_div(cols, 16) <= INT32_MAX &&
         most / 16 + r.E <= INT32_MAX && (most / kBM + r.E) * ceil_div(cols, 128) <= kLastTile;
}

// Offsets inside an expert's sub-blocks have 32 bits (see descriptor()).
bool fits_region(const Rows& r, int64_t row_bytes) {
  return !r.count || r.offset || (int64_t)r.R * r.M * row_bytes < kRange;
}

int64_t up(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

extern "C" {

int64_t ep_ffn_workspace_bytes(const ep_rows_t* rows, int32_t hidden, int32_t inter, int32_t format,
                               int32_t backward) {
  if (validate_rows(rows) != EP_OK || !valid_width(hidden, format) || !valid_width(inter, format))
    return -1;
  if (backward != 0 && (backward != 1 || format != EP_WEIGHT_BF16)) return -1;
  const int64_t cap = rows->capacity;
  if (format == EP_WEIGHT_INT8)
    return up(cap * hidden) + up(cap * 2 * inter) + up(cap * inter) + 2 * up(cap * 4);
  return up(cap * 2 * inter) + (backward ? up(cap * 4 * inter) : 0);
}

int ep_ffn(const ep_rows_t* rows, const ep_ffn_args_t* a, void* stream) {
  int rc = validate_rows(rows);
  if (rc != EP_OK) return rc;
  if (!a || a->w13.format != a->w2.format) return EP_ERR_INVALID_ARG;
  const int format = a->w13.format, H = a->hidden, I = a->inter;
  if (!valid_width(H, format) || !valid_width(I, format)) return EP_ERR_INVALID_ARG;
  if (rows->max_rows == 0) return EP_OK;
  const bool i8 = format == EP_WEIGHT_INT8;
  if (!a->x || !a->y || !a->workspace || !a->w13.data || !a->w2.data ||
      (i8 && (!a->w13.scales || !a->w2.scales)) || !aligned16(a->x) || !aligned16(a->y) ||
      !aligned16(a->gate_up) || !aligned16(a->w13.data) || !aligned16(a->w2.data) ||
      !aligned(a->workspace, 256))
    return EP_ERR_INVALID_ARG;
  const int bytes = i8 ? 1 : 2;
  const int64_t cap = rows->capacity;
  if (overlap(a->gate_up, cap * 4 * I, a->x, cap * 2 * H) ||
      overlap(a->gate_up, cap * 4 * I, a->y, cap * 2 * H) || !aligned(a->w13.scales, i8 ? 4 : 1) ||
      !aligned(a->w2.scales, i8 ? 4 : 1))
    return EP_ERR_INVALID_ARG;
  const Rows r = device_rows(rows);
  if (!fits_region(r, (int64_t)H * 2) || !fits_region(r, (int64_t)I * 2) ||
      !few_enough(r, std::max(H, 2 * I)))
    return EP_ERR_INVALID_ARG;
  rc = check_device();
  if (rc != EP_OK) return rc;
  hipStream_t st = (hipStream_t)stream;
  uint8_t* ws = (uint8_t*)a->workspace;
  uint8_t* h = ws;
  uint8_t* xq = h + up(cap * 2 * I);
  uint8_t* hq = xq + up(cap * H);
  float* sx = (float*)(hq + up(cap * I));
  float* sh = (float*)((uint8_t*)sx + up(cap * 4));
  EP_LOG("ffn experts=%d max_rows=%d H=%d I=%d int8=%d", r.E, rows->max_rows, H, I, (int)i8);
  Product p{};
  p.rows = r;
  p.b = (const uint8_t*)a->w13.data;
  p.k = p.b_row = H * bytes;
  p.b_expert = (int64_t)2 * I * p.k;
  p.n = I;
  p.far = I;
  const StoreGate gate{(uint16_t*)h, (uint16_t*)a->gate_up, I, sx, (const float*)a->w13.scales};
  rc = i8 ? run_int8(p, gate, rows->max_rows, a->x, xq, sx, st)
          : run_bf16(p, gate, rows->max_rows, a->x, st);
  if (rc != EP_OK) return rc;
  p.b = (const uint8_t*)a->w2.data;
  p.k = p.b_row = I * bytes;
  p.b_expert = (int64_t)H * p.k;
  p.n = H;
  p.far = 0;
  const StoreRows out{(uint16_t*)a->y, H, sh, (const float*)a->w2.scales};
  return i8 ? run_int8(p, out, rows->max_rows, h, hq, sh, st)
            : run_bf16(p, out, rows->max_rows, h, st);
}

int ep_ffn_backward(const ep_rows_t* rows, const ep_ffn_grad_args_t* a, void* stream) {
  int rc = validate_rows(rows);
  if (rc != EP_OK) return rc;
  if (!a || !valid_width(a->hidden, EP_WEIGHT_BF16) || !valid_width(a->inter, EP_WEIGHT_BF16))
    return EP_ERR_INVALID_ARG;
  const int H = a->hidden, I = a->inter;
  const Rows r = device_rows(rows);
  if (r.count && !r.offset) return EP_ERR_INVALID_ARG;   // low-latency sub-blocks
  const int64_t cap = rows->capacity, w13_bytes = (int64_t)r.E * 4 * I * H;
  const struct { const void* p; int64_t n; } in[] = {{a->dy, cap * 2 * H}, {a->x, cap * 2 * H},
      {a->gate_up, cap * 4 * I}, {a->w13, w13_bytes}, {a->w2, w13_bytes / 2}},
      out[] = {{a->dx, cap * 2 * H}, {a->dw13, w13_bytes}, {a->dw2, w13_bytes / 2}};
  for (const auto& o : out)
    for (const auto& i : in)
      if (overlap(o.p, o.n, i.p, i.n)) return EP_ERR_INVALID_ARG;
  if (!few_enough(r, std::max(H, 2 * I)) ||
      r.E * (ceil_div(2 * I, kST) + ceil_div(I, kST)) * ceil_div(H, kST) > kLastTile)
    return EP_ERR_INVALID_ARG;
  const bool any = rows->max_rows > 0;
  if (!a->w13 || !a->w2 || !a->dw13 || !a->dw2 || !aligned(a->workspace, 256) ||
      (any && (!a->x || !a->dy || !a->gate_up || !a->dx || !a->workspace)) || !aligned16(a->x) ||
      !aligned16(a->dy) || !aligned16(a->gate_up) || !aligned16(a->dx) || !aligned16(a->w13) ||
      !aligned16(a->w2) || !aligned16(a->dw13) || !aligned16(a->dw2))
    return EP_ERR_INVALID_ARG;
  rc = check_device();
  if (rc != EP_OK) return rc;
  hipStream_t st = (hipStream_t)stream;
  uint8_t* h = (uint8_t*)a->workspace;
  uint8_t* dgu = any ? h + up(cap * 2 * I) : nullptr;
  EP_LOG("ffn_backward experts=%d max_rows=%d H=%d I=%d", r.E, rows->max_rows, H, I);
  Product p{};
  p.rows = r;
  if (any) {
    p.a = (const uint8_t*)a->dy;
    p.b = (const uint8_t*)a->w2;
    p.k = 2 * H;
    p.a_row = 2 * H;
    p.b_row = 2 * I;
    p.b_expert = (int64_t)2 * H * I;
    p.n = I;
    const StoreGateGrad gg{(const uint16_t*)a->gate_up, (uint16_t*)dgu, (uint16_t*)h, I};
    rc = run_grad<kRows>(p, gg, rows->max_rows, st);
    if (rc != EP_OK) return rc;
    p.a = dgu;
    p.b = (const uint8_t*)a->w13;
    p.k = 4 * I;
    p.a_row = 4 * I;
    p.b_row = 2 * H;
    p.b_expert = (int64_t)4 * H * I;
    p.n = H;
    const StoreRows dx{(uint16_t*)a->dx, H, nullptr, nullptr};
    rc = run_grad<kRows>(p, dx, rows->max_rows, st);
    if (rc != EP_OK) return rc;
  }
  if (!any) p.rows = Rows{nullptr, nullptr, 0, r.E, 1, 0, 0};   // no rows: zeros
  p.a = dgu;
  p.b = (const uint8_t*)a->x;
  p.a_row = 4 * I;
  p.b_row = 2 * H;
  p.m = 2 * I;
  p.n = H;
  p.also = Outer{(const uint8_t*)a->dy, h, 2 * H, 2 * I, H, I};
  const StoreMatrix out_w{(uint16_t*)a->dw13, (uint16_t*)a->dw2, r.E, 2 * I, H, H, I};
  return run_grad<kOuter>(p, out_w, rows->max_rows, st);
}

int64_t ep_integer_workspace_bytes(const ep_rows_t* rows, int32_t cols) {
  if (validate_rows(rows) != EP_OK || !valid_width(cols, EP_WEIGHT_INT8)) return -1;
  return up(rows->capacity * cols) + up(rows->capacity * 4);
}

int ep_integer_linear(const ep_rows_t* rows, const ep_integer_args_t* a, void* stream) {
  int rc = validate_rows(rows);
  if (rc != EP_OK) return rc;
  if (!a || !valid_width(a->cols, EP_WEIGHT_INT8) || a->out_rows < 1 ||
      a->out_rows > EP_MAX_HIDDEN || a->w.format != EP_WEIGHT_INT8)
    return EP_ERR_INVALID_ARG;
  if (rows->max_rows == 0) return EP_OK;
  const int C = a->cols, O = a->out_rows;
  if (!a->x || !a->y || !a->w.data || !a->w.scales || !aligned16(a->x) || !aligned16(a->y) ||
      !aligned16(a->w.data) || !aligned(a->workspace, 256) || (!a->x_scales && !a->workspace) ||
      !aligned(a->w.scales, 4) || !aligned(a->x_scales, 4) ||
      overlap(a->y, rows->capacity * 2 * O, a->x, rows->capacity * C * (a->x_scales ? 1 : 2)))
    return EP_ERR_INVALID_ARG;
  const Rows r = device_rows(rows);
  if (!fits_region(r, C)) return EP_ERR_INVALID_ARG;
  if (!few_enough(r, O)) return EP_ERR_INVALID_ARG;
  rc = check_device();
  if (rc != EP_OK) return rc;
  hipStream_t st = (hipStream_t)stream;
  EP_LOG("integer_linear experts=%d max_rows=%d cols=%d out=%d", r.E, rows->max_rows, C, O);
  Product p{};
  p.rows = r;
  p.b = (const uint8_t*)a->w.data;
  p.k = p.b_row = C;
  p.b_expert = (int64_t)O * C;
  p.n = O;
  StoreRows out{(uint16_t*)a->y, O, a->x_scales, (const float*)a->w.scales};
  if (a->x_scales) {
    p.a = (const uint8_t*)a->x;
    p.a_row = C;
    return run_rows<StoreRows, true>(p, out, rows->max_rows, st);
  }
  uint8_t* codes = (uint8_t*)a->workspace;
  float* scales = (float*)(codes + up(rows->capacity * C));
  out.sx = scales;
  return run_int8(p, out, rows->max_rows, a->x, codes, scales, st);
}

}  // extern "C"
