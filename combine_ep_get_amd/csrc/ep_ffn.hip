// ep_ffn.hip -- the experts' feed-forward block on dispatched rows, its gradient, and
// products in 8-bit integers (include/ep_get.h states the contracts).
#include "ep_host.h"
#include "ep_rows.h"

#include <type_traits>

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

#define EP_LDS __attribute__((address_space(3)))

constexpr int kRange = 0x60000000;     // bytes that a buffer descriptor spans
constexpr int kAbsent = 0x7F000000;    // an offset outside of it: the load returns zeros
constexpr int kBN = 256;               // columns of a tile
constexpr int kGroupM = 8;             // row tiles that are neighbours in the order of tiles

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// How the operands lie in memory (D = A B^T, contraction over k):
//   kRowsT  A [row][k], B [column][k]     activations by a weight's rows
//   kRows   A [row][k], B [k][column]     activations by a weight's columns
//   kOuter  A [k][row], B [k][column]     a weight's gradient: k runs over an expert's rows
enum { kRowsT, kRows, kOuter };

struct Product {            // kernel argument
  Rows rows;
  const uint8_t* a;
  const uint8_t* b;
  int64_t a_row, b_row;     // bytes per row of a and b
  int64_t b_expert;         // bytes per expert of b (kRowsT, kRows)
  int k;                    // contraction: bytes of a row of a (kRowsT, kRows)
  int m, n;                 // D's rows (kOuter) and columns
  int far;                  // > 0: column j of a tile's second half is b's row far + n0/2 + j
};

// 16 bytes per lane from global memory straight to LDS, lane l's at base + 16 l.  In asm,
// because the compiler would wait for all such loads before the next read of LDS; the
// waits are written out at the loop.  The s_nop covers a descriptor word or base that a
// VALU instruction has just written (five wait states), which the compiler cannot see
// here, and m0.
__device__ __forceinline__ void load_lds(uint32_t lds, int offset, i32x4 desc) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(offset), "s"(desc)
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

__device__ __forceinline__ u32x4 pack8(const float* v) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    bf16x2 p = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
    r[i] = __builtin_bit_cast(uint32_t, p);
  }
  return r;
}

__device__ __forceinline__ void unpack8(u32x4 r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    v[2 * i] = __builtin_bit_cast(float, r[i] << 16);
    v[2 * i + 1] = __builtin_bit_cast(float, r[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ float sigmoid(float g) { return 1.f / (1.f + __expf(-g)); }

// ---------------------------------------------------------------- epilogues
// What becomes of eight neighbouring columns of a row of D.  `slot` is the row's slot
// (kOuter: its row of the expert's matrix), `e` the expert, `c` the first column.
struct StoreRows {
  static constexpr bool gate = false;
  uint16_t* y;
  int n;
  const float *sx, *sw;    // 8-bit products: scales per slot and per expert and column
  template <class T>
  __device__ __forceinline__ void operator()(int e, int slot, int c, const T* v, const T*) const {
    if (c >= n) return;
    float f[8];
    const int left = n - c;
    if constexpr (std::is_same_v<T, int>) {
      const float s = sx[slot];
      const float* w = sw + (int64_t)e * n + c;
#pragma unroll
      for (int i = 0; i < 8; i++) f[i] = (float)v[i] * s * (i < left ? w[i] : 0.f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) f[i] = v[i];
    }
    const u32x4 r = pack8(f);
    uint16_t* to = y + (int64_t)slot * n + c;
    if ((n & 7) == 0) {
      *(u32x4*)to = r;
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++)
        if (i < left) to[i] = (uint16_t)(r[i >> 1] >> (16 * (i & 1)));
    }
  }
};

struct StoreMatrix {       // kOuter: [e][m][n]
  static constexpr bool gate = false;
  uint16_t* y;
  int m, n;
  __device__ __forceinline__ void operator()(int e, int row, int c, const float* v,
                                             const float*) const {
    if (c >= n) return;
    *(u32x4*)(y + ((int64_t)e * m + row) * n + c) = pack8(v);
  }
};

// silu(gate) * up; the tile's columns are `c` of gate and of up.
struct StoreGate {
  static constexpr bool gate = true;
  uint16_t* h;             // [slot][inter]
  uint16_t* gu;            // [slot][2 inter] or NULL
  int inter;
  const float *sx, *sw;
  template <class T>
  __device__ __forceinline__ void operator()(int e, int slot, int c, const T* g, const T* u) const {
    if (c >= inter) return;
    float a[8], b[8], r[8];
    if constexpr (std::is_same_v<T, int>) {
      const float s = sx[slot];
      const float* w = sw + (int64_t)e * 2 * inter + c;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        a[i] = (float)g[i] * s * w[i];
        b[i] = (float)u[i] * s * w[inter + i];
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
  const uint16_t* gu;      // [slot][2 inter]
  uint16_t* dgu;           // [slot][2 inter]
  uint16_t* h;             // [slot][inter]
  int inter;
  __device__ __forceinline__ void operator()(int, int slot, int c, const float* v,
                                             const float*) const {
    if (c >= inter) return;
    const int64_t at = (int64_t)slot * 2 * inter + c;
    float g[8], u[8], dg[8], du[8], hh[8];
    unpack8(*(const u32x4*)(gu + at), g);
    unpack8(*(const u32x4*)(gu + at + inter), u);
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

// One operand's half tile in LDS: R rows by 128 bytes of k (16-byte chunk c of row r at
// c ^ (r & 7)), or, where k is the slow axis, 64 k by 128 columns (256 bytes; chunk c of
// row k at c ^ 4 (k & 3)): no two lanes of a read share a bank.
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

template <int KIND, class Epi, bool I8, int BM>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
void product_kernel(Product p, Epi epi) {
  constexpr int kHalfA = BM / 2 * 128, kHalfB = 16384;     // bytes
  constexpr int kStage = 2 * kHalfA + 2 * kHalfB;
  constexpr int NA = BM / 128, NB = 2;                     // loads per wavefront and half
  constexpr int WM = BM / 4, MB = WM / 32;                 // a wavefront's rows of a half
  constexpr bool kSlowA = KIND == kOuter, kSlowB = KIND != kRowsT;
  static_assert(KIND != kOuter || BM == 256, "k-major tiles of 128 rows only");
  using acc_t = typename Acc<I8>::type;
  using val_t = typename Acc<I8>::scalar;

  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage];
  __shared__ int first_tile[EP_MAX_EXPERTS + 1];
  __shared__ int slot_of_row[BM];

  const int tid = threadIdx.x, l = tid & 63, w = uniform(tid >> 6);
  const int wm = w >> 2, wn = w & 3;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(EP_LDS uint8_t*)lds;
  const int NT = KIND == kRowsT && p.far ? (p.n + 127) / 128 : (p.n + kBN - 1) / kBN;
  const int MT = (p.m + BM - 1) / BM;                      // kOuter
  int total;
  if constexpr (KIND == kOuter) {
    total = p.rows.E * MT * NT;
  } else {
    scan_tiles(p.rows, BM, first_tile);
    total = uniform(first_tile[p.rows.E]) * NT;
  }

  // where this lane's bytes of a load go, and where it reads
  const int chunk_k = (l & 7) ^ (l >> 3);                  // of 128 bytes of a row
  const int chunk_n = (l & 15) ^ ((l >> 4) << 2);          // of 128 columns of a k
  const int read_k = (l & 31) * 128 + ((((l >> 5) ^ (l & 7))) << 4);
  const int i16 = l & 15;
  auto read_n = [&](int chunk) {
    return ((l >> 5) * 8 + (i16 >> 2)) * 256 +
           (((chunk + ((l >> 4) & 1) * 2 + ((i16 & 3) >> 1)) ^ ((i16 >> 2) << 2)) << 4) +
           (i16 & 1) * 8;
  };
  int read_a[MB];
#pragma unroll
  for (int mb = 0; mb < MB; mb++)
    read_a[mb] = kSlowA ? read_n(wm * 8 + mb * 4) : (wm * WM + mb * 32) * 128 + read_k;
  const int read_b = kSlowB ? read_n(wn * 4) : wn * 32 * 128 + read_k;

  // workgroup ids go round robin over the 8 XCDs: give each XCD neighbouring tiles
  const int G = gridDim.x;
  const int me = G % 8 == 0 ? (blockIdx.x % 8) * (G / 8) + blockIdx.x / 8 : blockIdx.x;
  for (int tile = me; tile < total; tile += G) {
    // ---- which tile
    int e = 0, mt, nt, nrows, KT;
    int row0, slot0 = 0;
    const uint8_t *a0, *b0;
    if constexpr (KIND == kOuter) {
      e = tile / (MT * NT);
      const int r = tile - e * MT * NT;
      const int g = r / (kGroupM * NT), f = g * kGroupM, gs = min(kGroupM, MT - f);
      const int q = r - g * kGroupM * NT;
      mt = f + q % gs;
      nt = q / gs;
      row0 = mt * BM;
      nrows = min(BM, p.m - row0);
      const int cnt = uniform(p.rows.rows_of(e));
      KT = (cnt + 63) / 64;
      slot0 = uniform(p.rows.first_slot(e));
      a0 = p.a + (int64_t)slot0 * p.a_row + (int64_t)row0 * 2;
      b0 = p.b + (int64_t)slot0 * p.b_row + (int64_t)nt * kBN * 2;
      p.k = cnt;
    } else {
      e = find_expert(first_tile, p.rows.E, tile / NT);
      const int f0 = uniform(first_tile[e]), mts = uniform(first_tile[e + 1]) - f0;
      const int r = tile - f0 * NT;
      const int g = r / (kGroupM * NT), f = g * kGroupM, gs = min(kGroupM, mts - f);
      const int q = r - g * kGroupM * NT;
      mt = f + q % gs;
      nt = q / gs;
      row0 = mt * BM;
      nrows = min(BM, uniform(p.rows.rows_of(e)) - row0);
      if (tid < BM) slot_of_row[tid] = tid < nrows ? p.rows.slot(e, row0 + tid) : -1;
      slot0 = uniform(p.rows.base_slot(e, row0));
      a0 = p.a + (int64_t)slot0 * p.a_row;
      b0 = p.b + (int64_t)e * p.b_expert;
      if constexpr (KIND == kRowsT)
        b0 += (int64_t)nt * (p.far ? 128 : kBN) * p.b_row;
      else
        b0 += (int64_t)nt * kBN * 2;
      KT = (p.k + 127) / 128;
      __syncthreads();
    }

    // ---- offsets of this lane's loads from a0 and b0
    int off_a[2][NA], off_b[2][NB];
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
      for (int j = 0; j < NA; j++) {
        if constexpr (kSlowA) {
          const int c = h * 128 + chunk_n * 8;
          off_a[h][j] = c < nrows ? ((w * NA + j) * 4 + (l >> 4)) * (int)p.a_row + c * 2 : kAbsent;
        } else {
          const int s = slot_of_row[h * (BM / 2) + (w * NA + j) * 8 + (l >> 3)];
          off_a[h][j] = s >= 0 ? (int)((s - slot0) * p.a_row) + chunk_k * 16 : kAbsent;
        }
      }
#pragma unroll
      for (int j = 0; j < NB; j++) {
        if constexpr (kSlowB) {
          const int c = h * 128 + chunk_n * 8;
          off_b[h][j] = nt * kBN + c < p.n
                            ? ((w * NB + j) * 4 + (l >> 4)) * (int)p.b_row + c * 2 : kAbsent;
        } else {
          const int c = (w * NB + j) * 8 + (l >> 3);
          if (p.far)
            off_b[h][j] = nt * 128 + c < p.n ? (int)(c * p.b_row) + chunk_k * 16 : kAbsent;
          else
            off_b[h][j] = nt * kBN + h * 128 + c < p.n
                              ? (int)((c + h * 128) * p.b_row) + chunk_k * 16 : kAbsent;
        }
      }
    }

    const int64_t far = (int64_t)p.far * p.b_row;
    const int64_t step_a = kSlowA ? 64 * p.a_row : 128, step_b = kSlowB ? 64 * p.b_row : 128;
    auto load_a = [&](int t, int h) {
      const i32x4 d = descriptor(a0 + t * step_a);
      const uint32_t to = lds0 + (t & 1) * kStage + h * kHalfA + w * NA * 1024;
#pragma unroll
      for (int j = 0; j < NA; j++) {
        const bool in = kSlowA ? (w * NA + j) * 4 + (l >> 4) < p.k - t * 64
                               : chunk_k * 16 < p.k - t * 128;
        load_lds(to + j * 1024, in ? off_a[h][j] : kAbsent, d);
      }
    };
    // k of b's rows: p.k counts bytes of a's rows where those hold k
    const int k_b = KIND == kRows ? p.k / 2 : p.k;
    auto load_b = [&](int t, int h) {
      const i32x4 d = descriptor(b0 + t * step_b + h * far);
      const uint32_t to = lds0 + (t & 1) * kStage + 2 * kHalfA + h * kHalfB + w * NB * 1024;
#pragma unroll
      for (int j = 0; j < NB; j++) {
        const bool in = kSlowB ? (w * NB + j) * 4 + (l >> 4) < k_b - t * 64
                               : chunk_k * 16 < k_b - t * 128;
        load_lds(to + j * 1024, in ? off_b[h][j] : kAbsent, d);
      }
    };

    // ---- the loop.  Two groups of four wavefronts, one of each group on every SIMD,
    // half a phase apart: while one group's MFMAs run, the other reads its next
    // fragments and sends loads.  A half tile is loaded again as soon as both groups
    // have read it: its reads have returned (wait_lds) before the barrier behind which
    // the load is sent.
    acc_t acc[2][2][MB];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int j = 0; j < 2; j++)
#pragma unroll
        for (int k = 0; k < MB; k++) acc[i][j][k] = acc_t{};

    if (KT > 0) {
      load_b(0, 0);
      load_a(0, 0);
      load_b(0, 1);
      load_a(0, 1);
      load_b(1, 0);
      load_a(1, 0);
      load_b(1, 1);
      wait_loads<2 * NB + NA>();
      barrier();
      if (wm == 1) barrier();
      for (int t = 0; t < KT; t++) {
        const uint8_t* st = lds + (t & 1) * kStage;
        u32x4 fa[MB][4], fb[2][4];
        auto read_as = [&](int h) {
#pragma unroll
          for (int mb = 0; mb < MB; mb++)
#pragma unroll
            for (int ks = 0; ks < 4; ks++)
              fa[mb][ks] = fragment<kSlowA>(st + h * kHalfA, read_a[mb], ks);
        };
        auto read_bs = [&](int h) {
#pragma unroll
          for (int ks = 0; ks < 4; ks++)
            fb[h][ks] = fragment<kSlowB>(st + 2 * kHalfA + h * kHalfB, read_b, ks);
        };
        auto multiply = [&](int qm, int qn) {
          wait_lds();
          barrier();
          __builtin_amdgcn_s_setprio(1);
#pragma unroll
          for (int ks = 0; ks < 4; ks++)
#pragma unroll
            for (int mb = 0; mb < MB; mb++)
              acc[qm][qn][mb] = mfma<I8>(fb[qn][ks], fa[mb][ks], acc[qm][qn][mb]);
          __builtin_amdgcn_s_setprio(0);
          barrier();
        };
        read_bs(0);
        read_as(0);
        load_a(t + 1, 1);
        multiply(0, 0);
        read_bs(1);
        load_b(t + 2, 0);
        multiply(0, 1);
        read_as(1);
        load_a(t + 2, 0);
        multiply(1, 1);
        load_b(t + 2, 1);
        wait_loads<2 * NB + NA>();
        multiply(1, 0);
      }
      if (wm == 0) barrier();
      wait_loads<0>();
    }

    // ---- epilogue: through LDS, so that a lane has eight neighbouring columns
#pragma unroll
    for (int h = 0; h < 2; h++) {
      __syncthreads();
#pragma unroll
      for (int mb = 0; mb < MB; mb++) {
        const int row = wm * WM + mb * 32 + (l & 31);
#pragma unroll
        for (int qn = 0; qn < 2; qn++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int c = qn * 32 + wn * 8 + 2 * i + (l >> 5);
            u32x4 v;
#pragma unroll
            for (int j = 0; j < 4; j++)
              v[j] = __builtin_bit_cast(uint32_t, (val_t)acc[h][qn][mb][i * 4 + j]);
            *(u32x4*)(lds + row * 1024 + ((c ^ (l & 31)) << 4)) = v;
          }
      }
      __syncthreads();
      constexpr int kChunks = Epi::gate ? 16 : 32;
#pragma unroll 2
      for (int i = tid; i < BM / 2 * kChunks; i += 512) {
        const int r = i / kChunks, c = i % kChunks, x = r & 31;
        if (h * (BM / 2) + r >= nrows) break;
        val_t v[8], u[8];
        auto take = [&](int chunk, val_t* to) {
#pragma unroll
          for (int q = 0; q < 2; q++) {
            const u32x4 t = *(const u32x4*)(lds + r * 1024 + (((chunk + q) ^ x) << 4));
#pragma unroll
            for (int j = 0; j < 4; j++) to[q * 4 + j] = __builtin_bit_cast(val_t, (uint32_t)t[j]);
          }
        };
        take(2 * c, v);
        if constexpr (Epi::gate) take(32 + 2 * c, u);
        const int row = KIND == kOuter ? row0 + h * (BM / 2) + r : slot_of_row[h * (BM / 2) + r];
        epi(e, row, nt * (Epi::gate ? 128 : kBN) + c * 8, v, u);
      }
    }
    __syncthreads();
  }
}

template <int KIND, class Epi, bool I8, int BM>
void launch(const Product& p, const Epi& epi, int64_t tiles, hipStream_t st) {
  // one workgroup per CU at most: each takes more than half of a CU's LDS
  const int grid = (int)(tiles < 256 ? tiles : 256);
  product_kernel<KIND, Epi, I8, BM><<<dim3(grid), dim3(512), 0, st>>>(p, epi);
}

// Rows of D: row tiles are counted on the device; here only their upper bound.
template <int KIND, class Epi, bool I8>
int run_rows(const Product& p, const Epi& epi, int max_rows, int64_t tiles_n, hipStream_t st) {
  const int E = p.rows.E;
  const bool small = max_rows / E <= 160;
  const int bm = small ? 128 : 256;
  const int64_t tiles = ((int64_t)max_rows / bm + E) * tiles_n;
  if (small) launch<KIND, Epi, I8, 128>(p, epi, tiles, st);
  else launch<KIND, Epi, I8, 256>(p, epi, tiles, st);
  return check_launch("ep_ffn product");
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
  const Rows r = device_rows(rows);
  if (!fits_region(r, (int64_t)H * 2) || !fits_region(r, (int64_t)I * 2)) return EP_ERR_INVALID_ARG;
  rc = check_device();
  if (rc != EP_OK) return rc;
  hipStream_t st = (hipStream_t)stream;
  const int64_t cap = rows->capacity;
  uint8_t* ws = (uint8_t*)a->workspace;
  uint8_t* h = ws;
  uint8_t* xq = h + up(cap * 2 * I);
  uint8_t* hq = xq + up(cap * H);
  float* sx = (float*)(hq + up(cap * I));
  float* sh = (float*)((uint8_t*)sx + up(cap * 4));
  EP_LOG("ffn experts=%d max_rows=%d H=%d I=%d int8=%d", r.E, rows->max_rows, H, I, (int)i8);
  if (i8) {
    rc = quantize_rows(r, rows->max_rows, a->x, H, xq, sx, st);
    if (rc != EP_OK) return rc;
  }
  Product p{};
  p.rows = r;
  p.a = i8 ? xq : (const uint8_t*)a->x;
  p.b = (const uint8_t*)a->w13.data;
  p.k = H * bytes;
  p.a_row = p.b_row = p.k;
  p.b_expert = (int64_t)2 * I * p.k;
  p.n = I;
  p.far = I;
  const StoreGate gate{(uint16_t*)h, (uint16_t*)a->gate_up, I, sx, (const float*)a->w13.scales};
  rc = i8 ? run_rows<kRowsT, StoreGate, true>(p, gate, rows->max_rows, (I + 127) / 128, st)
          : run_rows<kRowsT, StoreGate, false>(p, gate, rows->max_rows, (I + 127) / 128, st);
  if (rc != EP_OK) return rc;
  if (i8) {
    rc = quantize_rows(r, rows->max_rows, h, I, hq, sh, st);
    if (rc != EP_OK) return rc;
  }
  p.a = i8 ? hq : h;
  p.b = (const uint8_t*)a->w2.data;
  p.k = I * bytes;
  p.a_row = p.b_row = p.k;
  p.b_expert = (int64_t)H * p.k;
  p.n = H;
  p.far = 0;
  const StoreRows out{(uint16_t*)a->y, H, sh, (const float*)a->w2.scales};
  return i8 ? run_rows<kRowsT, StoreRows, true>(p, out, rows->max_rows, (H + kBN - 1) / kBN, st)
            : run_rows<kRowsT, StoreRows, false>(p, out, rows->max_rows, (H + kBN - 1) / kBN, st);
}

int ep_ffn_backward(const ep_rows_t* rows, const ep_ffn_grad_args_t* a, void* stream) {
  int rc = validate_rows(rows);
  if (rc != EP_OK) return rc;
  if (!a || !valid_width(a->hidden, EP_WEIGHT_BF16) || !valid_width(a->inter, EP_WEIGHT_BF16))
    return EP_ERR_INVALID_ARG;
  const int H = a->hidden, I = a->inter;
  const Rows r = device_rows(rows);
  if (r.count && !r.offset) return EP_ERR_INVALID_ARG;   // low-latency sub-blocks
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
  uint8_t* dgu = h + up(rows->capacity * 2 * I);
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
    rc = run_rows<kRows, StoreGateGrad, false>(p, gg, rows->max_rows, (I + kBN - 1) / kBN, st);
    if (rc != EP_OK) return rc;
    p.a = dgu;
    p.b = (const uint8_t*)a->w13;
    p.k = 4 * I;
    p.a_row = 4 * I;
    p.b_row = 2 * H;
    p.b_expert = (int64_t)4 * H * I;
    p.n = H;
    const StoreRows dx{(uint16_t*)a->dx, H, nullptr, nullptr};
    rc = run_rows<kRows, StoreRows, false>(p, dx, rows->max_rows, (H + kBN - 1) / kBN, st);
    if (rc != EP_OK) return rc;
  }
  if (!any) p.rows = Rows{nullptr, nullptr, 0, r.E, 1, 0, 0};   // no rows: zeros
  p.a = dgu;
  p.b = (const uint8_t*)a->x;
  p.a_row = 4 * I;
  p.b_row = 2 * H;
  p.m = 2 * I;
  p.n = H;
  const StoreMatrix w13{(uint16_t*)a->dw13, 2 * I, H};
  launch<kOuter, StoreMatrix, false, 256>(
      p, w13, (int64_t)r.E * ((2 * I + 255) / 256) * ((H + 255) / 256), st);
  rc = check_launch("ep_ffn_backward dw13");
  if (rc != EP_OK) return rc;
  p.a = (const uint8_t*)a->dy;
  p.b = h;
  p.a_row = 2 * H;
  p.b_row = 2 * I;
  p.m = H;
  p.n = I;
  const StoreMatrix w2{(uint16_t*)a->dw2, H, I};
  launch<kOuter, StoreMatrix, false, 256>(
      p, w2, (int64_t)r.E * ((H + 255) / 256) * ((I + 255) / 256), st);
  return check_launch("ep_ffn_backward dw2");
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
      !aligned16(a->w.data) || !aligned(a->workspace, 256) || (!a->x_scales && !a->workspace))
    return EP_ERR_INVALID_ARG;
  const Rows r = device_rows(rows);
  if (!fits_region(r, C)) return EP_ERR_INVALID_ARG;
  const int64_t tiles_n = (O + kBN - 1) / kBN;
  if (((int64_t)rows->max_rows / 128 + r.E) * tiles_n > INT32_MAX) return EP_ERR_INVALID_ARG;
  rc = check_device();
  if (rc != EP_OK) return rc;
  hipStream_t st = (hipStream_t)stream;
  const uint8_t* xq = (const uint8_t*)a->x;
  const float* sx = a->x_scales;
  if (!sx) {
    uint8_t* q = (uint8_t*)a->workspace;
    float* s = (float*)(q + up(rows->capacity * C));
    rc = quantize_rows(r, rows->max_rows, a->x, C, q, s, st);
    if (rc != EP_OK) return rc;
    xq = q;
    sx = s;
  }
  EP_LOG("int8_linear experts=%d max_rows=%d cols=%d out=%d", r.E, rows->max_rows, C, O);
  Product p{};
  p.rows = r;
  p.a = xq;
  p.b = (const uint8_t*)a->w.data;
  p.k = C;
  p.a_row = p.b_row = C;
  p.b_expert = (int64_t)O * C;
  p.n = O;
  const StoreRows out{(uint16_t*)a->y, O, sx, (const float*)a->w.scales};
  return run_rows<kRowsT, StoreRows, true>(p, out, rows->max_rows, tiles_n, st);
}

}  // extern "C"
