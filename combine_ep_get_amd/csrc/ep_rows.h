// ep_rows.h -- the rows of each expert in a buffer (ep_rows_t): checks on the host, where
// they lie on the device, and what the sources that work on them share.
#ifndef EP_ROWS_H
#define EP_ROWS_H

#include "ep_host.h"

namespace ep {

struct Rows {            // kernel argument
  const int* offset;
  const int* count;
  int cap;
  int E, R, M;           // R sub-blocks of M rows per expert where there are no offsets
  int plain;             // rows of the one expert where there are no counts either

  // Rows of expert e: its region's, cut off at the ends of the buffer.  Of one that starts
  // before the buffer the first rows are lost, not the last.
  __device__ __forceinline__ int rows_of(int e) const {
    if (!count) return plain;
    if (offset) {
      const int64_t end = min((int64_t)offset[e] + count[e], (int64_t)cap);
      return (int)max((int64_t)0, end - first_slot(e));
    }
    int n = 0;
    for (int s = 0; s < R; s++) n += max(0, min(count[e * R + s], M));
    return n;
  }
  __device__ __forceinline__ int first_slot(int e) const {
    return offset ? max(0, min(offset[e], cap)) : 0;
  }
  // Slot of row r of expert e (r < rows_of(e)).
  __device__ __forceinline__ int slot(int e, int r) const {
    if (!count || offset) return first_slot(e) + r;
    for (int s = 0; s < R; s++) {
      const int n = max(0, min(count[e * R + s], M));
      if (r < n) return (e * R + s) * M + r;
      r -= n;
    }
    return e * R * M;      // not reached
  }
  // A slot at most as far before those of the rows r, r + 1, ... as 32 bits of bytes
  // reach (checked on the host).
  __device__ __forceinline__ int base_slot(int e, int r) const {
    return count && !offset ? e * R * M : first_slot(e) + r;
  }
};

// A row quantiser for other sources (ep_quantize_rows on the rows of Rows).
__attribute__((visibility("hidden"))) int quantize_rows(const Rows& rows, int max_rows,
                                                        const void* x, int cols, void* codes,
                                                        float* scales, hipStream_t st);

}  // namespace ep

namespace {

using ep::Rows;
using ep::quantize_rows;

// v[e + 1] for e < n: the sum of v[1] .. v[e + 1], by one wavefront.
template <class T>
__device__ __forceinline__ void scan(T* v, int n) {
  const int l = threadIdx.x & 63, per = (n + 63) / 64, from = l * per, to = min(n, from + per);
  int sum = 0;
  for (int e = from; e < to; e++) sum += v[e + 1];
  int before = sum;
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(before, d);
    if (l >= d) before += o;
  }
  before -= sum;
  for (int e = from; e < to; e++) {
    before += v[e + 1];
    v[e + 1] = (T)before;
  }
}

// The expert whose row tiles hold tile i, by every wavefront for itself.  One round of loads
// for up to 64 experts and no barrier: a table in LDS, and a search in it, made small
// calls about 3 us longer.
struct Found {
  int e, first, tiles;       // the expert, the row tiles before its own, its own
  int count, slot;           // its rows, the slot of its first
};
[[maybe_unused]] __device__ __forceinline__ bool find_rows(const Rows& rows, int tile, int i,
                                                           Found& f) {
  const int l = threadIdx.x & 63;
  int before = 0;
  for (int base = 0; base < rows.E; base += 64) {
    const int e = base + l;
    const int n = e < rows.E ? rows.rows_of(e) : 0;
    const int slot = e < rows.E ? rows.base_slot(e, 0) : 0;
    const int tiles = n / tile + (n % tile != 0);          // n may be all that an int holds
    int sum = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(sum, d);
      if (l >= d) sum += o;
    }
    const uint64_t beyond = __ballot(before + sum > i);
    if (beyond != 0) {
      const int at = __builtin_ctzll(beyond);
      f.e = base + at;
      f.tiles = __builtin_amdgcn_readlane(tiles, at);
      f.first = before + __builtin_amdgcn_readlane(sum, at) - f.tiles;
      f.count = __builtin_amdgcn_readlane(n, at);
      f.slot = __builtin_amdgcn_readlane(slot, at);
      return true;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  return false;
}

// What a workgroup that walks over many tiles keeps of the experts: their rows and first
// slots, and the row tiles before each, where a last tile of at most half the rows is
// counted apart.
struct Experts {
  int count[EP_MAX_EXPERTS], slot[EP_MAX_EXPERTS], first[EP_MAX_EXPERTS + 1];
  uint16_t first_short[EP_MAX_EXPERTS + 2];
  __device__ __forceinline__ void fill(const Rows& rows, int tile) {
    for (int e = threadIdx.x; e < rows.E; e += blockDim.x) {
      const int n = rows.rows_of(e), last = n % tile;
      const bool half = last > 0 && 2 * last <= tile;
      count[e] = n;
      slot[e] = rows.base_slot(e, 0);
      first[e + 1] = n / tile + (last > 0 && !half);
      first_short[e + 1] = half;
    }
    if (threadIdx.x == 0) first[0] = first_short[0] = 0;
    __syncthreads();
    if (threadIdx.x < 64) scan(first, rows.E);
    else if (threadIdx.x < 128) scan(first_short, rows.E);
    __syncthreads();
  }
};

// The expert whose tiles hold tile i: first[e] <= i < first[e + 1].
template <class T>
__device__ __forceinline__ int find_expert(const T* first, int E, int i) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__builtin_amdgcn_readfirstlane((int)first[mid]) <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

[[maybe_unused]] __device__ __forceinline__ void unpack8(u32x4 r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    v[2 * i] = __builtin_bit_cast(float, r[i] << 16);
    v[2 * i + 1] = __builtin_bit_cast(float, r[i] & 0xFFFF0000u);
  }
}

[[maybe_unused]] __device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}
[[maybe_unused]] __device__ __forceinline__ u32x4 pack8(const float* v) {
  return u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
}

// ---------------------------------------------------------------- rows as 8-bit integers
// The largest magnitude of eight bf16 values as bits: they are ordered as the values are,
// infinities and NaN last.
[[maybe_unused]] __device__ __forceinline__ uint32_t largest8(u32x4 r) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) top = max(top, max(r[i] & 0x7FFFu, (r[i] >> 16) & 0x7FFFu));
  return top;
}
[[maybe_unused]] __device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  return v;
}

// A row's scale, from its largest magnitude, and its codes.  fma(x, 1 / s, 1.5 2^23) leaves
// the nearest integer q of x * (1 / s) in its lowest bits.  That is off from x / s by less
// than 2^-16, so only where it is this near to a half may the exact quotient round
// otherwise: there the remainder x - q s decides, which is exact (q has 7 bits, s 24, x
// 8, and they cancel), halves to even.  Rows below 2^-100 are taken 2^64 times as large
// (exact), since 1 / s would overflow.
struct RowScale {
  float scale, s, inv, up;
  bool finite, tiny;
  static __device__ __forceinline__ RowScale of(uint32_t top) {
    RowScale r;
    const float amax = __builtin_bit_cast(float, top << 16);
    r.finite = top < 0x7F80u;
    r.tiny = amax < 0x1p-100f && top != 0;
    r.up = r.tiny ? 0x1p64f : 1.f;
    r.scale = top == 0 ? 1.f : amax / 127.f;
    r.s = r.scale * r.up;
    r.inv = 1.f / r.s;
    if (!r.finite) r.scale = __builtin_bit_cast(float, 0x7FC00000u);
    return r;
  }
  __device__ __forceinline__ u32x2 codes8(u32x4 raw) const {
    constexpr float kMagic = 12582912.f;
    float v[8], t[8], near = 0.f;
    unpack8(raw, v);
    if (tiny) {
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] *= up;
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
      t[i] = fmaf(v[i], inv, kMagic);
      near = fmaxf(near, fabsf(fmaf(v[i], inv, kMagic - t[i])));
    }
    if (near > 0.5f - 0x1p-14f) {
      const float half = 0.5f * s;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        float q = t[i] - kMagic;
        const float r = fmaf(-q, s, v[i]);
        const bool odd = ((int)q & 1) != 0;
        if (r > half || (r == half && odd)) q += 1.f;
        if (-r > half || (-r == half && odd)) q -= 1.f;
        t[i] = q + kMagic;
      }
    }
    if (!finite) return u32x2{0, 0};
    u32x2 out;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const uint32_t b0 = __builtin_bit_cast(uint32_t, t[4 * h]),
                     b1 = __builtin_bit_cast(uint32_t, t[4 * h + 1]),
                     b2 = __builtin_bit_cast(uint32_t, t[4 * h + 2]),
                     b3 = __builtin_bit_cast(uint32_t, t[4 * h + 3]);
      out[h] = (b0 & 0xFFu) | (b1 & 0xFFu) << 8 | (b2 & 0xFFu) << 16 | b3 << 24;
    }
    return out;
  }
};

[[maybe_unused]] bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }
[[maybe_unused]] bool aligned16(const void* p) { return aligned(p, 16); }

// Whether n bytes at p and m bytes at q share any (NULL: none).
[[maybe_unused]] bool overlap(const void* p, int64_t n, const void* q, int64_t m) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return p && q && n > 0 && m > 0 && a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

[[maybe_unused]] int validate_rows(const ep_rows_t* r) {
  if (!r || r->capacity < 0 || r->capacity > INT32_MAX || r->max_rows < 0 || r->num_experts < 1 ||
      r->num_experts > EP_MAX_EXPERTS || r->num_sources < 1 || r->num_sources > EP_MAX_RANKS)
    return EP_ERR_INVALID_ARG;
  if (r->offset && !r->count) return EP_ERR_INVALID_ARG;
  if (r->offset || !r->count) {
    if (r->num_sources != 1 || r->rows_per_source != 0) return EP_ERR_INVALID_ARG;
  } else if (r->rows_per_source < 1 ||
             (int64_t)r->num_experts * r->num_sources * r->rows_per_source > r->capacity) {
    return EP_ERR_INVALID_ARG;
  }
  if (!r->count && (r->num_experts != 1 || r->max_rows > r->capacity)) return EP_ERR_INVALID_ARG;
  if (!aligned(r->offset, 4) || !aligned(r->count, 4)) return EP_ERR_INVALID_ARG;
  return EP_OK;
}

[[maybe_unused]] Rows device_rows(const ep_rows_t* r) {
  return Rows{r->offset, r->count,           (int)r->capacity,
              r->num_experts, r->num_sources, r->rows_per_source, r->max_rows};
}

// A row width (hidden, inter, cols): whole 16-byte chunks, and within limits.
[[maybe_unused]] bool valid_width(int cols, int format) {
  if (format != EP_WEIGHT_BF16 && format != EP_WEIGHT_INT8) return false;
  return cols >= 1 && cols <= EP_MAX_CONTRACTION &&
         cols % (format == EP_WEIGHT_INT8 ? 16 : 8) == 0;
}

}  // namespace

#endif  // EP_ROWS_H
