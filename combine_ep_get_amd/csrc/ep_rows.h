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

  // Rows of expert e; counts and offsets are cut off where they leave the buffer.
  __device__ __forceinline__ int rows_of(int e) const {
    if (!count) return plain;
    if (offset) return max(0, min(count[e], cap - first_slot(e)));
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

// first[e] = row tiles of the experts before e, first[E] of all; by the whole workgroup.
[[maybe_unused]] __device__ __forceinline__ void scan_tiles(const Rows& rows, int tile,
                                                            int* first) {
  for (int e = threadIdx.x; e < rows.E; e += blockDim.x)
    first[e + 1] = (rows.rows_of(e) + tile - 1) / tile;
  if (threadIdx.x == 0) first[0] = 0;
  __syncthreads();
  if (threadIdx.x < 64) {
    const int per = (rows.E + 63) / 64, from = threadIdx.x * per,
              to = min(rows.E, from + per);
    int sum = 0;
    for (int e = from; e < to; e++) sum += first[e + 1];
    int before = sum;
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(before, d);
      if ((int)threadIdx.x >= d) before += v;
    }
    before -= sum;
    for (int e = from; e < to; e++) {
      before += first[e + 1];
      first[e + 1] = before;
    }
  }
  __syncthreads();
}

// The expert whose tiles hold tile i: first[e] <= i < first[e + 1].
[[maybe_unused]] __device__ __forceinline__ int find_expert(const int* first, int E, int i) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__builtin_amdgcn_readfirstlane(first[mid]) <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

[[maybe_unused]] bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }
[[maybe_unused]] bool aligned16(const void* p) { return aligned(p, 16); }

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
  if (((uintptr_t)r->offset | (uintptr_t)r->count) & 3) return EP_ERR_INVALID_ARG;
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
