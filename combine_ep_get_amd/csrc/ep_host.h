// ep_host.h -- host-side helpers that every source of libepget shares: logging,
// the architecture check, launch errors and the checks of a problem descriptor.
#ifndef EP_HOST_H
#define EP_HOST_H

#include <hip/hip_runtime.h>

#include <atomic>
#include <climits>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "ep_get.h"

namespace {

[[maybe_unused]] bool log_on() {
  static int v = -1;
  if (v < 0) {
    const char* e = getenv("EP_GET_LOG");
    v = (e && *e && *e != '0') ? 1 : 0;
  }
  return v == 1;
}

#define EP_LOG(...)                          \
  do {                                       \
    if (log_on()) {                          \
      fprintf(stderr, "[ep_get] " __VA_ARGS__); \
      fputc('\n', stderr);                   \
    }                                        \
  } while (0)

[[maybe_unused]] int check_device() {
  static std::atomic<int> cache[64];  // 0 unknown, 1 gfx950, 2 other
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return EP_ERR_HIP;
  int c = (dev >= 0 && dev < 64) ? cache[dev].load() : 0;
  if (c == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return EP_ERR_HIP;
    c = (strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    if (dev >= 0 && dev < 64) cache[dev].store(c);
  }
  return c == 1 ? EP_OK : EP_ERR_UNSUPPORTED;
}

[[maybe_unused]] int check_launch(const char* what) {
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) {
    EP_LOG("%s: %s", what, hipGetErrorString(e));
    return EP_ERR_HIP;
  }
  return EP_OK;
}

[[maybe_unused]] int64_t bound_of(const ep_problem_t* p) {
  return (int64_t)p->num_tokens * p->num_topk + (int64_t)p->num_experts * (p->expert_alignment - 1);
}

[[maybe_unused]] int validate_layout(const ep_problem_t* p) {
  if (!p) return EP_ERR_INVALID_ARG;
  const int N = p->num_tokens, K = p->num_topk, E = p->num_experts, R = p->num_ranks,
            A = p->expert_alignment;
  if (N < 0 || K < 1 || K > EP_MAX_TOPK || E < 1 || E > EP_MAX_EXPERTS || R < 1 ||
      R > EP_MAX_RANKS || R > E || A < 1)
    return EP_ERR_INVALID_ARG;
  if (E % R != 0 || N % R != 0) return EP_ERR_INVALID_ARG;
  if (p->topk_idx_bytes != 0 && p->topk_idx_bytes != 4 && p->topk_idx_bytes != 8)
    return EP_ERR_INVALID_ARG;
  if (p->cu_budget < 0) return EP_ERR_INVALID_ARG;
  if (bound_of(p) > INT32_MAX) return EP_ERR_INVALID_ARG;
  return EP_OK;
}

}  // namespace

#endif  // EP_HOST_H
