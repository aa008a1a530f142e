/*
 * Drives the host side of the entry points for the experts' block, its gradient,
 * combine's gradient and the 8-bit products with random and extreme descriptors, in a
 * build with host-only -fsanitize=address,undefined.  Run where no device is visible:
 * what validation accepts ends at the device check.  Test infrastructure only.
 */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "ep_get.h"

static uint64_t st = 0xD1B54A32D192ED03ull;
static uint32_t rnd(void) {
  st ^= st >> 12; st ^= st << 25; st ^= st >> 27;
  return (uint32_t)((st * 0x2545F4914F6CDD1Dull) >> 32);
}
static int32_t pick(void) {
  static const int32_t v[] = {-2147483647 - 1, -1, 0, 1, 2, 8, 16, 64, 128, 256, 344, 1024, 1025,
                              2048, 7168, 65536, 65552, 1 << 24, 2147483647};
  if (rnd() % 4) return v[rnd() % (sizeof v / sizeof v[0])];
  return (int32_t)(rnd() % 4096) * 16;
}
static int32_t width(void) { return rnd() % 8 ? 16 * (int32_t)(1 + rnd() % 512) : pick(); }
/* mostly regions far apart, sometimes close, misaligned or none */
static void* pointer(int i) {
  const uintptr_t at = ((uintptr_t)(i + 1) << 44) + (rnd() % 16 ? 0 : (rnd() % 64) * 4);
  return rnd() % 40 ? (void*)at : rnd() % 2 ? NULL : (void*)((uintptr_t)1 << 44);
}
static ep_weight_t weight(int i) {
  static const int32_t f[] = {EP_WEIGHT_BF16, EP_WEIGHT_INT8, EP_WEIGHT_BF16, EP_WEIGHT_INT8,
                              EP_WEIGHT_INT4, 7};
  ep_weight_t w = {pointer(i), pointer(i + 1), NULL, f[rnd() % (rnd() % 4 ? 2 : 6)], 0};
  return w;
}
#define FAIL(...) do { fprintf(stderr, __VA_ARGS__); fputc('\n', stderr); exit(1); } while (0)

int main(void) {
  int valid = 0;
  for (int i = 0; i < 300000; i++) {
    const int kind = rnd() % 3;
    ep_rows_t r = {kind == 0 ? pointer(0) : NULL, kind < 2 ? pointer(1) : NULL,
                   rnd() % 4 ? 1 + (int64_t)(rnd() % (1u << 30)) : pick(),
                   kind == 2 ? 1 : pick() % 1200, kind == 1 ? 1 + (int32_t)(rnd() % 8) : 1,
                   kind == 1 ? 1 + (int32_t)(rnd() % 512) : 0,
                   rnd() % 2 ? (int32_t)(rnd() % 70000) : pick()};
    if (rnd() % 16 == 0) r.num_sources = pick();
    if (rnd() % 16 == 0) r.rows_per_source = pick();
    const int32_t H = width(), I = width();
    const int format = rnd() % 2 ? EP_WEIGHT_INT8 : EP_WEIGHT_BF16, back = (int)(rnd() % 3);
    const int64_t ws = ep_ffn_workspace_bytes(&r, H, I, format, back);
    if (ws >= 0 && (ws % 256 || (double)ws < (double)r.capacity * 2 * I)) FAIL("workspace of %lld", (long long)ws);
    ep_ffn_args_t f = {pointer(2), weight(3), weight(5), pointer(7), rnd() % 2 ? pointer(8) : NULL,
                       pointer(9), H, I};
    const int rf = ep_ffn(&r, &f, NULL);
    if (rf == EP_OK && r.max_rows > 0) FAIL("a block without a device");
    ep_ffn_grad_args_t g = {pointer(2), pointer(3), pointer(4), pointer(5), pointer(6), pointer(7),
                            pointer(8), pointer(9), pointer(10), H, I};
    const int rg = ep_ffn_backward(&r, &g, NULL);
    if (rg == EP_OK) FAIL("a gradient without a device");
    ep_integer_args_t q = {pointer(2), rnd() % 2 ? pointer(3) : NULL, weight(4), pointer(6),
                           pointer(7), H, rnd() % 2 ? I : pick()};
    const int rq = ep_integer_linear(&r, &q, NULL);
    if (rq == EP_OK && r.max_rows > 0) FAIL("a product without a device");
    const int64_t n = pick();
    const int rz = ep_quantize_rows(n, H, pointer(2), pointer(3), pointer(4), NULL);
    if (rz == EP_OK && n != 0) FAIL("codes without a device");
    ep_problem_t p = {pick() % 5000, H, 1 + (int32_t)(rnd() % 34), 1 + (int32_t)(rnd() % 1030), 1, 1, 0,
                      4, 0};
    const int rc = ep_combine_backward(&p, pointer(2), pointer(3), pointer(4), pointer(5), pointer(6),
                                       pointer(7), pick(), NULL);
    if (rc == EP_OK && p.num_tokens > 0) FAIL("combine's gradient without a device");
    if (ep_integer_workspace_bytes(&r, H) >= 0 && H % 16) FAIL("a ragged row accepted");
    valid += (rf > EP_ERR_INVALID_ARG) + (rg > EP_ERR_INVALID_ARG) + (rq > EP_ERR_INVALID_ARG) +
             (rz > EP_ERR_INVALID_ARG) + (rc > EP_ERR_INVALID_ARG);
  }
  if (valid < 1000) FAIL("only %d accepted descriptors", valid);
  printf("host driver clean, %d accepted\n", valid);
  return 0;
}
