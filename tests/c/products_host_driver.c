/*
 * Drives the host side of the router's and the products' entry points with random
 * and extreme descriptors, in a build with host-only -fsanitize=address,undefined.
 * Run where no device is visible: what validation accepts ends at the device check.
 * Test infrastructure only.
 */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "ep_get.h"

static uint64_t st = 0x9E3779B97F4A7C15ull;
static uint32_t rnd(void) {
  st ^= st >> 12; st ^= st << 25; st ^= st >> 27;
  return (uint32_t)((st * 0x2545F4914F6CDD1Dull) >> 32);
}
static int32_t pick(void) {
  static const int32_t v[] = {-2147483647 - 1, -1, 0, 1, 2, 4, 8, 16, 32, 64, 128, 256, 257, 384,
                              1024, 1025, 7168, 65536, 65544, 1 << 24, 1 << 30, 2147483647};
  if (rnd() % 4) return v[rnd() % (sizeof v / sizeof v[0])];
  return (int32_t)(rnd() % 2000);
}
static void* pointer(void) {
  static const uintptr_t v[] = {256, 1 << 20, 1 << 30, 257, 260, 0};
  return (void*)v[rnd() % 8 < 6 ? rnd() % 3 : rnd() % 6];
}
static ep_weight_t weight(void) {
  static const int32_t groups[] = {32, 64, 128, 0, 48};
  ep_weight_t w = {pointer(), pointer(), rnd() % 2 ? pointer() : NULL, (int32_t)(rnd() % 4),
                   groups[rnd() % 5]};
  return w;
}
#define FAIL(...) do { fprintf(stderr, __VA_ARGS__); fputc('\n', stderr); exit(1); } while (0)

int main(void) {
  int valid = 0;
  for (int i = 0; i < 300000; i++) {
    ep_problem_t p = {pick() % 300, pick(), pick() % 40, pick(), 1, 1, 0, rnd() % 2 ? 8 : 4, 0};
    const int32_t inter = pick();
    const int64_t ws = ep_moe_workspace_bytes(&p, inter);
    if (ws >= 0 && (ws % 256 || ws > 2147483647ll)) FAIL("workspace of %lld bytes", (long long)ws);
    if (ws >= 0 && ws < (int64_t)p.num_tokens * p.num_topk * inter * 2) FAIL("workspace too small");
    ep_moe_args_t m = {pointer(), pointer(), pointer(), weight(), weight(), pointer(), pointer(), inter};
    const int rm = ep_moe_layer(&p, &m, NULL);
    if (rm == EP_OK) FAIL("a layer without a device");
    if (rm != EP_ERR_INVALID_ARG && ws < 0) FAIL("a layer accepted that has no workspace size");
    ep_weight_t w = weight();
    const int rl = ep_quant_linear(pick(), pick(), pick(), pointer(), &w, pointer(), NULL);
    if (rl == EP_OK) FAIL("a product without a device");
    ep_route_args_t r = {pointer(), pointer(), pointer(), pointer(), pick(), pick(), pick() % 40,
                         pick(), pick(), (int32_t)(rnd() % 4), (int32_t)(rnd() % 3),
                         (int32_t)(rnd() % 3), rnd() % 2 ? 2 : 4, rnd() % 2 ? 8 : 4, 1.f};
    const int rr = ep_route(&r, NULL);
    if (rr == EP_OK) FAIL("a routing without a device");
    valid += (rm != EP_ERR_INVALID_ARG) + (rl != EP_ERR_INVALID_ARG) + (rr != EP_ERR_INVALID_ARG);
  }
  if (valid < 100) FAIL("only %d accepted descriptors", valid);
  printf("host driver clean, %d accepted\n", valid);
  return 0;
}
