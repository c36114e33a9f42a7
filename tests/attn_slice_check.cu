// Checks csrc/attn_slice.h on the host: the slices of a cluster's warps cover the
// slots once and in order, up to the largest length, and stepping through a slice
// the way the kernel's loops do stays within an int.
#include <cstdio>
#include <random>

#include "attn_slice.h"

static long long checks = 0, failed = 0;
static void check(bool ok, const char* what, long long n, int c) {
  ++checks;
  if (!ok && failed++ < 20) std::printf("FAILED: %s (%lld slots, %d CTAs)\n", what, n, c);
}

static void run(long long n, int c) {
  constexpr int kWarps = 32;
  const long long slots = attn::slice_slots((int)n, c * kWarps);
  check(slots > 0 && slots % 128 == 0 && slots * c * kWarps >= n, "a slice holds its share", n, c);
  long long upto = 0;
  for (int w = 0; w < c * kWarps; ++w) {
    const long long j0 = attn::slice_begin((int)n, (int)slots, w), j1 = attn::slice_begin((int)n, (int)slots, w + 1);
    check(j0 == upto && j1 >= j0 && j1 - j0 <= slots && (j0 % 128 == 0 || j0 == n), "slices in order", n, c);
    // the loops go on by at most 512 slots and look at most 512 ahead
    check(j1 <= n && (j0 == j1 || j1 - 1 + 512 + 512 <= 0x7FFFFFFFll), "steps within an int", n, c);
    upto = j1;
  }
  check(upto == n, "every slot", n, c);
}

int main() {
  const long long most = 0x7FFFFFFFll - 2048;
  std::mt19937_64 g(1);
  for (int c = 1; c <= 16; c *= 2) {
    for (long long n = 1; n < 1500; ++n) run(n, c);
    for (long long k = 0; k < 70000; k += 61) run(most - k, c);
    for (int i = 0; i < 2000; ++i) run(1 + (long long)(g() % (unsigned long long)(g() % 2 ? most : 1000000)), c);
    run(most, c);
  }
  std::printf("%lld checks, %lld failed\n", checks, failed);
  return failed != 0;
}
