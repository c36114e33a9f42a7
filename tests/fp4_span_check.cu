// Checks csrc/fp4_span.h on the host against sets of bytes: rows of every small
// width, stride, number and distance, and the same far up in the address range.
#include <cstdio>
#include <initializer_list>
#include <vector>

#include "fp4_span.h"

using fp4::Span;

static long long checks = 0, failed = 0;

static bool plain(const Span& a, const Span& b) {
  std::vector<char> seen(400, 0);
  for (long long r = 0; r < a.rows; ++r)
    for (long long i = 0; i < a.width; ++i) seen[a.at + r * a.stride + i] = 1;
  for (long long r = 0; r < b.rows; ++r)
    for (long long i = 0; i < b.width; ++i)
      if (seen[b.at + r * b.stride + i]) return true;
  return false;
}

static void check(const Span& a, const Span& b) {
  const bool want = plain(a, b);
  for (long long base : {0ll, 0x7fff00000000ll}) {
    Span x = a, y = b;
    x.at += base, y.at += base;
    ++checks;
    if ((fp4::overlap(x, y) != want || fp4::overlap(y, x) != want) && failed++ < 20)
      std::printf("FAILED: %lld+%lldx%lld/%lld against %lld+%lldx%lld/%lld: %d\n", a.at, a.rows, a.width, a.stride, b.at,
                  b.rows, b.width, b.stride, want);
  }
}

int main() {
  for (long long wa = 1; wa <= 4; ++wa)
    for (long long sa = wa; sa <= 7; ++sa)
      for (long long ra = 1; ra <= 5; ++ra)
        for (long long wb = 1; wb <= 4; ++wb)
          for (long long sb = wb; sb <= 7; ++sb)
            for (long long rb = 1; rb <= 5; ++rb)
              for (long long at = 0; at <= 80; ++at) check(Span{40, wa, sa, ra, 0}, Span{at, wb, sb, rb, 0});

  // gate | up | out side by side, 2^24 rows: apart, and not when one is a byte wider
  const long long rows = 1 << 24, stride = 3 * 4096;
  auto side = [&](long long k, long long width) { return Span{(1ll << 40) + 4096 * k, width, stride, rows, 2}; };
  bool ok = !fp4::overlap(side(0, 4096), side(1, 4096)) && !fp4::overlap(side(2, 4096), side(0, 4096)) &&
            fp4::overlap(side(0, 4097), side(1, 4096)) && fp4::overlap(side(2, 4097), side(0, 4096));
  // where only the last row of one and the first of the other are near
  ok = ok && !fp4::overlap(side(0, 4096), side(3 * rows, 4096)) && fp4::overlap(side(0, 4096), side(3 * rows - 3, 4096));
  // a piece of memory among rows, and none
  ok = ok && fp4::overlap(fp4::piece((void*)(1ll << 40), 5), side(0, 4096)) && !fp4::overlap(fp4::piece(nullptr, 5), side(0, 4096)) &&
       !fp4::overlap(fp4::piece((void*)(1ll << 40), 0), side(0, 4096));
  // the same place is of rows of the same elements alone
  const Span a = fp4::rows_span((void*)4096, 3, 64, 128, 2), shifted = fp4::rows_span((void*)(4096 + 256), 3, 64, 128, 2);
  ok = ok && fp4::same_place(a, fp4::rows_span((void*)4096, 3, 64, 128, 2)) && !fp4::same_place(a, shifted) &&
       !fp4::same_place(a, fp4::rows_span((void*)4096, 3, 32, 64, 4)) && !fp4::same_place(a, fp4::rows_span((void*)4096, 3, 64, 136, 2)) &&
       !fp4::same_place(fp4::piece((void*)4096, 64), fp4::piece((void*)4096, 64)) &&
       fp4::same_place(fp4::rows_span((void*)4096, 1, 64, 128, 2), fp4::rows_span((void*)4096, 1, 64, 0, 2));
  const Span ins[2] = {a, side(0, 4096)}, same[2] = {a, side(1, 4096)}, moved[1] = {shifted}, twice[2] = {side(1, 64), side(1, 64)};
  ok = ok && fp4::apart(same, ins) && !fp4::apart(moved, ins) && !fp4::apart(twice, ins);
  checks += 1, failed += !ok;
  if (!ok) std::printf("FAILED: single cases\n");
  std::printf("%lld checks, %lld failed\n", checks, failed);
  return failed != 0;
}
