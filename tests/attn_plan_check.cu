// Walks the work division of attn_tree_decode (csrc/attn_plan.h) on the host
// the way the kernel's roles do, for many batches and numbers of parts: every
// tile of every unit is covered exactly once and in order, the parts are even,
// a part holds at most one piece that continues a unit and one that starts a
// divided unit (its two places in the workspace), and the pieces of a divided
// unit are found where the joining kernel looks for them.
#include <cstdio>
#include <map>
#include <random>
#include <tuple>
#include <vector>

#include "attn_plan.h"

using namespace attn;

static long long checks = 0, failed = 0;
static void check(bool ok, const char* what) {
  ++checks;
  if (!ok && failed++ < 20) std::printf("FAILED: %s\n", what);
}

static void run(const PlanDims& d, const std::vector<int>& len, const std::vector<int>& n, int grid) {
  long long total = 0;
  int levels = 0;
  for (size_t b = 0; b < len.size(); ++b)
    for (int level = 0; n[b] > 0 && level < row_groups(d, n[b]); ++level) {
      total += sequence_length(d, len[b], n[b], level);
      levels = level + 1 > levels ? level + 1 : levels;
    }
  const int parts = part_count(d, total, grid);
  check(parts <= grid && (parts < grid || total >= grid) && (total == 0) == (parts == 0), "parts");
  std::map<std::tuple<int, int, int>, int> reached;  // unit -> tiles covered so far
  std::map<std::tuple<int, int, int>, std::pair<int, int>> split;  // divided unit -> first part, pieces announced
  std::map<std::tuple<int, int, int>, int> pieces;
  long long most = 0, least = total;
  for (int c = 0; c < parts; ++c) {
    const long long t0 = part_begin(total, parts, c), t1 = part_begin(total, parts, c + 1);
    most = t1 - t0 > most ? t1 - t0 : most;
    least = t1 - t0 < least ? t1 - t0 : least;
    check(t0 < t1, "a part has work");
    check(part_of(total, parts, t0) == c && part_of(total, parts, t1 - 1) == c, "part_of");
    long long t = t0, base = 0;
    size_t b = 0;
    int level = 0, going_on = 0, starting = 0;
    while (t < t1) {
      while (t >= base + sequence_length(d, len[b], n[b], level)) {
        base += sequence_length(d, len[b], n[b], level);
        if (++b == len.size()) b = 0, ++level;
      }
      check(level < levels, "level in range");
      const Piece p = piece_at(d, len[b], n[b], base, t, t1);
      check(p.next > t && p.next <= t1, "goes on");
      t = p.next;
      if (p.kt0 >= p.kt1) continue;
      check(p.head >= 0 && p.head < d.kv_heads && level < row_groups(d, n[b]), "unit in range");
      check(p.kt0 >= 0 && p.kt0 < p.kt1 && p.kt1 <= p.tiles && p.tiles == key_tiles(d, len[b], n[b]), "tiles in range");
      const auto unit = std::make_tuple((int)b, p.head, level);
      check(reached[unit] == p.kt0, "tiles in order, once");
      reached[unit] = p.kt1;
      if (p.kt0 > 0) {
        ++going_on;
        check(split.count(unit) && split[unit].first + pieces[unit] == c, "a continued unit's pieces lie in successive parts");
        ++pieces[unit];
      } else if (p.kt1 < p.tiles) {
        ++starting;
        const int last = part_of(total, parts, p.first_tile + p.tiles - 1);
        split[unit] = {c, last - c + 1};
        pieces[unit] = 1;
      }
    }
    check(t == t1 && going_on <= 1 && starting <= 1, "two places a part");
  }
  check(parts == 0 || most - least <= 1, "even parts");
  for (size_t b = 0; b < len.size(); ++b)
    for (int h = 0; h < d.kv_heads && n[b] > 0; ++h)
      for (int r = 0; r < row_groups(d, n[b]); ++r) check(reached[std::make_tuple((int)b, h, r)] == key_tiles(d, len[b], n[b]), "every unit whole");
  for (auto& s : split) check(pieces[s.first] == s.second.second, "as many pieces as announced");
}

int main() {
  std::mt19937 g(1);
  auto in = [&](int a, int b) { return (int)(a + g() % (unsigned)(b - a + 1)); };
  for (int trial = 0; trial < 3000; ++trial) {
    PlanDims d{in(1, 8), in(1, 16), trial % 3 ? 256 : 128, trial % 2 ? 128 : 64, (int)(g() % 6), in(1, 5)};
    const int B = in(1, trial % 7 ? 6 : 60);
    std::vector<int> len(B), n(B);
    for (int b = 0; b < B; ++b) {
      len[b] = in(0, 3) == 0 ? in(0, 2) : in(0, trial % 5 ? 700 : 30000);
      n[b] = in(0, 4) == 0 ? 0 : in(1, trial % 4 ? 5 : 200);
    }
    run(d, len, n, in(0, 1) ? 152 : in(1, 300));
  }
  // lengths near the limit
  run(PlanDims{8, 8, 256, 128, 3, 5}, {2147481600 - 300, 2147480000, 5}, {100, 64, 0}, 152);
  std::printf("%lld checks, %lld failed\n", checks, failed);
  return failed != 0;
}
