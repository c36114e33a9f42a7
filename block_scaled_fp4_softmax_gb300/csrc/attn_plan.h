// How attn_tree_decode divides its work, for host and device.
//
// A unit is one (sequence, KV head, group of up to `unit_rows` query rows);
// a row is one token in flight and query head of the KV head's group.  Its
// work is the tiles of keys it looks at, and `cost` tiles' time for fetching
// the rows and writing the result, which stand before its first tile.  All
// units form one line that is cut into `parts` nearly equal ranges, one per
// CTA: every CTA gets the same share however ragged the batch is, and a long
// sequence is spread over as many CTAs as its share of the work.  A unit that a
// cut divides is joined from its pieces afterwards.
//
// The order on the line is row group (level), sequence, head.  The levels of a
// batch of like sequences are equally long, so the CTAs that take the second row
// group of some keys run beside those that take the first, and find the keys in
// L2: with the row groups of a head side by side instead, 8 sequences of 16384
// slots and 504 rows read K and V from HBM twice (134 us against 130).
#pragma once

#ifdef __CUDACC__
#define ATTN_HD __host__ __device__ __forceinline__
#else
#define ATTN_HD inline
#endif

namespace attn {

// a / b of non-negative numbers; the 32-bit division is several times cheaper
// and nearly always enough.
ATTN_HD long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (long long)((unsigned)a / (unsigned)b);
  return a / b;
}

struct PlanDims {
  int kv_heads, group;      // query heads of a KV head
  int unit_rows, tile;      // rows of a unit, keys of a tile
  int cost;                 // places of the line before a unit's first tile
  int least;                // places that a part has at least, if the line has them
};

ATTN_HD int row_groups(const PlanDims& d, int n) {
  return (int)quotient((long long)n * d.group + d.unit_rows - 1, d.unit_rows);
}
ATTN_HD int key_tiles(const PlanDims& d, int len, int n) { return (int)quotient((long long)len + n + d.tile - 1, d.tile); }
// Places of the units of a sequence on a level.
ATTN_HD long long sequence_length(const PlanDims& d, int len, int n, int level) {
  return n <= 0 || row_groups(d, n) <= level ? 0 : (long long)d.kv_heads * (d.cost + key_tiles(d, len, n));
}

// A line longer than this is refused (the products below stay within 64 bits).
constexpr long long kMaxLine = 1ll << 47;

// Into how many parts a line is cut for a grid.
ATTN_HD int part_count(const PlanDims& d, long long total, int grid) {
  const long long most = quotient(total + d.least - 1, d.least);
  return most < grid ? (int)most : grid;
}
// First place of part c, and the part that holds place t (at most 2^15 parts).
ATTN_HD long long part_begin(long long total, int parts, int c) { return quotient(total * c, parts); }
ATTN_HD int part_of(long long total, int parts, long long t) { return (int)quotient((t + 1) * parts - 1, total); }

// One piece of a unit: key tiles [kt0, kt1) of its `tiles` (none, if the part
// holds only places before the first tile).
struct Piece {
  int head;
  int kt0, kt1, tiles;
  long long first_tile;  // the place of the unit's tile 0
  long long next;        // where the part goes on
};

// The piece that starts at place `t` of the line and ends before `end`, where
// the sequence's first place on the level is `base`.
ATTN_HD Piece piece_at(const PlanDims& d, int len, int n, long long base, long long t, long long end) {
  Piece p;
  p.tiles = key_tiles(d, len, n);
  const long long u = quotient(t - base, p.tiles + d.cost);
  p.first_tile = base + u * (p.tiles + d.cost) + d.cost;
  const long long from = t - p.first_tile, to = end - p.first_tile;
  p.kt0 = from < 0 ? 0 : (int)from;
  p.kt1 = to < 0 ? 0 : to < p.tiles ? (int)to : p.tiles;
  p.next = to < p.tiles ? end : p.first_tile + p.tiles;
  p.head = (int)u;
  return p;
}

}  // namespace attn
