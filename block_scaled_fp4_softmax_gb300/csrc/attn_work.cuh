// The line of work that attn_plan.h describes, as the kernels walk it.
#pragma once

#include "attn.cuh"
#include "attn_plan.h"

namespace attn {

// What a kernel's CTA knows of the batch, in shared memory.
struct Share {
  long long scan[20], all[20];  // by warp
  long long base0;      // first place of sequence b0 on level0
  long long t0, t1;     // this CTA's places
  long long total;      // places of the line
  int b0, level0;       // the sequence and level that t0 lies in
  int parts;            // CTAs that have places
};

// Scans the batch with the whole block of THREADS threads: the CTA's range of
// the line and the sequence it starts in.  False if lens or cu are out of range
// (the same answer in every CTA).  Ends with a block barrier.
template <int THREADS>
__device__ bool take_share(const int32_t* __restrict__ cu, const int32_t* __restrict__ lens, int batch, int tokens,
                           long long cap, const PlanDims& d, Share& sh) {
  const int per = (batch + THREADS - 1) / THREADS;
  const int b0 = min((int)threadIdx.x * per, batch), b1 = min(b0 + per, batch);
  bool ok = __ldg(cu) == 0 && __ldg(cu + batch) == tokens;
  long long mine = 0, all = 0;  // this thread's sequences: on level 0, and on all levels
  for (int b = b0; b < b1; ++b) {
    const Seq s = sequence(cu, lens, b, tokens, cap);
    ok &= s.ok;
    if (!s.ok || s.n == 0) continue;
    const long long w = sequence_length(d, s.len, s.n, 0);
    mine += w;
    all += w * row_groups(d, s.n);
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = min(THREADS, (batch + per - 1) / per + 31) / 32;  // those that hold sequences
  long long upto = mine;
  auto scan = [&]() {  // upto: of the warp's threads up to this one
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, upto, k);
      if (lane >= k) upto += o;
    }
    if (lane == 31) sh.scan[warp] = upto;
  };
  if (warp < warps) {
    scan();
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) all += __shfl_xor_sync(0xffffffffu, all, k);
    if (lane == 0) sh.all[warp] = all;
  }
  if (!__syncthreads_and(ok)) return false;
  long long total = 0, length = 0;  // of the line, of the level
  for (int w = 0; w < warps; ++w) {
    if (w < warp) upto += sh.scan[w];
    length += sh.scan[w];
    total += sh.all[w];
  }
  if (total > kMaxLine) return false;
  const int parts = part_count(d, total, gridDim.x), c = blockIdx.x;
  const long long t0 = c < parts ? part_begin(total, parts, c) : 0;
  const long long t1 = c < parts ? part_begin(total, parts, c + 1) : 0;
  if (threadIdx.x == 0) sh.t0 = t0, sh.t1 = t1, sh.total = total, sh.parts = parts;
  int level = 0;
  long long before = 0;  // places of the levels below
  while (t0 < t1 && t0 >= before + length) {
    before += length;
    ++level;
    __syncthreads();
    mine = 0;
    for (int b = b0; b < b1; ++b) {
      const Seq s = sequence(cu, lens, b, tokens, cap);
      mine += sequence_length(d, s.len, s.n, level);
    }
    upto = mine;
    if (warp < warps) scan();
    __syncthreads();
    length = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) upto += sh.scan[w];
      length += sh.scan[w];
    }
  }
  upto += before;
  if (t0 < t1 && upto - mine <= t0 && t0 < upto) {
    long long base = upto - mine;
    int b = b0;
    for (;; ++b) {
      const Seq s = sequence(cu, lens, b, tokens, cap);
      const long long w = sequence_length(d, s.len, s.n, level);
      if (t0 < base + w) break;
      base += w;
    }
    sh.b0 = b;
    sh.level0 = level;
    sh.base0 = base;
  }
  __syncthreads();
  return true;
}

// The pieces of one CTA, in order; every role of a kernel walks them on its own.
struct Walk {
  const int32_t *cu, *lens;
  int batch, tokens;
  PlanDims d;
  long long base, t, t1;
  int b, level, number;  // sequence, row group, and pieces before this one
  Seq s;
  Piece p;
  int row0, rows;  // the unit's rows, counted from the first row of the sequence and KV head

  __device__ Walk(const int32_t* cu_, const int32_t* lens_, int batch_, int tokens_, const PlanDims& dims, const Share& sh)
      : cu(cu_), lens(lens_), batch(batch_), tokens(tokens_), d(dims), base(sh.base0), t(sh.t0), t1(sh.t1), b(sh.b0),
        level(sh.level0), number(-1) {
    if (t < t1) s = sequence(cu, lens, b, tokens, kMaxSlots);
  }
  __device__ bool next() {
    do {
      if (t >= t1) return false;
      long long w = sequence_length(d, s.len, s.n, level);
      while (t >= base + w) {
        base += w;
        if (++b == batch) b = 0, ++level;
        s = sequence(cu, lens, b, tokens, kMaxSlots);
        w = sequence_length(d, s.len, s.n, level);
      }
      p = piece_at(d, s.len, s.n, base, t, t1);
      t = p.next;
    } while (p.kt0 >= p.kt1);
    row0 = level * d.unit_rows;
    const long long left = (long long)s.n * d.group - row0;
    rows = left < d.unit_rows ? (int)left : d.unit_rows;
    ++number;
    return true;
  }
  __device__ bool whole() const { return p.kt0 == 0 && p.kt1 == p.tiles; }
};

// Which of slots k0 .. k0 + 31 token `i` of the sequence sees (bit j: slot
// k0 + j).  tree: the ancestor rows of all tokens, or NULL for a chain.
__device__ __forceinline__ uint32_t seen(const uint64_t* __restrict__ tree, int words, const Seq& s, int i, int k0) {
  const int old = s.len - k0, all = s.len + s.n - k0;
  if (old >= 32) return 0xFFFFFFFFu;
  const uint32_t below = all >= 32 ? 0xFFFFFFFFu : all <= 0 ? 0u : (1u << all) - 1u;
  const uint32_t committed = old <= 0 ? 0u : (1u << old) - 1u;
  const uint32_t drafts = tree ? tree_bits(tree + (long long)(s.first + i) * words, words, -old) : chain_bits(i, -old);
  return (committed | drafts) & below;
}

}  // namespace attn
