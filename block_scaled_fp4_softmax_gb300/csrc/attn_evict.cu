// Eviction from a paged cache by accumulated weight.
//
// Two launches.  select_kernel finds, for every sequence and KV head, which
// slots stay; move_kernel copies the kept rows from beyond the budget into
// the holes below it.
//
// Selection is a radix select on 32-bit keys whose unsigned order is the
// ranking (protected slots all ones, FP32 weights order-preserving, NaN 0),
// 11 + 11 + 10 bits a round, by one cluster of CTAs per (sequence, head).  All
// protected slots stay as a rule, whatever their order; where the first round finds
// that they alone fill the budget, the keys are formed anew, of the protected slots'
// weights and 0 for the others, and the rounds begin again.  Each
// CTA keeps its slice's keys in shared memory, so acc and slot_pos are read
// once; a round counts digits into a shared histogram, and every CTA adds up
// the cluster's histograms through distributed shared memory.  The result is
// the key of the last slot that stays and how many of the slots with just
// that key stay (the lowest ones).  Ranks of holes and movers then follow from
// two counts at the start of each warp's slots (keys above, keys equal):
// kept(x) = above(x) + min(equal(x), ties) slots below x stay, so x - kept(x)
// below the budget are holes and kept(x) - kept(budget) beyond it move.  No
// atomics decide an order: results are the same from call to call.
//
// What bounds it: three dependent rounds, each two barriers of the cluster and a
// scan (3000 cycles; 7000 in clusters of 16), and for many rows the copies, which
// are scattered rows of D elements.  Measured, with the copies: 16 ragged sequences of
// up to 16384 slots x 8 heads of 128 to 6144: 44 us (select 19, move 25 for 0.11 GB);
// 2 of 200003 x 2 heads of 64 to 131072: 40 us (25, 16); 1 of 2500 x 4 heads: 13 us.
#include <cooperative_groups.h>

#include "attn.cuh"
#include "attn_slice.h"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 16;  // beyond 8 the kernel has to allow it, and the device to have room
constexpr int kMaxKeys = 44 * 1024;  // keys of one CTA's slice held in shared memory

struct EvictArgs {
  attn_cache c;
  const float* acc;
  const int32_t* slot_pos;
  int slot_cap;
  const int32_t *lens, *next_pos;
  int budget, sinks, recent;
  float* acc_out;
  int32_t* pos_out;
  int32_t* lens_out;
  int32_t* counts;  // [batch x kv_heads] moves
  int32_t* src;     // [batch x kv_heads x budget] mover slots, ascending
  int32_t* dst;     // the same: hole slots
  int32_t* st;
};

// `of_held`: of the protected slots' weights (NaN 1), 0 for the others.
__device__ __forceinline__ uint32_t rank_key(float w, int pos, int sinks, long long recent_from, bool of_held) {
  const bool held = pos < sinks || pos >= recent_from;
  if (held != of_held) return held ? 0xFFFFFFFFu : 0u;
  if (w != w) return of_held ? 1u : 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

struct alignas(16) Shared {
  uint32_t hist[3][kBins];
  uint32_t total[kBins];  // the cluster's histogram, where it is added up in slices
  uint32_t part[kThreads];  // of this CTA's slice: sums over two CTAs each
  uint32_t warp_sum[kWarps];
  int4 counts[kWarps];  // above, equal, above below the budget, equal below the budget
  int2 before[kWarps];       // above and equal in the CTA's warps before
  int4 of_cta[kMaxCluster];  // the same four counts of each CTA
  uint32_t digit, rest;
};

// KEYS: the slice's keys fit in shared memory; otherwise each pass reads acc
// and slot_pos again.  A warp owns `sub` consecutive slots and takes 128 at a
// time, four to a lane.  VEC: rows of acc and slot_pos are 16-byte aligned.
template <bool KEYS, bool VEC>
__global__ void __launch_bounds__(kThreads) select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint4 s_all[];
  Shared& sh = *reinterpret_cast<Shared*>(s_all);
  uint32_t* s_keys = reinterpret_cast<uint32_t*>(&sh + 1);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), r = (int)cluster.block_rank();
  const int problem = blockIdx.x / C, b = problem / a.c.kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < 3 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
  moe::pdl_wait();
  moe::pdl_launch_dependents();
  const int n = __ldg(a.lens + b), K = a.budget;
  const long long recent_from = (long long)__ldg(a.next_pos + b) - a.recent;
  const long long base = (long long)problem * a.slot_cap;
  const float* __restrict__ acc = a.acc + base;
  const int32_t* __restrict__ pos = a.slot_pos + base;
  const long long most = (long long)a.c.max_pages * a.c.page_size;
  const bool bad = n < 0 || n > a.slot_cap || n > most;
  if (r == 0 && threadIdx.x == 0 && problem % a.c.kv_heads == 0) {
    a.lens_out[b] = n < 0 ? 0 : n < K ? n : K;
    if (bad) moe::status_or(a.st, ATTN_DEV_BAD_LENGTH);
  }
  if (bad || n <= K) {  // the whole cluster takes this branch together
    const int m = n < 0 ? 0 : bad ? min(min(n, K), a.slot_cap) : n;
    const int share = attn::slice_slots(m, C * kWarps), w = r * kWarps + warp, end = attn::slice_begin(m, share, w + 1);
    for (int c0 = attn::slice_begin(m, share, w); c0 < end; c0 += 128) {
      float old[4];
      int at[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int j = c0 + 32 * q + lane;
        old[q] = __uint_as_float(0x7FC00000u), at[q] = -1;
        if (!bad && j < end) old[q] = acc[j], at[q] = pos[j];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int j = c0 + 32 * q + lane;
        if (j < end) a.acc_out[base + j] = old[q], a.pos_out[base + j] = at[q];
      }
    }
    if (r == 0 && threadIdx.x == 0) a.counts[problem] = 0;
    return;
  }
  const int sub = attn::slice_slots(n, C * kWarps);
  const int j0 = attn::slice_begin(n, sub, r * kWarps + warp), j1 = attn::slice_begin(n, sub, r * kWarps + warp + 1);
  uint32_t* keys = s_keys + warp * sub;
  auto fetch = [&](int j, float4& w, int4& p) {  // slots j .. j + 3; nothing past the end
    w = make_float4(0.f, 0.f, 0.f, 0.f);
    p = make_int4(0, 0, 0, 0);
    if (VEC && j + 4 <= n) {
      w = *reinterpret_cast<const float4*>(acc + j);
      p = *reinterpret_cast<const int4*>(pos + j);
      return;
    }
    if (j < n) w.x = acc[j], p.x = pos[j];
    if (j + 1 < n) w.y = acc[j + 1], p.y = pos[j + 1];
    if (j + 2 < n) w.z = acc[j + 2], p.z = pos[j + 2];
    if (j + 3 < n) w.w = acc[j + 3], p.w = pos[j + 3];
  };
  bool of_held = false;
  auto key_of = [&](float w, int p) { return rank_key(w, p, a.sinks, recent_from, of_held); };
  auto keys_of = [&](const float4& w, const int4& p) {
    return make_uint4(key_of(w.x, p.x), key_of(w.y, p.y), key_of(w.z, p.z), key_of(w.w, p.w));
  };
  auto keys_at = [&](int j) {
    if (KEYS) return *reinterpret_cast<const uint4*>(keys + (j - j0));
    float4 w;
    int4 p;
    fetch(j, w, p);
    return keys_of(w, p);
  };
  // keys into shared memory; what lies below the budget goes to the outputs as it
  // is (a mover overwrites what is dropped there)
  constexpr int kAhead = 4;
  for (int c0 = j0; c0 < j1; c0 += 128 * kAhead) {
    float4 w[kAhead];
    int4 p[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) fetch(c0 + 128 * q + 4 * lane < j1 ? c0 + 128 * q + 4 * lane : n, w[q], p[q]);
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int j = c0 + 128 * q + 4 * lane;
      if (j >= j1) continue;
      if (KEYS) *reinterpret_cast<uint4*>(keys + (j - j0)) = keys_of(w[q], p[q]);
      if (VEC && j + 4 <= K) {
        *reinterpret_cast<float4*>(a.acc_out + base + j) = w[q];
        *reinterpret_cast<int4*>(a.pos_out + base + j) = p[q];
      } else {
        if (j < K) a.acc_out[base + j] = w[q].x, a.pos_out[base + j] = p[q].x;
        if (j + 1 < K) a.acc_out[base + j + 1] = w[q].y, a.pos_out[base + j + 1] = p[q].y;
        if (j + 2 < K) a.acc_out[base + j + 2] = w[q].z, a.pos_out[base + j + 2] = p[q].z;
        if (j + 3 < K) a.acc_out[base + j + 3] = w[q].w, a.pos_out[base + j + 3] = p[q].w;
      }
    }
  }
  __syncthreads();

  uint32_t prefix = 0, rest = (uint32_t)K;  // slots still to be placed among those with this prefix
  for (int round = 0; round < 3; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
    const int bits = round == 2 ? 10 : 11;
    const uint32_t above = round == 0 ? 0u : 0xFFFFFFFFu << (shift + bits);
    uint32_t* const hist = sh.hist[of_held ? (round + 1) % 3 : round];  // one that is all zeros
    for (int j = j0 + 4 * lane; j < j1; j += 128) {
      const uint4 v = keys_at(j);
      const uint32_t k[4] = {v.x, v.y, v.z, v.w};
      const int live = j1 - j;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < live && (k[q] & above) == prefix)
          atomicAdd(&hist[(k[q] >> shift) & ((1u << bits) - 1u)], 1u);
    }
    cluster.sync();
    if (of_held && round == 0)  // no CTA looks at the first histogram any more
      for (int i = threadIdx.x; i < kBins; i += kThreads) sh.hist[0][i] = 0;
    // thread i: bins kBins - 1 - 2i and the one below, over the cluster.  Up to four
    // CTAs each read all histograms; more share the bins out and hand the sums
    // round (16 CTAs reading 16 histograms took 12000 cycles a round).
    const int hi = kBins - 1 - 2 * threadIdx.x;
    uint32_t n_hi = 0, n_lo = 0;
    if (C <= 4) {
      for (int q = 0; q < C; ++q) {
        const uint32_t* other = cluster.map_shared_rank(hist, q);
        const uint2 v = *reinterpret_cast<const uint2*>(other + hi - 1);
        n_lo += v.x;
        n_hi += v.y;
      }
    } else {
      const int slice = kBins / C, half = C / 2;  // threads: bin of the slice x pair of CTAs
      const int bin = r * slice + (int)threadIdx.x % slice, pair = threadIdx.x / slice;
      sh.part[threadIdx.x] = cluster.map_shared_rank(hist, pair)[bin] +
                             cluster.map_shared_rank(hist, pair + half)[bin];
      __syncthreads();
      uint32_t sum = 0;
      for (int q = 0; q < half; ++q) sum += sh.part[q * slice + (int)threadIdx.x % slice];
      cluster.map_shared_rank(&sh.total[0], pair)[bin] = sum;
      cluster.map_shared_rank(&sh.total[0], pair + half)[bin] = sum;
      cluster.sync();
      n_lo = sh.total[hi - 1];
      n_hi = sh.total[hi];
    }
    uint32_t scan = n_hi + n_lo;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, scan, d);
      if (lane >= d) scan += up;
    }
    if (lane == 31) sh.warp_sum[warp] = scan;
    __syncthreads();
    uint32_t lower = lane < warp ? sh.warp_sum[lane] : 0u;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) lower += __shfl_xor_sync(0xffffffffu, lower, d);
    const uint32_t upto = lower + scan, before_hi = upto - n_hi - n_lo, before_lo = upto - n_lo;
    if (before_hi < rest && rest <= before_lo) sh.digit = hi, sh.rest = rest - before_hi;
    else if (before_lo < rest && rest <= upto) sh.digit = hi - 1, sh.rest = rest - before_lo;
    __syncthreads();
    prefix |= sh.digit << shift;
    rest = sh.rest;
    if (round == 0 && !of_held && prefix >> shift == kBins - 1) {  // (no weight has this digit)
      of_held = true;
      if (KEYS)
        for (int j = j0 + 4 * lane; j < j1; j += 128) {
          float4 w;
          int4 p;
          fetch(j, w, p);
          *reinterpret_cast<uint4*>(keys + (j - j0)) = keys_of(w, p);
        }
      prefix = 0, rest = (uint32_t)K, round = -1;
    }
  }
  // slots with a key above `prefix` stay, and the first `rest` of those equal to it
  int4 cnt = make_int4(0, 0, 0, 0);
  for (int c0 = j0; c0 < j1; c0 += 128) {
    const int j = c0 + 4 * lane, live = j1 - j;
    const uint4 v = live > 0 ? keys_at(j) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t k[4] = {v.x, v.y, v.z, v.w};
    int gt = 0, eq = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      gt += q < live && k[q] > prefix;
      eq += q < live && k[q] == prefix;
    }
    cnt.x += gt;
    cnt.y += eq;
    if (c0 + 128 <= K) {
      cnt.z += gt, cnt.w += eq;
    } else if (c0 < K) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        cnt.z += q < live && j + q < K && k[q] > prefix;
        cnt.w += q < live && j + q < K && k[q] == prefix;
      }
    }
  }
  cnt.x = __reduce_add_sync(0xffffffffu, cnt.x);
  cnt.y = __reduce_add_sync(0xffffffffu, cnt.y);
  cnt.z = __reduce_add_sync(0xffffffffu, cnt.z);
  cnt.w = __reduce_add_sync(0xffffffffu, cnt.w);
  if (lane == 0) sh.counts[warp] = cnt;
  cluster.sync();
  if (warp < C) {  // a warp to a CTA, a lane to a warp of it
    const int4 v = *cluster.map_shared_rank(&sh.counts[lane], warp);
    int2 in = make_int2(v.x, v.y);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int ux = __shfl_up_sync(0xffffffffu, in.x, d), uy = __shfl_up_sync(0xffffffffu, in.y, d);
      if (lane >= d) in.x += ux, in.y += uy;
    }
    if (warp == r) sh.before[lane] = make_int2(in.x - v.x, in.y - v.y);
    const int low = __reduce_add_sync(0xffffffffu, v.z), low_equal = __reduce_add_sync(0xffffffffu, v.w);
    if (lane == 31) sh.of_cta[warp] = make_int4(in.x, in.y, low, low_equal);
  }
  __syncthreads();
  int above = sh.before[warp].x, equal = sh.before[warp].y, low = 0, low_equal = 0;
  for (int q = 0; q < C; ++q) {
    const int4 v = sh.of_cta[q];
    if (q < r) above += v.x, equal += v.y;
    low += v.z;
    low_equal += v.w;
  }
  const int ties = (int)rest;
  const int kept_low = low + min(low_equal, ties);  // kept slots below the budget
  if (r == 0 && threadIdx.x == 0) a.counts[problem] = K - kept_low;
  int32_t* src = a.src + (long long)problem * K;
  int32_t* dst = a.dst + (long long)problem * K;
  // here a lane takes every 32nd slot: what the warp writes lies side by side
  const uint32_t lower_lanes = (1u << lane) - 1u;
  for (int c0 = j0; c0 < j1; c0 += 128) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = c0 + 32 * q + lane;
      const bool live = j < j1;
      uint32_t key = 0u;
      if (live) key = KEYS ? keys[j - j0] : key_of(acc[j], pos[j]);
      const bool gt = live && key > prefix, eq = live && key == prefix;
      const uint32_t all_gt = __ballot_sync(0xffffffffu, gt), all_eq = __ballot_sync(0xffffffffu, eq);
      const int eq_before = equal + __popc(all_eq & lower_lanes);
      const bool kept = gt || (eq && eq_before < ties);
      const int kept_before = above + __popc(all_gt & lower_lanes) + min(eq_before, ties);
      if (live) {
        if (j >= K) {
          if (kept) src[kept_before - kept_low] = j;
        } else if (!kept) {
          dst[j - kept_before] = j;
        }
      }
      above += __popc(all_gt);
      equal += __popc(all_eq);
    }
  }
  cluster.sync();  // no CTA leaves while another may still read its shared memory
}

constexpr int kMoveThreads = 256;

constexpr int kBatch = 128;  // moves a block takes at a time
constexpr int kMoves = 4;    // moves of a group whose loads are in flight together

// A thread looks up where each move of a batch leads from and to, and moves the
// weight and position; then a group of LANES lanes copies a row of k and of v.
template <int LANES>
__global__ void __launch_bounds__(kMoveThreads, 4) move_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int kGroups = kMoveThreads / LANES;
  static_assert(kBatch % (kGroups * kMoves) == 0 || kBatch < kGroups * kMoves, "whole rounds");
  __shared__ long long s_from[kBatch], s_to[kBatch];  // -1: no move
  moe::pdl_wait();
  const int problem = blockIdx.y, b = problem / a.c.kv_heads, h = problem - b * a.c.kv_heads;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int n = __ldg(a.counts + problem);
  const long long base = (long long)problem * a.slot_cap;
  const int32_t* src = a.src + (long long)problem * a.budget;
  const int32_t* dst = a.dst + (long long)problem * a.budget;
  const bool mine = lane * 8 < a.c.head_dim;
  uint16_t* const k = static_cast<uint16_t*>(a.c.k) + lane * 8;
  uint16_t* const v = static_cast<uint16_t*>(a.c.v) + lane * 8;
  for (int i0 = blockIdx.x * kBatch; i0 < n; i0 += gridDim.x * kBatch) {
    __syncthreads();
    if (threadIdx.x < kBatch) {
      long long from = -1, to = -1;
      if (i0 + (int)threadIdx.x < n) {
        const int s = __ldg(src + i0 + threadIdx.x), d = __ldg(dst + i0 + threadIdx.x);
        const float w = a.acc[base + s];
        const int p = a.slot_pos[base + s];
        from = attn::slot_offset(a.c, b, s, h), to = attn::slot_offset(a.c, b, d, h);
        const bool good = from >= 0 && to >= 0;
        if (!good) moe::status_or(a.st, ATTN_DEV_BAD_PAGE), from = -1;
        a.acc_out[base + d] = good ? w : __uint_as_float(0x7FC00000u);
        a.pos_out[base + d] = p;
      }
      s_from[threadIdx.x] = from;
      s_to[threadIdx.x] = to;
    }
    __syncthreads();
#pragma unroll 1
    for (int m0 = group; m0 < kBatch; m0 += kGroups * kMoves) {
      long long from[kMoves];
      uint4 x[kMoves], y[kMoves];
#pragma unroll
      for (int m = 0; m < kMoves; ++m) {
        from[m] = m0 + m * kGroups < kBatch ? s_from[m0 + m * kGroups] : -1;
        if (mine && from[m] >= 0) {
          x[m] = *reinterpret_cast<const uint4*>(k + from[m]);
          y[m] = *reinterpret_cast<const uint4*>(v + from[m]);
        }
      }
#pragma unroll
      for (int m = 0; m < kMoves; ++m)
        if (mine && from[m] >= 0) {
          const long long to = s_to[m0 + m * kGroups];
          *reinterpret_cast<uint4*>(k + to) = x[m];
          *reinterpret_cast<uint4*>(v + to) = y[m];
        }
    }
  }
}

template <int LANES>
int launch_move(const EvictArgs& a, int problems, int sms, cudaStream_t st) {
  // no more blocks than the budget's rows need, nor than a few waves
  const long long per = ((long long)a.budget + kBatch - 1) / kBatch, most = (16ll * sms + problems - 1) / problems;
  return moe::launch_pdl(move_kernel<LANES>, dim3((unsigned)(per < most ? per : most), problems), dim3(kMoveThreads), 0, st, a);
}

// Whether clusters of 16 CTAs with `smem` bytes each can run on the current
// device; asked once per device (for the largest slice).
template <bool KEYS, bool VEC>
bool sixteen_fit() {
  static std::atomic<int> known[moe::kMaxDevices];  // 0: not asked, 1: no, 2: yes
  const int d = moe::current_device();
  if (d < 0) return false;
  int k = known[d].load(std::memory_order_acquire);
  if (k == 0) {
    const size_t smem = sizeof(Shared) + (KEYS ? (size_t)kMaxKeys * 4 : 0);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    const bool yes =
        cudaFuncSetAttribute(select_kernel<KEYS, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess &&
        cudaFuncSetAttribute(select_kernel<KEYS, VEC>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, select_kernel<KEYS, VEC>, &cfg) == cudaSuccess && n > 0;
    if (!yes) (void)cudaGetLastError();
    known[d].store(k = yes ? 2 : 1, std::memory_order_release);
  }
  return k == 2;
}

template <bool KEYS, bool VEC>
int launch_select(const EvictArgs& a, int problems, int C, size_t smem, cudaStream_t st) {
  static moe::SmemGrant grant;
  if (!moe::grant_smem(select_kernel<KEYS, VEC>, smem, grant)) return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(problems * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_kernel<KEYS, VEC>, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <bool VEC>
int select(const EvictArgs& a, int problems, int sms, cudaStream_t st) {
  // one CTA a problem, more while SMs are idle and a CTA has more than two rounds of slots
  int C = 1;
  while (C < kMaxCluster && problems * C < sms && a.slot_cap > 2 * kThreads * C) C *= 2;
  auto slots = [&](int c) { return (long long)attn::slice_slots(a.slot_cap, c * kWarps) * kWarps; };  // of a CTA
  const bool keys = slots(C) <= kMaxKeys;
  if (C == 16 && !(keys ? sixteen_fit<true, VEC>() : sixteen_fit<false, VEC>())) C = 8;
  return slots(C) <= kMaxKeys ? launch_select<true, VEC>(a, problems, C, sizeof(Shared) + (size_t)slots(C) * 4, st)
                              : launch_select<false, VEC>(a, problems, C, sizeof(Shared), st);
}

bool overlap(const void* a, size_t n, const void* b, size_t m) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + m && y < x + n;
}

size_t counts_bytes(const attn_cache& c) { return ((size_t)c.batch * c.kv_heads * 4 + 15) & ~(size_t)15; }

}  // namespace

extern "C" {

size_t attn_cache_evict_workspace(const attn_cache* cache, int budget) {
  attn_cache c;
  if (attn::check_cache(cache, c) || budget <= 0) return 0;
  return counts_bytes(c) + (size_t)c.batch * c.kv_heads * budget * 8;
}

int attn_cache_evict(const attn_cache* cache, const float* acc, const int32_t* slot_pos, int slot_cap,
                     const int32_t* lens, const int32_t* next_pos, int budget, int sinks, int recent, float* acc_out,
                     int32_t* slot_pos_out, int32_t* lens_out, void* workspace, size_t ws_bytes, int32_t* dev_status,
                     void* stream) {
  EvictArgs a;
  if (const int rc = attn::check_cache(cache, a.c)) return rc;
  if (!acc || !slot_pos || !lens || !next_pos || !acc_out || !slot_pos_out || !lens_out || !workspace ||
      slot_cap <= 0 || budget <= 0 || sinks < 0 || recent < 0)
    return MOE_ERR_INVALID_ARG;
  const long long problems = (long long)a.c.batch * a.c.kv_heads;
  if (slot_cap > attn::kMaxSlots || problems > 65535) return MOE_ERR_UNSUPPORTED;
  // the CTAs of a sequence read its inputs while others write
  const size_t all = (size_t)problems * slot_cap * 4, each = (size_t)a.c.batch * 4;
  if (overlap(acc_out, all, acc, all) || overlap(slot_pos_out, all, slot_pos, all) ||
      overlap(lens_out, each, lens, each) || overlap(lens_out, each, next_pos, each))
    return MOE_ERR_INVALID_ARG;
  if (!moe::aligned16(workspace)) return MOE_ERR_ALIGNMENT;
  if (ws_bytes < attn_cache_evict_workspace(cache, budget)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  a.acc = acc, a.slot_pos = slot_pos, a.slot_cap = slot_cap, a.lens = lens, a.next_pos = next_pos;
  a.budget = budget, a.sinks = sinks, a.recent = recent;
  a.acc_out = acc_out, a.pos_out = slot_pos_out, a.lens_out = lens_out, a.st = dev_status;
  a.counts = static_cast<int32_t*>(workspace);
  a.src = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + counts_bytes(a.c));
  a.dst = a.src + problems * budget;
  const int sms = moe::device_info().sms;
  if (sms <= 0) return MOE_ERR_CUDA;
  const cudaStream_t st = (cudaStream_t)stream;
  const bool vec = slot_cap % 4 == 0 && moe::aligned16(acc) && moe::aligned16(slot_pos) && moe::aligned16(acc_out) &&
                   moe::aligned16(slot_pos_out);
  const int rc = vec ? select<true>(a, (int)problems, sms, st) : select<false>(a, (int)problems, sms, st);
  if (rc) return rc;
  if (a.c.head_dim <= 32) return launch_move<4>(a, (int)problems, sms, st);
  if (a.c.head_dim <= 64) return launch_move<8>(a, (int)problems, sms, st);
  if (a.c.head_dim <= 128) return launch_move<16>(a, (int)problems, sms, st);
  return launch_move<32>(a, (int)problems, sms, st);
}

}  // extern "C"
