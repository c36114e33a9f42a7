// Eviction from a paged cache by accumulated weight.
//
// Two launches.  select_kernel finds, for every sequence and KV head, which
// slots stay; move_kernel copies the kept rows from beyond the budget into
// the holes below it.
//
// Selection is a radix select on 32-bit keys whose unsigned order is the
// ranking (protected slots all ones, FP32 weights order-preserving, NaN 0),
// 11 + 11 + 10 bits a round, by one cluster of CTAs per (sequence, head).  Each
// CTA keeps its slice's keys in shared memory, so acc and slot_pos are read
// once; a round counts digits into a shared histogram, and every CTA adds up
// the cluster's histograms through distributed shared memory.  The result is
// the key of the last slot that stays and how many of the slots with just
// that key stay (the lowest ones).  Ranks of holes and movers then follow from
// two counts at the start of each warp's slots (keys above, keys equal):
// kept(x) = above(x) + min(equal(x), ties) slots below x stay, so x - kept(x)
// below the budget are holes and kept(x) - kept(budget) beyond it move.  No
// atomics decide an order: results are the same from call to call.
#include <cooperative_groups.h>

#include "attn.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxKeys = 48 * 1024;  // keys of one CTA's slice held in shared memory

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

__device__ __forceinline__ uint32_t rank_key(float w, int pos, int sinks, long long recent_from) {
  if (pos < sinks || pos >= recent_from) return 0xFFFFFFFFu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

struct alignas(16) Shared {
  uint32_t hist[3][kBins];
  uint32_t warp_sum[kWarps];
  int4 counts[kWarps];  // above, equal, above below the budget, equal below the budget
  int2 before[kWarps];
  int2 at_budget;
  uint32_t digit, rest;
};

// KEYS: the slice's keys fit in shared memory; otherwise each pass reads acc
// and slot_pos again.
template <bool KEYS>
__global__ void __launch_bounds__(kThreads) select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint4 s_all[];
  Shared& sh = *reinterpret_cast<Shared*>(s_all);
  uint32_t* s_keys = reinterpret_cast<uint32_t*>(&sh + 1);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), r = (int)cluster.block_rank();
  const int problem = blockIdx.x / C, b = problem / a.c.kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = __ldg(a.lens + b), K = a.budget;
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
    for (int j = r * kThreads + threadIdx.x; j < m; j += C * kThreads) {
      a.acc_out[base + j] = bad ? __uint_as_float(0x7FC00000u) : acc[j];
      a.pos_out[base + j] = bad ? -1 : pos[j];
    }
    if (r == 0 && threadIdx.x == 0) a.counts[problem] = 0;
    return;
  }
  const long long recent_from = (long long)__ldg(a.next_pos + b) - a.recent;
  const int sub = ((n + C * kWarps - 1) / (C * kWarps) + 31) & ~31;  // slots of a warp
  const int j0 = min((r * kWarps + warp) * sub, n), j1 = min(j0 + sub, n);
  uint32_t* keys = s_keys + warp * sub;
  for (int i = threadIdx.x; i < 3 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
  if (KEYS) {
#pragma unroll 8
    for (int j = j0 + lane; j < j1; j += 32) keys[j - j0] = rank_key(acc[j], pos[j], a.sinks, recent_from);
  }
  auto key_of = [&](int j) { return KEYS ? keys[j - j0] : rank_key(acc[j], pos[j], a.sinks, recent_from); };
  __syncthreads();

  uint32_t prefix = 0, rest = (uint32_t)K;  // slots still to be placed among those with this prefix
  for (int round = 0; round < 3; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
    const int bits = round == 2 ? 10 : 11;
    const uint32_t above = round == 0 ? 0u : 0xFFFFFFFFu << (shift + bits);
    for (int c0 = j0; c0 < j1; c0 += 32) {
      const uint32_t k = c0 + lane < j1 ? key_of(c0 + lane) : 0u;
      const bool in = c0 + lane < j1 && (k & above) == prefix;
      const uint32_t digit = (k >> shift) & ((1u << bits) - 1u);
      // many slots share a digit (weights that are 0, protected slots): one
      // add for a warp that holds a single one
      const unsigned act = __ballot_sync(0xffffffffu, in);
      if (act == 0) continue;
      const int leader = __ffs(act) - 1;
      const uint32_t first = __shfl_sync(0xffffffffu, digit, leader);
      if (__all_sync(0xffffffffu, !in || digit == first)) {
        if (lane == leader) atomicAdd(&sh.hist[round][digit], (unsigned)__popc(act));
      } else if (in) {
        atomicAdd(&sh.hist[round][digit], 1u);
      }
    }
    cluster.sync();
    // thread i: bins kBins - 1 - 2i and the one below, over the cluster
    const int hi = kBins - 1 - 2 * threadIdx.x;
    uint32_t n_hi = 0, n_lo = 0;
    for (int q = 0; q < C; ++q) {
      const uint32_t* other = cluster.map_shared_rank(&sh.hist[round][0], q);
      const uint2 v = *reinterpret_cast<const uint2*>(other + hi - 1);
      n_lo += v.x;
      n_hi += v.y;
    }
    uint32_t scan = n_hi + n_lo;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, scan, d);
      if (lane >= d) scan += up;
    }
    if (lane == 31) sh.warp_sum[warp] = scan;
    __syncthreads();
    uint32_t lower = 0;
    for (int w = 0; w < warp; ++w) lower += sh.warp_sum[w];
    const uint32_t upto = lower + scan, before_hi = upto - n_hi - n_lo, before_lo = upto - n_lo;
    if (before_hi < rest && rest <= before_lo) sh.digit = hi, sh.rest = rest - before_hi;
    else if (before_lo < rest && rest <= upto) sh.digit = hi - 1, sh.rest = rest - before_lo;
    __syncthreads();
    prefix |= sh.digit << shift;
    rest = sh.rest;
  }
  // slots with a key above `prefix` stay, and the first `rest` of those equal to it
  int4 cnt = make_int4(0, 0, 0, 0);
  for (int j = j0 + lane; j < j1; j += 32) {
    const uint32_t k = key_of(j);
    cnt.x += k > prefix;
    cnt.y += k == prefix;
    cnt.z += k > prefix && j < K;
    cnt.w += k == prefix && j < K;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    cnt.x += __shfl_xor_sync(0xffffffffu, cnt.x, d);
    cnt.y += __shfl_xor_sync(0xffffffffu, cnt.y, d);
    cnt.z += __shfl_xor_sync(0xffffffffu, cnt.z, d);
    cnt.w += __shfl_xor_sync(0xffffffffu, cnt.w, d);
  }
  if (lane == 0) sh.counts[warp] = cnt;
  cluster.sync();
  if (warp == 0) {  // lane = warp of a CTA; prefix over the cluster in slot order
    int2 run = make_int2(0, 0), at = make_int2(0, 0);
    for (int q = 0; q < C; ++q) {
      const int4 v = *cluster.map_shared_rank(&sh.counts[lane], q);
      int2 in = make_int2(v.x, v.y);
      at.x += v.z;
      at.y += v.w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int ux = __shfl_up_sync(0xffffffffu, in.x, d), uy = __shfl_up_sync(0xffffffffu, in.y, d);
        if (lane >= d) in.x += ux, in.y += uy;
      }
      if (q == r) sh.before[lane] = make_int2(run.x + in.x - v.x, run.y + in.y - v.y);
      run.x += __shfl_sync(0xffffffffu, in.x, 31);
      run.y += __shfl_sync(0xffffffffu, in.y, 31);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      at.x += __shfl_xor_sync(0xffffffffu, at.x, d);
      at.y += __shfl_xor_sync(0xffffffffu, at.y, d);
    }
    if (lane == 0) sh.at_budget = at;
  }
  __syncthreads();
  const int ties = (int)rest;
  const int kept_low = sh.at_budget.x + min(sh.at_budget.y, ties);  // kept slots below the budget
  if (r == 0 && threadIdx.x == 0) a.counts[problem] = K - kept_low;
  int above = sh.before[warp].x, equal = sh.before[warp].y;
  int32_t* src = a.src + (long long)problem * K;
  int32_t* dst = a.dst + (long long)problem * K;
  const unsigned below_me = (1u << lane) - 1u;
  for (int c0 = j0; c0 < j1; c0 += 32) {
    const int j = c0 + lane;
    const uint32_t k = j < j1 ? key_of(j) : 0u;
    const bool gt = j < j1 && k > prefix, eq = j < j1 && k == prefix;
    const unsigned m_gt = __ballot_sync(0xffffffffu, gt), m_eq = __ballot_sync(0xffffffffu, eq);
    const int eq_rank = equal + __popc(m_eq & below_me);
    const bool kept = gt || (eq && eq_rank < ties);
    const int kept_before = above + __popc(m_gt & below_me) + min(eq_rank, ties);
    if (j < j1) {
      if (j < K) {
        if (kept) {
          a.acc_out[base + j] = acc[j];
          a.pos_out[base + j] = pos[j];
        } else {
          dst[j - kept_before] = j;
        }
      } else if (kept) {
        src[kept_before - kept_low] = j;
      }
    }
    above += __popc(m_gt);
    equal += __popc(m_eq);
  }
  cluster.sync();  // no CTA leaves while another may still read its shared memory
}

constexpr int kMoveThreads = 256;

// One group of LANES lanes copies one moved row of k and of v.
template <int LANES>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int kGroups = kMoveThreads / LANES;
  const int problem = blockIdx.y, b = problem / a.c.kv_heads, h = problem % a.c.kv_heads;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int n = __ldg(a.counts + problem);
  const long long base = (long long)problem * a.slot_cap;
  const int32_t* src = a.src + (long long)problem * a.budget;
  const int32_t* dst = a.dst + (long long)problem * a.budget;
  const bool mine = lane * 8 < a.c.head_dim;
  for (int i = blockIdx.x * kGroups + group; i < n; i += gridDim.x * kGroups) {
    const int s = __ldg(src + i), d = __ldg(dst + i);
    const long long from = attn::slot_offset(a.c, b, s, h), to = attn::slot_offset(a.c, b, d, h);
    const bool bad = from < 0 || to < 0;
    if (!bad && mine) {
      const uint16_t* k = static_cast<const uint16_t*>(a.c.k) + lane * 8;
      const uint16_t* v = static_cast<const uint16_t*>(a.c.v) + lane * 8;
      const uint4 x = *reinterpret_cast<const uint4*>(k + from), y = *reinterpret_cast<const uint4*>(v + from);
      *reinterpret_cast<uint4*>(const_cast<uint16_t*>(k) + to) = x;
      *reinterpret_cast<uint4*>(const_cast<uint16_t*>(v) + to) = y;
    }
    if (lane == 0) {
      if (bad) moe::status_or(a.st, ATTN_DEV_BAD_PAGE);
      a.acc_out[base + d] = bad ? __uint_as_float(0x7FC00000u) : a.acc[base + s];
      a.pos_out[base + d] = a.slot_pos[base + s];
    }
  }
}

template <int LANES>
int launch_move(const EvictArgs& a, int problems, int sms, cudaStream_t st) {
  constexpr int kGroups = kMoveThreads / LANES;
  // no more blocks than the budget's rows need, nor than a few waves
  long long per = (a.budget + kGroups - 1) / kGroups, most = (16ll * sms + problems - 1) / problems;
  move_kernel<LANES><<<dim3((unsigned)(per < most ? per : most), problems), kMoveThreads, 0, st>>>(a);
  return moe::launch_status();
}

template <bool KEYS>
int launch_select(const EvictArgs& a, int problems, int C, size_t smem, cudaStream_t st) {
  static moe::SmemGrant grant;
  if (!moe::grant_smem(select_kernel<KEYS>, smem, grant)) return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(problems * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_kernel<KEYS>, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
      slot_cap <= 0 || budget <= 0 || sinks < 0 || recent < 0 || acc == acc_out || slot_pos == slot_pos_out ||
      lens == lens_out)
    return MOE_ERR_INVALID_ARG;
  const long long problems = (long long)a.c.batch * a.c.kv_heads;
  if (slot_cap > attn::kMaxSlots || problems > 65535) return MOE_ERR_UNSUPPORTED;
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
  int C = 1;
  while (C < kMaxCluster && problems * C < sms && slot_cap > 1024 * C) C *= 2;
  const int sub = ((slot_cap + C * kWarps - 1) / (C * kWarps) + 31) & ~31;
  const bool keys = sub * kWarps <= kMaxKeys;
  const int rc = keys ? launch_select<true>(a, (int)problems, C, sizeof(Shared) + (size_t)sub * kWarps * 4, st)
                      : launch_select<false>(a, (int)problems, C, sizeof(Shared), st);
  if (rc) return rc;
  if (a.c.head_dim <= 32) return launch_move<4>(a, (int)problems, sms, st);
  if (a.c.head_dim <= 64) return launch_move<8>(a, (int)problems, sms, st);
  if (a.c.head_dim <= 128) return launch_move<16>(a, (int)problems, sms, st);
  return launch_move<32>(a, (int)problems, sms, st);
}

}  // extern "C"
