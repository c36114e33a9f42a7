// Products of FP4 matrices with many rows of x: pairs of CTAs that make one tile of
// 256 rows of x by BN columns of y between them (cta_group::2).
//
// Each CTA of a pair holds its 128 rows of x and half of the tile's rows of w, so
// that w's codes come to an SM once for 256 rows; the first of the two issues the MMAs of
// both.  A persistent pair walks over tiles; its ring of chunks (fp4_linear.cu) runs
// on from tile to tile, and the epilogue warps (16, 12 or 8 for 256, 192 or 128 columns) take the
// sums from TMEM into registers at once, so that the next tile's products start while they write.
//
// Barriers: full (the copies of both CTAs, at the first), empty and sums_full (commits, to
// both CTAs), sums_empty (the epilogue warps of both CTAs, at the first).
//
// What bounds it: the copies into shared memory.  A chunk of a tile of 256 x 256 in NVFP4 is 38 KB for each SM and
// 512 cycles of MMAs; with the copies it takes 626 (62 bytes a cycle and SM), with the copies announced
// but not made 512.  MXFP4's 35 KB take 610 (59).  Copies of scales to TMEM and the issue hide beside the MMAs.
// Narrower tiles have more bytes an MMA and pay where they fill the rounds of tiles better.
// The MMA is the one of 64 columns a step, two thirds of the one of 96 that the card's FP4 peak is quoted with.
// Measured (library GEMM in BF16 1.96 PFLOP/s):
//   16384 x 8192 x 8192   NVFP4   315 to 339 us, 6.5 to 7.0 PFLOP/s (the card's clocks differ)
//   4096 x 8192 x 8192    NVFP4    85 us, 6.5 PFLOP/s        MXFP4   83 us, 6.6 PFLOP/s
//   2451 x 4096 x 5760    MXFP4    27 us, 4.2 PFLOP/s (4 rounds of 300 tiles of 192 columns)
//   256 x 2560 x 8192     NVFP4    9.3 us
// A launch costs 6 to 7 us beside its chunks: set-up, first copies, the last tile's epilogue.
#include "fp4_mma.cuh"

using namespace moe::tc;
using namespace fp4;

namespace {

constexpr int kEpilogueWarps = 16, kTmaWarp = 16, kMmaWarp = 17, kThreads = 576;

template <int FMT, int BN_>
struct Cfg {
  static constexpr int BN = BN_;                                // columns of y of a tile
  static constexpr bool NV = FMT == MOE_FMT_NVFP4;
  static constexpr int COPIES = NV ? 4 : 2;                     // tiles of scales of a chunk and 128 rows
  static constexpr int W_TILES = (BN + 127) / 128;              // 128 rows of w's scales; both CTAs take all
  static constexpr int X_BYTES = 128 * 128, W_BYTES = BN / 2 * 128, S_BYTES = COPIES * 512;
  static constexpr int SLOT = X_BYTES + W_BYTES + (1 + W_TILES) * S_BYTES;
  static constexpr int STAGE = kEpilogueWarps * 32 * 64;        // 64 bytes of 32 rows for each epilogue warp
  static constexpr int ROOM = (227 * 1024 - 1024 - STAGE - 256) / SLOT;
  static constexpr int SLOTS = ROOM < 8 ? ROOM : 8;
  static constexpr int SX_COLS = COPIES * 4, SW_COLS = SX_COLS * W_TILES;
  // TMEM holds the scales of as many chunks as the ring: where a slot's copies have
  // landed, the products that took the scales before it have been made.
  static constexpr int S_COL = BN;
  static constexpr int TMEM = 512;
  static constexpr int SHARE = 64;                              // columns of an epilogue warp
  static_assert(S_COL + SLOTS * (SX_COLS + SW_COLS) <= TMEM, "TMEM");
  static_assert(SLOT % 1024 == 0, "the swizzle's alignment");
  static_assert(BN % 64 == 0, "tiles of scales may start in the middle of 128 rows");
};

struct Control {
  uint64_t full[8], empty[8];
  uint64_t sums_full, sums_empty, drain;
  uint32_t tmem;
  int abort, peer_abort;  // a wait has run out, in this CTA or in the other one
  int loaded;             // chunks whose copies the CTA has issued, at its end
};
template <class C>
constexpr size_t smem_bytes() {
  return 1024 + (size_t)C::SLOTS * C::SLOT + C::STAGE + sizeof(Control);
}
static_assert(sizeof(Control) <= 256, "Cfg::ROOM");

// Which tile of the grid of tiles comes i-th: blocks of 8 tiles of rows, so that the
// tiles that run at a time share both operands in L2.
struct Tile {
  int t0, n0;
  __device__ __forceinline__ Tile(int i, int t_tiles, int n_tiles, int BN) {
    const int group = i / (8 * n_tiles), first = group * 8, rows = min(8, t_tiles - first);
    const int k = i - group * 8 * n_tiles;
    t0 = (first + k % rows) * 256;
    n0 = k / rows * BN;
  }
};

__device__ __forceinline__ void commit_both(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// `stage`: 64 bytes of each of 32 rows, in pieces of 16 bytes that are swizzled.
__device__ __forceinline__ uint4* staged(uint8_t* stage, int row, int piece) {
  return reinterpret_cast<uint4*>(stage + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
}

// Writes what the warp has staged, the first `rows` rows and `left` columns of it, so that its
// stores are whole sectors, four lanes to a row: with rows written by their own threads the
// epilogue held up the next tile's copies for some 4000 cycles.
__device__ __forceinline__ void write_staged(uint8_t* stage, int lane, bool vector, uint8_t* to, long long step, int item,
                                             int rows, int left) {
  __syncwarp();
  if (vector && left * item >= 64) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 8 * k + (lane >> 2), c = lane & 3;
      if (r < rows) *reinterpret_cast<uint4*>(to + r * step + 16 * c) = *staged(stage, r, c);
    }
  } else {  // the edge of y, or rows that do not lie on 16 bytes: 32 or 16 elements a row
    // (eight rows at a time: 504 x 2560 x 50257 43 us, one after the other 45)
    const int per = 64 / item, first = lane / per, c = lane % per;
    auto row = [&](int r) { return reinterpret_cast<const uint8_t*>(staged(stage, r, (c * item) >> 4)) + ((c * item) & 15); };
    if (c < left && item == 4) {
#pragma unroll 8
      for (int k = 0; k < 16; ++k)
        if (const int r = first + 2 * k; r < rows)
          *reinterpret_cast<uint32_t*>(to + r * step + 4 * c) = *reinterpret_cast<const uint32_t*>(row(r));
    } else if (c < left) {
#pragma unroll 8
      for (int r = 0; r < 32; ++r)
        if (r < rows) *reinterpret_cast<uint16_t*>(to + r * step + 2 * c) = *reinterpret_cast<const uint16_t*>(row(r));
    }
  }
  __syncwarp();
}

struct WideArgs {
  LinearArgs l;
  CUtensorMap w_scales_map, x_scales_map;
  int t_tiles, n_tiles;
  int vector;  // y may be written 16 bytes at a time
};

template <int FMT, int BN>
__global__ void __launch_bounds__(kThreads, 1) wide_kernel(const __grid_constant__ WideArgs args) {
  const LinearArgs& a = args.l;
  const int t_tiles = args.t_tiles, n_tiles = args.n_tiles;
  using C = Cfg<FMT, BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Control& ctl = *reinterpret_cast<Control*>(ring + (size_t)C::SLOTS * C::SLOT + C::STAGE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int all = t_tiles * n_tiles;
  const int chunks = (a.cols + kChunk - 1) / kChunk;
  const int tiles = scale_tiles(a.cols, FMT);

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    mbar_init(&ctl.sums_full, 1 + a.extra);
    mbar_init(&ctl.sums_empty, 2 * 4 * (BN / C::SHARE));
    mbar_init(&ctl.drain, 1);
    ctl.abort = ctl.peer_abort = 0;
    mbar_fence_init();
    attn::prefetch_map(&a.w_map);
    attn::prefetch_map(&a.x_map);
    attn::prefetch_map(&args.w_scales_map);
    attn::prefetch_map(&args.x_scales_map);
  }
  __syncthreads();
  cluster_sync();  // the barriers of both CTAs are set up
  // (as in fp4_linear.cu: TMEM is taken between the kernel before and the one behind)
  moe::pdl_wait();
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem)),
                 "r"(C::TMEM)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  moe::pdl_launch_dependents();
  const uint32_t tmem = ctl.tmem;
  volatile int* abort_flag = &ctl.abort;

  if (warp == kTmaWarp) {
    if (lane == 0) {
      bool alive = true;
      int i = 0;  // chunks so far
      for (int at = pair; at < all && alive; at += pairs) {
        const Tile tile(at, t_tiles, n_tiles, BN);
        const int t0 = tile.t0 + 128 * rank, n0 = tile.n0;
        for (int c = 0; c < chunks; ++c, ++i) {
          const int slot = i % C::SLOTS;
          alive = cluster_wait(&ctl.empty[slot], ((i / C::SLOTS) & 1) ^ 1, a.wait_cycles, abort_flag, a.st);
          if (!alive) break;
          // Both CTAs' copies are counted at the first one's barrier.  A box of scales may
          // reach into the next rows' tiles or past the last: nothing takes those.
          if (rank == 0) mbar_arrive_expect_tx(&ctl.full[slot], 2 * C::SLOT);
          const uint32_t bar = peer_address(smem_u32(&ctl.full[slot]), 0);
          const uint32_t x = smem_u32(ring + (size_t)slot * C::SLOT), w = x + C::X_BYTES, s = w + C::W_BYTES;
          const int kt = c * C::COPIES;
          load_pair(&a.x_map, x, bar, c * (kChunk / 2), t0);
          load_pair(&a.w_map, w, bar, c * (kChunk / 2), n0 + BN / 2 * rank);
          load_pair(&args.x_scales_map, s, bar, 0, (t0 >> 7) * tiles + kt);
#pragma unroll
          for (int k = 0; k < C::W_TILES; ++k)
            load_pair(&args.w_scales_map, s + (1 + k) * C::S_BYTES, bar, 0, ((n0 >> 7) + k) * tiles + kt);
        }
      }
      ctl.loaded = i;
      // the commits that free the last slots have arrived: none is under way at the CTA's end
      for (int k = max(0, i - C::SLOTS); k < i && alive; ++k)
        alive = cluster_wait(&ctl.empty[k % C::SLOTS], (k / C::SLOTS) & 1, a.wait_cycles, abort_flag, a.st);
    }
    __syncwarp();
  } else if (warp == kMmaWarp && rank == 1) {
    // (the first CTA's issues for both)
  } else if (warp == kMmaWarp) {
    // The warp walks and waits as one and its elected lane issues: with what it issues
    // in a branch of one lane's own, each of these instructions took 67 cycles, 1075 a
    // chunk, twice the time of its products.
    const bool leader = attn::elect_lane();
    bool alive = true;
    int slot = 0, done = 0;  // of the ring; tiles so far
    uint32_t round = 0;      // parity of the ring's rounds
    const uint64_t x_desc = sw128_kmajor_desc(smem_u32(ring)), w_desc = sw128_kmajor_desc(smem_u32(ring) + C::X_BYTES);
    const uint64_t s_desc = scales_desc(smem_u32(ring) + C::X_BYTES + C::W_BYTES);
    for (int at = pair; at < all && alive; at += pairs, ++done) {
      if (done > 0)
        alive = __all_sync(0xffffffffu, cluster_wait(&ctl.sums_empty, (done - 1) & 1, a.wait_cycles, abort_flag, a.st));
      // a tile that starts in the middle of 128 rows of w takes their scales from there
      const uint32_t skip = Tile(at, t_tiles, n_tiles, BN).n0 % 128 / 32;
      for (int c = 0; c < chunks && alive; ++c) {
        alive = __all_sync(0xffffffffu, cluster_wait(&ctl.full[slot], round, a.wait_cycles, abort_flag, a.st));
        if (!alive) break;
        fence_after_sync();
        if (leader) {
          const uint32_t off = (uint32_t)slot * (C::SLOT >> 4);
          const uint32_t set = tmem + C::S_COL + slot * (C::SX_COLS + C::SW_COLS);
          auto step = [&](int k) {
            const int copy = C::NV ? k : k / 2, id = C::NV ? 0 : 2 * (k & 1);
            const uint32_t sx = set + 4 * copy, sw = set + C::SX_COLS + 4 * C::W_TILES * copy;
            if (id == 0) {
              copy_scales<2>(sx, s_desc + off + copy * 32);
#pragma unroll
              for (int q = 0; q < C::W_TILES; ++q)
                copy_scales<2>(sw + 4 * q, s_desc + off + ((1 + q) * C::S_BYTES >> 4) + copy * 32);
            }
            mma_fp4<FMT, 2>(tmem, x_desc + off + 2 * k, w_desc + off + 2 * k, idesc_fp4<FMT>(256, BN, id), sx, sw + skip,
                            c > 0 || k > 0);
          };
          if (a.cols - c * kChunk >= kChunk) {
#pragma unroll
            for (int k = 0; k < kChunk / 64; ++k) step(k);
          } else {
            const int steps = (a.cols - c * kChunk + 63) / 64;
#pragma unroll
            for (int k = 0; k < kChunk / 64 - 1; ++k)
              if (k < steps) step(k);
            if (steps == kChunk / 64) step(kChunk / 64 - 1);
          }
          commit_both(&ctl.empty[slot]);
          if (c == chunks - 1) commit_both(&ctl.sums_full);
        }
        __syncwarp();
        if (++slot == C::SLOTS) slot = 0, round ^= 1;
      }
    }
    // ... nor an arrival of the other CTA's epilogue
    if (alive && done > 0) cluster_wait(&ctl.sums_empty, (done - 1) & 1, a.wait_cycles, abort_flag, a.st);
    __syncwarp();
    // TMEM and the ring go back only when every MMA has completed
    if (leader) {
      asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&ctl.drain))
                   : "memory");
      attn::bounded_wait(&ctl.drain, 0, attn::kDrainCycles, nullptr, a.st);
    }
    __syncwarp();
  } else {
    // Four warps to the 128 rows of 64 columns each.  They take the sums as they are into
    // registers and free their place, before any arithmetic: the next tile's products
    // wait for that (some 3000 cycles when they scaled and rounded first).
    const int first = (warp >> 2) * C::SHARE;
    const uint32_t sums = tmem + ((uint32_t)((warp & 3) * 32) << 16) + first;
    uint8_t* stage = ring + (size_t)C::SLOTS * C::SLOT + warp * (32 * 64);
    const int item = element_bytes(a.y_type);
    const long long step = a.y_stride * item;
    // Factors of a tile: of the lane's row, and of columns `lane` and `lane + 32` of the warp's,
    // which the others get by shuffles.  Those of the next tile are fetched while this
    // one's sums are awaited.
    struct Factors {
      float row, scale[2], add[2];
    };
    auto factors = [&](int at) {
      Factors f = {1.f, {1.f, 1.f}, {0.f, 0.f}};
      if (at >= all) return f;
      const Tile tile(at, t_tiles, n_tiles, BN);
      const int t = tile.t0 + 128 * rank + (warp & 3) * 32 + lane;
      if (a.x_row && t < a.t) f.row = __ldg(a.x_row + t);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int n = tile.n0 + first + 32 * k + lane;
        if (a.w_row && n < a.n) f.scale[k] = __ldg(a.w_row + n);
        if (a.bias && n < a.n) f.add[k] = __ldg(a.bias + n);
      }
      return f;
    };
    bool alive = true;
    int done = 0;
    Factors next = factors(pair);
    for (int at = pair; at < all && first < BN; at += pairs, ++done) {
      const Tile tile(at, t_tiles, n_tiles, BN);
      const int t0 = tile.t0 + 128 * rank + (warp & 3) * 32, n0 = tile.n0 + first;
      Factors f = next;
      next = factors(at + pairs);
      alive = alive && __all_sync(0xffffffffu, cluster_wait(&ctl.sums_full, done & 1, a.wait_cycles, abort_flag, a.st));
      fence_after_sync();
      float v[C::SHARE];
      attn::tmem_ld32(sums, v);
      attn::tmem_ld32(sums + 32, v + 32);
      attn::tmem_ld_wait32(v);
      attn::tmem_ld_wait32(v + 32);
      fence_before_sync();
      __syncwarp();
      if (lane == 0 && alive) arrive_relaxed_at(&ctl.sums_empty, 0);
      if (!alive) f.row = kNaN;
      const int rows = min(32, a.t - t0), left = a.n - n0;
      uint8_t* y = static_cast<uint8_t*>(a.y) + (t0 * a.y_stride + n0) * item;
      if (rows <= 0 || left <= 0) continue;
      auto scaled = [&](int i) {  // column i of the lane's row
        const float c = __shfl_sync(0xffffffffu, f.scale[i >> 5], i & 31);
        const float b = a.bias ? __shfl_sync(0xffffffffu, f.add[i >> 5], i & 31) : 0.f;
        return fmaf(v[i] * f.row, c, b);
      };
      if (a.y_type != FP4_FP32) {
#pragma unroll
        for (int i = 0; i < C::SHARE; i += 32) {
          if (i >= left) break;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = scaled(i + 8 * k + e);
            *staged(stage, lane, k) = a.y_type == FP4_BF16 ? attn::pack8<attn::Brain>(q) : attn::pack8<attn::Half>(q);
          }
          write_staged(stage, lane, args.vector, y + 2 * i, step, 2, rows, left - i);
        }
      } else {
#pragma unroll
        for (int i = 0; i < C::SHARE; i += 16) {
          if (i >= left) break;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float q[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) q[e] = scaled(i + 4 * k + e);
            *staged(stage, lane, k) = *reinterpret_cast<const uint4*>(q);
          }
          write_staged(stage, lane, args.vector, y + 4 * i, step, 4, rows, left - i);
        }
      }
    }
  }
  // No CTA's shared memory or TMEM is in use by the other any more: all copies have landed, all
  // MMAs have completed and all arrivals have come, unless a wait has run out in one of the two.  That
  // one says so to the other before it arrives.
  __syncthreads();
  const bool gave_up = *abort_flag;
  if (gave_up) {
    if (threadIdx.x == 0) set_peer_word(smem_u32(&ctl.peer_abort), rank ^ 1, 1);
    cluster_sync();
  } else {
    cluster_sync_relaxed();
  }
  if (gave_up || *(volatile int*)&ctl.peer_abort) {
    cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
      // One CTA may have stopped a few copies before the other: what the barriers still expect
      // of it is struck off, what they do not expect is added.
      const int mine = ctl.loaded, other = (int)peer_word(smem_u32(&ctl.loaded), 1);
      for (int k = max(0, max(mine, other) - C::SLOTS); k < max(mine, other); ++k) {
        uint64_t* bar = &ctl.full[k % C::SLOTS];
        if (k >= other)
          asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(C::SLOT)
                       : "memory");
        if (k >= mine) mbar_arrive_expect_tx(bar, C::SLOT);
        attn::bounded_wait(bar, (k / C::SLOTS) & 1, attn::kDrainCycles, nullptr, a.st);
      }
    }
    __syncthreads();
    cluster_sync();
  }
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM) : "memory");
}

template <int FMT, int BN>
int launch(LinearArgs& a, const fp4_matrix& x, const fp4_matrix& w, int sms, cudaStream_t st) {
  using C = Cfg<FMT, BN>;
  static moe::SmemGrant grant;
  const long long t_tiles = (a.t + 255) / 256, n_tiles = (a.n + BN - 1) / BN;
  if (t_tiles * n_tiles > 0x3FFFFFFF || 8 * n_tiles > 0x3FFFFFFF) return MOE_ERR_UNSUPPORTED;
  WideArgs args = {a, {}, {}, (int)t_tiles, (int)n_tiles, 0};
  args.vector = moe::aligned16(a.y) && a.y_stride * element_bytes(a.y_type) % 16 == 0;
  if (const int rc = codes_map(x, 128, &args.l.x_map)) return rc;
  if (const int rc = codes_map(w, BN / 2, &args.l.w_map)) return rc;
  if (const int rc = scales_map(x, &args.x_scales_map)) return rc;
  if (const int rc = scales_map(w, &args.w_scales_map)) return rc;
  if (!moe::grant_smem(wide_kernel<FMT, BN>, smem_bytes<C>(), grant)) return MOE_ERR_CUDA;
  const int pairs = (int)(t_tiles * n_tiles < sms / 2 ? t_tiles * n_tiles : sms / 2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<C>();
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, wide_kernel<FMT, BN>, args) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// The width of a tile that gives the least time: rounds of tiles over the pairs, each of
// its chunks (NVFP4's 626, 580 and 500 cycles, which the copies take; MXFP4's are 610, 558 and 494, and the
// widths that come out below were its best ones too) and some 2500 cycles between
// tiles.  With 256, 192 and 128 columns a tile, in us:
//   512 x 9728 x 2560 17.5 17.1 15.5 (one round of each)    504 x 4096 x 5120 11.7 11.1 14.5
//   4096 x 4096 x 5120 36.8 39.2 47.9 (5, 6, 9 rounds)      2451 x 2880 x 4096 20.9 19.1 23.8
//   1024 x 4096 x 4096 12.0 16.6 14.9 (1, 2, 2 rounds)      8192 x 2560 x 7680 62.3 69.9 88.7
template <int FMT>
int by_width(LinearArgs& a, const fp4_matrix& x, const fp4_matrix& w, int sms, cudaStream_t st) {
  const int widths[3] = {256, 192, 128}, cycles[3] = {626, 580, 500};
  long long best = 1ll << 62;
  int width = 0;
  for (int i = 0; i < 3; ++i) {
    const int b = widths[i];
    const long long tiles = (long long)((a.t + 255) / 256) * ((a.n + b - 1) / b), rounds = (tiles + sms / 2 - 1) / (sms / 2);
    const long long cost = rounds * ((a.cols + kChunk - 1) / kChunk * cycles[i] + 2500);
    if (cost < best) best = cost, width = b;
  }
  return width == 256 ? launch<FMT, 256>(a, x, w, sms, st) : width == 192 ? launch<FMT, 192>(a, x, w, sms, st)
                                                                           : launch<FMT, 128>(a, x, w, sms, st);
}

}  // namespace

namespace fp4 {

int launch_wide(LinearArgs& a, const fp4_matrix& x, const fp4_matrix& w, int sms, cudaStream_t st) {
  return w.format == MOE_FMT_NVFP4 ? by_width<MOE_FMT_NVFP4>(a, x, w, sms, st) : by_width<MOE_FMT_MXFP4>(a, x, w, sms, st);
}

}  // namespace fp4
