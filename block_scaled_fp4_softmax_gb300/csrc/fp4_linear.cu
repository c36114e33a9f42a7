// Products of two FP4 matrices on the 5th-generation tensor cores, whose MMA takes
// e2m1 operands and their block scales (kind::mxf4nvf4, 64 columns a step).
//
//   D[n, t] = sum_k w[n, k] x[t, k]      weights on the M side, 128 rows a tile
//
// Chunks of 256 columns go through a ring in shared memory: codes by TMA (128 bytes a
// row, 128-byte swizzle), block scales by bulk copies (they lie in memory as
// the tensor core wants them, 512 bytes for 128 rows x 4 blocks), from where
// tcgen05.cp takes them to TMEM beside the sums.
//
// Few rows of x are bound by the weights' bytes.  A persistent CTA walks over tiles; its
// ring runs on from tile to tile, and a tile's sums are written while the next one's are
// made (two places in TMEM).  Where there are fewer tiles than SMs, a tile's columns are split
// over a cluster of CTAs, whose sums meet in distributed shared memory in a fixed order.
//
// Up to 16 rows of x stay in shared memory for all tiles (HELD), if they fit.  One or two rows of
// up to 32768 elements in all are quantised by each CTA itself, which saves a launch (2 us on the host)
// and 0.5 to 1 us of the GPU; with four rows it would cost 0.5 to 1.6.
//
// What bounds it: the weights' bytes, 0.5625 of an element, from HBM; below some 20 MB of them the
// chain of launch, loads, products and the exchange (4.1 us with next to no weights, 5.2 with a
// cluster).  Measured, NVFP4, matrices of x, copy bandwidth 6.68 TB/s:
//   7 x 2560 x 200000    51 us, 5.7 TB/s        7 x 2560 x 50257     17 us, 4.2 TB/s (393 tiles: three
//   16 x 2560 x 8192     6.8 us                 rounds of 152 SMs, the last with 89 of them)
//   504 x 4096 x 1024 (MXFP4, four CTAs a tile)   8.8 us
#include <math.h>

#include "fp4_mma.cuh"
#include "fp4_quantize.cuh"

using namespace moe::tc;
using namespace fp4;

namespace {

constexpr int kThreads = 192;  // warps 0-3: epilogue; 4: copies; 5: MMA
constexpr int kTmaWarp = 4, kMmaWarp = 5;
constexpr int kMaxRaw = 32768, kMaxRawRows = 2;  // elements and rows of x that every CTA quantises for itself

template <int FMT, int BN_, bool HELD>
struct Cfg {
  static constexpr int BN = BN_;                               // rows of x of a tile
  static constexpr bool NV = FMT == MOE_FMT_NVFP4;
  static constexpr int COPIES = NV ? 4 : 2;                    // tiles of scales of a chunk
  static constexpr int W_BYTES = 128 * 128, X_BYTES = BN * 128, S_BYTES = COPIES * 512;
  static constexpr int X_PART = X_BYTES + S_BYTES;             // a chunk of x with its scales
  static constexpr int SLOT = W_BYTES + S_BYTES + (HELD ? 0 : X_PART);
  static constexpr int MOST = 10;                              // slots
  static constexpr int S_COLS = COPIES * 4;                    // TMEM columns of a chunk's scales, of either side
  // TMEM holds two tiles' sums, and the scales of as many chunks as the ring: where a
  // slot's copies have landed, the products that took the scales before it have been made.
  static constexpr int SUMS = BN <= 32 ? 32 : BN, S_COL = 2 * SUMS;
  static_assert(SLOT % 1024 == 0 && X_PART % 1024 == 0, "the swizzle's alignment");
  static constexpr int slots_of(int bytes) {
    const int n = bytes / SLOT, m = (512 - S_COL) / (2 * S_COLS);
    return n < m ? (n < MOST ? n : MOST) : (m < MOST ? m : MOST);
  }
};

struct Control {
  uint64_t full[10], empty[10], sums_full[2], sums_empty[2], x_full, drain;
  uint32_t tmem;
  int abort;
  uint32_t row_top[4][kMaxRawRows];
  // factors of the CTA's rows of x, and with a cluster of its tile's columns of y
  alignas(16) float x_row[128];
  alignas(16) float w_row[128], bias[128];
};
constexpr int kRoom = 227 * 1024 - 1024 - (int)sizeof(Control);  // for the ring and the held rows

// Quantises all of x for the CTA's chunks c0 .. c1 - 1, as fp4_quantize does, with the four
// epilogue warps: all on one row, two on each of two.
template <int FMT, int TYPE>
__device__ void hold_raw(const LinearArgs& a, Control& ctl, uint8_t* held, int part, int x_bytes, int c0, int c1) {
  constexpr bool NV = FMT == MOE_FMT_NVFP4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  static_assert(kMaxRawRows == 2, "the warps' shares");
  const int share = a.t == 1 ? 4 : 2, mine = warp % share, t = warp / share;  // warps of a row, which of them, the row
  const int first = (mine * 32 + lane) * 8, width = share * 256;
  auto load = [&](int col, float(&v)[8]) {
    Raw<TYPE> raw;
    if (col < a.cols) raw.load(a.raw.data, t * a.raw.stride + col);
    else raw.zero();
    raw.floats(v);
  };
  RowScale scale;
  if (NV) {
    uint32_t top = 0;
#pragma unroll 4
    for (int col = first; col < a.cols; col += width) {
      float v[8];
      load(col, v);
      const float b = max_abs(max_abs(v[0], v[1], v[2]), max_abs(v[3], v[4], v[5]), max_abs(v[6], v[7], 0.f));
      top = max(top, __float_as_uint(b));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) ctl.row_top[mine][t] = top;
    named_sync(1, 128);
    for (int k = 0; k < share; ++k) top = max(top, ctl.row_top[k][t]);
    scale = row_scale(top);
  }
  if (mine == 0 && lane == 0) ctl.x_row[t] = scale.value();
  const int end = min(c1 * kChunk, (a.cols + 63) / 64 * 64);  // whole words of NVFP4's scales
#pragma unroll 4
  for (int from = c0 * kChunk; from < end; from += width) {
    const int col = from + first;
    float v[8];
    load(col, v);
    uint32_t top = block_top<NV>(v), word[1];
    if (NV && scale.tiny) scale_first(scale, v, top);
    const uint32_t four = quantize<NV>(v, top, scale, lane, col < a.cols, word);
    if (col >= c1 * kChunk) continue;
    uint8_t* at = held + (size_t)(col / kChunk - c0) * part;
    const int b = col % kChunk / 2;  // byte of the row's 128
    *reinterpret_cast<uint32_t*>(at + t * 128 + (((b >> 4) ^ (t & 7)) << 4) + (b & 15)) = word[0];
    if ((lane & (kScaleLanes<NV, 8> - 1)) == 0)
      *reinterpret_cast<uint32_t*>(at + x_bytes + col % kChunk / (8 * kScaleLanes<NV, 8>) * 512 + t * 16) = four;
  }
  fence_proxy_async();
  named_sync(1, 128);
}

// Grid: min(SMs, tiles) CTAs, or split * tiles in clusters of `split`; tiles = ceil(n / 128)
// * ceil(t / BN).
template <int FMT, int BN, bool HELD>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ LinearArgs a, int split,
                                                            int slots, int tmem_columns) {
  using C = Cfg<FMT, BN, HELD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (the rank in the cluster, by an expression that the compiler knows to be the same for the
  // warp: with a loop whose bounds it did not, what the MMA warp issues took four times as long)
  const int rank = blockIdx.x % split;
  const int t_tiles = (a.t + BN - 1) / BN, all = (a.n + 127) / 128 * t_tiles;
  const int first = blockIdx.x / split, step = gridDim.x / split;
  const int chunks = (a.cols + kChunk - 1) / kChunk;
  const int c0 = chunks * rank / split, c1 = chunks * (rank + 1) / split;
  const int tiles = scale_tiles(a.cols, FMT);
  uint8_t* held = ring + (size_t)slots * C::SLOT;
  Control& ctl = *reinterpret_cast<Control*>(held + (HELD ? (size_t)(c1 - c0) * C::X_PART : 0));
  auto n_of = [&](int tile) { return tile / t_tiles * 128; };
  auto t_of = [&](int tile) { return tile % t_tiles * BN; };

  // copies of a chunk of w; all of the slot's are announced
  auto load_w = [&](int slot, int tile, int c) {
    const uint32_t at = smem_u32(ring + (size_t)slot * C::SLOT);
    const int kt = c * C::COPIES, bytes = min(C::COPIES, tiles - kt) * 512;
    mbar_arrive_expect_tx(&ctl.full[slot], C::W_BYTES + bytes + (HELD ? 0 : C::X_BYTES + bytes));
    load_codes(&a.w_map, at, &ctl.full[slot], c * (kChunk / 2), n_of(tile));
    bulk_g2s(at + C::W_BYTES, a.w_scales + ((size_t)(n_of(tile) >> 7) * tiles + kt) * 512, bytes, &ctl.full[slot]);
  };
  auto load_x = [&](uint32_t at, uint64_t* bar, int tile, int c) {
    const int kt = c * C::COPIES, bytes = min(C::COPIES, tiles - kt) * 512;
    load_codes(&a.x_map, at, bar, c * (kChunk / 2), t_of(tile));
    bulk_g2s(at + C::X_BYTES, a.x_scales + ((size_t)(t_of(tile) >> 7) * tiles + kt) * 512, bytes, bar);
  };
  const int ahead = a.early ? min(slots, c1 - c0) : 0;  // chunks whose part of w does not wait
  if (threadIdx.x == 32 * kTmaWarp) {
    for (int i = 0; i < slots; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.sums_full[i], 1 + a.extra);
      mbar_init(&ctl.sums_empty[i], 4);
    }
    mbar_init(&ctl.x_full, 1);
    mbar_init(&ctl.drain, 1);
    ctl.abort = 0;
    mbar_fence_init();
    attn::prefetch_map(&a.w_map);
    if (!a.raw.data) attn::prefetch_map(&a.x_map);
    for (int i = 0; i < ahead; ++i) load_w(i, first, c0 + i);
  }
  // TMEM is taken only when the kernel before has ended, and before the next one may
  // start: CTAs that wait for one another's kernels never hold what the others need.
  moe::pdl_wait();
  if (warp == kMmaWarp) tmem_alloc(&ctl.tmem, tmem_columns);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  moe::pdl_launch_dependents();
  const uint32_t tmem = ctl.tmem;
  volatile int* abort_flag = &ctl.abort;

  if (warp == kTmaWarp) {
    if (lane == 0) {
      bool alive = true;
      if (HELD && !a.raw.data) {
        uint32_t bytes = 0;
        for (int c = c0; c < c1; ++c) bytes += C::X_BYTES + min(C::COPIES, tiles - c * C::COPIES) * 512;
        mbar_arrive_expect_tx(&ctl.x_full, bytes);
        for (int c = c0; c < c1; ++c) load_x(smem_u32(held + (size_t)(c - c0) * C::X_PART), &ctl.x_full, first, c);
      }
      int filled = 0, slot = 0;
      uint32_t round = 1;
      for (int tile = first; tile < all && alive; tile += step)
        for (int c = c0; c < c1; ++c, ++filled) {
          alive = attn::bounded_wait(&ctl.empty[slot], round, a.wait_cycles, abort_flag, a.st);
          if (!alive) break;
          if (filled >= ahead) load_w(slot, tile, c);
          if (!HELD) load_x(smem_u32(ring + (size_t)slot * C::SLOT) + C::W_BYTES + C::S_BYTES, &ctl.full[slot], tile, c);
          if (++slot == slots) slot = 0, round ^= 1;
        }
      // every copy has landed before the CTA's shared memory goes away
      for (int i = max(0, filled - slots); i < filled; ++i)
        attn::bounded_wait(&ctl.full[i % slots], (i / slots) & 1, attn::kDrainCycles, nullptr, a.st);
      if (HELD && !a.raw.data) attn::bounded_wait(&ctl.x_full, 0, attn::kDrainCycles, nullptr, a.st);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // (the warp walks and waits as one, its elected lane issues; see fp4_linear_wide.cu)
    const bool leader = attn::elect_lane();
    const uint64_t w_desc = sw128_kmajor_desc(smem_u32(ring)), ws_desc = scales_desc(smem_u32(ring) + C::W_BYTES);
    const uint32_t x_at = HELD ? smem_u32(held) : smem_u32(ring) + C::W_BYTES + C::S_BYTES;
    const uint64_t x_desc = sw128_kmajor_desc(x_at), xs_desc = scales_desc(x_at + C::X_BYTES);
    bool alive = !HELD || __all_sync(0xffffffffu, attn::bounded_wait(&ctl.x_full, 0, a.wait_cycles, abort_flag, a.st));
    int slot = 0, done = 0;
    uint32_t round = 0;
    for (int tile = first; tile < all && alive; tile += step, ++done) {
      const int place = done & 1;
      if (done >= 2)
        alive = __all_sync(0xffffffffu, attn::bounded_wait(&ctl.sums_empty[place], ((done >> 1) - 1) & 1, a.wait_cycles,
                                                           abort_flag, a.st));
      for (int c = c0; c < c1 && alive; ++c) {
        alive = __all_sync(0xffffffffu, attn::bounded_wait(&ctl.full[slot], round, a.wait_cycles, abort_flag, a.st));
        if (!alive) break;
        fence_after_sync();
        if (leader) {
          const uint32_t off = (uint32_t)slot * (C::SLOT >> 4);
          const uint32_t x_off = HELD ? (uint32_t)(c - c0) * (C::X_PART >> 4) : off;
          const uint32_t set = tmem + C::S_COL + slot * 2 * C::S_COLS, sums = tmem + place * C::SUMS;
          const int steps = min(kChunk, a.cols - c * kChunk + 63) / 64;
#pragma unroll
          for (int k = 0; k < kChunk / 64; ++k) {
            if (k >= steps) break;
            const int copy = C::NV ? k : k / 2, id = C::NV ? 0 : 2 * (k & 1);
            const uint32_t sw = set + 4 * copy, sx = sw + C::S_COLS;
            if (id == 0) {
              copy_scales<1>(sw, ws_desc + off + copy * 32);
              copy_scales<1>(sx, xs_desc + x_off + copy * 32);
            }
            mma_fp4<FMT, 1>(sums, w_desc + off + 2 * k, x_desc + x_off + 2 * k, idesc_fp4<FMT>(128, BN, id), sw, sx,
                            c > c0 || k > 0);
          }
          mma_commit(&ctl.empty[slot]);
          if (c == c1 - 1) mma_commit(&ctl.sums_full[place]);
        }
        __syncwarp();
        if (++slot == slots) slot = 0, round ^= 1;
      }
    }
    // TMEM and the ring go back only when every MMA has completed
    if (leader) {
      mma_commit(&ctl.drain);
      attn::bounded_wait(&ctl.drain, 0, attn::kDrainCycles, nullptr, a.st);
    }
    __syncwarp();
  } else {
    if (HELD && a.raw.data) {
      if (a.raw.type == FP4_BF16) hold_raw<FMT, FP4_BF16>(a, ctl, held, C::X_PART, C::X_BYTES, c0, c1);
      else if (a.raw.type == FP4_FP16) hold_raw<FMT, FP4_FP16>(a, ctl, held, C::X_PART, C::X_BYTES, c0, c1);
      else hold_raw<FMT, FP4_FP32>(a, ctl, held, C::X_PART, C::X_BYTES, c0, c1);
      if (threadIdx.x == 0) mbar_arrive(&ctl.x_full);
    }
    // The factors are fetched while the sums are awaited: one load for each row of x behind them
    // took 40 ns a row, and the columns' behind a cluster's exchange a trip to HBM.  (All of
    // the CTA's tiles have the same rows of x: more than one tile of them goes to clusters only.)
    if (!a.raw.data && threadIdx.x < BN) {
      const int t = t_of(first) + threadIdx.x;
      ctl.x_row[threadIdx.x] = a.x_row && t < a.t ? __ldg(a.x_row + t) : 1.f;
    }
    if (split > 1) {
      const int n = n_of(first) + threadIdx.x;
      ctl.w_row[threadIdx.x] = a.w_row && n < a.n ? __ldg(a.w_row + n) : 1.f;
      ctl.bias[threadIdx.x] = a.bias && n < a.n ? __ldg(a.bias + n) : 0.f;
    }
    named_sync(1, 128);
    bool alive = true;
    int done = 0;
    for (int tile = first; tile < all; tile += step, ++done) {
      const int place = done & 1, n = n_of(tile) + threadIdx.x, t0 = t_of(tile);
      float scale = a.w_row && n < a.n ? __ldg(a.w_row + n) : 1.f;
      const float add = a.bias && n < a.n ? __ldg(a.bias + n) : 0.f;
      alive = alive && __all_sync(0xffffffffu, attn::bounded_wait(&ctl.sums_full[place], (done >> 1) & 1, a.wait_cycles,
                                                                  abort_flag, a.st));
      fence_after_sync();
      if (split > 1) break;  // (of one tile; below)
      if (!alive) scale = kNaN;
      const uint32_t sums = tmem + place * C::SUMS + ((uint32_t)(warp * 32) << 16);
      const int rows = min(BN, a.t - t0);
      uint8_t* y = static_cast<uint8_t*>(a.y) + (t0 * a.y_stride + n) * element_bytes(a.y_type);
      const long long next = a.y_stride * element_bytes(a.y_type);
#pragma unroll 1
      for (int j = 0; j < rows; j += 16) {
        uint32_t r[16];
        tmem_ld16(sums + j, r);
        tmem_ld_wait();
        if (j + 16 >= rows) {  // the tile's sums have been read
          fence_before_sync();
          __syncwarp();
          if (lane == 0 && alive) mbar_arrive(&ctl.sums_empty[place]);
        }
        float row[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(row + 4 * i) = *reinterpret_cast<const float4*>(ctl.x_row + j + 4 * i);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (j + i >= rows || n >= a.n) break;
          store_one(y + (j + i) * next, 0, a.y_type, fmaf(__uint_as_float(r[i]) * row[i], scale, add));
        }
      }
    }
  }
  if (split > 1) {
    __syncthreads();  // no copy is under way any more, and nobody gives up from here on
    const bool ok = !*abort_flag;
    if (warp < 4) {
      const uint32_t sums = tmem + ((uint32_t)(warp * 32) << 16);
      float* part = reinterpret_cast<float*>(ring);  // [BN][128], where the chunks were
#pragma unroll 1
      for (int j = 0; j < BN; j += 16) {
        uint32_t r[16];
        tmem_ld16(sums + j, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(j + i) * 128 + threadIdx.x] = ok ? __uint_as_float(r[i]) : kNaN;
      }
      fence_before_sync();
    }
    cluster_sync();
    // A thread adds up 4 columns of y of a row of x; 4 of those at a time, as a word of
    // another CTA is some 500 cycles away (128 rows of x, 2 CTAs: one at a time took 20 us).
    const int n0 = n_of(first), t0 = t_of(first);
    const int q0 = BN * rank / split * 32, q1 = min(BN * (rank + 1) / split, a.t - t0) * 32;
    const int item = element_bytes(a.y_type);
    constexpr int U = 4;
    for (int q = q0 + threadIdx.x; q < q1; q += U * kThreads) {
      float4 v[U] = {};
      for (int k = 0; k < split; ++k) {
        float4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = peer_float4(smem_u32(ring) + (uint32_t)min(q + u * kThreads, q1 - 1) * 16, k);
#pragma unroll
        for (int u = 0; u < U; ++u) v[u].x += w[u].x, v[u].y += w[u].y, v[u].z += w[u].z, v[u].w += w[u].w;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = q + u * kThreads, j = at >> 5, n = n0 + (at & 31) * 4;
        if (at >= q1) break;
        const float row = ctl.x_row[j];
        const float4 scale = *reinterpret_cast<const float4*>(ctl.w_row + (at & 31) * 4);
        const float4 add = *reinterpret_cast<const float4*>(ctl.bias + (at & 31) * 4);
        const uint32_t out[4] = {__float_as_uint(fmaf(v[u].x * row, scale.x, add.x)),
                                 __float_as_uint(fmaf(v[u].y * row, scale.y, add.y)),
                                 __float_as_uint(fmaf(v[u].z * row, scale.z, add.z)),
                                 __float_as_uint(fmaf(v[u].w * row, scale.w, add.w))};
        uint8_t* y = static_cast<uint8_t*>(a.y) + ((t0 + j) * a.y_stride + n) * item;
        if (((uintptr_t)y & (4 * item - 1)) == 0 && n + 4 <= a.n) {
          if (item == 4) {
            *reinterpret_cast<uint4*>(y) = make_uint4(out[0], out[1], out[2], out[3]);
          } else {
            auto two = [&](int e) {
              const float lo = __uint_as_float(out[e]), hi = __uint_as_float(out[e + 1]);
              return a.y_type == FP4_BF16 ? attn::Brain::down(lo, hi) : attn::Half::down(lo, hi);
            };
            *reinterpret_cast<uint2*>(y) = make_uint2(two(0), two(2));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < a.n) store_one(y, e, a.y_type, __uint_as_float(out[e]));
        }
      }
    }
    cluster_sync_relaxed();  // the others have read this CTA's part
  }
  fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, tmem_columns);
}

constexpr size_t kHalf = 113 * 1024;  // of an SM's shared memory: two CTAs find room

// How many clusters of 2, 4 or 8 CTAs with so much shared memory run at the same time: a
// GPC's SMs need not be a multiple of four (of 152 SMs, with one CTA to each, 36
// clusters of 4 and 15 of 8; 512 x 2048 x 512 with 16 clusters of 8 took 13.9 us, not 7.3).  Looked up
// once per device, for a kernel of its own: the others' grants of shared memory differ.
__global__ void __launch_bounds__(kThreads, 1) nothing_kernel() {}
int clusters_at_once(int split, bool half) {
  static std::atomic<int> known[moe::kMaxDevices][2][3];
  static moe::SmemGrant grant;
  const int d = moe::current_device();
  if (d < 0) return 0;
  std::atomic<int>& entry = known[d][half][split >> 2];
  int n = entry.load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (!moe::grant_smem(nothing_kernel, 2 * kHalf, grant)) return 0;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(split);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = half ? kHalf : 2 * kHalf;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, nothing_kernel, &cfg) != cudaSuccess) return 0;
  entry.store(n, std::memory_order_relaxed);
  return n;
}

// What a launch takes.
template <int FMT, int BN, bool HELD>
struct Plan {
  using C = Cfg<FMT, BN, HELD>;
  int split, clusters, slots, columns;
  size_t smem;

  // Over how many CTAs a tile's columns are split: as many as still give each tile a
  // cluster of its own at the same time.  With up to 16 rows of x the exchange takes as long as three
  // chunks, and that many have to go elsewhere (one CTA against two, 1 x 8192 columns of y:
  // 3 chunks 4.2 and 5.2 us, 6 chunks 5.7 and 5.7, 10 chunks 8.1 and 6.7); with more the cluster shares
  // the rows' epilogue too (32 rows: 2 chunks 4.7 and 4.7, 6 chunks 6.7 and 5.7).
  Plan(const LinearArgs& a, int sms) {
    const int chunks = chunks_of(a);
    const long long tiles = tiles_of(a);
    set(a, 1, sms);
    for (int k = 2; k <= 8 && 2 * split <= chunks && tiles * k <= sms; k *= 2) {
      Plan next = *this;
      next.set(a, k, sms);
      if (tiles > clusters_at_once(k, next.smem <= kHalf)) break;
      *this = next;
    }
    if (BN <= 16 && chunks - (chunks + split - 1) / split < 3) set(a, 1, sms);
  }
  static int chunks_of(const LinearArgs& a) { return (a.cols + kChunk - 1) / kChunk; }
  static long long tiles_of(const LinearArgs& a) { return (long long)((a.n + 127) / 128) * ((a.t + BN - 1) / BN); }

 private:
  void set(const LinearArgs& a, int split_, int sms) {
    split = split_;
    const int most = (chunks_of(a) + split - 1) / split;  // chunks of a CTA
    const long long tiles = tiles_of(a);
    clusters = (int)(tiles < sms / split ? tiles : sms / split);
    const int held = HELD ? most * C::X_PART : 0;
    slots = held < kRoom ? C::slots_of(kRoom - held) : 0;
    // no more than a CTA's tiles have chunks, but room for the sums that a cluster exchanges
    const long long work = (tiles + clusters - 1) / clusters * most;
    const int least = split > 1 ? (BN * 512 + C::SLOT - 1) / C::SLOT : 1;
    if (slots > work) slots = (int)(work < least ? least : work);
    // Two CTAs on an SM, of clusters in two streams, must not wait for each other's TMEM: as
    // many as shared memory lets in have to find theirs.  So half of TMEM goes with half of
    // the shared memory or more, and all of it with more than half.
    smem = 1024 + (size_t)slots * C::SLOT + held + sizeof(Control);
    columns = smem <= kHalf && C::S_COL + slots * 2 * C::S_COLS <= 256 ? 256 : 512;
    if (smem <= kHalf) smem = columns == 256 ? kHalf : kHalf + 1024;
  }
};

template <int FMT, int BN, bool HELD>
int launch(LinearArgs& a, const fp4_matrix* x, const fp4_matrix& w, const Plan<FMT, BN, HELD>& p, cudaStream_t st) {
  static moe::SmemGrant grant;
  if (p.tiles_of(a) > 0x3FFFFFFF) return MOE_ERR_UNSUPPORTED;
  if (const int rc = codes_map(w, 128, &a.w_map)) return rc;
  if (x)
    if (const int rc = codes_map(*x, BN, &a.x_map)) return rc;
  if (!moe::grant_smem(linear_kernel<FMT, BN, HELD>, p.smem, grant)) return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.clusters * p.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, linear_kernel<FMT, BN, HELD>, a, p.split, p.slots, p.columns) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

// Whether the rows of x stay in shared memory: up to 16, if they leave a ring of six slots.
template <int FMT>
bool holds(const LinearArgs& a, const Plan<FMT, 16, true>& p) {
  using C = Cfg<FMT, 16, true>;
  return a.t <= 16 && C::slots_of(kRoom - (p.chunks_of(a) + p.split - 1) / p.split * C::X_PART) >= 6;
}
bool holds(const LinearArgs& a, int format, int sms) {
  return format == MOE_FMT_NVFP4 ? holds<MOE_FMT_NVFP4>(a, {a, sms}) : holds<MOE_FMT_MXFP4>(a, {a, sms});
}

// x NULL: a.raw, which is held.
template <int FMT>
int launch(LinearArgs& a, const fp4_matrix* x, const fp4_matrix& w, int sms, cudaStream_t st) {
  if (a.t <= 16) {
    const Plan<FMT, 16, true> p(a, sms);
    if (holds<FMT>(a, p)) return launch(a, x, w, p, st);
  }
  if (!x) return MOE_ERR_UNSUPPORTED;  // (no call gets here)
  if (a.t <= 16) return launch<FMT, 16, false>(a, x, w, {a, sms}, st);
  if (a.t <= 32) return launch<FMT, 32, false>(a, x, w, {a, sms}, st);
  if (a.t <= 64) return launch<FMT, 64, false>(a, x, w, {a, sms}, st);
  // More rows: pairs of CTAs, unless there are so few tiles that each can have four CTAs or more, and
  // columns enough to share (504 x 8192 x 1024: 10.8 us against 13.9 of the pairs, 512 x 2048 x 512 7.3
  // and 7.7, 504 x 1024 x 1024 7.2 and 6.7; with two to a tile the pairs are faster, 1024 x 4096
  // x 1024 11.9 and 10.8, 96 x 2560 x 8192 10.4 and 9.7, and more so with one, 160 x 2560 x 8192 17.5 and 9.3).
  const Plan<FMT, 128, false> p(a, sms);
  return p.split >= 4 && a.cols > 7 * kChunk ? launch(a, x, w, p, st) : launch_wide(a, *x, w, sms, st);
}

// Where fp4_linear_rows keeps its quantised rows.
struct Layout {
  size_t scales, row_scale, bytes;
};
Layout layout(int rows, int cols, int format) {
  Layout l;
  l.scales = ((size_t)rows * cols / 2 + 255) & ~(size_t)255;
  l.row_scale = l.scales + fp4_scale_bytes(rows, cols, format);
  l.bytes = l.row_scale + (size_t)rows * sizeof(float);
  return l;
}

int check_output(const Rows& y, int rows, int cols) {
  if (!y.data && rows > 0 && cols > 0) return MOE_ERR_INVALID_ARG;
  if (y.type != FP4_BF16 && y.type != FP4_FP16 && y.type != FP4_FP32) return MOE_ERR_UNSUPPORTED;
  if ((uintptr_t)y.data % element_bytes(y.type)) return MOE_ERR_ALIGNMENT;
  if (rows > 1 && (y.stride < cols || y.stride >= (1ll << 38))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// What the kernels are told, but for x.
LinearArgs arguments(const fp4_matrix& w, const float* bias, const Rows& y, int rows, int32_t* dev_status) {
  LinearArgs a = {};
  a.w_scales = static_cast<const uint8_t*>(w.scales), a.w_row = w.row_scale, a.bias = bias;
  a.n = w.rows, a.t = rows, a.cols = w.cols;
  a.y = y.data, a.y_stride = rows > 1 ? y.stride : 0, a.y_type = y.type;
  a.wait_cycles = attn::wait_cycles(), a.extra = (int)moe::barrier_extra(), a.st = dev_status;
  return a;
}
int launch(LinearArgs& a, const fp4_matrix* x, const fp4_matrix& w, int sms, cudaStream_t st) {
  if (x) a.x_scales = static_cast<const uint8_t*>(x->scales), a.x_row = x->row_scale;
  return w.format == MOE_FMT_NVFP4 ? launch<MOE_FMT_NVFP4>(a, x, w, sms, st) : launch<MOE_FMT_MXFP4>(a, x, w, sms, st);
}

}  // namespace

extern "C" {

int fp4_linear(const fp4_matrix* x, const fp4_matrix* w, const float* bias, void* y, long long y_stride, int y_type,
               int32_t* dev_status, void* stream) {
  if (const int rc = check_matrix(x)) return rc;
  if (const int rc = check_matrix(w)) return rc;
  if (x->cols != w->cols || x->format != w->format) return MOE_ERR_INVALID_ARG;
  const Rows out = rows_of(y, y_stride, y_type);
  if (const int rc = check_output(out, x->rows, w->rows)) return rc;
  if ((uintptr_t)bias & 3u) return MOE_ERR_ALIGNMENT;
  if (x->rows == 0 || w->rows == 0) return MOE_OK;
  const Span outs[] = {span_of(out, x->rows, w->rows, false), piece(dev_status, 4)};
  const Span ins[] = {codes_span(*x), scales_span(*x), row_scale_span(*x),
                      codes_span(*w), scales_span(*w), row_scale_span(*w), piece(bias, 4ll * w->rows)};
  if (!apart(outs, ins)) return MOE_ERR_INVALID_ARG;
  const int sms = moe::device_info().sms;
  if (sms <= 0) return MOE_ERR_CUDA;
  LinearArgs a = arguments(*w, bias, out, x->rows, dev_status);
  return launch(a, x, *w, sms, (cudaStream_t)stream);
}

size_t fp4_linear_rows_workspace(const fp4_matrix* w, int rows) {
  if (!w || rows < 0 || !shape_ok(rows, w->cols, w->format)) return 0;
  return layout(rows, w->cols, w->format).bytes + 16;
}

int fp4_linear_rows(const void* x, long long x_stride, int x_type, int rows, const fp4_matrix* w, const float* bias,
                    void* y, long long y_stride, int y_type, void* workspace, size_t ws_bytes, int32_t* dev_status,
                    void* stream) {
  if (rows < 0) return MOE_ERR_INVALID_ARG;
  if (const int rc = check_matrix(w)) return rc;
  if (!shape_ok(rows, w->cols, w->format)) return MOE_ERR_UNSUPPORTED;
  const Rows in = rows_of(x, x_stride, x_type), out = rows_of(y, y_stride, y_type);
  if (const int rc = check_rows(in, rows, w->cols, true)) return rc;
  if (const int rc = check_output(out, rows, w->rows)) return rc;
  if ((uintptr_t)bias & 3u) return MOE_ERR_ALIGNMENT;
  if (rows == 0 || w->rows == 0) return MOE_OK;
  if (!workspace) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned16(workspace)) return MOE_ERR_ALIGNMENT;
  const Layout l = layout(rows, w->cols, w->format);
  if (ws_bytes < l.bytes) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const Span outs[] = {span_of(out, rows, w->rows, false), piece(workspace, (long long)l.bytes), piece(dev_status, 4)};
  const Span ins[] = {span_of(in, rows, w->cols, false), codes_span(*w), scales_span(*w), row_scale_span(*w),
                      piece(bias, 4ll * w->rows)};
  if (!apart(outs, ins)) return MOE_ERR_INVALID_ARG;
  const int sms = moe::device_info().sms;
  if (sms <= 0) return MOE_ERR_CUDA;
  LinearArgs a = arguments(*w, bias, out, rows, dev_status);
  if (rows <= kMaxRawRows && rows * w->cols <= kMaxRaw && holds(a, w->format, sms)) {
    a.raw = in;
    if (rows == 1) a.raw.stride = 0;
    return launch(a, nullptr, *w, sms, (cudaStream_t)stream);
  }
  uint8_t* at = static_cast<uint8_t*>(workspace);
  const fp4_matrix m = {at, at + l.scales,
                        w->format == MOE_FMT_NVFP4 ? reinterpret_cast<float*>(at + l.row_scale) : nullptr, rows,
                        w->cols, w->format};
  if (const int rc = fp4_quantize(x, x_stride, x_type, &m, stream)) return rc;
  a.early = 1;  // the kernel before writes x alone, and has waited for those before it
  return launch(a, &m, *w, sms, (cudaStream_t)stream);
}

}  // extern "C"
