// Attention of the tokens in flight over a paged cache, on the 5th-generation
// tensor cores.
//
// Rows (token in flight x query head of a KV head) are the M side of both
// products; a piece of work is up to 256 rows against a run of key tiles:
//
//   S = Q . K^T            Q in shared memory, K tile by TMA        -> TMEM
//   P = exp2(S c - m)      one thread per row: running maximum and sum -> TMEM (16 bits)
//   O += P . V             P from TMEM, V tile by TMA               -> TMEM
//
// What bounds it: K and V are read once per 256 rows (128 for wide heads), so a
// few rows are HBM bound, whatever part of the 128 MMA rows they fill (a tile of
// 128 keys is 64 KB at D = 128: about 2800 cycles of an SM's share of HBM, and 1024
// of MMA); from some 200 rows the MMAs and the exponentials bound it.
//
// Measured, BF16 (copy bandwidth 6.69 TB/s, library GEMM 1.90 PFLOP/s):
//   32 sequences of 16384 slots, 4 x 8 heads of 128  177 us, 6.1 TB/s
//   32 ragged ones of 1024 .. 8192, the same         72 us, 4.4 TB/s
//   8 of 16384, 504 rows, D = 128                   125 us, 1.08 PFLOP/s
//   1 of 300001, 136 rows, D = 256 (FP16)           166 us, 3.7 TB/s
//   1 of 1000, 4 rows, D = 128                       16 us
// Of the ragged batch's time some 20 us do not grow with the bytes: launch, plan and
// first loads 6 to 8, changes of piece 2 to 5, the join 8 to 11.  With 504 rows the tensor pipe is active
// for half of the time: an MMA of Q and K takes 85 cycles (65 alone, with no copies
// into the shared memory that both operands come from), one of P and V 70; taking out
// the exponentials and maxima gains 2 us, halving either product 10.  With wide heads
// and a second row group K and V come from L2 twice, 8.2 TB/s in all, and neither the
// products nor the softmax show in the time.
//
// Two streams of tiles run through one CTA, each with its own S and O in TMEM
// and its own warpgroup, so that one's softmax runs under the other's MMAs.
// With more than 128 rows the streams are the two halves of the rows over the
// same keys; otherwise they are the even and the odd key tiles over the same
// rows, and their O, m, l are joined at the end of the piece.  Heads wider
// than 128 leave TMEM for one O: one stream with two S buffers.
//
// The MMAs are issued S(i + 1) before O(i), so a softmax always has the other
// tile's S product running beside it.  The running maximum moves only when a
// row's scores outgrow it by kLag (in powers of two): O is rescaled rarely.
// For FP16 the weights carry a factor 2^kLift, which keeps those down to
// 2^-24 of the largest out of FP16's subnormals; it cancels with the sum.
//
// Work division: attn_plan.h.  Pieces of a divided unit go to the workspace
// (unscaled O, m, l) and join_kernel adds them up in their order, so results
// repeat bit for bit.
//
// What a row must not see: scores are replaced by -inf, and values that could
// reach the product with weight 0 (slots past the end of the sequence, NaN or
// infinite elements of drafts) are zeroed in shared memory; the latter are put
// back, for the rows that do see them, when the piece is written.
#include "attn_tma.cuh"
#include "attn_work.cuh"

using namespace moe::tc;

namespace {

// Warps 0-3, 4-7: softmax of streams 0, 1; 8: TMA; 9: MMA (10, 11 fill up the
// warpgroup, whose registers go to the other two: they hold a row of S each, and
// spilling a few of them cost 10% of the whole kernel's time).
constexpr int kThreads = 384;
constexpr int kRegsSoftmax = 208;
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr float kNaN = __builtin_nanf("");

struct TreeArgs {
  const void* q;
  long long q_stride;
  const int32_t *cu, *lens;
  int tokens, q_heads;
  const uint64_t* tree;
  int tree_words;
  float scale;
  attn_cache c;
  attn::Maps maps;
  long long wait_cycles;
  int extra;  // arrivals that never come, on p_full
  void* out;
  float* lse;
  int32_t* st;
  struct Split* splits;  // [parts]
  float* ml;             // [parts][2][rows][2]
  float4* o;             // [parts][2][DP / 4][rows]
};

// The divided unit whose first piece ends part c, if there is one.
struct Split {
  int pieces;  // 0: none
  int first, n, head, row0, rows;
};

template <int DP_>
struct Cfg {
  static constexpr int DP = DP_;
  static constexpr int STREAMS = DP <= 128 ? 2 : 1;
  static constexpr int BN = DP <= 128 ? 128 : 64;      // keys of a tile
  static constexpr int ROWS = 128 * STREAMS;           // rows of a unit
  static constexpr int SLOT = BN * DP * 2;             // bytes of a K or V tile
  static constexpr int SLOTS = DP == 64 ? 10 : 5;
  static constexpr int QTILE = 128 * DP * 2;
  static constexpr int PANEL = BN * 128;               // 64 elements of a tile's rows
  static constexpr int S_COL = 0, O_COL = 2 * BN;      // S buffers, then O of each stream
  static constexpr int TMEM = 512;
  // fetching the rows and writing the result: some 8000 cycles, of which a tile
  // takes 2700 (1400 at half the width)
  static constexpr int UNIT_COST = DP == 64 ? 5 : 3;
  static constexpr int REGS_OTHER = STREAMS == 2 ? 88 : 144;  // of a warpgroup that runs no softmax
  static_assert(STREAMS * kRegsSoftmax + (3 - STREAMS) * REGS_OTHER <= 3 * 168, "168 registers a thread at launch");
  static_assert(O_COL + STREAMS * DP <= TMEM, "TMEM");
  static constexpr size_t OFF_Q = 0;
  static constexpr size_t OFF_RING = OFF_Q + (size_t)STREAMS * QTILE;
  static constexpr size_t OFF_CTRL = OFF_RING + (size_t)SLOTS * SLOT;
};

struct Control {
  uint64_t full[10], empty[10];
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2];
  uint64_t q_full, qk_done, pv_done, drain;
  attn::Share share;
  uint32_t tmem;
  int abort;
  int bad_page[8];   // piece number, at index piece % 8, that met a bad page
  int dirty[2][8];   // ... whose drafts' values hold NaN or infinity, by cleaning stream
  float2 ml[128];    // stream 1's m and l for the join
};
template <class C>
constexpr size_t smem_bytes() {
  return 1024 + C::OFF_CTRL + sizeof(Control);
}
static_assert(smem_bytes<Cfg<64>>() <= 232448 && smem_bytes<Cfg<128>>() <= 232448 && smem_bytes<Cfg<256>>() <= 232448,
              "shared memory");

template <class E>
struct Weight {  // P = exp2(s - m + kLift), m lagging the maximum by up to kLag
  static constexpr float kLift = 0.f, kLag = 8.f;
};
template <>
struct Weight<attn::Half> {
  static constexpr float kLift = 10.f, kLag = 5.f;
};

template <class C>
__device__ __forceinline__ attn::PlanDims plan_dims(const TreeArgs& a) {
  // A piece of R rows writes and reads back R * D * 8 bytes, as much as R / 64 tiles
  // at D = 128: pieces of many rows are not cut as short as those of few.
  const int G = a.q_heads / a.c.kv_heads;
  const long long rows = (long long)a.tokens * G / a.c.batch;  // of an average sequence
  const int least = 1 + (int)(rows < C::ROWS ? rows : C::ROWS) / 64;
  return attn::PlanDims{a.c.kv_heads, G, C::ROWS, C::BN, C::UNIT_COST, least};
}

// Adds the NaN and infinite elements of a piece's drafts, which the products
// took as zeros, to the result of a row that sees them.  `skip`: slots of the tiles
// that another stream took, of every two tiles from slot k0 on (-1: none).
// Element d of the row is out[(d / 4) * step + d % 4].
template <int BN, class T, class O>
__device__ __noinline__ void put_back(const TreeArgs& a, attn::Seq s, int b, int head, int token, int d0, int d1,
                                      int k0, int skip, O* out, int step) {
  for (int dr = d0; dr < d1; ++dr) {
    if ((((s.len + dr - k0) / BN) & 1) == skip) continue;
    const long long off = attn::slot_offset(a.c, b, s.len + dr, head);
    if (off < 0 || !(attn::seen(a.tree, a.tree_words, s, token, s.len + dr) & 1u)) continue;
    const T* v = static_cast<const T*>(a.c.v) + off;
    for (int d = 0; d < a.c.head_dim; ++d) {
      const float e = (float)v[d];
      if (!isfinite(e)) out[d / 4 * step + d % 4] = (O)((float)out[d / 4 * step + d % 4] + e);
    }
  }
}

template <class E, int DP>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const __grid_constant__ TreeArgs a) {
  using C = Cfg<DP>;
  using T = typename E::T;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sRing = smem + C::OFF_RING;
  Control& ctl = *reinterpret_cast<Control*>(smem + C::OFF_CTRL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int D = a.c.head_dim, G = a.q_heads / a.c.kv_heads;
  const int panels = (D + 63) / 64;
  constexpr int kWorkers = 128 * C::STREAMS;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&ctl.s_full[x], 1);
      mbar_init(&ctl.p_half[x], 4);
      mbar_init(&ctl.p_full[x], 4 + a.extra);
      mbar_init(&ctl.o_full[x], 1);
    }
    mbar_init(&ctl.q_full, kWorkers);
    mbar_init(&ctl.qk_done, 1);
    mbar_init(&ctl.pv_done, 1);
    mbar_init(&ctl.drain, 1);
    ctl.abort = 0;
    for (int i = 0; i < 8; ++i) ctl.bad_page[i] = ctl.dirty[0][i] = ctl.dirty[1][i] = -1;
    mbar_fence_init();
    attn::prefetch_map(&a.maps.k);
    attn::prefetch_map(&a.maps.v);
  }
  moe::pdl_wait();
  moe::pdl_launch_dependents();
  const attn::PlanDims dims = plan_dims<C>(a);
  if (!attn::take_share<kThreads>(a.cu, a.lens, a.c.batch, a.tokens, (long long)a.c.max_pages * a.c.page_size, dims, ctl.share)) {  // (its barriers also publish the set-up above)
    if (threadIdx.x == 0) {
      if (blockIdx.x == 0) moe::status_or(a.st, ATTN_DEV_BAD_LENGTH);
      a.splits[blockIdx.x].pieces = 0;
    }
    const long long rows = (long long)a.tokens * a.q_heads, step = (long long)gridDim.x * kThreads;
    const float nan8[8] = {kNaN, kNaN, kNaN, kNaN, kNaN, kNaN, kNaN, kNaN};
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < rows * (D / 8); i += step)
      reinterpret_cast<uint4*>(a.out)[i] = attn::pack8<E>(nan8);
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; a.lse && i < rows; i += step) a.lse[i] = kNaN;
    return;
  }
  if (ctl.share.t0 >= ctl.share.t1) {
    if (threadIdx.x == 0) a.splits[blockIdx.x].pieces = 0;
    return;
  }
  if (warp == kMmaWarp) tmem_alloc(&ctl.tmem, C::TMEM);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = ctl.tmem;
  volatile int* abort_flag = &ctl.abort;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return attn::bounded_wait(bar, parity, a.wait_cycles, abort_flag, a.st);
  };
  // for what a warp does together: it goes on, or gives up, as one
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };

  // A role ends inside its branch: code behind the branches would run with either
  // number of registers.
  auto finish = [&]() {
    fence_before_sync();
    named_sync(0, kThreads);
  };
  if (warp >= 4 * C::STREAMS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHER));
    if (warp == kTmaWarp) {
      // ------------------------------------------------------------- TMA
      // Slots are filled K, V, K, V, ... in key order; lane i issues box i of
      // the tile's at most 32 (8-row boxes of two panels of 128 rows, or four of 64).
      attn::Walk w(a.cu, a.lens, a.c.batch, a.tokens, dims, ctl.share);
      int pos = 0;  // slots filled so far
      bool alive = true;
      const int box_rows = a.maps.box_rows, boxes = C::BN / box_rows;
      const int my_box = lane % boxes, my_panel = lane / boxes;
      while (alive && w.next()) {
        const int end = w.s.len + w.s.n;
        const int32_t* table = a.c.page_table + (size_t)w.b * a.c.max_pages;
        for (int j = w.p.kt0; j < w.p.kt1 && alive; ++j) {
          const int slot0 = j * C::BN, start = slot0 + my_box * box_rows;
          const int issued = min(boxes, (end - slot0 + box_rows - 1) / box_rows);
          int page = 0, row = 0;
          if (my_box < issued) {
            const int pi = start / a.c.page_size;
            page = __ldg(table + pi);
            row = start - pi * a.c.page_size;
            if ((unsigned)page >= (unsigned)a.c.pages) {
              page = a.c.pages;  // past the last: the copy delivers zeros
              ctl.bad_page[w.number & 7] = w.number;
              moe::status_or(a.st, ATTN_DEV_BAD_PAGE);
            }
          }
          __syncwarp();
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++pos) {
            const int slot = pos % C::SLOTS;
            alive = warp_wait(&ctl.empty[slot], ((pos / C::SLOTS) & 1) ^ 1);
            if (!alive) break;
            if (lane == 0) mbar_arrive_expect_tx(&ctl.full[slot], (uint32_t)(issued * box_rows * 128 * panels));
            __syncwarp();
            const uint32_t dst = smem_u32(sRing + (size_t)slot * C::SLOT) + (uint32_t)(my_box * box_rows * 128);
            if (my_box < issued)
              for (int p = my_panel; p < panels; p += 32 / boxes)
                attn::load_box(kv ? &a.maps.v : &a.maps.k, dst + p * C::PANEL, &ctl.full[slot], p * 64, row, w.p.head,
                               page, a.maps.head_inner);
          }
        }
      }
      // every copy has landed before the CTA's shared memory goes away
      if (lane == 0)
        for (int i = max(0, pos - C::SLOTS); i < pos; ++i) {
          attn::bounded_wait(&ctl.full[i % C::SLOTS], (i / C::SLOTS) & 1, attn::kDrainCycles, nullptr, a.st);
        }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ----------------------------------------------------------- MMA
      // The warp walks as one, its elected lane issues.  Every lane waits for itself and
      // they vote once a product, behind its MMAs, whether to go on (a vote after
      // every wait cost 8% of the whole kernel's time).  What it does between
      // the MMAs is kept short: at 128 keys and 128 elements a product takes 512 cycles,
      // and the tensor core idles while the next one's operands are worked out.
      const bool leader = attn::elect_lane();
      attn::Walk w(a.cu, a.lens, a.c.batch, a.tokens, dims, ctl.share);
      int k_slot = 0, k_round = 0, v_slot = 1, v_round = 0, pieces = 0;
      uint32_t p_odd = 0;  // bit x: an odd number of tiles' weights has been taken from S buffer x
      bool alive = true;
      const int k_steps = (D + 15) / 16, full_panels = k_steps / 4, rest = k_steps - 4 * full_panels;
      // a negative scale negates Q, the sums keep |scale|
      const uint32_t id_s = attn::idesc<E>(128, C::BN, false) | (a.scale < 0.f ? 1u << 13 : 0u);
      const uint32_t id_o = attn::idesc<E>(128, (D + 15) & ~15, true);
      const uint64_t q_desc = sw128_kmajor_desc(smem_u32(sQ)), k_desc = sw128_kmajor_desc(smem_u32(sRing));
      const uint64_t v_desc = attn::sw128_mnmajor_desc(smem_u32(sRing), C::PANEL);
      const uint32_t q_low = (uint32_t)q_desc, k_low = (uint32_t)k_desc, k_high = (uint32_t)(k_desc >> 32);
      const uint32_t v_low = (uint32_t)v_desc, v_high = (uint32_t)(v_desc >> 32);
      auto on = [](int& slot, int& round) {  // K and V alternate in the ring
        slot += 2;
        if (slot >= C::SLOTS) slot -= C::SLOTS, ++round;
      };
      while (alive && w.next()) {
        const bool both = C::STREAMS == 2 && w.rows > 128;  // two row tiles over the same keys
        const int tiles = w.p.kt1 - w.p.kt0, items = both ? 2 * tiles : tiles;
        alive = warp_wait(&ctl.q_full, pieces & 1);
        if (!alive) break;
        fence_after_sync();
        auto qk = [&](int it) {
          const int x = it & 1;
          bool ok = true;  // of this lane's waits; the vote behind the MMAs makes it the warp's
          if (!both || x == 0) {
            ok = wait(&ctl.full[k_slot], k_round & 1);
            fence_after_sync();
          }
          if (leader && ok) {
            uint32_t ql = q_low + (both && x ? C::QTILE >> 4 : 0), kl = k_low + (uint32_t)k_slot * (C::SLOT >> 4);
            const uint32_t d = tmem + C::S_COL + x * C::BN;
            uint32_t more = 0;
            for (int p = 0; p < full_panels; ++p, ql += (128 * 128) >> 4, kl += C::PANEL >> 4) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk, more = 1)
                mma_bf16(d, attn::make_desc(k_high, ql + 2 * kk), attn::make_desc(k_high, kl + 2 * kk), id_s, more);
            }
            for (int kk = 0; kk < rest; ++kk, more = 1)
              mma_bf16(d, attn::make_desc(k_high, ql + 2 * kk), attn::make_desc(k_high, kl + 2 * kk), id_s, more);
            mma_commit(&ctl.s_full[x]);
            if (!both || x == 1) mma_commit(&ctl.empty[k_slot]);
            if (it == items - 1) mma_commit(&ctl.qk_done);
          }
          if (!both || x == 1) on(k_slot, k_round);
          return __all_sync(0xffffffffu, ok) != 0;
        };
        auto pv = [&](int it) {
          const int x = it & 1, st = C::STREAMS == 2 ? x : 0;  // whose O
          const uint32_t o = tmem + C::O_COL + st * DP, p = tmem + C::S_COL + x * C::BN;
          const uint32_t vl = v_low + (uint32_t)v_slot * (C::SLOT >> 4), seen = (p_odd >> x) & 1;
          const uint32_t more = it >= C::STREAMS;
          p_odd ^= 1u << x;
          bool ok = (both && x != 0) || wait(&ctl.full[v_slot], v_round & 1);
          ok = ok && wait(&ctl.p_half[x], seen);
          fence_after_sync();
          if (leader && ok) {
#pragma unroll
            for (int kk = 0; kk < C::BN / 32; ++kk)
              attn::mma_ts(o, p + kk * 8, attn::make_desc(v_high, vl + kk * (2048 >> 4)), id_o, kk ? 1 : more);
          }
          __syncwarp();
          ok = ok && wait(&ctl.p_full[x], seen);
          fence_after_sync();
          if (leader && ok) {
#pragma unroll
            for (int kk = C::BN / 32; kk < C::BN / 16; ++kk)
              attn::mma_ts(o, p + kk * 8, attn::make_desc(v_high, vl + kk * (2048 >> 4)), id_o, 1);
            if (!both || x == 1) mma_commit(&ctl.empty[v_slot]);
            if (C::STREAMS == 1) mma_commit(&ctl.pv_done);
            if (it >= items - C::STREAMS) mma_commit(&ctl.o_full[st]);
          }
          if (!both || x == 1) on(v_slot, v_round);
          return __all_sync(0xffffffffu, ok) != 0;
        };
        alive = qk(0);
        for (int it = 0; it < items && alive; ++it) {
          if (it + 1 < items) alive = qk(it + 1);
          alive = alive && pv(it);
        }
        ++pieces;
      }
      // every MMA has completed before TMEM goes back
      __syncwarp();
      if (leader) {
        mma_commit(&ctl.drain);
        attn::bounded_wait(&ctl.drain, 0, attn::kDrainCycles, nullptr, a.st);
      }
      __syncwarp();
    }
    finish();
    if (warp == kMmaWarp) tmem_dealloc(tmem, C::TMEM);
    return;
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    {
      // ----------------------------------------------------------- softmax
      const int st = warp >> 2, wl = warp & 3;
      const int r_tile = wl * 32 + lane;  // this thread's row of its 128
      const uint32_t lane_base = (uint32_t)(wl * 32) << 16;
      const uint32_t o_addr = tmem + lane_base + C::O_COL + st * DP;
      const float c2 = fabsf(a.scale) * 1.4426950408889634f;
      constexpr float kLift = Weight<E>::kLift, kLag = Weight<E>::kLag;
      attn::Walk w(a.cu, a.lens, a.c.batch, a.tokens, dims, ctl.share);
      int pos = 0, s_seen[2] = {0, 0}, o_seen = 0, pieces = 0, pv_seen = 0;
      bool alive = true;
      if (threadIdx.x == 0) a.splits[blockIdx.x].pieces = 0;
      while (w.next()) {
        const bool both = C::STREAMS == 2 && w.rows > 128;
        const int tiles = w.p.kt1 - w.p.kt0, items = both ? 2 * tiles : tiles;
        const int tile_row0 = both ? 128 * st : 0;  // first row of this warpgroup's row tile
        // ---- Q into shared memory, zeros past D
        alive = alive && (pieces == 0 || warp_wait(&ctl.qk_done, (pieces - 1) & 1));
        {
          const int n_rows = min(128, w.rows - tile_row0);
          const uint32_t dst = smem_u32(sQ) + (both ? st * C::QTILE : 0);
          const int me = both ? threadIdx.x & 127 : threadIdx.x, step = (both ? 128 : kWorkers) / 8;
          const int ch = me & 7;  // 8 lanes copy 128 contiguous bytes
          const T* q = static_cast<const T*>(a.q) + (long long)w.s.first * a.q_stride + (long long)w.p.head * G * D + ch * 8;
          const int first = w.row0 + tile_row0 + (me >> 3), step_tok = step / G, step_g = step - step_tok * G;
          int tok = first / G, g = first - tok * G;
          for (int r = me >> 3; r < n_rows && alive; r += step) {
            const T* src = q + tok * a.q_stride + g * D;
            for (int p = 0; p < panels; ++p) {
              const bool inside = p * 64 + ch * 8 < D;
              cp_async16(dst + attn::sw128_offset(r, p * 8 + ch, 128), inside ? src + p * 64 : src, inside ? 16u : 0u);
            }
            tok += step_tok, g += step_g;
            if (g >= G) g -= G, ++tok;
          }
          cp_async_commit();
          cp_async_wait<0>();
          fence_proxy_async();
          if (alive) mbar_arrive(&ctl.q_full);
        }
        const bool active = wl * 32 < w.rows - tile_row0;  // whether the warp has rows at all
        const int row = w.row0 + tile_row0 + r_tile;       // of the sequence and head
        const int token = min(row / G, w.s.n - 1);
        const bool real = row < w.row0 + w.rows;
        float m = -INFINITY, l = 0.f;  // m in powers of two
        int done = 0;
        // Where a wait has given up, the loop still runs to its end without waiting, so
        // that the warpgroups meet at every barrier; but it announces nothing any more, and
        // no product is made of rows, weights or values that are not what they should be.
        for (int it = (C::STREAMS == 2 ? st : 0); it < items; it += C::STREAMS) {
          const int x = it & 1, tile = both ? it >> 1 : it;
          const int k0 = (w.p.kt0 + tile) * C::BN;
          const uint32_t s_addr = tmem + lane_base + C::S_COL + x * C::BN;
          const bool edge = k0 + C::BN > w.s.len;
          // ---- clean V where the tile reaches past the committed slots
          if (edge && (!both || st == 0)) {
            const int ps = pos + 2 * tile + 1;
            alive = alive && warp_wait(&ctl.full[ps % C::SLOTS], (ps / C::SLOTS) & 1);
            uint8_t* v = sRing + (size_t)(ps % C::SLOTS) * C::SLOT;
            const int lo = max(0, w.s.len - k0), hi = w.s.len + w.s.n - k0;
            const int chunks = panels * 8;
            for (int i = lo * chunks + (threadIdx.x & 127); alive && i < C::BN * chunks; i += 128) {
              const int r = i / chunks, ch = i - r * chunks;
              uint4* at = reinterpret_cast<uint4*>(v + attn::sw128_offset(r, ch, C::BN));
              if (r >= hi) {
                *at = make_uint4(0u, 0u, 0u, 0u);
              } else {
                uint32_t e[4] = {at->x, at->y, at->z, at->w};
                bool changed = false;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const float2 f = E::up(e[q]);
                  if (!isfinite(f.x)) e[q] &= 0xFFFF0000u, changed = true;
                  if (!isfinite(f.y)) e[q] &= 0x0000FFFFu, changed = true;
                }
                if (changed) {
                  *at = make_uint4(e[0], e[1], e[2], e[3]);
                  ctl.dirty[st][w.number & 7] = w.number;
                }
              }
            }
            fence_proxy_async();
          }
          alive = alive && warp_wait(&ctl.s_full[x], s_seen[x]++ & 1);
          fence_after_sync();
          if (active) {
            float s[C::BN];
#pragma unroll
            for (int i = 0; i < C::BN; i += 32) attn::tmem_ld32(s_addr + i, s + i);
#pragma unroll
            for (int i = 0; i < C::BN; i += 32) attn::tmem_ld_wait32(s + i);
            if (edge) {
#pragma unroll
              for (int i = 0; i < C::BN; i += 32) {
                const uint32_t bits = attn::seen(a.tree, a.tree_words, w.s, token, k0 + i);
#pragma unroll
                for (int q = 0; q < 32; ++q) s[i + q] = (bits >> q) & 1u ? s[i + q] : -INFINITY;
              }
            }
            float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < C::BN; i += 8)
#pragma unroll
              for (int q = 0; q < 4; ++q) t[q] = attn::max3(t[q], s[i + 2 * q], s[i + 2 * q + 1]);
            const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * c2;
            // the first tile takes its maximum; later ones move it only by more than kLag
            const bool grow = real && top > (done ? m + kLag : m);
            if (__any_sync(0xffffffffu, grow)) {
              const float m1 = grow ? top : m;
              if (done) {
                if (C::STREAMS == 1) {  // O still takes the tile before: wait for that product
                  alive = alive && warp_wait(&ctl.pv_done, (pv_seen + done - 1) & 1);
                  fence_after_sync();
                }
                const float f = m == -INFINITY ? 0.f : attn::exp2_fast(m - m1);
                l *= f;
                float o[32];
#pragma unroll 1
                for (int i = 0; i < DP; i += 32) {
                  attn::tmem_ld32(o_addr + i, o);
                  attn::tmem_ld_wait32(o);
#pragma unroll
                  for (int q = 0; q < 32; ++q) o[q] *= f;
                  attn::tmem_st32(o_addr + i, o);
                }
              }
              m = m1;
            }
            const float bias = kLift - (m == -INFINITY ? 0.f : m);
            const float2 c22 = make_float2(c2, c2), b22 = make_float2(bias, bias), ones = make_float2(1.f, 1.f);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            auto weights = [&](const float* u, int i) {  // 32 columns from i
              uint32_t pk[16];
#pragma unroll
              for (int q = 0; q < 32; q += 2) {
                float2 e = moe::ffma2(make_float2(u[q], u[q + 1]), c22, b22);
                e.x = attn::exp2_fast(e.x);
                e.y = attn::exp2_fast(e.y);
                sum[(q >> 1) & 1] = moe::ffma2(e, ones, sum[(q >> 1) & 1]);
                pk[q >> 1] = E::down(e.x, e.y);
              }
              attn::tmem_st16(s_addr + i / 2, pk);
              if (i + 32 == C::BN / 2) {  // the first half may go into its product
                attn::tmem_st_wait();
                fence_before_sync();
                __syncwarp();
                if (lane == 0 && alive) mbar_arrive(&ctl.p_half[x]);
              }
            };
#pragma unroll
            for (int i = 0; i < C::BN; i += 32) weights(s + i, i);
            attn::tmem_st_wait();
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          } else if (lane == 0 && alive) {
            mbar_arrive(&ctl.p_half[x]);
          }
          ++done;
          fence_before_sync();
          __syncwarp();
          if (lane == 0 && alive) mbar_arrive(&ctl.p_full[x]);
        }
        pv_seen += done;
        if (l != l && m == -INFINITY) m = 0.f;  // only NaN scores: not to be mistaken for a row that saw nothing
        // ---- the piece's result
        if (done > 0 && alive) {
          alive = warp_wait(&ctl.o_full[st], o_seen & 1);
          fence_after_sync();
        }
        o_seen += done > 0;
        const bool whole = w.whole();
        // Streams over different keys of a whole unit are joined here: stream 1 hands
        // its O over in Q's second tile, which is unused then and holds all
        // columns of 64 rows or half of them of 128.
        const bool join = C::STREAMS == 2 && !both && tiles > 1 && whole;
        if (both || join) named_sync(1, kWorkers);  // the other stream's flags are final
        const bool dirty = ctl.dirty[0][w.number & 7] == w.number || ctl.dirty[1][w.number & 7] == w.number;
        if (!alive || ctl.bad_page[w.number & 7] == w.number) l = kNaN, m = 0.f;
        const int d0 = max(w.p.kt0 * C::BN - w.s.len, 0), d1 = min(w.p.kt1 * C::BN - w.s.len, w.s.n);  // its drafts
        auto read_o = [&](int col, float* o) {
          attn::tmem_ld32(o_addr + col, o);
          attn::tmem_ld_wait32(o);
        };
        if (!whole) {
          const size_t slot = (size_t)blockIdx.x * 2 + (w.p.kt0 == 0);
          const int at = 128 * st + r_tile;
          if (active) {
            // l < 0: the stream had no tile of the piece, its place in the workspace holds nothing
            if (real) reinterpret_cast<float2*>(a.ml)[slot * C::ROWS + at] = make_float2(m, done > 0 || l != l ? l : -1.f);
            float4* dst = a.o + slot * (DP / 4) * C::ROWS + at;
#pragma unroll 1
            for (int col = 0; col < D && done > 0; col += 32) {
              float o[32];
              read_o(col, o);
              if (real) {
#pragma unroll
                for (int q = 0; q < 32; q += 4)
                  if (col + q < D) dst[(col + q) / 4 * C::ROWS] = make_float4(o[q], o[q + 1], o[q + 2], o[q + 3]);
              }
              __syncwarp();
            }
            if (dirty && real && done > 0) {
              put_back<C::BN, T>(a, w.s, w.b, w.p.head, token, d0, d1, w.p.kt0 * C::BN, C::STREAMS == 1 || both ? -1 : 1 - st,
                                 reinterpret_cast<float*>(dst), 4 * C::ROWS);
            }
            __syncwarp();
          }
          if (threadIdx.x == 0 && w.p.kt0 == 0) {
            Split s;
            s.pieces = attn::part_of(ctl.share.total, ctl.share.parts, w.p.first_tile + w.p.tiles - 1) - blockIdx.x + 1;
            s.first = w.s.first, s.n = w.s.n, s.head = w.p.head, s.row0 = w.row0, s.rows = w.rows;
            a.splits[blockIdx.x] = s;
          }
        } else {
          float* exch = reinterpret_cast<float*>(sQ + C::QTILE);
          const int exch_rows = w.rows <= 64 ? 64 : 128;
          const int span = join && exch_rows == 128 ? DP / 2 : DP;
          const int tok = row / G;
          const long long out_row = (long long)(w.s.first + tok) * a.q_heads + w.p.head * G + (row - tok * G);
          float f0 = 1.f, f1 = 0.f, inv = 0.f;
          if (join && st == 1) ctl.ml[r_tile] = make_float2(m, l);
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += span) {
            if (join) {
              if (st == 1 && active) {
#pragma unroll 1
                for (int col = 0; col < span; col += 32) {
                  float o[32];
                  read_o(c0 + col, o);
#pragma unroll
                  for (int q = 0; q < 32; ++q) exch[(col + q) * exch_rows + r_tile] = o[q];
                }
              }
              named_sync(1, kWorkers);
            }
            if (active && (both || st == 0)) {
              if (c0 == 0) {
                if (join) {
                  const float2 other = ctl.ml[r_tile];
                  const float top = fmaxf(m, other.x);
                  f0 = m == -INFINITY ? 0.f : attn::exp2_fast(m - top);
                  f1 = other.x == -INFINITY ? 0.f : attn::exp2_fast(other.x - top);
                  l = l * f0 + other.y * f1;
                  m = top;
                }
                inv = l == 0.f ? 0.f : 1.f / l;
                if (real && a.lse) a.lse[out_row] = l == 0.f ? -INFINITY : (m - kLift) * 0.6931471805599453f + logf(l);
              }
#pragma unroll 1
              for (int col = 0; col < span && c0 + col < D; col += 32) {
                float o[32];
                read_o(c0 + col, o);
                if (join) {
#pragma unroll
                  for (int q = 0; q < 32; ++q) o[q] = o[q] * f0 + exch[(col + q) * exch_rows + r_tile] * f1;
                }
                if (real) {
#pragma unroll
                  for (int q = 0; q < 32; q += 8) {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = o[q + e] * inv;
                    if (c0 + col + q < D)
                      *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + out_row * D + c0 + col + q) = attn::pack8<E>(y);
                  }
                }
                __syncwarp();
              }
            }
            if (join) named_sync(1, kWorkers);
          }
          if (dirty && real && active && (both || st == 0)) {
            put_back<C::BN, T>(a, w.s, w.b, w.p.head, token, d0, d1, 0, -1, static_cast<T*>(a.out) + out_row * D, 4);
          }
          __syncwarp();
        }
        fence_before_sync();  // O has been read before the next piece's first P is announced
        pos += 2 * tiles;
        ++pieces;
      }
    }
    finish();
  }
}

// Adds up the pieces of divided units.  Block (part, y, z) takes rows 32 y .. 32 y +
// 31 of the unit, a lane to a row, and the z-th of SLICES parts of the columns.
// The warps first share the pieces (m and l, turned into factors in shared
// memory), then the columns.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;

template <class E, int DP, int SLICES>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ TreeArgs a) {
  using C = Cfg<DP>;
  using T = typename E::T;
  constexpr int kMine = DP / 4 / kJoinWarps / SLICES;  // columns of a lane, by fours
  const int first = 4 * (threadIdx.x >> 5) + 32 * kMine * blockIdx.z;
  constexpr int kChunk = 32;  // pieces whose factors are held at a time
  __shared__ float s_top[kJoinWarps][32], s_l[kJoinWarps][32], s_factor[kChunk][32];
  moe::pdl_wait();
  const int part = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Split s = a.splits[part];
  if (s.pieces == 0) return;
  const int D = a.c.head_dim, G = a.q_heads / a.c.kv_heads;
  // streams over different keys of the same rows have a place each
  const int streams = C::STREAMS == 2 && s.rows <= 128 ? 2 : 1, n = s.pieces * streams;
  const float2* ml = reinterpret_cast<const float2*>(a.ml);
  for (int r0 = blockIdx.y * 32; r0 < s.rows; r0 += gridDim.y * 32) {
    const bool real = r0 + lane < s.rows;
    const int r = real ? r0 + lane : r0;
    auto place = [&](int i) {  // of piece i's row among all rows of the workspace
      return ((size_t)(part + i / streams) * 2 + (i < streams)) * C::ROWS + r + (i % streams) * 128;
    };
    // one look at every piece's m and l: a running maximum, and the sum under it
    float top = -INFINITY, l = 0.f;
#pragma unroll 4
    for (int i = warp; i < n; i += kJoinWarps) {
      const float2 v = ml[place(i)];
      const float m = fmaxf(top, v.x);
      if (m != -INFINITY) l = l * attn::exp2_fast(top - m) + (v.x == -INFINITY ? 0.f : v.y * attn::exp2_fast(v.x - m));
      top = m;
    }
    s_top[warp][lane] = top;
    s_l[warp][lane] = l;
    __syncthreads();
    top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_top[w][lane]);
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w)
      if (s_top[w][lane] != -INFINITY) l += s_l[w][lane] * attn::exp2_fast(s_top[w][lane] - top);
    float y[4 * kMine] = {};  // columns first + 32 k ..
    for (int i0 = 0; i0 < n; i0 += kChunk) {
      const int count = min(kChunk, n - i0);
      for (int i = warp; i < count; i += kJoinWarps) {
        const float2 v = ml[place(i0 + i)];
        s_factor[i][lane] = v.x != -INFINITY ? attn::exp2_fast(v.x - top) : v.y < 0.f ? -1.f : 0.f;
      }
      __syncthreads();
#pragma unroll 8
      for (int i = 0; i < count; ++i) {
        const float f = s_factor[i][lane];
        const size_t at = place(i0 + i), slot = at / C::ROWS;
        const float4* o = a.o + (slot * (DP / 4) + first / 4) * C::ROWS + (at - slot * C::ROWS);
#pragma unroll
        for (int k = 0; k < kMine; ++k)
          // 0 counts: of a seen key with an infinite value 0 * inf is NaN
          if (!(f < 0.f) && first + 32 * k < D) {
            const float4 v = o[(size_t)k * kJoinWarps * C::ROWS];
            y[4 * k] += v.x * f, y[4 * k + 1] += v.y * f, y[4 * k + 2] += v.z * f, y[4 * k + 3] += v.w * f;
          }
      }
      __syncthreads();
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int row = s.row0 + r, tok = row / G;
    const long long out_row = (long long)(s.first + tok) * a.q_heads + s.head * G + (row - tok * G);
    if (first == 0 && real && a.lse)
      a.lse[out_row] = l == 0.f ? -INFINITY : (top - Weight<E>::kLift) * 0.6931471805599453f + logf(l);
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int d = first + 32 * k;
      if (real && d < D)
        *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + out_row * D + d) =
            make_uint2(E::down(y[4 * k] * inv, y[4 * k + 1] * inv), E::down(y[4 * k + 2] * inv, y[4 * k + 3] * inv));
    }
  }
}

struct Layout {
  size_t ml, o, bytes;
};
Layout layout(int sms, int DP, int rows) {
  Layout w;
  w.ml = ((size_t)sms * sizeof(Split) + 255) & ~(size_t)255;
  w.o = w.ml + (size_t)sms * 2 * rows * sizeof(float2);
  w.bytes = w.o + (size_t)sms * 2 * rows * DP * sizeof(float);
  return w;
}
Layout layout(int sms, int head_dim) {
  return head_dim <= 64    ? layout(sms, 64, Cfg<64>::ROWS)
         : head_dim <= 128 ? layout(sms, 128, Cfg<128>::ROWS)
                           : layout(sms, 256, Cfg<256>::ROWS);
}

template <class E, int DP>
int launch(TreeArgs& a, int sms, cudaStream_t st) {
  using C = Cfg<DP>;
  static moe::SmemGrant grant;
  if (const int rc = attn::make_maps(a.c, C::BN, a.maps)) return rc;
  if (!moe::grant_smem(tree_kernel<E, DP>, smem_bytes<C>(), grant)) return MOE_ERR_CUDA;
  // rows of an average sequence; a block goes on with the rows 32 join_blocks on
  const long long rows = ((long long)a.tokens + a.c.batch - 1) / a.c.batch * (a.q_heads / a.c.kv_heads);
  const int join_blocks = rows >= C::ROWS ? C::ROWS / 32 : (int)(rows + 31) / 32;
  if (const int rc = moe::launch_pdl(tree_kernel<E, DP>, dim3(sms), dim3(kThreads), smem_bytes<C>(), st, a)) return rc;
  const long long units = (long long)a.c.batch * a.c.kv_heads * ((rows + C::ROWS - 1) / C::ROWS);
  // 32 columns a block where the blocks with work are all resident at once, four to an
  // SM: few units have many pieces each (1 sequence of 300001 slots, 136 rows, D = 256:
  // 174 us without slices, 163 with; 8 sequences of 504 rows: 123 without, 126 with)
  constexpr int kSlices = DP / 32;
  if (units * join_blocks * kSlices <= 4 * sms)
    return moe::launch_pdl(join_kernel<E, DP, kSlices>, dim3(sms, join_blocks, kSlices), dim3(kJoinThreads), 0, st, a);
  return moe::launch_pdl(join_kernel<E, DP, 1>, dim3(sms, join_blocks), dim3(kJoinThreads), 0, st, a);
}

template <class E>
int launch(TreeArgs& a, int sms, cudaStream_t st) {
  if (a.c.head_dim <= 64) return launch<E, 64>(a, sms, st);
  if (a.c.head_dim <= 128) return launch<E, 128>(a, sms, st);
  return launch<E, 256>(a, sms, st);
}

}  // namespace

extern "C" {

size_t attn_tree_decode_workspace(const attn_cache* cache) {
  attn_cache c;
  if (attn::check_cache(cache, c)) return 0;
  const int sms = moe::device_info().sms;
  return sms > 0 ? layout(sms, c.head_dim).bytes : 0;
}

int attn_tree_decode(const void* q, long long q_stride, const int32_t* cu, const int32_t* lens, int tokens,
                     int q_heads, const uint64_t* tree, int tree_words, double scale, const attn_cache* cache,
                     void* out, float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  TreeArgs a;
  if (const int rc = attn::check_cache(cache, a.c)) return rc;
  if (const int rc = attn::check_queries(a.c, q, q_stride, cu, lens, tokens, q_heads, tree, tree_words)) return rc;
  if (!attn::rows_fit(a.c, tokens, q_heads)) return MOE_ERR_UNSUPPORTED;
  if ((!out && tokens > 0) || !workspace) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned16(out) || !moe::aligned16(workspace)) return MOE_ERR_ALIGNMENT;
  if (!(fabs(scale) >= 1e-30 && fabs(scale) <= 1e30)) return MOE_ERR_INVALID_ARG;
  if (tokens == 0) return MOE_OK;
  if (ws_bytes < 16) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const int sms = moe::device_info().sms;
  if (sms <= 0) return MOE_ERR_CUDA;
  const Layout w = layout(sms, a.c.head_dim);
  if (ws_bytes < w.bytes) return MOE_ERR_WORKSPACE_TOO_SMALL;
  a.q = q, a.q_stride = q_stride, a.cu = cu, a.lens = lens, a.tokens = tokens, a.q_heads = q_heads;
  a.wait_cycles = attn::wait_cycles(), a.extra = (int)moe::barrier_extra();
  a.tree = tree, a.tree_words = tree_words, a.scale = (float)scale, a.out = out, a.lse = lse, a.st = dev_status;
  a.splits = static_cast<Split*>(workspace);
  a.ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.ml);
  a.o = reinterpret_cast<float4*>(static_cast<char*>(workspace) + w.o);
  const cudaStream_t st = (cudaStream_t)stream;
  return a.c.dtype == ATTN_BF16 ? launch<attn::Brain>(a, sms, st) : launch<attn::Half>(a, sms, st);
}

}  // extern "C"
