// The softmax weight each cached slot received, on the tensor cores.
//
//   S^T = K . Q^T   (128 slots x up to 128 rows at a time, TMEM)
//   acc_out[slot] = decay * acc[slot] + sum over rows of exp2(c S - lse)
//
// The slots are the M side: a thread owns one slot (a TMEM lane) and adds up
// its row of S^T itself, so the sum over rows needs no exchange between threads
// and has a fixed order.  K is read once, by TMA, in panels of 64 elements x 128
// slots; Q (all rows of a sequence and KV head, up to 128 KB) stays in shared
// memory for the whole run of tiles.
//
// What bounds it: K alone for a few rows (HBM); with R rows a tile of 128 slots
// costs 128 R exponentials, which passes the time of its 32 KB (D = 128) at some
// 100 rows, and the MMAs (128 R D products) run beside them.  Four warpgroups
// share the chunks of two tiles, each with an S buffer of its own: while one
// waits for its next product, three keep the exponential units busy.
//
// Measured: 8 sequences of 16384 slots and 504 rows, D = 128, BF16: 78 us, 0.87
// PFLOP/s, 3.4 exponentials a ns (the units could do 9); a single-token step of two
// short caches: 7 us.  Of a CTA's 137000 cycles there, 62000 go to issuing MMAs, 36000
// to waiting for an S buffer, 16000 for K, 11000 to the start and Q.  Reading the
// biases (a shared-memory word for every row and warp, beside the operands of the
// MMAs) costs 11 us, the exponentials 12, half of the MMAs 7; none of them alone
// is the bound.
//
// Rows are padded to 32 with copies of the pass's first row under a bias of
// -FLT_MAX: whatever the score, infinities and NaN included, a copy adds nothing
// that its original does not add too (zeros under -inf would make NaN of an
// infinite key).  Rows with lse = -inf, whose score may be anything, are picked out
// one by one; the passes that hold some are flagged.
//
// Work division: attn_plan.h, with units of all rows of a sequence and KV
// head; tiles are independent, so a cut unit needs no joining.  More rows than
// Q's room holds are taken in passes over the piece's tiles; each pass adds to
// what the same thread wrote in the one before.
#include <float.h>

#include "attn_tma.cuh"
#include "attn_work.cuh"

using namespace moe::tc;

namespace {

// Warpgroups 0, 1: even and odd chunks of the even tiles; 2, 3: of the odd
// tiles; then a warp each for TMA and MMA.
constexpr int kThreads = 576;
constexpr int kWorkers = 512;
constexpr int kTmaWarp = 16, kMmaWarp = 17;
constexpr int kTile = 128;               // slots of a tile
constexpr int kChunk = 128;              // rows of one MMA and S buffer
constexpr int kPanel = kTile * 128;      // bytes of 64 elements of a tile
constexpr int kSlots = 5;                // panels in the ring
constexpr int kQBytes = 128 * 1024;
constexpr int kMaxRows = kQBytes / 128;  // rows that Q's room holds at D <= 64
constexpr float kNaN = __builtin_nanf("");

struct WeightArgs {
  const void* q;
  long long q_stride;
  const float* lse;
  const int32_t *cu, *lens;
  int tokens, q_heads;
  const uint64_t* tree;
  int tree_words;
  float c2;         // |scale| in powers of two, rounded
  double lse_to_2;  // c2 / |scale|: what lse has to be multiplied with to go with c2
  bool negative;    // the scale
  attn_cache c;
  attn::Maps maps;
  long long wait_cycles;
  int extra;  // arrivals that never come, on s_free
  const float* acc;
  float decay;
  float* acc_out;
  int slot_cap;
  int32_t* st;
};

struct Control {
  uint64_t full[kSlots], empty[kSlots];
  uint64_t s_full[4], s_free[4];  // one S buffer for each warpgroup
  uint64_t q_full, qk_done, drain;
  attn::Share share;
  uint32_t tmem;
  int abort;
  int left_out[2];  // whether rows of a pass add nothing, by turns
  float odd[2][2][kTile];  // [tile parity][even, odd of its tiles]: sums of the odd chunks
  alignas(16) float bias[kMaxRows];  // -lse in powers of two; +inf: the row adds nothing
};
constexpr size_t kOffRing = kQBytes, kOffCtrl = kOffRing + (size_t)kSlots * kPanel;
constexpr size_t kSmem = 1024 + kOffCtrl + sizeof(Control);
static_assert(kSmem <= 232448, "shared memory");

template <class E>
__global__ void __launch_bounds__(kThreads, 1) weights_kernel(const __grid_constant__ WeightArgs a) {
  using T = typename E::T;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + kOffRing;
  Control& ctl = *reinterpret_cast<Control*>(smem + kOffCtrl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int D = a.c.head_dim, G = a.q_heads / a.c.kv_heads;
  const int panels = (D + 63) / 64;
  const int q_rows = (kMaxRows / panels) & ~31;  // rows of one pass
  const bool paired = 2 * panels < kSlots;       // two tiles of K at once leave room for a next panel

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.s_free[i], 128 + a.extra);
    }
    mbar_init(&ctl.q_full, kWorkers);
    mbar_init(&ctl.qk_done, 1);
    mbar_init(&ctl.drain, 1);
    ctl.abort = ctl.left_out[0] = ctl.left_out[1] = 0;
    mbar_fence_init();
    attn::prefetch_map(&a.maps.k);
  }
  moe::pdl_wait();
  moe::pdl_launch_dependents();
  const attn::PlanDims dims{a.c.kv_heads, G, 0x7FFFFFFF, kTile, 2, 1};
  const long long most = (long long)a.c.max_pages * a.c.page_size;
  if (!attn::take_share<kThreads>(a.cu, a.lens, a.c.batch, a.tokens, most < a.slot_cap ? most : a.slot_cap, dims,
                                  ctl.share)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) moe::status_or(a.st, ATTN_DEV_BAD_LENGTH);
    const long long n = (long long)a.c.batch * a.c.kv_heads * a.slot_cap;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kThreads)
      a.acc_out[i] = kNaN;
    return;
  }
  // sequences with nothing in flight only decay
  for (int b = warp; b < a.c.batch; b += kThreads / 32) {
    const attn::Seq s = attn::sequence(a.cu, a.lens, b, a.tokens, attn::kMaxSlots);
    if (s.n > 0) continue;
    for (int h = 0; h < a.c.kv_heads; ++h) {
      const long long base = ((long long)b * a.c.kv_heads + h) * a.slot_cap;
      for (long long j = (long long)blockIdx.x * 32 + lane; j < s.len; j += (long long)gridDim.x * 32)
        a.acc_out[base + j] = a.decay * a.acc[base + j];
    }
  }
  if (ctl.share.t0 >= ctl.share.t1) return;
  if (warp == kMmaWarp) tmem_alloc(&ctl.tmem, 512);
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
  auto passes = [&](const attn::Walk& w) { return (w.rows + q_rows - 1) / q_rows; };

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------- TMA
    attn::Walk w(a.cu, a.lens, a.c.batch, a.tokens, dims, ctl.share);
    int pos = 0;
    bool alive = true;
    const int box_rows = a.maps.box_rows, boxes = kTile / box_rows;  // at most 16
    while (alive && w.next()) {
      const int end = w.s.len + w.s.n;
      const int32_t* table = a.c.page_table + (size_t)w.b * a.c.max_pages;
      const int n_pass = passes(w);
      for (int pass = 0; pass < n_pass && alive; ++pass) {
        for (int j = w.p.kt0; j < w.p.kt1 && alive; ++j) {
          const int slot0 = j * kTile, start = slot0 + lane * box_rows;
          const int issued = min(boxes, (end - slot0 + box_rows - 1) / box_rows);
          int page = 0, row = 0;
          if (lane < issued) {
            const int pi = start / a.c.page_size;
            page = __ldg(table + pi);
            row = start - pi * a.c.page_size;
            if ((unsigned)page >= (unsigned)a.c.pages) {
              page = a.c.pages;  // past the last: zeros; the slots' own threads see the page number too
              moe::status_or(a.st, ATTN_DEV_BAD_PAGE);
            }
          }
          for (int p = 0; p < panels; ++p, ++pos) {
            const int slot = pos % kSlots;
            alive = warp_wait(&ctl.empty[slot], ((pos / kSlots) & 1) ^ 1);
            if (!alive) break;
            if (lane == 0) mbar_arrive_expect_tx(&ctl.full[slot], (uint32_t)(issued * box_rows * 128));
            __syncwarp();
            if (lane < issued)
              attn::load_box(&a.maps.k, smem_u32(sRing + (size_t)slot * kPanel) + (uint32_t)(lane * box_rows * 128),
                             &ctl.full[slot], p * 64, row, w.p.head, page, a.maps.head_inner);
          }
        }
      }
    }
    if (lane == 0)  // every copy has landed before the CTA's shared memory goes away
      for (int i = max(0, pos - kSlots); i < pos; ++i)
        attn::bounded_wait(&ctl.full[i % kSlots], (i / kSlots) & 1, attn::kDrainCycles, nullptr, a.st);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------- MMA
    // The warp walks and waits as one; its elected lane issues.
    const bool leader = attn::elect_lane();
    attn::Walk w(a.cu, a.lens, a.c.batch, a.tokens, dims, ctl.share);
    int slot0 = 0, round0 = 0;          // ring slot of the pass's first panel, and how often the ring had turned
    int loads = 0;
    uint32_t used = 0;                  // bit b: buffer b has been used an odd number of times
    bool alive = true;
    const int k_steps = (D + 15) / 16;
    const uint64_t q_desc = sw128_kmajor_desc(smem_u32(sQ)), k_desc = sw128_kmajor_desc(smem_u32(sRing));
    const uint32_t high = (uint32_t)(q_desc >> 32), q_low = (uint32_t)q_desc, k_low = (uint32_t)k_desc;
    const uint32_t negate = a.negative ? 1u << 13 : 0u;  // a negative scale negates K, the sums keep |scale|
    while (alive && w.next()) {
      const int tiles = w.p.kt1 - w.p.kt0, n_pass = passes(w);
      for (int pass = 0; pass < n_pass && alive; ++pass) {
        const int rows = min(q_rows, w.rows - pass * q_rows), chunks = (rows + kChunk - 1) / kChunk;
        alive = warp_wait(&ctl.q_full, loads++ & 1);
        fence_after_sync();
        // chunks g and g + 1 in one product: a slot's elements are read once for both
        auto product = [&](int tile, int first_slot, int first_round, int g) {
          const int buf = 2 * (tile & 1);
          const bool second = g + 1 < chunks, last = g + 2 >= chunks;
          if (!warp_wait(&ctl.s_free[buf], ((used >> buf) & 1) ^ 1)) return false;
          if (second && !warp_wait(&ctl.s_free[buf + 1], ((used >> (buf + 1)) & 1) ^ 1)) return false;
          used ^= (second ? 3u : 1u) << buf;
          const int n = min(2 * kChunk, ((rows - g * kChunk) + 31) & ~31);
          const uint32_t id = attn::idesc<E>(kTile, n, false) | negate;
          const uint32_t d = tmem + buf * kChunk;
          int slot = first_slot, round = first_round;
          for (int p = 0; p < panels; ++p) {
            if (g == 0 && !warp_wait(&ctl.full[slot], round & 1)) return false;
            fence_after_sync();
            if (leader) {
              uint32_t kl = k_low + (uint32_t)slot * (kPanel >> 4);
              uint32_t ql = q_low + (uint32_t)(p * q_rows + g * kChunk) * (128 >> 4);
              const int steps = min(4, k_steps - 4 * p);
              if (steps == 4) {  // unrolled, the MMAs leave at the tensor core's pace
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma_bf16(d, attn::make_desc(high, kl + 2 * kk), attn::make_desc(high, ql + 2 * kk), id, (p | kk) != 0);
              } else {
                for (int kk = 0; kk < steps; ++kk)
                  mma_bf16(d, attn::make_desc(high, kl + 2 * kk), attn::make_desc(high, ql + 2 * kk), id, (p | kk) != 0);
              }
              if (last) mma_commit(&ctl.empty[slot]);
            }
            __syncwarp();
            if (++slot == kSlots) slot = 0, ++round;
          }
          if (leader) {
            mma_commit(&ctl.s_full[buf]);
            if (second) mma_commit(&ctl.s_full[buf + 1]);
            if (last && tile == tiles - 1) mma_commit(&ctl.qk_done);
          }
          __syncwarp();
          return true;
        };
        auto advance = [&](int& slot, int& round) {
          slot += panels;
          if (slot >= kSlots) slot -= kSlots, ++round;
        };
        for (int t = 0; t < tiles && alive; t += paired ? 2 : 1) {
          int slot1 = slot0, round1 = round0;
          advance(slot1, round1);
          const bool two = paired && t + 1 < tiles;
          for (int g = 0; g < chunks && alive; g += 2) {
            alive = product(t, slot0, round0, g);
            if (two) alive = alive && product(t + 1, slot1, round1, g);
          }
          slot0 = slot1, round0 = round1;
          if (two) advance(slot0, round0);
        }
      }
    }
    if (leader) {
      mma_commit(&ctl.drain);
      attn::bounded_wait(&ctl.drain, 0, attn::kDrainCycles, nullptr, a.st);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- sums
    const int buf = warp >> 2, x = buf >> 1, odd = buf & 1, wl = warp & 3;
    const uint32_t lane_base = (uint32_t)(wl * 32) << 16;
    const float c2 = a.c2;
    const float2 c22 = make_float2(c2, c2), ones = make_float2(1.f, 1.f);
    attn::Walk w(a.cu, a.lens, a.c.batch, a.tokens, dims, ctl.share);
    int loads = 0, used = 0;
    bool alive = true;
    while (w.next()) {
      const int n_pass = passes(w);
      const long long base = ((long long)w.b * a.c.kv_heads + w.p.head) * a.slot_cap;
      for (int pass = 0; pass < n_pass; ++pass) {
        const int r0 = pass * q_rows, rows = min(q_rows, w.rows - r0), chunks = (rows + kChunk - 1) / kChunk;
        alive = alive && (loads == 0 || warp_wait(&ctl.qk_done, (loads - 1) & 1));
        ++loads;
        named_sync(1, kWorkers);  // both warpgroups are done with the biases
        {
          const int padded = (rows + 31) & ~31, ch = threadIdx.x & 7;  // 8 lanes copy 128 contiguous bytes
          const uint32_t dst = smem_u32(sQ);
          const T* q = static_cast<const T*>(a.q) + (long long)w.s.first * a.q_stride + (long long)w.p.head * G * D + ch * 8;
          const int first = r0 + (threadIdx.x >> 3), step = kWorkers / 8, step_tok = step / G, step_g = step - step_tok * G;
          int tok = first / G, g = first - tok * G;
          // who has given up leaves Q alone and does not announce it: no product is made of
          // rows that are not what they should be
          for (int r = threadIdx.x >> 3; r < padded && alive; r += step) {
            const T* src = r < rows ? q + tok * a.q_stride + g * D : q + r0 / G * a.q_stride + r0 % G * D;
            for (int p = 0; p < panels; ++p) {
              const bool inside = p * 64 + ch * 8 < D;
              cp_async16(dst + attn::sw128_offset(r, p * 8 + ch, q_rows), inside ? src + p * 64 : src, inside ? 16u : 0u);
            }
            tok += step_tok, g += step_g;
            if (g >= G) g -= G, ++tok;
          }
          cp_async_commit();
          for (int r = threadIdx.x; r < padded; r += kWorkers) {
            float bias = -FLT_MAX;
            if (r < rows) {
              const int row = r0 + r, tok = row / G, g = row - tok * G;
              const float lse = a.lse[(long long)(w.s.first + tok) * a.q_heads + w.p.head * G + g];
              // in FP64: the rounding of c2 cancels where weights are large, instead of adding up
              // over all rows
              bias = (float)(-(double)lse * a.lse_to_2);
              if (lse == -INFINITY) ctl.left_out[loads & 1] = 1;
            }
            ctl.bias[r] = bias;
          }
          cp_async_wait<0>();
          fence_proxy_async();
          named_sync(1, kWorkers);
          if (alive) mbar_arrive(&ctl.q_full);
        }
        const bool left_out = ctl.left_out[loads & 1] != 0;
        if (threadIdx.x == 0) ctl.left_out[(loads + 1) & 1] = 0;  // read by all before this pass began
        for (int j = w.p.kt0 + x; j < w.p.kt1; j += 2) {
          const int k0 = j * kTile + wl * 32, slot = k0 + lane;
          const bool mine = !odd && slot < w.s.len + w.s.n;
          // loaded here, used behind the sums: a use any earlier would stall the warp
          float before = 0.f;
          int page = 0;
          if (mine) {
            page = __ldg(a.c.page_table + (size_t)w.b * a.c.max_pages + slot / a.c.page_size);
            if (pass > 0) before = a.acc_out[base + slot];
            else if (slot < w.s.len) before = a.acc[base + slot];
          }
          const bool edge = k0 + 32 > w.s.len;  // some of the warp's slots are drafts or past the end
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          for (int g = odd; g < chunks && alive; g += 2) {
            alive = warp_wait(&ctl.s_full[buf], used++ & 1);
            if (!alive) break;
            fence_after_sync();
            const int n = min(kChunk, ((rows - g * kChunk) + 31) & ~31);
            const uint32_t from = tmem + lane_base + buf * kChunk;
            uint32_t sa[16];
            if (!edge && !left_out) {
              // 16 columns are on their way from TMEM while the 16 before are added up
              uint32_t sb[16];
              auto add = [&](const uint32_t (&s)[16], int half, int i) {
                const float4* bias = reinterpret_cast<const float4*>(ctl.bias + g * kChunk + i + half);
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                  const float4 bb = bias[e >> 2];
                  const uint32_t* x = s + half + e;
                  float2 u = moe::ffma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), c22, make_float2(bb.x, bb.y));
                  float2 v = moe::ffma2(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])), c22, make_float2(bb.z, bb.w));
                  u.x = attn::exp2_fast(u.x), u.y = attn::exp2_fast(u.y);
                  v.x = attn::exp2_fast(v.x), v.y = attn::exp2_fast(v.y);
                  sum[0] = moe::ffma2(u, ones, sum[0]);
                  sum[1] = moe::ffma2(v, ones, sum[1]);
                }
              };
              tmem_ld16(from, sa);
              attn::tmem_ld_wait16(sa, sum);
#pragma unroll 1
              for (int i = 0; i < n; i += 32) {
                tmem_ld16(from + i + 16, sb);
                add(sa, 0, i);
                attn::tmem_ld_wait16(sb, sum);
                add(sa, 8, i);
                tmem_ld16(from + min(i + 32, n - 16), sa);
                add(sb, 0, i + 16);
                attn::tmem_ld_wait16(sa, sum);
                add(sb, 8, i + 16);
              }
            } else {
#pragma unroll 1
              for (int i = 0; i < n; i += 16) {
                tmem_ld16(from + i, sa);
                attn::tmem_ld_wait16(sa, sum);
                // lane e looks up what row e sees of the warp's 32 slots
                const int row = r0 + g * kChunk + i + (lane & 15);
                const uint32_t bits = row < r0 + rows ? attn::seen(a.tree, a.tree_words, w.s, row / G, k0) : 0u;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const uint32_t of_row = __shfl_sync(0xffffffffu, bits, e);
                  const float b = ctl.bias[g * kChunk + i + e];
                  const float p = attn::exp2_fast(fmaf(__uint_as_float(sa[e]), c2, b));
                  if (((of_row >> lane) & 1u) && b != INFINITY) (e & 1 ? sum[0].y : sum[0].x) += p;
                }
              }
            }
            fence_before_sync();
            mbar_arrive(&ctl.s_free[buf]);
          }
          float total = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          if (chunks > 1) {  // the odd chunks' sums; the next tile's take the other place
            float* from = ctl.odd[x][(j >> 1) & 1];
            if (odd) from[wl * 32 + lane] = alive ? total : kNaN;
            named_sync(2 + x, 256);
            if (!odd) total += from[wl * 32 + lane];
          }
          if (mine) {
            const bool bad = (unsigned)page >= (unsigned)a.c.pages;
            a.acc_out[base + slot] = bad || !alive ? kNaN : (pass > 0 ? before : a.decay * before) + total;
          }
        }
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <class E>
int launch(WeightArgs& a, int sms, cudaStream_t st) {
  static moe::SmemGrant grant;
  if (const int rc = attn::make_maps(a.c, kTile, a.maps)) return rc;
  if (!moe::grant_smem(weights_kernel<E>, kSmem, grant)) return MOE_ERR_CUDA;
  return moe::launch_pdl(weights_kernel<E>, dim3(sms), dim3(kThreads), kSmem, st, a);
}

}  // namespace

extern "C" int attn_cache_weights(const void* q, long long q_stride, const float* lse, const int32_t* cu,
                                  const int32_t* lens, int tokens, int q_heads, const uint64_t* tree, int tree_words,
                                  double scale, const attn_cache* cache, const float* acc, double decay,
                                  float* acc_out, int slot_cap, int32_t* dev_status, void* stream) {
  WeightArgs a;
  if (const int rc = attn::check_cache(cache, a.c)) return rc;
  if (const int rc = attn::check_queries(a.c, q, q_stride, cu, lens, tokens, q_heads, tree, tree_words)) return rc;
  if (!attn::rows_fit(a.c, tokens, q_heads)) return MOE_ERR_UNSUPPORTED;
  if ((!lse && tokens > 0) || !acc || !acc_out || slot_cap <= 0 || !(fabs(scale) >= 1e-30 && fabs(scale) <= 1e30))
    return MOE_ERR_INVALID_ARG;
  const int sms = moe::device_info().sms;
  if (sms <= 0) return MOE_ERR_CUDA;
  a.q = q, a.q_stride = q_stride, a.lse = lse, a.cu = cu, a.lens = lens, a.tokens = tokens, a.q_heads = q_heads;
  a.wait_cycles = attn::wait_cycles(), a.extra = (int)moe::barrier_extra();
  a.tree = tree, a.tree_words = tree_words, a.acc = acc, a.decay = (float)decay;
  a.acc_out = acc_out, a.slot_cap = slot_cap, a.st = dev_status;
  a.c2 = (float)(fabs(scale) * 1.4426950408889634), a.lse_to_2 = (double)a.c2 / fabs(scale), a.negative = scale < 0.0;
  const cudaStream_t st = (cudaStream_t)stream;
  return a.c.dtype == ATTN_BF16 ? launch<attn::Brain>(a, sms, st) : launch<attn::Half>(a, sms, st);
}
