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
// Few rows of x are bound by the weights' bytes: a tile's columns are split over a
// cluster of CTAs, whose sums meet in distributed shared memory in a fixed order.
#include <math.h>

#include "fp4_mma.cuh"

using namespace moe::tc;
using namespace fp4;

namespace {

constexpr int kThreads = 192;  // warps 0-3: epilogue; 4: copies; 5: MMA
constexpr int kTmaWarp = 4, kMmaWarp = 5;

template <int FMT, int BN_>
struct Cfg {
  static constexpr int BN = BN_;                               // rows of x of a tile
  static constexpr bool NV = FMT == MOE_FMT_NVFP4;
  static constexpr int COPIES = NV ? 4 : 2;                    // tiles of scales of a chunk
  static constexpr int W_BYTES = 128 * 128, X_BYTES = BN * 128, S_BYTES = COPIES * 512;
  static constexpr int SLOT = W_BYTES + X_BYTES + 2 * S_BYTES;
  // two CTAs to an SM: one's loads run while the other starts or ends
  static constexpr int SLOTS = (113 * 1024 - 3072) / SLOT;
  static constexpr int S_COLS = COPIES * 4;                    // TMEM columns of a chunk's scales, of either side
  // TMEM holds the scales of as many chunks as the ring: where a slot's copies have
  // landed, the products that took the scales before it have been made.
  static constexpr int S_COL = BN <= 32 ? 32 : BN;             // first of them, behind the sums
  static constexpr int TMEM = S_COL + SLOTS * 2 * S_COLS <= 128 ? 128 : 256;
  static_assert(S_COL + SLOTS * 2 * S_COLS <= TMEM, "TMEM");
  static_assert(SLOTS >= 3 && SLOTS * SLOT >= BN * 128 * 4, "ring");
};

struct Control {
  uint64_t full[8], empty[8], done, drain;
  uint32_t tmem;
  int abort;
};

template <class C>
constexpr size_t smem_bytes(int slots) {
  return 1024 + (size_t)slots * C::SLOT + sizeof(Control);
}

// Grid: split * ceil(n / 128) * ceil(t / BN), in clusters of `split`.
template <int FMT, int BN>
__global__ void __launch_bounds__(kThreads, 2) linear_kernel(const __grid_constant__ LinearArgs a, int split,
                                                            int slots) {
  using C = Cfg<FMT, BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Control& ctl = *reinterpret_cast<Control*>(ring + (size_t)slots * C::SLOT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = split > 1 ? (int)cluster_rank() : 0;
  const int t_tiles = (a.t + BN - 1) / BN, tile = blockIdx.x / split;
  const int n0 = tile / t_tiles * 128, t0 = tile % t_tiles * BN;
  const int chunks = (a.cols + kChunk - 1) / kChunk;
  const int c0 = chunks * rank / split, c1 = chunks * (rank + 1) / split;
  const int tiles = fp4::scale_tiles(a.cols, FMT);

  auto load_w = [&](int slot, int c) {  // ... and announces all of the chunk's copies
    const uint32_t at = smem_u32(ring + (size_t)slot * C::SLOT);
    const int kt = c * C::COPIES, bytes = min(C::COPIES, tiles - kt) * 512;
    mbar_arrive_expect_tx(&ctl.full[slot], C::W_BYTES + C::X_BYTES + 2 * bytes);
    load_codes(&a.w_map, at, &ctl.full[slot], c * (kChunk / 2), n0);
    bulk_g2s(at + C::W_BYTES + C::X_BYTES, a.w_scales + ((size_t)(n0 >> 7) * tiles + kt) * 512, bytes, &ctl.full[slot]);
  };
  auto load_x = [&](int slot, int c) {
    const uint32_t at = smem_u32(ring + (size_t)slot * C::SLOT);
    const int kt = c * C::COPIES, bytes = min(C::COPIES, tiles - kt) * 512;
    load_codes(&a.x_map, at + C::W_BYTES, &ctl.full[slot], c * (kChunk / 2), t0);
    bulk_g2s(at + C::W_BYTES + C::X_BYTES + C::S_BYTES, a.x_scales + ((size_t)(t0 >> 7) * tiles + kt) * 512, bytes,
             &ctl.full[slot]);
  };
  const int ahead = a.early ? min(slots, c1 - c0) : 0;  // chunks whose part of w does not wait
  if (threadIdx.x == 32 * kTmaWarp) {
    for (int i = 0; i < slots; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    mbar_init(&ctl.done, 1 + a.extra);
    mbar_init(&ctl.drain, 1);
    ctl.abort = 0;
    mbar_fence_init();
    attn::prefetch_map(&a.w_map);
    attn::prefetch_map(&a.x_map);
    for (int i = 0; i < ahead; ++i) load_w(i, c0 + i);
  }
  // TMEM is taken only when the kernel before has ended, and before the next one may
  // start: CTAs that wait for one another's kernels never hold what the others need.
  moe::pdl_wait();
  if (warp == kMmaWarp) tmem_alloc(&ctl.tmem, C::TMEM);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  moe::pdl_launch_dependents();
  const uint32_t tmem = ctl.tmem;
  volatile int* abort_flag = &ctl.abort;

  if (warp == kTmaWarp) {
    if (lane == 0) {
      bool alive = true;
      int filled = 0;
      for (int c = c0; c < c1; ++c, ++filled) {
        const int slot = filled % slots;
        alive = attn::bounded_wait(&ctl.empty[slot], ((filled / slots) & 1) ^ 1, a.wait_cycles, abort_flag, a.st);
        if (!alive) break;
        if (filled >= ahead) load_w(slot, c);
        load_x(slot, c);
      }
      // every copy has landed before the CTA's shared memory goes away
      for (int i = max(0, filled - slots); i < filled; ++i)
        attn::bounded_wait(&ctl.full[i % slots], (i / slots) & 1, attn::kDrainCycles, nullptr, a.st);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // (the warp walks and waits as one, its elected lane issues; see fp4_linear_wide.cu)
    const bool leader = attn::elect_lane();
    const uint64_t w_desc = sw128_kmajor_desc(smem_u32(ring)), x_desc = sw128_kmajor_desc(smem_u32(ring) + C::W_BYTES);
    const uint64_t s_desc = scales_desc(smem_u32(ring) + C::W_BYTES + C::X_BYTES);
    for (int c = c0, i = 0; c < c1; ++c, ++i) {
      const int slot = i % slots;
      const bool ok = attn::bounded_wait(&ctl.full[slot], (i / slots) & 1, a.wait_cycles, abort_flag, a.st);
      if (!__all_sync(0xffffffffu, ok)) break;
      fence_after_sync();
      const uint32_t off = (uint32_t)slot * (C::SLOT >> 4);
      const uint32_t set = tmem + C::S_COL + slot * 2 * C::S_COLS;
      const int steps = min(kChunk, a.cols - c * kChunk + 63) / 64;
      if (leader) {
#pragma unroll
        for (int k = 0; k < kChunk / 64; ++k) {
          if (k >= steps) break;
          const int copy = C::NV ? k : k / 2, id = C::NV ? 0 : 2 * (k & 1);
          const uint32_t sw = set + 4 * copy, sx = sw + C::S_COLS;
          if (id == 0) {
            copy_scales<1>(sw, s_desc + off + copy * 32);
            copy_scales<1>(sx, s_desc + off + (C::S_BYTES >> 4) + copy * 32);
          }
          mma_fp4<FMT, 1>(tmem, w_desc + off + 2 * k, x_desc + off + 2 * k, idesc_fp4<FMT>(128, BN, id), sw, sx,
                          i > 0 || k > 0);
        }
        mma_commit(&ctl.empty[slot]);
      }
      __syncwarp();
    }
    if (leader) {
      mma_commit(&ctl.done);
      // TMEM goes back only when every MMA has completed
      mma_commit(&ctl.drain);
      attn::bounded_wait(&ctl.drain, 0, attn::kDrainCycles, nullptr, a.st);
    }
    __syncwarp();
  } else {
    attn::bounded_wait(&ctl.done, 0, a.wait_cycles, abort_flag, a.st);
    __syncwarp();
  }
  __syncthreads();  // no copy is under way any more, and nobody gives up from here on
  const bool ok = !*abort_flag;
  if (warp < 4) {
    fence_after_sync();
    const uint32_t sums = tmem + ((uint32_t)(warp * 32) << 16);
    const int n = n0 + threadIdx.x;
    const float scale = a.w_row && n < a.n ? __ldg(a.w_row + n) : 1.f;
    const float add = a.bias && n < a.n ? __ldg(a.bias + n) : 0.f;
    auto put = [&](int j, float v) {
      const int t = t0 + j;
      if (n >= a.n || t >= a.t) return;
      if (a.x_row) v *= __ldg(a.x_row + t);
      store_one(a.y, t * a.y_stride + n, a.y_type, ok ? fmaf(v, scale, add) : kNaN);
    };
    float* part = reinterpret_cast<float*>(ring);  // [BN][128], where the chunks were
#pragma unroll 1
    for (int j = 0; j < BN; j += 16) {
      uint32_t r[16];
      tmem_ld16(sums + j, r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float v = __uint_as_float(r[i]);
        if (split == 1) put(j + i, v);
        else part[(j + i) * 128 + threadIdx.x] = ok ? v : kNaN;
      }
    }
    fence_before_sync();
  }
  if (split > 1) {
    cluster_sync();
    // A thread adds up 4 columns of y of a row of x; 4 of those at a time, as a word of
    // another CTA is some 500 cycles away (128 rows of x, 2 CTAs: one at a time took 20 us).
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
        const int at = q + u * kThreads, t = t0 + (at >> 5), n = n0 + (at & 31) * 4;
        if (at >= q1) break;
        const float row = a.x_row ? __ldg(a.x_row + t) : 1.f;
        const float f[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        uint32_t out[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float scale = a.w_row && n + e < a.n ? __ldg(a.w_row + n + e) : 1.f;
          const float add = a.bias && n + e < a.n ? __ldg(a.bias + n + e) : 0.f;
          out[e] = __float_as_uint(fmaf(f[e] * row, scale, add));
        }
        uint8_t* y = static_cast<uint8_t*>(a.y) + (t * a.y_stride + n) * item;
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
    cluster_sync();  // the others have read this CTA's part
  }
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, C::TMEM);
}

template <int FMT, int BN>
int launch(LinearArgs& a, const fp4_matrix& x, const fp4_matrix& w, int sms, cudaStream_t st) {
  using C = Cfg<FMT, BN>;
  static moe::SmemGrant grant;
  if (const int rc = codes_map(w, 128, &a.w_map)) return rc;
  if (const int rc = codes_map(x, BN, &a.x_map)) return rc;
  if (!moe::grant_smem(linear_kernel<FMT, BN>, smem_bytes<C>(C::SLOTS), grant)) return MOE_ERR_CUDA;
  const int n_tiles = (a.n + 127) / 128, t_tiles = (a.t + BN - 1) / BN, chunks = (a.cols + kChunk - 1) / kChunk;
  // the split that leaves the busiest SM the fewest chunks
  int split = 1;
  long long best = 1ll << 62;
  for (int s = 1; s <= 8 && s <= chunks; s *= 2) {
    const long long waves = ((long long)n_tiles * t_tiles * s + sms - 1) / sms, cost = waves * ((chunks + s - 1) / s + 1);
    if (cost < best) best = cost, split = s;
  }
  const int slots = C::SLOTS;
  const long long blocks = (long long)n_tiles * t_tiles * split;
  if (blocks > 0x7FFFFFFF) return MOE_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<C>(slots);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, linear_kernel<FMT, BN>, a, split, slots) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int FMT>
int launch(LinearArgs& a, const fp4_matrix& x, const fp4_matrix& w, int sms, cudaStream_t st) {
  if (a.t <= 16) return launch<FMT, 16>(a, x, w, sms, st);
  if (a.t <= 32) return launch<FMT, 32>(a, x, w, sms, st);
  if (a.t <= 64) return launch<FMT, 64>(a, x, w, sms, st);
  if (a.t > 256) return launch_wide(a, x, w, sms, st);
  return launch<FMT, 128>(a, x, w, sms, st);
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

// `early`: the kernel before on the stream writes x alone, and waited for those before it.
int product(const fp4_matrix* x, const fp4_matrix* w, const float* bias, const Rows& y, int32_t* dev_status, void* stream,
            bool early) {
  if (const int rc = fp4::check_matrix(x)) return rc;
  if (const int rc = fp4::check_matrix(w)) return rc;
  if (x->cols != w->cols || x->format != w->format) return MOE_ERR_INVALID_ARG;
  if (const int rc = check_output(y, x->rows, w->rows)) return rc;
  if ((uintptr_t)bias & 3u) return MOE_ERR_ALIGNMENT;
  if (x->rows == 0 || w->rows == 0) return MOE_OK;
  const int sms = moe::device_info().sms;
  if (sms <= 0) return MOE_ERR_CUDA;
  LinearArgs a;
  a.w_scales = static_cast<const uint8_t*>(w->scales), a.x_scales = static_cast<const uint8_t*>(x->scales);
  a.w_row = w->row_scale, a.x_row = x->row_scale, a.bias = bias;
  a.n = w->rows, a.t = x->rows, a.cols = x->cols;
  a.y = y.data, a.y_stride = x->rows > 1 ? y.stride : 0, a.y_type = y.type;
  a.wait_cycles = attn::wait_cycles(), a.extra = (int)moe::barrier_extra(), a.st = dev_status;
  a.early = early;
  return w->format == MOE_FMT_NVFP4 ? launch<MOE_FMT_NVFP4>(a, *x, *w, sms, (cudaStream_t)stream)
                                    : launch<MOE_FMT_MXFP4>(a, *x, *w, sms, (cudaStream_t)stream);
}

}  // namespace

extern "C" {

int fp4_linear(const fp4_matrix* x, const fp4_matrix* w, const float* bias, void* y, long long y_stride, int y_type,
               int32_t* dev_status, void* stream) {
  return product(x, w, bias, rows_of(y, y_stride, y_type), dev_status, stream, false);
}

size_t fp4_linear_rows_workspace(const fp4_matrix* w, int rows) {
  if (!w || rows < 0 || !fp4::shape_ok(rows, w->cols, w->format)) return 0;
  return layout(rows, w->cols, w->format).bytes + 16;
}

int fp4_linear_rows(const void* x, long long x_stride, int x_type, int rows, const fp4_matrix* w, const float* bias,
                    void* y, long long y_stride, int y_type, void* workspace, size_t ws_bytes, int32_t* dev_status,
                    void* stream) {
  if (rows < 0) return MOE_ERR_INVALID_ARG;
  if (const int rc = fp4::check_matrix(w)) return rc;
  if (!fp4::shape_ok(rows, w->cols, w->format)) return MOE_ERR_UNSUPPORTED;
  const Rows out = rows_of(y, y_stride, y_type);
  if (const int rc = check_rows(rows_of(x, x_stride, x_type), rows, w->cols, true)) return rc;
  if (const int rc = check_output(out, rows, w->rows)) return rc;
  if ((uintptr_t)bias & 3u) return MOE_ERR_ALIGNMENT;
  if (rows == 0 || w->rows == 0) return MOE_OK;
  if (!workspace) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned16(workspace)) return MOE_ERR_ALIGNMENT;
  const Layout l = layout(rows, w->cols, w->format);
  if (ws_bytes < l.bytes) return MOE_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  const fp4_matrix m = {at, at + l.scales,
                        w->format == MOE_FMT_NVFP4 ? reinterpret_cast<float*>(at + l.row_scale) : nullptr, rows,
                        w->cols, w->format};
  if (const int rc = fp4_quantize(x, x_stride, x_type, &m, stream)) return rc;
  return product(&m, w, bias, out, dev_status, stream, true);
}

}  // extern "C"
