// What the kernels of FP4 products share: arguments, the block-scaled MMA and its
// scales, copies, and the CTAs of a cluster.
#pragma once

#include "attn_tma.cuh"
#include "fp4.cuh"

namespace fp4 {

constexpr int kChunk = 256;  // columns of a ring slot
constexpr float kNaN = __builtin_nanf("");

struct LinearArgs {
  CUtensorMap w_map, x_map;
  const uint8_t *w_scales, *x_scales;
  const float *w_row, *x_row, *bias;
  int n, t, cols;  // columns of y, rows of y, summed columns
  void* y;
  long long y_stride;
  int y_type;
  long long wait_cycles;
  int extra;  // arrivals that never come, on the barrier of the sums
  int early;  // w may be read before the kernel before this one has ended
  Rows raw;   // .data, where there is no matrix of x: its rows, to be quantised
  int32_t* st;
};

// Instruction descriptor of kind::mxf4nvf4: e2m1 operands, both K-major.
// `id`: which bytes of the scales' words a step of two scales a row takes.
template <int FMT>
__device__ constexpr uint32_t idesc_fp4(int M, int N, int id) {
  return ((uint32_t)id << 4)                         // bytes of B's scales
         | (1u << 7) | (1u << 10)                    // A and B: e2m1
         | ((uint32_t)(N >> 3) << 17)                // N / 8
         | (FMT == MOE_FMT_MXFP4 ? 1u << 23 : 0u)    // scales: UE8M0, or E4M3
         | ((uint32_t)(M >> 4) << 24)                // M / 16
         | ((uint32_t)id << 29);                     // bytes of A's scales
}

// Descriptor of 512 bytes of scales: 32 rows of 16 bytes, no swizzle.
__device__ __forceinline__ uint64_t scales_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(128 >> 4) << 32;  // next 8 rows
  d |= (uint64_t)1 << 46;           // descriptor version
  return d;
}
// ... to 32 lanes x 4 columns of TMEM, the same for each of the four warps' lanes.
// With GROUP = 2 in both CTAs of the pair, each from its own shared memory.
template <int GROUP>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (GROUP == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T, each with its scales in TMEM.
#define FP4_MMA(GROUP, VEC)                                                                                        \
  asm volatile(                                                                                                    \
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                           \
      "tcgen05.mma.cta_group::" GROUP ".kind::mxf4nvf4.block_scale.scale_vec::" VEC " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"( \
          d),                                                                                                      \
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)                                                \
      : "memory")
template <int FMT, int GROUP>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                        uint32_t accumulate) {
  if constexpr (FMT == MOE_FMT_NVFP4 && GROUP == 1) FP4_MMA("1", "4X");
  else if constexpr (FMT == MOE_FMT_NVFP4) FP4_MMA("2", "4X");
  else if constexpr (GROUP == 1) FP4_MMA("1", "2X");
  else FP4_MMA("2", "2X");
}
#undef FP4_MMA

// 128 bytes from x of `box` rows from row y on; what lies outside reads as zeros.
__device__ __forceinline__ void load_codes(const CUtensorMap* m, uint32_t dst, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(m), "r"(x), "r"(y), "r"(moe::tc::smem_u32(bar))
      : "memory");
}

// The same for a CTA of a pair, whose copies are counted at the first CTA's barrier
// (`bar`: its address in the cluster).
__device__ __forceinline__ void load_pair(const CUtensorMap* m, uint32_t dst, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same for the order of execution alone: what was written before need not be seen by the
// others (a release waits for every store that is under way, some 1300 cycles behind an epilogue).
__device__ __forceinline__ void cluster_sync_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// What CTA `rank` of the cluster has at an address of this one's shared memory.
__device__ __forceinline__ uint32_t peer_address(uint32_t saddr, int rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(saddr), "r"(rank));
  return at;
}
__device__ __forceinline__ uint32_t peer_word(uint32_t saddr, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_address(saddr, rank)) : "memory");
  return v;
}

// Arrives at CTA `rank`'s barrier, when nothing in memory has to be seen behind it
// (TMEM that has been read): a release of what the thread wrote before takes some 1500 cycles.
__device__ __forceinline__ void arrive_relaxed_at(uint64_t* bar, int rank) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                   peer_address(moe::tc::smem_u32(bar), rank))
               : "memory");
}
// attn::bounded_wait for a barrier at which other CTAs of the cluster arrive.
__device__ __forceinline__ bool cluster_wait(uint64_t* bar, uint32_t parity, long long limit, volatile int* abort,
                                             int32_t* st) {
  auto test = [&]() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(moe::tc::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
  };
  for (int i = 0; i < 64; ++i)
    if (test()) return true;
  const long long from = clock64();
  while (!test()) {
    if (*abort) return false;
    if (clock64() - from > limit) {
      moe::status_or(st, MOE_DEV_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ void set_peer_word(uint32_t saddr, int rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_address(saddr, rank)), "r"(v) : "memory");
}
// (volatile alone: behind the barriers of the cluster, but several at a time)
__device__ __forceinline__ float4 peer_float4(uint32_t saddr, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(peer_address(saddr, rank)));
  return v;
}

__device__ __forceinline__ void store_one(void* y, long long at, int type, float v) {
  if (type == FP4_FP32) static_cast<float*>(y)[at] = v;
  else if (type == FP4_BF16) static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16(v);
  else static_cast<__half*>(y)[at] = __float2half(v);
}

inline int make_map(CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* base, cuuint64_t width,
                    cuuint64_t bytes, cuuint64_t rows, int box_width, int box_rows, CUtensorMap* m) {
  const attn::MapEncoder encode = attn::map_encoder();
  if (!encode) return MOE_ERR_CUDA;
  const cuuint64_t dims[2] = {width, rows}, strides[1] = {bytes};
  const cuuint32_t boxes[2] = {(cuuint32_t)box_width, (cuuint32_t)box_rows}, one[2] = {1, 1};
  const CUresult rc = encode(m, type, 2, const_cast<void*>(base), dims, strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                             swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return rc == CUDA_SUCCESS ? MOE_OK : MOE_ERR_UNSUPPORTED;
}
// `box` rows of a chunk's codes.
inline int codes_map(const fp4_matrix& m, int box, CUtensorMap* map) {
  return make_map(CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, m.codes, m.cols / 2, m.cols / 2, m.rows,
                  kChunk / 2, box, map);
}
// A chunk's scales of 128 rows: consecutive tiles of 512 bytes.
inline int scales_map(const fp4_matrix& m, CUtensorMap* map) {
  const long long tiles = (long long)((m.rows + 127) / 128) * scale_tiles(m.cols, m.format);
  return make_map(CU_TENSOR_MAP_DATA_TYPE_UINT32, CU_TENSOR_MAP_SWIZZLE_NONE, m.scales, 128, 512, tiles, 128,
                  m.format == MOE_FMT_NVFP4 ? 4 : 2, map);
}

// fp4_linear with many rows of x (fp4_linear_wide.cu).
int launch_wide(LinearArgs& a, const fp4_matrix& x, const fp4_matrix& w, int sms, cudaStream_t st);

}  // namespace fp4
