// Tensor-map and tcgen05 pieces that the attention kernels share.
#pragma once

#include <cuda.h>

#include "attn.cuh"
#include "tcgen05.cuh"

namespace attn {

// ---------------------------------------------------------------------------
// Host: one tensor map for K and one for V.  Both view the cache as
// (element, row, head, page), the two middle axes in the order of their
// strides; a copy takes a box of 64 elements x `box_rows` rows of one head and
// page into shared memory with the 128-byte swizzle.
// ---------------------------------------------------------------------------
struct Maps {
  CUtensorMap k, v;
  int box_rows;    // rows of one copy: the largest power of two that divides a page, at most `tile`
  int head_inner;  // heads lie closer together than rows
};

// Cycles of a wait in the kernels: at most 2.07 of them are a ns.
inline long long wait_cycles() { return 2 * (long long)moe::wait_limit_ns(); }
// ... of one behind which shared memory or TMEM is given up: some 2 s, whatever the others' limit.
constexpr long long kDrainCycles = 4000000000ll;

typedef CUresult (*MapEncoder)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// The driver's cuTensorMapEncodeTiled, looked up once; NULL where there is none.
inline MapEncoder map_encoder() {
  static std::atomic<void*> entry{nullptr};
  void* f = entry.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
            cudaSuccess || found != cudaDriverEntryPointSuccess || !f)
      return nullptr;
    entry.store(f, std::memory_order_release);
  }
  return reinterpret_cast<MapEncoder>(f);
}

inline int make_map(const attn_cache& c, void* base, int box_rows, bool head_inner, CUtensorMap* m) {
  const MapEncoder encode = map_encoder();
  if (!encode) return MOE_ERR_CUDA;
  const cuuint64_t rows = c.page_size, heads = c.kv_heads;
  const cuuint64_t sr = (cuuint64_t)c.row_stride * 2, sh = (cuuint64_t)c.head_stride * 2;
  const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, head_inner ? heads : rows, head_inner ? rows : heads,
                              (cuuint64_t)c.pages};
  const cuuint64_t strides[3] = {head_inner ? sh : sr, head_inner ? sr : sh, (cuuint64_t)c.page_stride * 2};
  const cuuint32_t br = (cuuint32_t)box_rows;
  const cuuint32_t box[4] = {64, head_inner ? 1 : br, head_inner ? br : 1, 1}, one[4] = {1, 1, 1, 1};
  const CUresult rc = encode(
      m, c.dtype == ATTN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, base, dims,
      strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return rc == CUDA_SUCCESS ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

inline int make_maps(const attn_cache& c, int tile, Maps& m) {
  m.box_rows = c.page_size & -c.page_size;
  if (m.box_rows > tile) m.box_rows = tile;
  m.head_inner = c.head_stride < c.row_stride && c.kv_heads > 1;
  if (const int rc = make_map(c, c.k, m.box_rows, m.head_inner, &m.k)) return rc;
  return make_map(c, c.v, m.box_rows, m.head_inner, &m.v);
}

// ---------------------------------------------------------------------------
// Device
// ---------------------------------------------------------------------------

// Waits for the barrier's phase.  The first tries run without a clock, whose
// reads are slow; after `limit` cycles, or once another role of the CTA has given
// up (*abort), the wait gives up too: MOE_DEV_TIMEOUT, *abort set, false.  Lanes of
// a warp may part here, one by one: what a warp does together takes a vote.
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity, long long limit, volatile int* abort,
                                             int32_t* st) {
  for (int i = 0; i < 64; ++i)
    if (moe::tc::mbar_test(bar, parity)) return true;
  const long long from = clock64();
  while (!moe::tc::mbar_test(bar, parity)) {
    if (abort && *abort) return false;
    if (clock64() - from > limit) {
      moe::status_or(st, MOE_DEV_TIMEOUT);
      if (abort) *abort = 1;
      return false;
    }
  }
  return true;
}

// One box: 64 elements from x (a multiple of 64), `box_rows` rows from `row`
// of one head and page.  A page number past the last reads as zeros.
__device__ __forceinline__ void load_box(const CUtensorMap* m, uint32_t dst, uint64_t* bar, int x, int row, int head,
                                         int page, bool head_inner) {
  const int a = head_inner ? head : row, b = head_inner ? row : head;
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst), "l"(m), "r"(x), "r"(a), "r"(b), "r"(page), "r"(moe::tc::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// Descriptor of an operand whose other index is contiguous (the keys' rows of
// V as the K side of a product): rows of 64 elements (128 bytes, swizzled),
// 8-row groups 1024 bytes apart, the next 64 elements `panel` bytes on.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr, uint32_t panel) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(panel >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// The words of a descriptor: the high one is the same wherever the tile lies,
// the low one holds the address and advances by (bytes >> 4).
__device__ __forceinline__ uint64_t make_desc(uint32_t high, uint32_t low) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(low), "r"(high));
  return d;
}

// kind::f16 instruction descriptor, A K-major; B K-major or (b_mn) contiguous
// along N.
template <class E>
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool b_mn);
template <>
__host__ __device__ constexpr uint32_t idesc<Half>(int M, int N, bool b_mn) {
  return moe::tc::idesc_f16_f32(M, N) | (b_mn ? 1u << 16 : 0u);
}
template <>
__host__ __device__ constexpr uint32_t idesc<Brain>(int M, int N, bool b_mn) {
  return moe::tc::idesc_bf16_f32(M, N) | (b_mn ? 1u << 16 : 0u);
}

// True for one lane of a converged warp.
__device__ __forceinline__ bool elect_lane() {
  uint32_t yes;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
  return yes != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 TMEM lanes x 32 columns; thread i: lane base + i.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr)
      : "memory");
}
// Waits for the loads of this thread; naming the registers keeps every use of
// them behind the wait.
__device__ __forceinline__ void tmem_ld_wait32(float* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
        "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
        "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]),
        "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])
      :
      : "memory");
}
// The same for 16 columns; what has been added up into `done` before it in the
// source stays before it, so that the arithmetic on one group of columns covers
// the loads of the next.
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16], float2 (&done)[2]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
        "+f"(done[0].x), "+f"(done[0].y), "+f"(done[1].x), "+f"(done[1].y)
      :
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* r) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(r);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(u[0]), "r"(u[1]),
      "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]),
      "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]), "r"(u[19]), "r"(u[20]),
      "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]), "r"(u[28]), "r"(u[29]),
      "r"(u[30]), "r"(u[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(u[0]), "r"(u[1]), "r"(u[2]),
      "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]),
      "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Byte offset of 16-byte chunk `c` (8 elements) of row `r` in a swizzled tile
// of `rows` rows, 64-element panels one after the other.
__device__ __forceinline__ uint32_t sw128_offset(int r, int c, int rows) {
  return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

}  // namespace attn
