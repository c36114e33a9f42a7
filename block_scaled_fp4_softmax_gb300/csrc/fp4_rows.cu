// What stands between FP4 products: quantisation, SwiGLU and the norms around a
// residual sum, row by row, and the way back to 16 or 32 bits.
//
// A row belongs to `threads` consecutive threads; a thread holds NB units of W columns, unit
// u = j * threads + t.  A block of 16 or 32 columns is 1, 2 or 4 neighbouring lanes, four
// scales (one 32-bit word of the tiled layout) are four times as many.  The row stays in registers between
// its reductions: each element is read once and written once.  (Above 8192 columns the norm has
// 64 registers a thread for four operands of 32 columns and keeps some of them in local memory: up to 252 bytes a
// thread with a residual and a block in FP32, 8 to 40 with 16-bit residuals.  Nothing else spills but
// SwiGLU of FP32 above 16384 columns, 64 bytes.)
//
// Units are of 8 columns, so that the loads and stores of a warp are contiguous.  The quantiser takes
// 16: then one lane works out a block's scale instead of two (or two instead of four), and the loads of 32
// bytes a lane meet in L1 (69 us became 56 in the first case below).  SwiGLU and the norm hold two to
// four operands of a unit and gain nothing by that (97 us for 96, 70 for 65 with NVFP4 below).
//
// What bounds these: HBM, or for 16-bit rows into FP4 the issue slots beside it; for few rows
// the launch and the row's reductions.  Measured, copy bandwidth 6.68 TB/s, bytes as they have to be moved:
//   NVFP4 of 16384 x 8192 in BF16              56 us, 6.1 TB/s     of 50257 x 2560 in FP32   84 us, 7.0 TB/s
//   MXFP4 of 19608 x 4096 in FP16              30 us, 6.7 TB/s     back to BF16              32 us, 6.4 TB/s
//   SwiGLU of 19608 x 5760 in BF16, to BF16    95 us, 7.1 TB/s     to NVFP4                  92 us, 5.6 TB/s
//   norms of 19608 x 4096 in BF16 round a block in FP32, a gate for each element   168 us, 6.7 TB/s
//   the same in FP32 throughout: 4096 x 8192   96 us, 6.3 TB/s     2048 x 16384             133 us, 4.5 TB/s
//   19608 x 2560 in BF16, one norm, to BF16    62 us, 6.5 TB/s     to NVFP4                  66 us, 5.0 TB/s
//   scales of 50257 x 2560 in NVFP4, laid out  13 us, 1.2 TB/s     of 65536 x 8192           54 us, 1.3 TB/s
//   one row of 2560: 1.4 us quantised, 2.1 through SwiGLU, 4.1 through both norms
#include <math.h>

#include <type_traits>

#include "fp4_quantize.cuh"

using namespace fp4;

namespace {

// 8 elements rounded to `type` and written.
__device__ __forceinline__ void store8(void* base, long long at, int type, const float (&f)[8]) {
  if (type == FP4_FP32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[1] = make_float4(f[4], f[5], f[6], f[7]);
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (type == FP4_BF16) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    } else {
      const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Where a thread stands: blockDim.x threads (a multiple of 32) to a row, blockDim.y
// rows to a block.
template <int W>
struct PlaceOf {
  int t, threads, row, cols;
  bool live;
  __device__ PlaceOf(int rows, int cols_) : t(threadIdx.x), threads(blockDim.x), cols(cols_) {
    row = blockIdx.x * blockDim.y + threadIdx.y;
    live = row < rows;
  }
  __device__ __forceinline__ int col(int j) const { return (j * threads + t) * W; }
  __device__ __forceinline__ bool in(int j) const { return live && col(j) < cols; }
};
using Place = PlaceOf<8>;

// Reduction over a row's threads, in a fixed order; every thread gets the result.
// `slots` is used once in a kernel.  All threads of the block call it.
typedef uint32_t Slots[8][32];

__device__ __forceinline__ uint32_t row_max(uint32_t v, Slots& slots) {
  v = __reduce_max_sync(0xffffffffu, v);
  if (blockDim.x == 32) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) slots[threadIdx.y][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < (int)blockDim.x / 32 ? slots[threadIdx.y][lane] : 0u;
  return __reduce_max_sync(0xffffffffu, v);
}
__device__ __forceinline__ float row_sum(float v, Slots& slots) {
  v = moe::warp_sum(v);
  if (blockDim.x == 32) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) slots[threadIdx.y][threadIdx.x >> 5] = __float_as_uint(v);
  __syncthreads();
  v = lane < (int)blockDim.x / 32 ? __uint_as_float(slots[threadIdx.y][lane]) : 0.f;
  return moe::warp_sum(v);
}

// ---------------------------------------------------------------------------
// Quantisation of a row in registers; every thread of the block takes part, with
// zeros past the row's end.
// ---------------------------------------------------------------------------

template <int NB, bool NV, int W>
__device__ __forceinline__ void to_fp4(const fp4_matrix& m, const PlaceOf<W>& p, float (&v)[NB][W], Slots& slots) {
  uint32_t top[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) top[j] = block_top<NV>(v[j]);
  RowScale scale;
  if (NV) {
    uint32_t a = top[0];
#pragma unroll
    for (int j = 1; j < NB; ++j) a = max(a, top[j]);
    scale = row_scale(row_max(a, slots));
    if (p.t == 0 && p.live) m.row_scale[p.row] = scale.value();
    if (scale.tiny) {
#pragma unroll
      for (int j = 0; j < NB; ++j) scale_first(scale, v[j], top[j]);
    }
  } else if (m.row_scale && p.t == 0 && p.live) {
    m.row_scale[p.row] = 1.f;
  }
  const int tiles = scale_tiles(m.cols, NV ? MOE_FMT_NVFP4 : MOE_FMT_MXFP4);
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    uint32_t words[W / 8];
    const bool in = p.in(j);
    const uint32_t four = quantize<NV>(v[j], top[j], scale, p.t & 31, in, words);
    if (in) {
      uint8_t* to = static_cast<uint8_t*>(m.codes) + ((size_t)p.row * m.cols + p.col(j)) / 2;
      if constexpr (W == 16) *reinterpret_cast<uint2*>(to) = make_uint2(words[0], words[1]);
      else *reinterpret_cast<uint32_t*>(to) = words[0];
      if ((p.t & (kScaleLanes<NV, W> - 1)) == 0)
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(m.scales) +
                                     scale_word(p.row, p.col(j) / (W * kScaleLanes<NV, W>), tiles)) = four;
    }
  }
}

// ---------------------------------------------------------------------------
// Kernels
// ---------------------------------------------------------------------------

struct QuantizeArgs {
  fp4::Rows x;
  fp4_matrix m;
};

// (16 elements a unit: what is done for a block is done by one thread or two)
template <int NB, int TYPE, bool NV>
__global__ void __launch_bounds__(512) quantize_kernel(const __grid_constant__ QuantizeArgs a) {
  __shared__ Slots slots;
  const PlaceOf<16> p(a.m.rows, a.m.cols);
  moe::pdl_wait();
  moe::pdl_launch_dependents();
  Raw<TYPE> raw[NB][2];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (p.in(j)) raw[j][k].load(a.x.data, p.row * a.x.stride + p.col(j) + 8 * k);
      else raw[j][k].zero();
    }
  float v[NB][16];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int k = 0; k < 2; ++k) raw[j][k].floats(*reinterpret_cast<float(*)[8]>(&v[j][8 * k]));
  to_fp4<NB, NV>(a.m, p, v, slots);
}

// g / (1 + exp(-g)), the reciprocal from a quarter of the sum: for g between -88.7 and -87.3 the sum is above
// 2^126 and its reciprocal subnormal, to 2^-22 at worst, while the quotient is not (g = -88: -5e-37).  Past them
// exp(-g) is above 2^128, and the quotient -0.  (rcp.approx without .ftz: 116 us for 92 into NVFP4.)
__device__ __forceinline__ float silu(float g) {
  float e;  // exp(-g) / 4, the exponential of 2 within 2 ulp; below 2^-126 it is 0
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(g, -1.44269504f, -2.f)));
  return g * (0.25f * reciprocal(0.25f + e));
}

struct SwigluArgs {
  fp4::Rows gate, up, out;  // out.data, m.codes: NULL where not wanted
  fp4_matrix m;
  int rows, cols;
};

template <int NB, int TYPE>
__global__ void __launch_bounds__(NB <= 2 ? 256 : 512) swiglu_kernel(const __grid_constant__ SwigluArgs a) {
  __shared__ Slots slots;
  const Place p(a.rows, a.cols);
  moe::pdl_wait();
  moe::pdl_launch_dependents();
  Raw<TYPE> g[NB], u[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    if (p.in(j)) {
      g[j].load(a.gate.data, p.row * a.gate.stride + p.col(j));
      u[j].load(a.up.data, p.row * a.up.stride + p.col(j));
    } else {
      g[j].zero(), u[j].zero();
    }
  }
  float v[NB][8];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    float up[8];
    g[j].floats(v[j]);
    u[j].floats(up);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = silu(v[j][i]) * up[i];
    if (a.out.data && p.in(j)) store8(a.out.data, p.row * a.out.stride + p.col(j), a.out.type, v[j]);
  }
  if (!a.m.codes) return;
  if (a.m.format == MOE_FMT_NVFP4) to_fp4<NB, true>(a.m, p, v, slots);
  else to_fp4<NB, false>(a.m, p, v, slots);
}

struct NormArgs {
  fp4::Rows r, y, gate, r_out, h;  // .data NULL: not there
  int gate_cols;
  const float *post_weight, *weight;
  float scale, eps;
  int rows, cols;
  fp4_matrix m;  // .codes NULL: not wanted
};

__device__ __forceinline__ void load_weights(const float* w, int col, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w + col)), b = __ldg(reinterpret_cast<const float4*>(w + col) + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

__device__ __forceinline__ float one_element(const fp4::Rows& x, long long at) {
  if (x.type == FP4_FP32) return __ldg(static_cast<const float*>(x.data) + at);
  const uint16_t b = __ldg(static_cast<const uint16_t*>(x.data) + at);
  return x.type == FP4_BF16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
}

template <int NB, int R_TYPE, int Y_TYPE>
__global__ void __launch_bounds__(256 * NB) norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ Slots slots[3];
  const Place p(a.rows, a.cols);
  const float per = 1.f / (float)a.cols;
  moe::pdl_wait();
  moe::pdl_launch_dependents();
  Raw<R_TYPE> r[NB];
  Raw<Y_TYPE> y[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    if (p.in(j)) r[j].load(a.r.data, p.row * a.r.stride + p.col(j));
    else r[j].zero();
    if (a.y.data && p.in(j)) y[j].load(a.y.data, p.row * a.y.stride + p.col(j));
    else y[j].zero();
  }
  float v[NB][8];
  float factor = a.scale;
  if (a.y.data) {
    if (a.gate.data && a.gate_cols == 1 && p.live) factor *= one_element(a.gate, p.row * a.gate.stride);
#pragma unroll
    for (int j = 0; j < NB; ++j) y[j].floats(v[j]);
    if (a.post_weight) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(v[j][i], v[j][i], sum);
      const float f = 1.f / sqrtf(row_sum(sum, slots[0]) * per + a.eps);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if (!p.in(j)) continue;
        float w[8];
        load_weights(a.post_weight, p.col(j), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * f * w[i];
      }
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    float x[8];
    r[j].floats(x);
    if (a.y.data) {
      float g[8];
      if (a.gate.data && a.gate_cols != 1 && p.in(j)) {
        Raw<Y_TYPE> raw;
        raw.load(a.gate.data, p.row * a.gate.stride + p.col(j));
        raw.floats(g);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = 1.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf(factor * g[i], v[j][i], x[i]);
    }
    if (a.r_out.data && p.in(j)) store8(a.r_out.data, p.row * a.r_out.stride + p.col(j), R_TYPE, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[j][i] = x[i];
      sum = fmaf(x[i], x[i], sum);
    }
  }
  const float f = 1.f / sqrtf(row_sum(sum, slots[1]) * per + a.eps);
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    if (!p.in(j)) continue;
    if (a.weight) {
      float w[8];
      load_weights(a.weight, p.col(j), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * f * w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] *= f;
    }
    if (a.h.data) store8(a.h.data, p.row * a.h.stride + p.col(j), a.h.type, v[j]);
  }
  if (!a.m.codes) return;
  if (a.m.format == MOE_FMT_NVFP4) to_fp4<NB, true>(a.m, p, v, slots[2]);
  else to_fp4<NB, false>(a.m, p, v, slots[2]);
}

struct DequantizeArgs {
  fp4_matrix m;
  fp4::Rows out;
};

template <int NB, int TYPE, bool NV>
__global__ void __launch_bounds__(NB <= 2 ? 256 : 512) dequantize_kernel(const __grid_constant__ DequantizeArgs a) {
  const Place p(a.m.rows, a.m.cols);
  moe::pdl_wait();
  moe::pdl_launch_dependents();
  const int tiles = fp4::scale_tiles(p.cols, NV ? MOE_FMT_NVFP4 : MOE_FMT_MXFP4);
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.m.codes) + (size_t)p.row * p.cols / 2);
  const uint8_t* scales = static_cast<const uint8_t*>(a.m.scales) + fp4::scale_word(p.row, 0, tiles);
  const float row = p.live && a.m.row_scale ? __ldg(a.m.row_scale + p.row) : 1.f;
  uint32_t c[NB], b[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    if (!p.in(j)) continue;
    const int block = p.col(j) / (NV ? 16 : 32);
    c[j] = __ldg(codes + p.col(j) / 8);
    b[j] = __ldg(scales + (size_t)(block >> 2) * 512 + (block & 3));
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    if (!p.in(j)) continue;
    // code * block scale is exact: at most 2 + 4 significant bits, of NVFP4 within FP16
    // too; of MXFP4 within FP32, with its subnormals, up to a scale of 2^125
    uint32_t s2 = 0;
    if (NV) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"((uint16_t)(b[j] | b[j] << 8)));
    const float scale = NV ? 1.f : moe::ue8m0_to_f32(min(b[j], 252u));
    const float2 scales2 = make_float2(scale, scale), row2 = make_float2(row, row), none = make_float2(-0.f, -0.f);
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h = moe::e2m1x2_to_f16x2(c[j] >> (8 * i));
      if (NV) {
        const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&s2));
        h = *reinterpret_cast<const uint32_t*>(&v);
      }
      float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
      if (!NV) v = moe::ffma2(v, scales2, none);
      v = moe::ffma2(v, row2, none);
      f[2 * i] = v.x, f[2 * i + 1] = v.y;
    }
    if (!NV && b[j] > 252u) {  // what is left of the scale: 6 * 2^126 overflows, times the row's factor it need not
      const float left = b[j] == 255u ? __uint_as_float(0x7FC00000u) : b[j] == 254u ? 4.f : 2.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= left;
    }
    store8(a.out.data, p.row * a.out.stride + p.col(j), TYPE, f);
  }
}

// A thread to the four scales of a row's tile.  What bounds it: words that are scattered by 16 bytes and
// four loads of a byte for each (1.3 TB/s); once for a weight matrix.
__global__ void __launch_bounds__(256) tile_scales_kernel(const uint8_t* __restrict__ in, int rows, int blocks,
                                                          int tiles, uint8_t* __restrict__ out) {
  moe::pdl_wait();
  moe::pdl_launch_dependents();
  const long long words = (long long)rows * tiles, step = (long long)gridDim.x * blockDim.x;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += step) {
    const int r = (int)(i / tiles), kt = (int)(i - (long long)r * tiles);
    uint32_t four = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int b = kt * 4 + k;
      if (b < blocks) four |= (uint32_t)__ldg(in + (long long)r * blocks + b) << (8 * k);
    }
    *reinterpret_cast<uint32_t*>(out + fp4::scale_word(r, kt, tiles)) = four;
  }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------

// Units of a thread, and the block's shape: one row, or several short ones.
struct Shape {
  int nb;
  dim3 grid, block;
  void set(int rows, int cols, int units, int width = 8) {
    nb = units;
    const int threads = (cols + width * nb * 32 - 1) / (width * nb * 32) * 32;
    const int per = threads >= 256 ? 1 : threads == 32 ? 8 : 256 / threads;
    block = dim3(threads, per);
    grid = dim3((rows + per - 1) / per);
  }
};
// Of kernels that hold a row or two in registers: with many rows 4 units of a thread,
// as what is done once for a row (its reduction, its exponent) is some 50 instructions of
// every thread; with few of them as many threads as there may be.
struct LightShape : Shape {
  LightShape(int rows, int cols) { set(rows, cols, cols > 16384 ? 8 : cols > 4096 || (rows >= 1024 && cols >= 1024) ? 4 : cols > 2048 ? 2 : 1); }
};
template <class F>
int by_units(const LightShape& s, F f) {
  return s.nb == 1   ? f(std::integral_constant<int, 1>())
         : s.nb == 2 ? f(std::integral_constant<int, 2>())
         : s.nb == 4 ? f(std::integral_constant<int, 4>())
                     : f(std::integral_constant<int, 8>());
}
// ... and of the quantiser, in units of 16.
struct QuantizeShape : Shape {
  QuantizeShape(int rows, int cols) {
    set(rows, cols, cols > 16384 ? 4 : cols > 8192 || (rows >= 1024 && cols >= 1024) ? 2 : 1, 16);
  }
};
template <class F>
int by_units(const QuantizeShape& s, F f) {
  return s.nb == 1 ? f(std::integral_constant<int, 1>()) : s.nb == 2 ? f(std::integral_constant<int, 2>())
                                                                   : f(std::integral_constant<int, 4>());
}
// Of the norm's, whose threads hold four operands of each unit.
struct HeavyShape : Shape {
  HeavyShape(int rows, int cols) { set(rows, cols, cols <= 2048 ? 1 : cols <= 8192 ? 2 : 4); }
};
template <class F>
int by_units(const HeavyShape& s, F f) {
  return s.nb == 1 ? f(std::integral_constant<int, 1>()) : s.nb == 2 ? f(std::integral_constant<int, 2>())
                                                                   : f(std::integral_constant<int, 4>());
}

template <class F>
int by_type(int type, F f) {
  return type == FP4_BF16   ? f(std::integral_constant<int, FP4_BF16>())
         : type == FP4_FP16 ? f(std::integral_constant<int, FP4_FP16>())
                            : f(std::integral_constant<int, FP4_FP32>());
}

// The stride of a single row is of no account.
void one_row(fp4::Rows& x, int rows) {
  if (rows == 1) x.stride = 0;
}

}  // namespace

extern "C" {

size_t fp4_scale_bytes(int rows, int cols, int format) {
  if (!fp4::shape_ok(rows, cols, format)) return 0;
  return (size_t)((rows + 127) / 128) * fp4::scale_tiles(cols, format) * 512;
}

int fp4_tile_scales(const uint8_t* scales, int rows, int cols, int format, uint8_t* tiled, void* stream) {
  if (rows < 0) return MOE_ERR_INVALID_ARG;
  if (!fp4::shape_ok(rows, cols, format)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!scales || !tiled) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned16(tiled)) return MOE_ERR_ALIGNMENT;
  const int tiles = fp4::scale_tiles(cols, format);
  const fp4::Span outs[] = {fp4::piece(tiled, (long long)fp4_scale_bytes(rows, cols, format))};
  const fp4::Span ins[] = {fp4::piece(scales, (long long)rows * (cols / fp4::block_of(format)))};
  if (!fp4::apart(outs, ins)) return MOE_ERR_INVALID_ARG;
  const long long blocks = ((long long)rows * tiles + 255) / 256;
  return moe::launch_pdl(tile_scales_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0,
                         (cudaStream_t)stream, scales, rows, cols / fp4::block_of(format), tiles, tiled);
}

int fp4_quantize(const void* x, long long x_stride, int x_type, const fp4_matrix* out, void* stream) {
  if (!out) return MOE_ERR_INVALID_ARG;
  QuantizeArgs a{fp4::rows_of(x, x_stride, x_type), *out};
  if (const int rc = fp4::check_target(out, out->rows, out->cols)) return rc;
  if (const int rc = fp4::check_rows(a.x, out->rows, out->cols, true)) return rc;
  if (out->rows == 0) return MOE_OK;
  one_row(a.x, out->rows);
  const fp4::Span outs[] = {fp4::codes_span(*out), fp4::scales_span(*out), fp4::row_scale_span(*out)};
  const fp4::Span ins[] = {fp4::span_of(a.x, out->rows, out->cols, false)};
  if (!fp4::apart(outs, ins)) return MOE_ERR_INVALID_ARG;
  const QuantizeShape s(out->rows, out->cols);
  return by_units(s, [&](auto nb) {
    return by_type(x_type, [&](auto type) {
      return moe::launch_pdl(out->format == MOE_FMT_NVFP4 ? quantize_kernel<nb, type, true> : quantize_kernel<nb, type, false>,
                             s.grid, s.block, 0, (cudaStream_t)stream, a);
    });
  });
}

int fp4_dequantize(const fp4_matrix* m, void* out, long long out_stride, int out_type, void* stream) {
  if (const int rc = fp4::check_matrix(m)) return rc;
  DequantizeArgs a{*m, fp4::rows_of(out, out_stride, out_type)};
  if (const int rc = fp4::check_rows(a.out, m->rows, m->cols, true)) return rc;
  if (m->rows == 0) return MOE_OK;
  one_row(a.out, m->rows);
  const fp4::Span outs[] = {fp4::span_of(a.out, m->rows, m->cols, false)};
  const fp4::Span ins[] = {fp4::codes_span(*m), fp4::scales_span(*m), fp4::row_scale_span(*m)};
  if (!fp4::apart(outs, ins)) return MOE_ERR_INVALID_ARG;
  const LightShape s(m->rows, m->cols);
  return by_units(s, [&](auto nb) {
    return by_type(out_type, [&](auto type) {
      return moe::launch_pdl(
          m->format == MOE_FMT_NVFP4 ? dequantize_kernel<nb, type, true> : dequantize_kernel<nb, type, false>, s.grid,
          s.block, 0, (cudaStream_t)stream, a);
    });
  });
}

int fp4_swiglu(const void* gate, long long gate_stride, const void* up, long long up_stride, int type, int rows,
               int cols, void* out, long long out_stride, int out_type, const fp4_matrix* m, void* stream) {
  if (rows < 0 || (!out && !m && rows > 0)) return MOE_ERR_INVALID_ARG;
  if (!fp4::shape_ok(rows, cols, MOE_FMT_NVFP4)) return MOE_ERR_UNSUPPORTED;
  SwigluArgs a{fp4::rows_of(gate, gate_stride, type), fp4::rows_of(up, up_stride, type),
               fp4::rows_of(out, out_stride, out_type), m ? *m : fp4_matrix{}, rows, cols};
  if (const int rc = fp4::check_rows(a.gate, rows, cols, true)) return rc;
  if (const int rc = fp4::check_rows(a.up, rows, cols, true)) return rc;
  if (out)
    if (const int rc = fp4::check_rows(a.out, rows, cols, false)) return rc;
  if (m)
    if (const int rc = fp4::check_target(m, rows, cols)) return rc;
  if (rows == 0) return MOE_OK;
  one_row(a.gate, rows), one_row(a.up, rows), one_row(a.out, rows);
  const fp4::Span outs[] = {fp4::span_of(a.out, rows, cols, true), fp4::codes_span(a.m), fp4::scales_span(a.m), fp4::row_scale_span(a.m)};
  const fp4::Span ins[] = {fp4::span_of(a.gate, rows, cols, true), fp4::span_of(a.up, rows, cols, true)};
  if (!fp4::apart(outs, ins)) return MOE_ERR_INVALID_ARG;
  const LightShape s(rows, cols);
  return by_units(s, [&](auto nb) {
    return by_type(type, [&](auto t) {
      return moe::launch_pdl(swiglu_kernel<nb, t>, s.grid, s.block, 0, (cudaStream_t)stream, a);
    });
  });
}

int fp4_block_norm(const void* r, long long r_stride, int r_type, const void* y, long long y_stride, int y_type,
                   const float* post_weight, const void* gate, long long gate_stride, int gate_cols, double scale,
                   const float* weight, double eps, int rows, int cols, void* r_out, long long r_out_stride, void* h,
                   long long h_stride, int h_type, const fp4_matrix* m, void* stream) {
  if (rows < 0 || (!h && !m && rows > 0) || !(eps >= 0.) || !(eps <= 1e30) || !(fabs(scale) <= 1e30))
    return MOE_ERR_INVALID_ARG;
  if (!y && rows > 0 && (post_weight || gate)) return MOE_ERR_INVALID_ARG;
  if (!fp4::shape_ok(rows, cols, MOE_FMT_NVFP4)) return MOE_ERR_UNSUPPORTED;
  NormArgs a{fp4::rows_of(r, r_stride, r_type), fp4::rows_of(y, y_stride, y_type),
             fp4::rows_of(gate, gate_stride, y_type), fp4::rows_of(r_out, r_out_stride, r_type),
             fp4::rows_of(h, h_stride, h_type), gate_cols, post_weight, weight, (float)scale, (float)eps, rows, cols,
             m ? *m : fp4_matrix{}};
  if (const int rc = fp4::check_rows(a.r, rows, cols, true)) return rc;
  if (y)
    if (const int rc = fp4::check_rows(a.y, rows, cols, true)) return rc;
  if (!moe::aligned16(post_weight) || !moe::aligned16(weight)) return MOE_ERR_ALIGNMENT;
  if (gate) {
    if (gate_cols != 1 && gate_cols != cols) return MOE_ERR_INVALID_ARG;
    if (gate_cols == 1) {
      if ((uintptr_t)gate % fp4::element_bytes(y_type)) return MOE_ERR_ALIGNMENT;
      if (gate_stride < 0 || gate_stride >= (1ll << 38)) return MOE_ERR_INVALID_ARG;
    } else if (const int rc = fp4::check_rows(a.gate, gate_stride == 0 ? 1 : rows, cols, true)) {
      return rc;
    }
  }
  if (r_out)
    if (const int rc = fp4::check_rows(a.r_out, rows, cols, true)) return rc;
  if (h)
    if (const int rc = fp4::check_rows(a.h, rows, cols, false)) return rc;
  if (m)
    if (const int rc = fp4::check_target(m, rows, cols)) return rc;
  if (rows == 0) return MOE_OK;
  for (fp4::Rows* x : {&a.r, &a.y, &a.gate, &a.r_out, &a.h}) one_row(*x, rows);
  const fp4::Span outs[] = {fp4::span_of(a.r_out, rows, cols, true), fp4::span_of(a.h, rows, cols, true), fp4::codes_span(a.m),
                            fp4::scales_span(a.m), fp4::row_scale_span(a.m)};
  const fp4::Span ins[] = {fp4::span_of(a.r, rows, cols, true), fp4::span_of(a.y, rows, cols, true),
                           gate_cols == cols ? fp4::span_of(a.gate, gate_stride == 0 ? 1 : rows, cols, true)
                                             : fp4::span_of(a.gate, rows, 1, false),
                           fp4::piece(post_weight, 4ll * cols), fp4::piece(weight, 4ll * cols)};
  if (!fp4::apart(outs, ins)) return MOE_ERR_INVALID_ARG;
  const HeavyShape s(rows, cols);
  return by_units(s, [&](auto nb) {
    return by_type(r_type, [&](auto rt) {
      return by_type(y ? y_type : FP4_BF16, [&](auto yt) {
        return moe::launch_pdl(norm_kernel<nb, rt, yt>, s.grid, s.block, 0, (cudaStream_t)stream, a);
      });
    });
  });
}

}  // extern "C"
