// Quantisation of W = 8 or 16 elements of a row by a thread, whose neighbours have the
// elements beside them: a block of 16 or 32 columns is 1, 2 or 4 neighbouring lanes, four
// scales (one word of the tiled layout) are four times as many.  The whole warp takes part.
#pragma once

#include "fp4.cuh"

namespace fp4 {

// 2^(bits of the exponent field), field from 1 to 254.
__device__ __forceinline__ float power_field(int field) { return __uint_as_float((uint32_t)field << 23); }

// 8 elements of a type as they lie in memory (plain loads: a residual may be overwritten
// in place).
template <int TYPE>
struct Raw {
  uint4 q;
  __device__ __forceinline__ void load(const void* base, long long at) {
    q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
  }
  __device__ __forceinline__ void zero() { q = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = TYPE == FP4_BF16 ? make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u))
                                        : __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = v.x, f[2 * i + 1] = v.y;
    }
  }
};
template <>
struct Raw<FP4_FP32> {
  float4 q[2];
  __device__ __forceinline__ void load(const void* base, long long at) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    q[0] = p[0], q[1] = p[1];
  }
  __device__ __forceinline__ void zero() { q[0] = q[1] = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    f[0] = q[0].x, f[1] = q[0].y, f[2] = q[0].z, f[3] = q[0].w;
    f[4] = q[1].x, f[5] = q[1].y, f[6] = q[1].z, f[7] = q[1].w;
  }
};

// 1 / x within an ulp, 0 where that is below 2^-126.
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 8 floats -> a word of e2m1 codes, the first in the lowest nibble.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&f)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}
// The larger of |a|, |b|, |c|; NaN if there is one.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <bool NV, int W>
constexpr int kBlockLanes = (NV ? 16 : 32) / W;  // lanes that have a block
template <bool NV, int W>
constexpr int kScaleLanes = 4 * kBlockLanes<NV, W>;  // ... whose blocks' scales share a word

// The largest magnitude of the block as a bit pattern: in that order infinities and
// NaN are above all numbers.
template <bool NV, int W>
__device__ __forceinline__ uint32_t block_top(const float (&v)[W]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < W; i += 2) a = max_abs(a, v[i], v[i + 1]);
  uint32_t t = __float_as_uint(a);
#pragma unroll
  for (int k = 1; k < kBlockLanes<NV, W>; k *= 2) t = max(t, __shfl_xor_sync(0xffffffffu, t, k));
  return t;
}

// 2^E of an NVFP4 row.
struct RowScale {
  float up = 1.f, down = 1.f;  // 2^E, 2^-E
  bool bad = false;            // an infinity or a NaN in the row
  bool tiny = false;           // 2^-E / (a block's scale) would not be finite: the row is scaled first
  __device__ __forceinline__ float value() const { return bad ? __uint_as_float(0x7FC00000u) : up; }
};
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  RowScale s;
  s.bad = top >= 0x7F800000u;
  // top = f * 2^e: 2688 = 1.3125 * 2^11
  const int e = max(-126, (int)(top >> 23) - 127 - 11 + ((top & 0x7FFFFFu) > 0x280000u));
  s.up = power_field(127 + e), s.down = power_field(127 - e);
  s.tiny = e < -110;
  return s;
}
template <int W>
__device__ __forceinline__ void scale_first(const RowScale& s, float (&v)[W], uint32_t& top) {
  top = __float_as_uint(__uint_as_float(top) * s.down);
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] *= s.down;
}

// Codes of the elements (`words`), and the scales of this lane's block and its neighbours':
// the word is the one of the first of kScaleLanes lanes.  `in`: the elements exist.  A row that
// is tiny has been scaled before.
template <bool NV, int W>
__device__ __forceinline__ uint32_t quantize(const float (&v)[W], uint32_t top, const RowScale& row, int lane, bool in,
                                             uint32_t (&words)[W / 8]) {
  uint32_t scale, keep, turn = 0;  // masks of the codes: all or nothing, and their signs
  float q[W];
  if (NV) {
    // Quotients by Markstein's theorem: from a correctly rounded reciprocal and a
    // quotient within an ulp, one residual gives the correctly rounded quotient (ties
    // of e2m1 included), at a third of the cost of divisions.
    const float up = row.tiny ? 1.f : row.up, down = row.tiny ? 1.f : row.down;
    const float a = __uint_as_float(top) * down, sixth = 1.f / 6.f, b = a * sixth;
    scale = row.bad ? 0u : moe::f32_to_e4m3_rn_sat(fmaf(fmaf(-6.f, b, a), sixth, b));
    const float s = moe::e4m3x2_to_f32x2(scale).x;
    // 1 / s of a number of four bits: one step of Newton's method rounds it correctly
    const float y0 = reciprocal(s), y = fmaf(fmaf(-s, y0, 1.f), y0, y0);
    // Of the negated quotients, so that the residual is x - s q without a negation of x and a
    // zero keeps its sign; the codes' signs are turned round at the end.
    const float2 minus = make_float2(-y * down, -y * down), s2 = make_float2(s * up, s * up);
    const float2 none = make_float2(-0.f, -0.f);
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      const float2 x = make_float2(v[i], v[i + 1]), q0 = moe::ffma2(x, minus, none);
      const float2 z = moe::ffma2(moe::ffma2(q0, s2, x), minus, q0);
      q[i] = z.x, q[i + 1] = z.y;
    }
    turn = 0x88888888u;
    keep = scale != 0u ? 0xFFFFFFFFu : 0u;
  } else {
    // 6 = 1.5 * 2^2
    const bool bad = top >= 0x7F800000u;
    scale = bad ? 255u : (uint32_t)max(0, (int)(top >> 23) - 2 + ((top & 0x7FFFFFu) > 0x400000u));
    const float mult = power_field(254 - (int)min(scale, 253u));
#pragma unroll
    for (int i = 0; i < W; ++i) q[i] = v[i] * mult;
    keep = bad ? 0u : 0xFFFFFFFFu;
  }
#pragma unroll
  for (int i = 0; i < W / 8; ++i) {
    const float(&part)[8] = *reinterpret_cast<const float(*)[8]>(q + 8 * i);
    words[i] = (to_e2m1x8(part) ^ turn) & keep;
  }
  if (!in) scale = 0;
  constexpr int kStep = kBlockLanes<NV, W>;
  uint32_t four = scale << (8 * ((lane / kStep) & 3));
  four |= __shfl_xor_sync(0xffffffffu, four, kStep);
  four |= __shfl_xor_sync(0xffffffffu, four, 2 * kStep);
  return four;
}

}  // namespace fp4
